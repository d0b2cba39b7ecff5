// mla_project.cu -- the products with every head's own matrix that attention in
// the latent space needs before and after:
//
//   pa_mla_query   out[t, h, :512]  = q[t, h, :128] W_uk[h]     (128 x 512)
//                  out[t, h, 512:]  = q[t, h, 128:] turned by the token's angles
//   pa_mla_output  out[t, h]        = W_uv[h] o[t, h]           (128 x 512)
//
// With few tokens the weights are what is read, with many the activations; the
// products themselves stay far below the tensor cores' rate.  128 tokens are the
// rows of an MMA.  W_uk lies with its columns contiguous (an MN-major operand),
// W_uv with the summed dimension contiguous, so both are read as they are loaded.
#include <algorithm>

#include "cache4.cuh"
#include "pa_launch.h"
#include "pa_mla.h"
#include "pa_ptx.cuh"
#include "prefill_common.cuh"

namespace pa {
namespace {

constexpr int kTokens = 128;
constexpr int kTokenBytes = kTokens * 128;  // 64 elements of 128 tokens

// The rotary parts of 32 tokens of a head, a warp's: 4 lanes a token, 8 pairs each, so that a load or store touches whole
// sectors of 8 tokens.  All of the warp's loads are in flight before the first angle is asked for.
template <bool kF16, bool kInterleaved>
__device__ __forceinline__ void turn_rows(const MlaProjectArgs& a, int h, int tok0, int lane) {
    const int rj = lane & 3;
    const int ra = kInterleaved ? 16 * rj : 8 * rj, rb = kInterleaved ? 16 * rj + 8 : 32 + 8 * rj;
    uint4 lo[4], hi[4];
    int at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tok = tok0 + 8 * i + (lane >> 2);
        at[i] = -1;
        if (tok >= a.total) continue;
        at[i] = a.cos_sin != nullptr ? __ldg(&a.positions[tok]) : 0;
        const uint16_t* src = a.in + (long long)tok * a.in_stride + (long long)h * (kMlaNope + kMlaRope) + kMlaNope;
        lo[i] = __ldg(reinterpret_cast<const uint4*>(src + ra));
        hi[i] = __ldg(reinterpret_cast<const uint4*>(src + rb));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (at[i] < 0) continue;
        if (a.cos_sin != nullptr) {
            if (at[i] >= a.max_position) {
                atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
                continue;
            }
            float c[8], s[8], v[16];
            const float4* t = reinterpret_cast<const float4*>(a.cos_sin + (long long)at[i] * kMlaRope + 8 * rj);
            *reinterpret_cast<float4*>(&c[0]) = __ldg(t);
            *reinterpret_cast<float4*>(&c[4]) = __ldg(t + 1);
            *reinterpret_cast<float4*>(&s[0]) = __ldg(t + 8);
            *reinterpret_cast<float4*>(&s[4]) = __ldg(t + 9);
            uint32_t u[8] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w, hi[i].x, hi[i].y, hi[i].z, hi[i].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) unpack16x2(u[k], kF16, v[2 * k], v[2 * k + 1]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int f = kInterleaved ? 2 * k : k, g = kInterleaved ? 2 * k + 1 : 8 + k;
                const float y = v[f] * c[k] - v[g] * s[k], z = v[g] * c[k] + v[f] * s[k];
                v[f] = y;
                v[g] = z;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = pack16x2(v[2 * k], v[2 * k + 1], kF16);
            lo[i] = make_uint4(u[0], u[1], u[2], u[3]);
            hi[i] = make_uint4(u[4], u[5], u[6], u[7]);
        }
        uint16_t* dst = a.out + (long long)(tok0 + 8 * i + (lane >> 2)) * a.out_stride + (long long)h * kMlaRow + kMlaLatent;
        *reinterpret_cast<uint4*>(dst + ra) = lo[i];
        *reinterpret_cast<uint4*>(dst + rb) = hi[i];
    }
}

// ----------------------------------------------------------------- query

// kLarge: a CTA an SM takes a run of (head, 128 tokens), all 512 columns of a head's weights in shared memory until the
// head changes.  Otherwise two CTAs an SM take 256 columns of one tile each.  Results leave by TMA from 64-column buffers
// of two groups of 4 warps: two buffers each, or one in the place of the one tile's tokens, which are multiplied by then.
// Rotary parts are turned meanwhile, by warps of their own or by the first group before it has results to wait for.
//
// Bound by memory: 1 token x 128 heads is 17 MB of weights in 5.7 us (2.9 TB/s, of which the launch and the first
// loads' latency are over half), 64 x 128 29 MB in 7.3 us (4.0 TB/s), 1999 x 64 205 MB in 40.7 us, 147 MB of them
// written: a plain fill of as many bytes takes 39 us (3.8 TB/s), one of 1 GB runs at 4.0 TB/s.  Tiles of 128 columns, three CTAs an
// SM, took 7.1 and 9.8 us for the first two; three groups of one buffer and a token tile ahead 42 us for the third,
// weights loaded for every tile and heads side by side in time 45.
template <bool kLarge>
struct Query {
    static constexpr int kCols = kLarge ? kMlaLatent : 256, kParts = kMlaLatent / kCols;
    static constexpr int kStages = 2, kGroups = 2, kDeep = kLarge ? 2 : 1, kRotaryWarps = kLarge ? 4 : 0;
    static constexpr int kWBytes = kCols * kMlaNope * 2;
    static constexpr int kAOff = kWBytes, kOutOff = kAOff + (kLarge ? kStages * kTokenBytes : 0);
    static constexpr int kEnd = kOutOff + kGroups * kDeep * kTokenBytes;
    static constexpr int kPer = 4, kSlots = kCols / 64 / kPer;  // tensor memory: slots of kPer x 64 columns
    static_assert(kGroups <= kPer, "every group has a part of every slot");
    static_assert(kLarge || (kSlots == 1 && kGroups <= kStages), "a result is there once all tokens are multiplied");
    struct Small {
        uint64_t w_full[kSlots], w_empty, a_full[kStages], a_empty[kStages], d_full[kSlots], d_empty[kSlots];
        uint32_t tmem_base;
        int abort;
    };
    static constexpr int kSmem = kEnd + (int)sizeof(Small);
};
// loads, MMAs, 4 warps for each buffer of results, those for the rotary part
template <bool kLarge>
constexpr int kQueryThreads = 64 + 128 * Query<kLarge>::kGroups + 32 * Query<kLarge>::kRotaryWarps;
static_assert(Query<true>::kSmem <= 232448 && Query<false>::kSmem <= 115712, "one CTA an SM, two");

template <bool kLarge, bool kF16, bool kInterleaved>
__global__ void __launch_bounds__(kQueryThreads<kLarge>, kLarge ? 1 : 2)
    mla_query_kernel(const __grid_constant__ MlaProjectArgs a, const __grid_constant__ CUtensorMap map_in,
                     const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_out) {
    using L = Query<kLarge>;
    extern __shared__ __align__(1024) uint8_t sm[];
    typename L::Small& sh = *reinterpret_cast<typename L::Small*>(sm + L::kEnd);
    volatile int* const abort_sh = &sh.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = (a.total + kTokens - 1) / kTokens;
    // units (head, part) x tiles: this CTA's run
    const int items = a.heads * L::kParts * tiles;
    const int first = (int)((long long)items * blockIdx.x / gridDim.x), last = (int)((long long)items * (blockIdx.x + 1) / gridDim.x);
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kSlots; ++s) mbar_init(&sh.w_full[s], 1);
        mbar_init(&sh.w_empty, 1);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&sh.a_full[s], 1);
            mbar_init(&sh.a_empty[s], 1);
        }
        for (int s = 0; s < L::kSlots; ++s) {
            mbar_init(&sh.d_full[s], 1);
            mbar_init(&sh.d_empty[s], 4 * L::kGroups);
        }
        *abort_sh = 0;
        fence_barrier_init();
        tma_prefetch_map(&map_in);
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_out);
    }
    grid_dependency_wait();
    allow_dependents_launch();
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, L::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sh.tmem_base;
    bool ok = true;

    if (warp == 0) {
        if (elect_one()) {  // ---- loads
            int unit = -1;
            uint32_t m = 0, units = 0;
            for (int i = first; i < last && ok; ++i) {
                const int u = i / tiles, h = u / L::kParts, part = u % L::kParts, tok0 = (i - u * tiles) * kTokens;
                if (u != unit) {
                    if (units > 0) ok = mbar_wait(&sh.w_empty, (units - 1) & 1, abort_sh, a.wait_ns);
                    if (!ok) break;
#pragma unroll 1
                    for (int q = 0; q < L::kSlots; ++q) {
                        mbar_arrive_expect_tx(&sh.w_full[q], L::kPer * kTokenBytes);
                        for (int c = L::kPer * q; c < L::kPer * (q + 1); ++c)
                            tma_load_3d(sm + c * kTokenBytes, &map_w, &sh.w_full[q], part * L::kCols + c * 64, 0, h);
                    }
                    unit = u;
                    ++units;
                }
                for (int k = 0; k < 2 && ok; ++k, ++m) {
                    const uint32_t s = m % L::kStages;
                    ok = mbar_wait(&sh.a_empty[s], ((m / L::kStages) & 1) ^ 1, abort_sh, a.wait_ns);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&sh.a_full[s], kTokenBytes);
                    tma_load_3d(sm + L::kAOff + s * kTokenBytes, &map_in, &sh.a_full[s], 64 * k, h, tok0);
                }
            }
            // every copy issued lands before the CTA may exit
            if (units > 0)
                for (int q = 0; q < L::kSlots; ++q) mbar_wait(&sh.w_full[q], (units - 1) & 1, nullptr, a.wait_ns);
            for (uint32_t s = 0; s < (uint32_t)L::kStages && s < m; ++s)
                mbar_wait(&sh.a_full[s], ((m - 1 - (m - 1 - s) % L::kStages) / L::kStages) & 1, nullptr, a.wait_ns);
        }
    } else if (warp == 1) {
        if (elect_one()) {  // ---- MMAs
            constexpr uint32_t idesc = idesc_f16(kTokens, 64 * L::kPer, !kF16, false, true);
            const uint64_t ad = sdesc_sw128(smem_u32(sm + L::kAOff), 16, 1024), wd = sdesc_sw128(smem_u32(sm), kTokenBytes, 1024);
            const uint32_t a_lo = (uint32_t)ad, w_lo = (uint32_t)wd, a_hi = (uint32_t)(ad >> 32), w_hi = (uint32_t)(wd >> 32);
            int unit = -1;
            uint32_t n = 0, units = 0, steps = 0;
            for (int i = first; i < last && ok; ++i, ++n) {
                const int u = i / tiles;
                const bool fresh = u != unit;
                if (fresh) {
                    unit = u;
                    ++units;
                }
                uint32_t a0[2];
                for (uint32_t k = 0; k < 2; ++k) {
                    const uint32_t m = 2 * n + k, s = m % L::kStages;
                    if (ok) ok = mbar_wait(&sh.a_full[s], (m / L::kStages) & 1, abort_sh, a.wait_ns);
                    a0[k] = a_lo + s * (kTokenBytes >> 4);
                }
                if (!ok) break;
#pragma unroll 1
                for (int q = 0; q < L::kSlots; ++q, ++steps) {
                    if (fresh) ok = mbar_wait(&sh.w_full[q], (units - 1) & 1, abort_sh, a.wait_ns);
                    if (ok) ok = mbar_wait(&sh.d_empty[q], (n & 1) ^ 1, abort_sh, a.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t w0 = w_lo + (uint32_t)(q * L::kPer) * (kTokenBytes >> 4), dt = tbase + q * 64 * L::kPer;
                    mma_ss_w<0>(dt, a0[0], a_hi, w0, w_hi, idesc);
#pragma unroll
                    for (int k = 1; k < 8; ++k)
                        mma_ss_w<1>(dt, a0[k / 4] + (k & 3) * 2, a_hi, w0 + k * 128, w_hi, idesc);
                    mma_commit(&sh.d_full[q]);
                }
                if (!ok) break;
                for (uint32_t k = 0; k < 2; ++k) mma_commit(&sh.a_empty[(2 * n + k) % L::kStages]);
                if (i + 1 == last || (i + 1) / tiles != u) mma_commit(&sh.w_empty);
            }
            // (MMAs in flight end before the results are read, or after a timeout with their barriers)
            if (!ok && n > 0) mbar_wait(&sh.a_empty[(2 * n - 1) % L::kStages], ((2 * n - 1) / L::kStages) & 1, nullptr, a.wait_ns);
        }
    } else if (warp < 2 + 4 * L::kGroups) {
        // ---- the result, a token a thread; each group of 4 warps has kDeep buffers and every kGroups-th 64 columns
        const uint32_t group = (warp - 2) >> 2;
        const int q4 = warp & 3, row = q4 * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16, bar_id = 1 + group;
        const bool issuer = threadIdx.x == 64 + 128 * group;
        const bool wide = aligned32(a.out) && a.out_stride % 16 == 0;
        uint8_t* buffer = sm + L::kOutOff + group * L::kDeep * kTokenBytes;
        bool late = false, bad = false;  // this thread's wait ended at its limit, one of the group's
        uint32_t n = 0;
        for (int i = first; i < last && !bad; ++i, ++n) {
            const int u = i / tiles, h = u / L::kParts, part = u % L::kParts, tok0 = (i - u * tiles) * kTokens, tok = tok0 + row;
            if (!kLarge && group == 0 && part == L::kParts - 1) turn_rows<kF16, kInterleaved>(a, h, tok0 + 32 * (warp - 2), lane);
            bool write = tok < a.total;
            if (a.cos_sin != nullptr && write) {
                const int pos = __ldg(&a.positions[tok]);
                write = pos >= 0 && pos < a.max_position;
            }
            // tokens that are padding are left as they were: the tile is then written row by row, as one of few tokens is
            const bool by_rows = bar_or(bar_id, 128, !write && tok < a.total) || a.total - tok0 < 16;
            uint16_t* const dst = a.out + (long long)(write ? tok : 0) * a.out_stride + (long long)h * kMlaRow + part * L::kCols;
#pragma unroll 1
            for (int c = 0; c < L::kCols / 64; ++c) {  // 64 columns
                const int q = c / L::kPer;
                // (each waits for every slot of every tile, its first chunk or not: no slot runs two ahead of it)
                if (c % L::kPer == 0) late |= !mbar_wait(&sh.d_full[q], n & 1, abort_sh, a.wait_ns);
                if ((n * (L::kCols / 64) + c) % L::kGroups != group) continue;
                if (issuer) bulk_wait_read<L::kDeep - 1>();
                bad = bar_or(bar_id, 128, late);  // the buffer is free
                if (bad) break;
                tc_fence_after();
                uint32_t o[64];
                uint32_t (&o0)[32] = *reinterpret_cast<uint32_t (*)[32]>(&o[0]);
                uint32_t (&o1)[32] = *reinterpret_cast<uint32_t (*)[32]>(&o[32]);
                tmem_ld_x32(tbase + lane_addr + c * 64, o0);
                tmem_ld_x32(tbase + lane_addr + c * 64 + 32, o1);
                tmem_ld_wait();
                reg_fence(o0);
                reg_fence(o1);
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && c % L::kPer + L::kGroups >= L::kPer) mbar_arrive(&sh.d_empty[q]);  // the group's last of the slot
                uint32_t w[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) w[k] = pack16x2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]), kF16);
                if (by_rows) {
                    if (write) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            store_sector(dst + c * 64 + 16 * k, Sector{make_uint4(w[8 * k], w[8 * k + 1], w[8 * k + 2], w[8 * k + 3]),
                                         make_uint4(w[8 * k + 4], w[8 * k + 5], w[8 * k + 6], w[8 * k + 7])}, wide);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4*>(buffer + row * 128 + ((k ^ (row & 7)) << 4)) =
                            make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    fence_proxy_async_smem();
                    named_bar_sync(bar_id, 128);
                    if (issuer) {
                        tma_store_3d(&map_out, buffer, part * L::kCols + c * 64, h, tok0);
                        bulk_commit();
                    }
                    if (L::kDeep == 2) buffer = sm + L::kOutOff + ((buffer - (sm + L::kOutOff)) ^ kTokenBytes);
                }
            }
        }
        if (issuer) bulk_wait_read<0>();  // (the buffer is not read any more; what was written is there when the grid ends)
        ok = !bad && !late;
    } else {
        // ---- the rotary part, 32 tokens a warp
        const int w = warp - 2 - 4 * L::kGroups;
        for (int i = first; i < last; ++i) {
            const int u = i / tiles;
            if (u % L::kParts == L::kParts - 1) turn_rows<kF16, kInterleaved>(a, u / L::kParts, (i - u * tiles) * kTokens + 32 * w, lane);
        }
    }
    if (!ok) {
        *abort_sh = 1;
        atomicCAS(a.status, 0, PA_ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, L::kCols);
    }
}

// ----------------------------------------------------------------- output

// A CTA an SM takes a run of groups of 32 tokens, head by head, with a head's 128 KB of weights in shared memory, the
// run in tiles of up to 128 tokens whose 64-element pieces pass through a ring.  32 tokens are the unit so that SMs get
// equal shares: only the groups of a tile that are the CTA's own are loaded, and written a token a thread.  (Rows of a
// tile that were not loaded hold what was there; a row of a product depends on its own row alone.)
//
// Bound by memory: 64 tokens x 128 heads are 27 MB in 5.4 us (5.1 TB/s), 1499 x 32 66 MB in 13.4 us (4.9 TB/s, 1.2 of
// it because SMs are given 12 groups or none).  A CTA a tile, two an SM, its weights streamed along with the tokens,
// took 6.1 and 16.8 us.
struct Output {
    static constexpr int kGroup = kMlaOutputGroup, kSteps = kMlaLatent / 64, kStages = 5;
    static constexpr int kWBytes = kSteps * kTokenBytes;  // 64 elements of a head's 128 rows, eight times
    static constexpr int kAOff = kWBytes, kEnd = kAOff + kStages * kTokenBytes;
    struct Small {
        uint64_t w_full[kSteps], w_empty[kSteps], a_full[kStages], a_empty[kStages], d_full[2], d_empty[2];
        uint32_t tmem_base;
        int abort;
    };
    static constexpr int kSmem = kEnd + (int)sizeof(Small);
    static constexpr int kThreads = 192;  // loads, MMAs, 4 warps for the results
};
static_assert(Output::kSmem <= 232448, "a CTA an SM");

// The tiles of a CTA's run of groups, in order.
struct OutputRun {
    int at, end, per_head, total;
    int h, tok0, rows;  // the tile: its head, first token, and how many tokens are loaded
    __device__ __forceinline__ OutputRun(const MlaProjectArgs& a)
        : per_head((a.total + Output::kGroup - 1) / Output::kGroup), total(a.total), h(0), tok0(0), rows(0) {
        const long long groups = (long long)a.heads * per_head;
        at = (int)(groups * blockIdx.x / gridDim.x);
        end = (int)(groups * (blockIdx.x + 1) / gridDim.x);
    }
    __device__ __forceinline__ bool next() {
        if (at >= end) return false;
        h = at / per_head;
        const int first = at - h * per_head, n = min(min(kTokens / Output::kGroup, per_head - first), end - at);
        tok0 = first * Output::kGroup;
        rows = n * Output::kGroup;
        at += n;
        return true;
    }
};

template <bool kF16>
__global__ void __launch_bounds__(Output::kThreads, 1) mla_output_kernel(const __grid_constant__ MlaProjectArgs a,
                                                                         const __grid_constant__ CUtensorMap map_in,
                                                                         const __grid_constant__ CUtensorMap map_w) {
    using L = Output;
    extern __shared__ __align__(1024) uint8_t sm[];
    L::Small& sh = *reinterpret_cast<L::Small*>(sm + L::kEnd);
    volatile int* const abort_sh = &sh.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kSteps; ++s) {
            mbar_init(&sh.w_full[s], 1);
            mbar_init(&sh.w_empty[s], 1);
        }
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&sh.a_full[s], 1);
            mbar_init(&sh.a_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.d_full[s], 1);
            mbar_init(&sh.d_empty[s], 4);
        }
        *abort_sh = 0;
        fence_barrier_init();
        tma_prefetch_map(&map_in);
        tma_prefetch_map(&map_w);
    }
    grid_dependency_wait();
    allow_dependents_launch();
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, 2 * kMlaValue);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sh.tmem_base;
    bool ok = true;

    OutputRun run(a);
    if (warp == 0) {
        if (elect_one()) {  // ---- loads
            int head = -1;
            uint32_t m = 0, heads = 0;
            uint32_t last_w = 0;  // how many of the newest head's pieces were asked for
            while (ok && run.next()) {
                const bool fresh = run.h != head;
                if (fresh) {
                    head = run.h;
                    ++heads;
                    last_w = 0;
                }
#pragma unroll 1
                for (int k = 0; k < L::kSteps; ++k, ++m) {
                    if (fresh) {
                        if (heads > 1) ok = mbar_wait(&sh.w_empty[k], heads & 1, abort_sh, a.wait_ns);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&sh.w_full[k], kTokenBytes);
                        tma_load_3d(sm + k * kTokenBytes, &map_w, &sh.w_full[k], 64 * k, 0, head);
                        last_w = (uint32_t)k + 1;
                    }
                    const uint32_t s = m % L::kStages;
                    ok = mbar_wait(&sh.a_empty[s], ((m / L::kStages) & 1) ^ 1, abort_sh, a.wait_ns);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&sh.a_full[s], run.rows * 128);
                    for (int r = 0; r < run.rows; r += L::kGroup)
                        tma_load_3d(sm + L::kAOff + s * kTokenBytes + r * 128, &map_in, &sh.a_full[s], 64 * k, head, run.tok0 + r);
                }
            }
            // every copy issued lands before the CTA may exit
            for (uint32_t k = 0; k < (uint32_t)L::kSteps && heads > 0; ++k)
                if (k < last_w || heads > 1) mbar_wait(&sh.w_full[k], (k < last_w ? heads - 1 : heads) & 1, nullptr, a.wait_ns);
            for (uint32_t s = 0; s < (uint32_t)L::kStages && s < m; ++s)
                mbar_wait(&sh.a_full[s], ((m - 1 - (m - 1 - s) % L::kStages) / L::kStages) & 1, nullptr, a.wait_ns);
        }
    } else if (warp == 1) {
        if (elect_one()) {  // ---- MMAs
            constexpr uint32_t idesc = idesc_f16(kTokens, kMlaValue, !kF16, false, false);
            const uint64_t ad = sdesc_sw128(smem_u32(sm + L::kAOff), 16, 1024), wd = sdesc_sw128(smem_u32(sm), 16, 1024);
            const uint32_t a_lo = (uint32_t)ad, w_lo = (uint32_t)wd, a_hi = (uint32_t)(ad >> 32), w_hi = (uint32_t)(wd >> 32);
            int head = -1;
            uint32_t n = 0, m = 0, heads = 0;
            for (bool more = run.next(); more && ok; ++n) {
                const bool fresh = run.h != head;
                if (fresh) {
                    head = run.h;
                    ++heads;
                }
                more = run.next();  // (the one after this one)
                const bool leaves = !more || run.h != head;
                const uint32_t slot = n & 1, dt = tbase + slot * kMlaValue;
                ok = mbar_wait(&sh.d_empty[slot], ((n >> 1) & 1) ^ 1, abort_sh, a.wait_ns);
#pragma unroll 1
                for (int k = 0; k < L::kSteps && ok; ++k, ++m) {
                    const uint32_t s = m % L::kStages;
                    if (fresh) ok = mbar_wait(&sh.w_full[k], (heads - 1) & 1, abort_sh, a.wait_ns);
                    if (ok) ok = mbar_wait(&sh.a_full[s], (m / L::kStages) & 1, abort_sh, a.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a0 = a_lo + s * (kTokenBytes >> 4), w0 = w_lo + k * (kTokenBytes >> 4);
                    if (k == 0)
                        mma_ss_w<0>(dt, a0, a_hi, w0, w_hi, idesc);
                    else
                        mma_ss_w<1>(dt, a0, a_hi, w0, w_hi, idesc);
#pragma unroll
                    for (int i = 1; i < 4; ++i) mma_ss_w<1>(dt, a0 + i * 2, a_hi, w0 + i * 2, w_hi, idesc);
                    mma_commit(&sh.a_empty[s]);
                    if (leaves) mma_commit(&sh.w_empty[k]);
                }
                if (ok) mma_commit(&sh.d_full[slot]);
            }
            // MMAs in flight end before the CTA does
            if (!ok && m > 0) mbar_wait(&sh.a_empty[(m - 1) % L::kStages], ((m - 1) / L::kStages) & 1, nullptr, a.wait_ns);
        }
    } else {
        // ---- the result, a token a thread
        const int q4 = warp & 3, row = q4 * 32 + lane;
        const bool wide = aligned32(a.out) && a.out_stride % 16 == 0;
        for (uint32_t n = 0; ok && run.next(); ++n) {
            const int tok = run.tok0 + row;
            const bool write = row < run.rows && tok < a.total;
            uint16_t* const dst = a.out + (long long)(write ? tok : 0) * a.out_stride + (long long)run.h * kMlaValue;
            const uint32_t slot = n & 1;
            ok = mbar_wait(&sh.d_full[slot], (n >> 1) & 1, abort_sh, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kMlaValue / 64; ++c) {
                uint32_t o[64];
                uint32_t (&o0)[32] = *reinterpret_cast<uint32_t (*)[32]>(&o[0]);
                uint32_t (&o1)[32] = *reinterpret_cast<uint32_t (*)[32]>(&o[32]);
                const uint32_t at = tbase + ((uint32_t)(q4 * 32) << 16) + slot * kMlaValue + c * 64;
                tmem_ld_x32(at, o0);
                tmem_ld_x32(at + 32, o1);
                tmem_ld_wait();
                reg_fence(o0);
                reg_fence(o1);
                if (c + 1 == kMlaValue / 64) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.d_empty[slot]);
                }
                if (!write) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i] = pack16x2(__uint_as_float(o[16 * k + 2 * i]), __uint_as_float(o[16 * k + 2 * i + 1]), kF16);
                    store_sector(dst + c * 64 + 16 * k, Sector{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])}, wide);
                }
            }
        }
    }
    if (!ok) {
        *abort_sh = 1;
        atomicCAS(a.status, 0, PA_ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, 2 * kMlaValue);
    }
}

template <bool kLarge, bool kF16, bool kInterleaved>
cudaError_t launch_query(const MlaProjectArgs& a, long long ctas, const CUtensorMap* maps, cudaStream_t stream) {
    using L = Query<kLarge>;
    auto kernel = mla_query_kernel<kLarge, kF16, kInterleaved>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_dynamic_smem(kernel, L::kSmem, configured);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, dim3((unsigned)ctas), dim3(kQueryThreads<kLarge>), L::kSmem, stream, a, maps[0], maps[1], maps[2]);
}

template <bool kF16, bool kInterleaved>
cudaError_t launch_query_size(const MlaProjectArgs& a, const CUtensorMap* maps, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long items = (long long)a.heads * ((a.total + kTokens - 1) / kTokens);
    // (with 128 heads and one tile both take the same time, 5.8 us for 1 token and 7.3 for 64; from there on SMs keep
    // weights, below it halves reach twice as many SMs)
    if (items >= 2 * sms) return launch_query<true, kF16, kInterleaved>(a, sms, maps, stream);
    return launch_query<false, kF16, kInterleaved>(a, items * Query<false>::kParts, maps, stream);
}

// How many CTAs: parts of one head each, so that none loads two heads' weights, or all SMs with equal shares, where the
// longest share is then shorter by more than those weights, as long as 4 groups.  Measured at 32 heads of 1499 tokens
// (12 groups against 10): 13.4 us and 13.7 us.
int output_ctas(int heads, int total, int sms) {
    const long long per_head = (total + Output::kGroup - 1) / Output::kGroup;
    const long long groups = heads * per_head, equal = (groups + sms - 1) / sms;
    if (heads >= sms) return sms;
    const long long parts = std::min<long long>(sms / heads, per_head), whole = (per_head + parts - 1) / parts;
    return (int)(whole <= equal + 4 ? heads * parts : std::min<long long>(sms, groups));
}

template <bool kF16>
cudaError_t launch_output(const MlaProjectArgs& a, const CUtensorMap* maps, cudaStream_t stream) {
    auto kernel = mla_output_kernel<kF16>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_dynamic_smem(kernel, Output::kSmem, configured);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, dim3((unsigned)output_ctas(a.heads, a.total, sms)), dim3(Output::kThreads), Output::kSmem, stream, a,
                             maps[0], maps[1]);
}

}  // namespace

cudaError_t launch_mla_query(const MlaProjectArgs& a, const CUtensorMap* maps, cudaStream_t stream) {
    if (a.f16) return a.interleaved ? launch_query_size<true, true>(a, maps, stream) : launch_query_size<true, false>(a, maps, stream);
    return a.interleaved ? launch_query_size<false, true>(a, maps, stream) : launch_query_size<false, false>(a, maps, stream);
}

cudaError_t launch_mla_output(const MlaProjectArgs& a, const CUtensorMap* maps, cudaStream_t stream) {
    return a.f16 ? launch_output<true>(a, maps, stream) : launch_output<false>(a, maps, stream);
}

}  // namespace pa
