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
#include "cache4.cuh"
#include "pa_launch.h"
#include "pa_mla.h"
#include "pa_ptx.cuh"
#include "prefill_common.cuh"

namespace pa {
namespace {

constexpr int kTokens = 128;
constexpr int kTokenBytes = kTokens * 128;  // 64 elements of 128 tokens

// A query's rotary part of one token, in whole sectors where the addresses allow it.
template <bool kF16, bool kInterleaved>
__device__ __forceinline__ void turn_row(const uint16_t* src, uint16_t* dst, const float* cs, bool wide_in, bool wide_out) {
    Sector in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i] = load_sector(src + 16 * i, wide_in);
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // 16 pairs: sectors 2i, 2i + 1 or i, i + 2
        Sector& lo = in[kInterleaved ? 2 * i : i];
        Sector& hi = in[kInterleaved ? 2 * i + 1 : i + 2];
        if (cs != nullptr) {
            uint32_t u[16] = {lo.lo.x, lo.lo.y, lo.lo.z, lo.lo.w, lo.hi.x, lo.hi.y, lo.hi.z, lo.hi.w,
                              hi.lo.x, hi.lo.y, hi.lo.z, hi.lo.w, hi.hi.x, hi.hi.y, hi.hi.z, hi.hi.w};
            float v[32], c[16], s[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                *reinterpret_cast<float4*>(&c[4 * k]) = __ldg(reinterpret_cast<const float4*>(cs + 16 * i) + k);
                *reinterpret_cast<float4*>(&s[4 * k]) = __ldg(reinterpret_cast<const float4*>(cs + 32 + 16 * i) + k);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) unpack16x2(u[k], kF16, v[2 * k], v[2 * k + 1]);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int f = kInterleaved ? 2 * k : k, g = kInterleaved ? 2 * k + 1 : 16 + k;
                const float y = v[f] * c[k] - v[g] * s[k], z = v[g] * c[k] + v[f] * s[k];
                v[f] = y;
                v[g] = z;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) u[k] = pack16x2(v[2 * k], v[2 * k + 1], kF16);
            lo = Sector{make_uint4(u[0], u[1], u[2], u[3]), make_uint4(u[4], u[5], u[6], u[7])};
            hi = Sector{make_uint4(u[8], u[9], u[10], u[11]), make_uint4(u[12], u[13], u[14], u[15])};
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) store_sector(dst + 16 * i, in[i], wide_out);
}

// ----------------------------------------------------------------- query

// kLarge: a CTA an SM takes a run of (head, 128 tokens), all 512 columns of a head's weights in shared memory until the
// head changes; tokens come two tiles ahead.  Otherwise two CTAs an SM take 256 columns of one tile each.  Results leave
// by TMA from 64-column buffers; a token's rotary part is turned by warps of its own meanwhile.
template <bool kLarge>
struct Query {
    static constexpr int kCols = kLarge ? kMlaLatent : 256, kParts = kMlaLatent / kCols;
    static constexpr int kStages = kLarge ? 2 : 1, kBuffers = kLarge ? 2 : 1;
    static constexpr int kWBytes = kCols * kMlaNope * 2;
    static constexpr int kABytes = 2 * kTokenBytes;
    static constexpr int kAOff = kWBytes, kOutOff = kAOff + kStages * kABytes;
    static constexpr int kEnd = kOutOff + kBuffers * kTokenBytes;
    static constexpr int kSlots = kCols / 128;  // of tensor memory, 128 columns each
    struct Small {
        uint64_t w_full[kSlots], w_empty, a_full[kStages], a_empty[kStages], d_full[kSlots], d_empty[kSlots];
        uint32_t tmem_base;
        int abort;
    };
    static constexpr int kSmem = kEnd + (int)sizeof(Small);
};
// loads, MMAs, 4 warps for each buffer of results, 4 for the rotary part
template <bool kLarge>
constexpr int kQueryThreads = 192 + 128 * Query<kLarge>::kBuffers;
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
            mbar_init(&sh.d_empty[s], 8);
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
            uint32_t n = 0, units = 0;
            for (int i = first; i < last && ok; ++i, ++n) {
                const int u = i / tiles, h = u / L::kParts, part = u % L::kParts, tok0 = (i - u * tiles) * kTokens;
                if (u != unit) {
                    if (units > 0) ok = mbar_wait(&sh.w_empty, (units - 1) & 1, abort_sh, a.wait_ns);
                    if (!ok) break;
#pragma unroll 1
                    for (int q = 0; q < L::kSlots; ++q) {
                        mbar_arrive_expect_tx(&sh.w_full[q], 2 * kTokenBytes);
                        for (int c = 2 * q; c < 2 * q + 2; ++c)
                            tma_load_3d(sm + c * kTokenBytes, &map_w, &sh.w_full[q], part * L::kCols + c * 64, 0, h);
                    }
                    unit = u;
                    ++units;
                }
                const uint32_t s = n % L::kStages;
                ok = mbar_wait(&sh.a_empty[s], ((n / L::kStages) & 1) ^ 1, abort_sh, a.wait_ns);
                if (!ok) break;
                mbar_arrive_expect_tx(&sh.a_full[s], L::kABytes);
                tma_load_3d(sm + L::kAOff + s * L::kABytes, &map_in, &sh.a_full[s], 0, h, tok0);
                tma_load_3d(sm + L::kAOff + s * L::kABytes + kTokenBytes, &map_in, &sh.a_full[s], 64, h, tok0);
            }
            // every copy issued lands before the CTA may exit
            if (units > 0)
                for (int q = 0; q < L::kSlots; ++q) mbar_wait(&sh.w_full[q], (units - 1) & 1, nullptr, a.wait_ns);
            for (uint32_t s = 0; s < (uint32_t)L::kStages && s < n; ++s)
                mbar_wait(&sh.a_full[s], ((n - 1 - (n - 1 - s) % L::kStages) / L::kStages) & 1, nullptr, a.wait_ns);
        }
    } else if (warp == 1) {
        if (elect_one()) {  // ---- MMAs
            constexpr uint32_t idesc = idesc_f16(kTokens, 128, !kF16, false, true);
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
                const uint32_t s = n % L::kStages;
                ok = mbar_wait(&sh.a_full[s], (n / L::kStages) & 1, abort_sh, a.wait_ns);
                if (!ok) break;
                const uint32_t a0 = a_lo + s * (L::kABytes >> 4);
#pragma unroll 1
                for (int q = 0; q < L::kSlots; ++q, ++steps) {  // slot q: columns 128 q of the part
                    if (fresh) ok = mbar_wait(&sh.w_full[q], (units - 1) & 1, abort_sh, a.wait_ns);
                    if (ok) ok = mbar_wait(&sh.d_empty[q], (n & 1) ^ 1, abort_sh, a.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t w0 = w_lo + (uint32_t)(q * 2) * (kTokenBytes >> 4), dt = tbase + q * 128;
                    mma_ss_w<0>(dt, a0, a_hi, w0, w_hi, idesc);
#pragma unroll
                    for (int k = 1; k < 8; ++k)
                        mma_ss_w<1>(dt, a0 + (uint32_t)((k / 4 * kTokenBytes) >> 4) + (k & 3) * 2, a_hi, w0 + k * 128, w_hi, idesc);
                    mma_commit(&sh.d_full[q]);
                }
                if (!ok) break;
                mma_commit(&sh.a_empty[s]);
                if (i + 1 == last || (i + 1) / tiles != u) mma_commit(&sh.w_empty);
            }
            // (MMAs in flight end before the results are read, or after a timeout with their barriers)
            if (!ok && n > 0) mbar_wait(&sh.a_empty[(n - 1) % L::kStages], ((n - 1) / L::kStages) & 1, nullptr, a.wait_ns);
        }
    } else if (warp < 2 + 4 * L::kBuffers) {
        // ---- the result, a token a thread; each group of 4 warps has a buffer and every kBuffers-th 64 columns
        const int group = (warp - 2) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16, bar_id = 1 + group;
        const bool issuer = threadIdx.x == 64 + 128 * group;
        const bool wide = aligned32(a.out) && a.out_stride % 16 == 0;
        uint8_t* const buffer = sm + L::kOutOff + group * kTokenBytes;
        bool bad = false;
        uint32_t n = 0;
        for (int i = first; i < last && !bad; ++i, ++n) {
            const int u = i / tiles, h = u / L::kParts, part = u % L::kParts, tok0 = (i - u * tiles) * kTokens, tok = tok0 + row;
            bool write = tok < a.total;
            if (a.cos_sin != nullptr && write) {
                const int pos = __ldg(&a.positions[tok]);
                write = pos >= 0 && pos < a.max_position;
            }
            // tokens that are padding are left as they were: the tile is then written row by row, as one of few tokens is
            const bool by_rows = bar_or(bar_id, 128, !write && tok < a.total) || a.total - tok0 < 16;
            uint16_t* const dst = a.out + (long long)(write ? tok : 0) * a.out_stride + (long long)h * kMlaRow + part * L::kCols;
#pragma unroll 1
            for (int c = group; c < L::kCols / 64; c += L::kBuffers) {  // 64 columns
                const int q = c / 2;
                bad = !mbar_wait(&sh.d_full[q], n & 1, abort_sh, a.wait_ns);
                if (issuer) bulk_wait_read<0>();
                bad = bar_or(bar_id, 128, bad);  // the buffer is free
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
                if (lane == 0) mbar_arrive(&sh.d_empty[q]);  // (both halves of its 128 columns do)
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
                }
            }
        }
        if (issuer) bulk_wait_read<0>();  // (the buffer is not read any more; what was written is there when the grid ends)
        ok = !bad;
    } else {
        // ---- the rotary part, a token a thread
        const int row = (warp - 2 - 4 * L::kBuffers) * 32 + lane;
        const bool wide_in = aligned32(a.in) && a.in_stride % 16 == 0, wide_out = aligned32(a.out) && a.out_stride % 16 == 0;
        for (int i = first; i < last; ++i) {
            const int u = i / tiles, h = u / L::kParts, tok = (i - u * tiles) * kTokens + row;
            if (u % L::kParts != L::kParts - 1 || tok >= a.total) continue;
            const float* cs = nullptr;
            if (a.cos_sin != nullptr) {
                const int pos = __ldg(&a.positions[tok]);
                if (pos >= a.max_position) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
                if (pos < 0 || pos >= a.max_position) continue;
                cs = a.cos_sin + (long long)pos * kMlaRope;
            }
            turn_row<kF16, kInterleaved>(a.in + (long long)tok * a.in_stride + (long long)h * (kMlaNope + kMlaRope) + kMlaNope,
                                         a.out + (long long)tok * a.out_stride + (long long)h * kMlaRow + kMlaLatent, cs, wide_in, wide_out);
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

// A CTA takes 128 tokens of a head; warp 0 loads and multiplies, one thread, warps 1-4 write, a token a thread.
constexpr int kOutStages = 3, kOutStageBytes = 2 * kTokenBytes;  // 64 elements of 128 tokens, and of 128 rows of weights
constexpr int kOutSteps = kMlaLatent / 64, kOutSmem = kOutStages * kOutStageBytes + 1024;
constexpr int kOutThreads = 160;

template <bool kF16>
__global__ void __launch_bounds__(kOutThreads) mla_output_kernel(const __grid_constant__ MlaProjectArgs a,
                                                                 const __grid_constant__ CUtensorMap map_in,
                                                                 const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kOutStages], empty[kOutStages], done;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_store;
    volatile int* abort_sh = &abort_store;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = (int)blockIdx.x, tok0 = (int)blockIdx.y * kTokens;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kOutStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&done, 1);
        *abort_sh = 0;
        fence_barrier_init();
        tma_prefetch_map(&map_in);
        tma_prefetch_map(&map_w);
    }
    grid_dependency_wait();
    allow_dependents_launch();
    if (warp == 0) {
        tmem_alloc(&tmem_base_sh, kMlaValue);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = tmem_base_sh;

    if (warp == 0) {
        if (lane == 0) {
            auto load = [&](int step) {
                const int slot = step % kOutStages;
                uint8_t* at = sm + slot * kOutStageBytes;
                mbar_arrive_expect_tx(&full[slot], kOutStageBytes);
                tma_load_3d(at + kTokenBytes, &map_w, &full[slot], step * 64, 0, h);
                tma_load_3d(at, &map_in, &full[slot], step * 64, h, tok0);
            };
            for (int step = 0; step < kOutStages; ++step) load(step);
            constexpr uint32_t idesc = idesc_f16(kTokens, kMlaValue, !kF16, false, false);
            bool ok = true;
            int loaded = kOutStages;
            for (int step = 0; step < kOutSteps && ok; ++step) {
                const int slot = step % kOutStages;
                ok = mbar_wait(&full[slot], (step / kOutStages) & 1, abort_sh, a.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = smem_u32(sm + slot * kOutStageBytes);
                const uint64_t ad = sdesc_sw128(at, 16, 1024), bd = sdesc_sw128(at + kTokenBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ss(tbase, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), idesc, step > 0 || kk > 0);
                if (step + 1 == kOutSteps) {
                    mma_commit(&done);
                } else if (loaded < kOutSteps) {
                    mma_commit(&empty[slot]);
                    ok = mbar_wait(&empty[slot], (step / kOutStages) & 1, abort_sh, a.wait_ns);
                    if (ok) load(loaded++);
                }
            }
            if (!ok) {
                *abort_sh = 1;
                atomicCAS(a.status, 0, PA_ERR_TIMEOUT);
                // copies and MMAs in flight end before the CTA does
                for (int s = 0; s < kOutStages; ++s) {
                    const int last = loaded - 1 - (loaded - 1 - s) % kOutStages;
                    mbar_wait(&full[s], (last / kOutStages) & 1, nullptr, a.wait_ns);
                }
                mma_commit(&done);
                mbar_wait(&done, 0, nullptr, a.wait_ns);
            }
        }
    } else {
        const int q4 = warp & 3, row = q4 * 32 + lane, tok = tok0 + row;
        const bool write = tok < a.total;
        uint16_t* const dst = a.out + (long long)(write ? tok : 0) * a.out_stride + (long long)h * kMlaValue;
        const bool wide = aligned32(a.out) && a.out_stride % 16 == 0;
        const bool ok = mbar_wait(&done, 0, abort_sh, a.wait_ns);
        if (__all_sync(0xffffffffu, ok) && __any_sync(0xffffffffu, write)) {
            tc_fence_after();
#pragma unroll 2
            for (int c = 0; c < kMlaValue / 32; ++c) {
                uint32_t o[32];
                tmem_ld_x32(tbase + ((uint32_t)(q4 * 32) << 16) + c * 32, o);
                tmem_ld_wait();
                reg_fence(o);
                if (write) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[i] = pack16x2(__uint_as_float(o[16 * k + 2 * i]), __uint_as_float(o[16 * k + 2 * i + 1]), kF16);
                        store_sector(dst + c * 32 + 16 * k,
                                     Sector{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])}, wide);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tbase, kMlaValue);
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
    if (items >= 2 * sms) return launch_query<true, kF16, kInterleaved>(a, sms, maps, stream);
    return launch_query<false, kF16, kInterleaved>(a, items * Query<false>::kParts, maps, stream);
}

template <bool kF16>
cudaError_t launch_output(const MlaProjectArgs& a, const CUtensorMap* maps, cudaStream_t stream) {
    auto kernel = mla_output_kernel<kF16>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_dynamic_smem(kernel, kOutSmem, configured);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)a.heads, (unsigned)((a.total + kTokens - 1) / kTokens));
    return launch_overlapped(kernel, grid, dim3(kOutThreads), kOutSmem, stream, a, maps[0], maps[1]);
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
