// decode_fp4.cu -- single-token attention over 4-bit pages (PA_KV_FP4_E2M1).
//
//   S^T[keys, heads] = K q^T,  P = softmax,  O^T[dims, heads] = V^T P^T
//
// 0.5625 byte per cached element, so at the copy rate of the memory one SM
// has about 100 cycles for 16 keys (K and V, D = 128): 4096 elements to turn
// into fp16.  That conversion, not the products, is what the kernel is built
// around.  It runs in registers, straight into the fragments of
// mma.m16n8k16: measured per SM and cycle, 64 lanes of e2m1x2 -> f16x2
// conversion, 64 of byte permutes, 64 of f16x2 products and half an MMA, so
// 16 keys need about 50 (conversions and permutes), 32 (scale products) and
// 32 (MMA, up to 8 heads) cycles on three different pipes.  Converting into
// shared memory for tcgen05 instead would write and read back 2 bytes per
// element, 4 times what the page itself takes, through a port of 128 bytes
// per cycle.
//
// Keys are the M dimension of S^T and dims that of O^T, so a page element is
// always an A operand (256 elements per MMA, where it would be 128 as a B
// operand) and up to 8 query heads of a KV group fill N = 8 (two tiles up to
// 16 heads).  The order of the dims within a product and of the keys within
// a 16-key block is free, and chosen so that a lane's share is contiguous:
//   K   lane (g, t) of row g takes dims [t D/4, (t + 1) D/4): one or two
//       scale blocks, one load per row;
//   V   lane (g, t) takes dims [g D/8, (g + 1) D/8) of 4 keys: inside one
//       scale block, one load per key.
// code * scale is exact in fp16, so nothing is lost before the fp32
// accumulators; P is rounded to fp16 (relative 2^-12) and q, scaled by a
// power of two per head, is exact but for elements 2^14 below its largest.
//
// Each warp streams its own pages (every fourth of the item's) through its
// own ring of whole-slab bulk copies and keeps its own running maximum, sum
// and output, so warps meet only at the end of an item, where the four
// results are merged through the warps' free page buffers.  Splits of one
// sequence are merged by the last CTA to finish one (pa_decode) or by
// combine_kernel.  Every wait is bounded.
#include <cstdint>

#include "fp4.cuh"
#include "pa_internal.h"
#include "pa_launch.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kItems = 64;  // items of a CTA decoded once, in the prologue
constexpr float kLn2 = 0.69314718055994531f;
// The running maximum is only raised when a logit (in bits) exceeds it by more
// than this: P then reaches 2^8 in fp16, and most steps rescale nothing.
constexpr float kSlack = 8.f;

template <int D>
struct Layout {
    static constexpr int kSlab = fp4_slab_bytes(D);
    static constexpr int kStage = 2 * kSlab;  // K slab, V slab
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kBytes = kWarps * kStages * kStage;
    static_assert(16 * D * 4 <= kStage, "a warp's output (16 heads) must fit a page buffer");
};

struct Item {
    int b, s, kvh, nsplit, split_base, p0, p1, seq_len;
};

__device__ __forceinline__ void record(int* status, int code) { atomicCAS(status, 0, code); }

__device__ Item load_item(const DecodeArgs& a, int idx, int items_off) {
    const int32_t* meta = a.meta;
    Item it;
    int b = __ldg(&meta[items_off + 2 * idx]);
    const int w = __ldg(&meta[items_off + 2 * idx + 1]);
    int s = w >> 16, kvh = w & 0xFFFF;
    bool ok = (unsigned)b < (unsigned)a.batch && kvh < a.num_kv_heads;
    if (!ok) b = 0;
    int nsplit = __ldg(&meta[kMetaHeader + b]);
    if (nsplit < 1 || s < 0 || s >= nsplit) ok = false;
    int len = max(__ldg(&a.seq_lens[b]), 0);
    int pages = (int)(((long long)len + kPage - 1) / kPage);
    if (pages > a.max_pages) {
        record(a.status, PA_ERR_DEVICE_BOUNDS);
        pages = a.max_pages;
        len = pages * kPage;
    }
    if (!ok) {
        record(a.status, PA_ERR_DEVICE_BOUNDS);
        nsplit = 1; s = 0; kvh = 0; pages = 0; len = 0;
    }
    it.b = b; it.s = s; it.kvh = kvh; it.nsplit = nsplit;
    it.split_base = __ldg(&meta[kMetaHeader + a.batch + b]);
    it.p0 = (int)(((long long)s * pages) / nsplit);
    it.p1 = (int)(((long long)(s + 1) * pages) / nsplit);
    it.seq_len = len;
    return it;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// the half2 of byte `byte` of w (compile-time after unrolling)
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int byte) {
    return byte == 0 ? e2m1x2_to_half2<0>(w) : byte == 1 ? e2m1x2_to_half2<1>(w)
         : byte == 2 ? e2m1x2_to_half2<2>(w) : e2m1x2_to_half2<3>(w);
}

__device__ __forceinline__ uint16_t to_bf16(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// Which row of its 16-key block logical key k (of a product) is: neighbours
// swap in every other pair, so that the four keys of one V load, and the two
// of one K load phase, alternate between the two 64-byte halves of a
// 128-byte line of shared memory.
__device__ __forceinline__ int key_row(int k) { return k ^ ((k >> 1) & 1); }

// D: head dim; NT: 8-head tiles of the group
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 3) decode_fp4_kernel(const __grid_constant__ DecodeArgs a) {
    using L = Layout<D>;
    constexpr int S = L::kStages;
    constexpr int KK = D / 16;             // MMA steps over the dims of QK; dim tiles of PV
    constexpr int KB = NT == 1 ? 4 : 2;    // 16-key blocks per softmax step
    constexpr int kWords = D / 32;         // 32-bit code words of a lane's share of a K row
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kWarps][S];
    __shared__ Item items_sh[kItems];
    __shared__ float red_m[kWarps][NT * 8], red_l[kWarps][NT * 8];
    __shared__ int abort_store, merge_now;
    __shared__ int scratch_at[kWarps];  // the page buffer that holds each warp's output
    volatile int* abort_sh = &abort_store;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * (S * L::kStage);
    uint64_t* bar = full[warp];
    if (lane < S) mbar_init(&bar[lane], 1);
    if (threadIdx.x == 0) {
        abort_store = 0;
        merge_now = 0;
    }
    fence_barrier_init();
    grid_dependency_wait();  // shared memory only up to here

    const int items_off = kMetaHeader + 2 * a.batch + 1 + __ldg(&a.meta[5]) + 1;
    int it_lo = 0, it_hi = 0;
    if ((int)blockIdx.x < __ldg(&a.meta[5])) {
        it_lo = __ldg(&a.meta[kMetaHeader + 2 * a.batch + 1 + blockIdx.x]);
        it_hi = __ldg(&a.meta[kMetaHeader + 2 * a.batch + 1 + blockIdx.x + 1]);
    }
    for (int i = threadIdx.x; i < min(it_hi - it_lo, kItems); i += kThreads) items_sh[i] = load_item(a, it_lo + i, items_off);
    __syncthreads();
    auto get_item = [&](int j) { return j - it_lo < kItems ? items_sh[j - it_lo] : load_item(a, j, items_off); };

    // ---- producer side of this warp's ring
    int pj = it_lo, pp = 0, pend = 0, pkvh = 0, id_base = 0, ids = 0;
    long long bt_row = 0;
    bool pdone = false;
    uint32_t issued = 0, consumed = 0;  // pages handed to / taken from the ring
    uint32_t dead = 0;                  // stages whose page id was out of range
    auto load_ids = [&]() {  // the ids of this warp's next 32 pages
        id_base = pp;
        const int i = pp + kWarps * lane;
        ids = i < pend ? __ldg(&a.block_table[bt_row + i]) : 0;
    };
    auto open_item = [&]() {
        while (pp >= pend) {
            if (pj >= it_hi) {
                pdone = true;
                return;
            }
            const Item it = get_item(pj++);
            pp = it.p0 + warp;
            pend = it.p1;
            pkvh = it.kvh;
            bt_row = (long long)it.b * a.max_pages;
            if (pp < pend) load_ids();
        }
    };
    auto issue = [&]() {  // the warp's next page into the next stage, which is free
        if (!pdone) open_item();
        if (pdone) return;
        if (pp - id_base >= 32 * kWarps) load_ids();
        const int id = __shfl_sync(0xffffffffu, ids, (pp - id_base) / kWarps);
        const uint32_t st = issued % S;
        const bool ok = (unsigned)id < (unsigned)a.num_pool_pages;
        dead = ok ? dead & ~(1u << st) : dead | (1u << st);
        if (lane == 0) {
            if (ok) {
                const long long off = ((long long)id * a.num_kv_heads + pkvh) * L::kSlab;
                mbar_arrive_expect_tx(&bar[st], 2 * L::kSlab);
                bulk_load(ring + st * L::kStage, a.k_pool + off, L::kSlab, &bar[st]);
                bulk_load(ring + st * L::kStage + L::kSlab, a.v_pool + off, L::kSlab, &bar[st]);
            } else {
                record(a.status, PA_ERR_DEVICE_BOUNDS);
                mbar_arrive(&bar[st]);
            }
        }
        ++issued;
        pp += kWarps;
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) issue();

    const int G = a.group;
    bool bad = false;
    for (int j = it_lo; j < it_hi; ++j) {
        const Item it = get_item(j);
        const int key_end = min(it.seq_len, it.p1 * kPage);

        // ---- the group's queries as B fragments: head g (and 8 + g), dims [t D/4, (t + 1) D/4)
        uint32_t q[NT][2 * KK];
        float sl2[NT][2];
        const float base_scale = a.scale_log2 * __ldg(&a.k_scale[it.kvh]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint4 raw[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0, 0, 0, 0);
            if (n * 8 + g < G) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    a.q + ((long long)it.b * a.num_q_heads + it.kvh * G + n * 8 + g) * D + t * (D / 4));
#pragma unroll
                for (int i = 0; i < D / 32; ++i) raw[i] = __ldg(src + i);
            }
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^e <= amax < 2^(e+1), kept where both 2^e and 2^-e are ordinary floats
            const int e = amax > 0.f && amax < INFINITY ? min(max((int)(__float_as_uint(amax) >> 23) - 127, -96), 96) : 0;
            const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    q[n][4 * i + k] =
                        pack_half2(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xFFFF0000u) * down);
            }
            // head 2t + i of the tile: its power of two sits in lane 4 (2t + i)
            sl2[n][0] = base_scale * __shfl_sync(0xffffffffu, up, 8 * t);
            sl2[n][1] = base_scale * __shfl_sync(0xffffffffu, up, 8 * t + 4);
        }

        float o[NT][KK][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < KK; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][i][k] = 0.f;
        }

        bool owed = false;  // the last page's stage is refilled after the merge
        uint8_t* scratch = ring;
        for (int p = it.p0 + warp; p < it.p1 && !bad; p += kWarps) {
            const uint32_t st = consumed % S;
            const bool landed = mbar_wait(&bar[st], (consumed / S) & 1, abort_sh, a.wait_ns);
            if (!__all_sync(0xffffffffu, landed)) {
                bad = true;
                break;
            }
            ++consumed;
            const uint8_t* kc = ring + st * L::kStage;
            const uint8_t* vc = kc + L::kSlab;
            const int live = (dead >> st) & 1u ? 0 : min(key_end - p * kPage, kPage);  // keys of this page
#pragma unroll
            for (int step = 0; step < 4 / KB; ++step) {
                const int r0 = step * KB * 16;
                if (r0 >= live) break;
                // ---- S^T = K q^T
                float s[NT][KB][4];
#pragma unroll
                for (int blk = 0; blk < KB; ++blk) {
                    const int row = r0 + blk * 16 + key_row(g);
                    uint32_t w[2][kWords], sc[2][kWords / 2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint8_t* src = kc + (row + 8 * i) * (D / 2) + t * (D / 8);
                        const uint8_t* scl = kc + kPage * (D / 2) + (row + 8 * i) * (D / 16);
                        if constexpr (D == 128) {
                            const uint4 v = *reinterpret_cast<const uint4*>(src);
                            w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
                            const uint32_t h = e4m3x2_to_half2(reinterpret_cast<const uint16_t*>(scl)[t]);
                            sc[i][0] = __byte_perm(h, 0, 0x1010);
                            sc[i][1] = __byte_perm(h, 0, 0x3232);
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(src);
                            w[i][0] = v.x; w[i][1] = v.y;
                            sc[i][0] = __byte_perm(e4m3x2_to_half2(scl[t]), 0, 0x1010);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) s[n][blk][k] = 0.f;
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const int wi = kk / 2, byte = (kk & 1) * 2;
                        const uint32_t a0 = mul2(code_pair(w[0][wi], byte), sc[0][wi / 2]);
                        const uint32_t a1 = mul2(code_pair(w[1][wi], byte), sc[1][wi / 2]);
                        const uint32_t a2 = mul2(code_pair(w[0][wi], byte + 1), sc[0][wi / 2]);
                        const uint32_t a3 = mul2(code_pair(w[1][wi], byte + 1), sc[1][wi / 2]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816(s[n][blk], a0, a1, a2, a3, q[n][2 * kk], q[n][2 * kk + 1]);
                    }
                }
                // ---- running softmax, in bits
                const bool tail = live < r0 + KB * 16;
                bool raise = false;
                float mx[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v = -INFINITY;
#pragma unroll
                        for (int blk = 0; blk < KB; ++blk)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float& x = s[n][blk][2 * r + i];
                                x *= sl2[n][i];
                                if (tail && r0 + blk * 16 + 8 * r + key_row(g) >= live) x = -INFINITY;
                                v = fmaxf(v, x);
                            }
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        mx[n][i] = v;
                        raise |= v > m[n][i] + kSlack || (m[n][i] == -INFINITY && v > -INFINITY);
                    }
                if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float mn = fmaxf(m[n][i], mx[n][i]);
                            const float alpha = mn == -INFINITY ? 1.f : ex2(m[n][i] - mn);
                            m[n][i] = mn;
                            l[n][i] *= alpha;
#pragma unroll
                            for (int k = 0; k < KK; ++k) {
                                o[n][k][i] *= alpha;
                                o[n][k][2 + i] *= alpha;
                            }
                        }
                }
                uint32_t pb[NT][KB][2];  // P as B fragments: head g, keys (2t, 2t + 1) and (2t + 8, 2t + 9)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
                    for (int blk = 0; blk < KB; ++blk)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float p0 = ex2(s[n][blk][2 * r] - m0), p1 = ex2(s[n][blk][2 * r + 1] - m1);
                            l[n][0] += p0;
                            l[n][1] += p1;
                            pb[n][blk][r] = transpose8x8(pack_half2(p0, p1));
                        }
                }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int blk = 0; blk < KB; ++blk) {
                    const int k0 = r0 + blk * 16 + key_row(2 * t), k1 = r0 + blk * 16 + key_row(2 * t + 1);
                    const int keys[4] = {k0, k1, k0 + 8, k1 + 8};
                    uint32_t w[4][D / 64], b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (D == 128) {
                            const uint2 v = *reinterpret_cast<const uint2*>(vc + keys[i] * 64 + g * 8);
                            w[i][0] = v.x;
                            w[i][1] = v.y;
                            b[i] = vc[kPage * 64 + keys[i] * 8 + g];
                        } else {
                            w[i][0] = *reinterpret_cast<const uint32_t*>(vc + keys[i] * 32 + g * 4);
                            b[i] = vc[kPage * 32 + keys[i] * 4 + (g >> 1)];
                        }
                        // a dead key's scale may be a NaN, which a zero P would not cancel
                        if (tail && keys[i] >= live) b[i] = 0;
                    }
                    const uint32_t s01 = e4m3x2_to_half2(b[0] | (b[1] << 8)), s23 = e4m3x2_to_half2(b[2] | (b[3] << 8));
#pragma unroll
                    for (int mt = 0; mt < KK; ++mt) {
                        const uint32_t h0 = code_pair(w[0][mt / 4], mt & 3), h1 = code_pair(w[1][mt / 4], mt & 3);
                        const uint32_t h2 = code_pair(w[2][mt / 4], mt & 3), h3 = code_pair(w[3][mt / 4], mt & 3);
                        const uint32_t a0 = mul2(__byte_perm(h0, h1, 0x5410), s01);
                        const uint32_t a1 = mul2(__byte_perm(h0, h1, 0x7632), s01);
                        const uint32_t a2 = mul2(__byte_perm(h2, h3, 0x5410), s23);
                        const uint32_t a3 = mul2(__byte_perm(h2, h3, 0x7632), s23);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816(o[n][mt], a0, a1, a2, a3, pb[n][blk][0], pb[n][blk][1]);
                    }
                }
            }
            __syncwarp();  // every lane is done with the stage
            if (p + kWarps < it.p1) issue();
            else {
                owed = true;
                scratch = ring + st * L::kStage;
            }
        }

        // ---- merge the four warps: maxima and sums, then the outputs through the free page buffers
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], off);
                if (g == 0) {
                    red_m[warp][n * 8 + 2 * t + i] = m[n][i];
                    red_l[warp][n * 8 + 2 * t + i] = l[n][i];
                }
            }
        if (owed) {
            float* so = reinterpret_cast<float*>(scratch);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int mt = 0; mt < KK; ++mt)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (n * 8 + 2 * t + i < G)
                            *reinterpret_cast<float2*>(so + (n * 8 + 2 * t + i) * D + g * (D / 8) + 2 * mt) =
                                make_float2(o[n][mt][i], o[n][mt][2 + i]);
        }
        if (lane == 0) scratch_at[warp] = (int)(scratch - smem);
        if (__syncthreads_or(bad || *abort_sh != 0)) {
            bad = true;
            break;
        }
        const bool partial = it.nsplit > 1;
        const long long head0 = (long long)it.kvh * G;
        const long long orow = partial ? (long long)(it.split_base + it.s) * a.num_q_heads + head0
                                       : (long long)it.b * a.num_q_heads + head0;
        const float vs = __ldg(&a.v_scale[it.kvh]);
        for (int idx = threadIdx.x; idx < G * D; idx += kThreads) {
            const int h = idx / D, d = idx % D;
            float mm = -INFINITY, ll = 0.f, val = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, red_m[w][h]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = red_m[w][h], lw = red_l[w][h];
                if (mw == -INFINITY && lw == 0.f) continue;  // no live key: nothing was written
                const float f = ex2(mw - mm);                // a NaN logit leaves a NaN sum, and so a NaN output
                ll = fmaf(f, lw, ll);
                val = fmaf(f, reinterpret_cast<const float*>(smem + scratch_at[w])[h * D + d], val);
            }
            val = ll == 0.f ? 0.f : val * (vs / ll);
            if (partial) a.o_part[(orow + h) * D + d] = val;
            else a.out[(orow + h) * D + d] = to_bf16(val);
            if (d == 0) {
                const float lse = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
                if (partial) a.lse_part[orow + h] = lse;
                else if (a.lse) a.lse[orow + h] = lse;
            }
        }
        fence_proxy_async_smem();  // the buffers go back to the async copies
        if (partial && a.counters) __threadfence();
        __syncthreads();
        if (owed) issue();
        if (partial && a.counters) {
            // the last split of the sequence to arrive merges them all, in split order:
            // lse = m + ln sum_s exp(lse_s - m), out = sum_s exp(lse_s - lse) o_s
            int* ctr = a.counters + (long long)it.b * a.num_kv_heads + it.kvh;
            if (threadIdx.x == 0) {
                int prev;
                asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(prev) : "l"(ctr) : "memory");
                merge_now = prev == it.nsplit - 1;
            }
            __syncthreads();
            if (merge_now) {
                __threadfence();
                const long long base = (long long)it.split_base * a.num_q_heads + head0;
                const long long row = (long long)it.b * a.num_q_heads + head0;
                for (int idx = threadIdx.x; idx < G * D; idx += kThreads) {
                    const int h = idx / D, d = idx % D;
                    float mm = -INFINITY, sum = 0.f, acc = 0.f;
                    for (int s = 0; s < it.nsplit; ++s) mm = fmaxf(mm, __ldcg(&a.lse_part[base + (long long)s * a.num_q_heads + h]));
                    for (int s = 0; s < it.nsplit; ++s) {
                        const long long pr = base + (long long)s * a.num_q_heads + h;
                        const float ls = __ldcg(&a.lse_part[pr]);
                        if (ls == -INFINITY) continue;
                        const float w = __expf(ls - mm);
                        sum += w;
                        acc = fmaf(w, __ldcg(&a.o_part[pr * D + d]), acc);
                    }
                    a.out[(row + h) * D + d] = to_bf16(sum == 0.f ? 0.f : acc / sum);
                    if (d == 0 && a.lse) a.lse[row + h] = sum == 0.f ? -INFINITY : mm + __logf(sum);
                }
                if (threadIdx.x == 0) *ctr = 0;
            }
        }
    }
    if (bad) {
        if (lane == 0) {
            *abort_sh = 1;
            record(a.status, PA_ERR_TIMEOUT);
            // every issued copy must land before the CTA may exit
            for (; consumed < issued; ++consumed) mbar_wait(&bar[consumed % S], (consumed / S) & 1, nullptr, a.wait_ns);
        }
    }
}

template <int D, int NT>
cudaError_t launch_d(const DecodeArgs& a, int grid, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = ensure_dynamic_smem(decode_fp4_kernel<D, NT>, Layout<D>::kBytes, done);
    if (e != cudaSuccess) return e;
    return launch_overlapped(decode_fp4_kernel<D, NT>, dim3((unsigned)grid), dim3(kThreads), Layout<D>::kBytes, stream, a);
}

}  // namespace

cudaError_t launch_decode_fp4(int head_dim, const DecodeArgs& a, int grid, cudaStream_t stream) {
    if (head_dim == 128) return a.group <= 8 ? launch_d<128, 1>(a, grid, stream) : launch_d<128, 2>(a, grid, stream);
    return a.group <= 8 ? launch_d<64, 1>(a, grid, stream) : launch_d<64, 2>(a, grid, stream);
}

}  // namespace pa
