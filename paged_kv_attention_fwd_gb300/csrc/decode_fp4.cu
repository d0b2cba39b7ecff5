// decode_fp4.cu -- single-token attention over 4-bit pages (PA_KV_FP4_E2M1).
//
//   S^T[keys, heads] = K q^T,  P = softmax,  O^T[dims, heads] = V^T P^T
//
// 0.5625 byte per cached element, so at the copy rate of the memory one SM
// has about 100 cycles for 16 keys (K and V, D = 128): 4096 elements to turn
// into fp16.  That conversion, not the products, is what the kernel is built
// around.  It runs in registers, straight into the fragments of
// mma.m16n8k16: measured per SM and cycle, 2 warp-wide e2m1x2 -> f16x2
// conversions, byte permutes or other integer operations in all, 2 f16x2
// products and half an MMA.  Converting into shared memory for tcgen05 instead
// would write and read back 2 bytes per element, 4 times what the page itself
// takes, through a port of 128 bytes per cycle.
//
// Keys are the M dimension of S^T and dims that of O^T, so a page element is
// always an A operand (256 elements per MMA, where it would be 128 as a B
// operand), and query heads fill N = 8.  The order of the dims within a
// product and of the keys within a 16-key block is free, and chosen so that a
// lane's share is contiguous:
//   K   lane (g, t) of row g takes dims [t D/4, (t + 1) D/4): one or two
//       scale blocks, one load per row;
//   V   lane (g, t) takes dims [g D/8, (g + 1) D/8) of 4 keys: inside one
//       scale block, one load per key.
// A byte of V holds two dims of one key, where an A operand wants two keys of
// one dim side by side.  Past 4 heads the words of two keys trade nibbles
// before the conversion (a shift and a select per 4 bytes).  Up to 4 heads,
// whose columns fill half of N, the contraction runs over (key, parity of the
// dim) instead, with one column of P^T per head for each parity, zero at the
// other: no trade, half the softmax (a lane holds one head) and half the
// output registers.  For 8 heads that costs 8 more MMAs per 16 keys and
// measured slower (57 sequences of 8192 keys: 98 us a call against 92).
//
// Measured: 57 sequences of 8192 keys, 8 KV heads, D = 128 (539 MB), 85 us a
// call with 4 query heads per KV head (6.3 TB/s, near the memory's rate), 87 with
// 8 (issue slots: 250 instructions per 16 keys, 12 warps an SM), 162 with 16
// (twice the MMAs, 8 warps an SM; 138 in two splits each, where the plan has 456
// whole sequences for 304 CTAs).  Shorter batches also see an item's ends (about 2.5 us), 3 us until
// the first pages are asked for, and 2 to 3 us of the merge kernel: 64 sequences
// of up to 4096 keys 37 us a call, where the bytes alone take 23.
//
// code * scale is exact in fp16, so nothing is lost before the fp32
// accumulators; P is rounded to fp16 -- relative 2^-11, and 2^-32 of the
// largest weight where that leaves fp16's normal range -- and q, scaled by a
// power of two per head, is exact but for elements 2^14 below its largest.
//
// Each warp streams its own pages (every fourth of the item's) through its
// own ring of whole-slab bulk copies and keeps its own running maximum, sum
// and output, so warps meet only at the end of an item, where the four
// results are merged through the warps' last page buffers.  Splits of one
// sequence are merged by a second, small kernel.  Every wait is bounded.
#include <cstdint>

#include "fp4.cuh"
#include "pa_step.h"
#include "pa_launch.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kItems = 64;  // items of a CTA decoded once, in the prologue
constexpr float kLn2 = 0.69314718055994531f;
// The running maximum is only raised when a logit (in bits) exceeds it by more
// than this, and most steps rescale nothing.  It is kept as a product q k, not as
// a logit: the difference of two products is exact where it matters, however large
// the logits are, and so P never passes 2^(kShift + kSlack) = 2^15.
constexpr float kSlack = 8.f;
// P and its sum are 2^kShift times the weights beside the running maximum, which
// fp16 has room for: of thousands of keys far below one, none is lost that is more
// than 2^-32 of it (2^-25 with no shift).
constexpr float kShift = 7.f;
constexpr float kNone = -3e38f;  // the running maximum before any key: finite, so that its differences are
constexpr float kLeastScale = 1e-37f;  // of a logit in bits to its product: kNone still lies below every logit

// D: head dim; NH: query heads of a KV group the kernel has room for (4, 8 or 16)
template <int D, int NH>
struct Layout {
    static constexpr int kSlab = fp4_slab_bytes(D);
    static constexpr int kStage = 2 * kSlab;  // K slab, V slab
    // CTAs of an SM.  Past 8 heads two with up to 255 registers a thread: three
    // spill (64 sequences of up to 8192 keys, 16 heads a group: 114 us a call, 98
    // with two).
    static constexpr int kCtas = fp4_ctas_per_sm(NH);
    static constexpr int kStages = (NH == 16 ? 3 : 2) * (D == 128 ? 1 : 2);
    static constexpr int kRing = kStages * kStage;  // of one warp
    static constexpr int kBytes = kWarps * kRing;
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

// the same with C = 0
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// a times the low or the high half of s (the product takes a broadcast half as it is)
template <bool kHigh>
__device__ __forceinline__ uint32_t mul2_by(uint32_t a, uint32_t s) {
    const __half2 x = *reinterpret_cast<const __half2*>(&a), y = *reinterpret_cast<const __half2*>(&s);
    const __half2 r = __hmul2(x, kHigh ? __high2half2(y) : __low2half2(y));
    return *reinterpret_cast<const uint32_t*>(&r);
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

// D: head dim; NH: query heads of a KV group it has room for (4, 8 or 16)
template <int D, int NH>
__global__ void __launch_bounds__(kThreads, Layout<D, NH>::kCtas) decode_fp4_kernel(const __grid_constant__ DecodeArgs a) {
    using L = Layout<D, NH>;
    constexpr int S = L::kStages;
    constexpr int KB = kPage / 16;                   // 16-key blocks of a page
    constexpr int KK = D / 16;                       // MMA steps over the dims of QK
    constexpr int NQ = NH == 16 ? 2 : 1;             // column tiles of S^T and O^T
    constexpr int MT = NH == 4 ? D / 32 : D / 16;    // row tiles of O^T
    constexpr int HL = NH / 4;                       // heads whose logits a lane holds
    constexpr int M4 = D / 32;                       // groups of 4 dims of a lane's output
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kWarps][S];
    __shared__ Item items_sh[kItems];
    __shared__ float red_m[kWarps][NH], red_l[kWarps][NH], red_scale[NH];  // the last one every warp's
    __shared__ int scratch_at[kWarps];  // the page buffer that holds each warp's output
    __shared__ int abort_store;
    volatile int* abort_sh = &abort_store;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, G = a.group;
    uint8_t* ring = smem + warp * L::kRing;
    uint64_t* bar = full[warp];
    if (lane < S) mbar_init(&bar[lane], 1);
    if (threadIdx.x == 0) abort_store = 0;
    fence_barrier_init();
    grid_dependency_wait();  // shared memory only up to here
    // The merge kernel may become resident as this one's CTAs leave.  Nothing
    // else may: a later decode let in early is dealt to the SMs in the order
    // they empty, which undoes the schedule's balance (64 sequences, no
    // splits: 53 us a call against 43).
    if (a.counters) allow_dependents_launch();

    const int32_t* indptr = a.meta + kMetaHeader + 2 * a.batch + 1;
    const int grid = __ldg(&a.meta[5]);  // at most gridDim.x
    int it_lo = __ldg(&indptr[blockIdx.x]), it_hi = __ldg(&indptr[blockIdx.x + 1]);
    if ((int)blockIdx.x >= grid) it_lo = it_hi = 0;
    const int items_off = kMetaHeader + 2 * a.batch + 1 + grid + 1;
    for (int i = threadIdx.x; i < min(it_hi - it_lo, kItems); i += kThreads) items_sh[i] = load_item(a, it_lo + i, items_off);
    __syncthreads();
    auto get_item = [&](int j) { return j - it_lo < kItems ? items_sh[j - it_lo] : load_item(a, j, items_off); };

    // Queries are read once and so come from memory: the first item's are asked for before the pages, behind which they
    // would wait (4 us of a call), the next one's while the warps merge.
    uint32_t raw[NQ][D / 8];  // as they lie in memory: the head of column g, dims of t
    auto load_q = [&](int j) {
        const Item it = get_item(j);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int h = NH == 4 ? g >> 1 : n * 8 + g;
            const uint4* src = reinterpret_cast<const uint4*>(
                a.q + ((long long)it.b * a.num_q_heads + it.kvh * G + h) * D + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 v = h < G ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                raw[n][4 * i] = v.x; raw[n][4 * i + 1] = v.y; raw[n][4 * i + 2] = v.z; raw[n][4 * i + 3] = v.w;
            }
        }
    };
    if (it_lo < it_hi) load_q(it_lo);

    // ---- filling the ring: a cursor over this warp's pages of all items
    int pj = it_lo - 1, pp = 0, pend = 0, pkvh = 0;
    int ids = 0, id_base = 0;     // ids of the warp's next 32 pages of item pj, one per lane
    int next_ids = 0;             // and of its first 32 of item pj + 1, on their way
    uint32_t fill_st = 0, dead = 0;  // next stage to fill; stages whose page id was out of range
    int in_ring = 0;
    auto first_ids = [&](int j) {
        if (j >= it_hi) return 0;
        const Item it = get_item(j);
        const int i = it.p0 + warp + kWarps * lane;
        return i < it.p1 ? __ldg(&a.block_table[(long long)it.b * a.max_pages + i]) : 0;
    };
    next_ids = first_ids(it_lo);
    auto fill = [&]() {  // the warp's next page into stage fill_st, which is free
        while (pp >= pend) {
            if (pj + 1 >= it_hi) return;
            const Item it = get_item(++pj);
            pp = id_base = it.p0 + warp;
            pend = it.p1;
            pkvh = it.kvh;
            ids = next_ids;
            next_ids = first_ids(pj + 1);
        }
        if (pp - id_base >= 32 * kWarps) {
            const Item it = get_item(pj);
            id_base = pp;
            const int i = pp + kWarps * lane;
            ids = i < pend ? __ldg(&a.block_table[(long long)it.b * a.max_pages + i]) : 0;
        }
        const int id = __shfl_sync(0xffffffffu, ids, (pp - id_base) / kWarps);
        const bool ok = (unsigned)id < (unsigned)a.num_pool_pages;
        dead = ok ? dead & ~(1u << fill_st) : dead | (1u << fill_st);
        if (lane == 0) {
            uint8_t* dst = ring + fill_st * L::kStage;
            if (ok) {
                const long long off = ((long long)id * a.num_kv_heads + pkvh) * L::kSlab;
                mbar_arrive_expect_tx(&bar[fill_st], 2 * L::kSlab);
                bulk_load(dst, a.k_pool + off, L::kSlab, &bar[fill_st]);
                bulk_load(dst + L::kSlab, a.v_pool + off, L::kSlab, &bar[fill_st]);
            } else {
                record(a.status, PA_ERR_DEVICE_BOUNDS);
                mbar_arrive(&bar[fill_st]);
            }
        }
        if (++fill_st == S) fill_st = 0;
        ++in_ring;
        pp += kWarps;
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) fill();

    // this lane's places in a slab, for the first 16-key block: K row, V keys
    const int krow = key_row(g), vkey0 = key_row(2 * t), vkey1 = key_row(2 * t + 1);
    const uint8_t* kbase = ring + krow * (D / 2) + t * (D / 8);
    const uint8_t* kscale = ring + kPage * (D / 2) + krow * (D / 16) + (D == 128 ? 2 * t : t);
    const uint8_t* vslab = ring + L::kSlab;
    // halves of a P pair (keys 2t, 2t + 1) with a zero beside them
    const uint32_t sel0 = g & 1 ? 0x1044u : 0x4410u, sel1 = g & 1 ? 0x3244u : 0x4432u;

    uint32_t st = 0, phase = 0;  // next stage to take
    bool bad = false;
    for (int j = it_lo; j < it_hi; ++j) {
        const Item it = get_item(j);
        const int key_end = min(it.seq_len, it.p1 * kPage);
        const float k_scale = __ldg(&a.k_scale[it.kvh]), vs = __ldg(&a.v_scale[it.kvh]);
        // logits in bits are products times |bits|: its sign goes into q, so that maxima can be taken of the products
        const float bits = fabsf(a.scale_log2 * k_scale);
        const uint32_t sign = __float_as_uint(a.scale_log2 * k_scale) & 0x80000000u;
        uint32_t q[NQ][2 * KK];  // B fragments
        float sl2[HL], o[NQ][MT][4], m[HL], l[HL];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[n][i] << 16)), fabsf(__uint_as_float(raw[n][i] & 0xFFFF0000u))));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^e <= amax < 2^(e+1), kept where both 2^e and 2^-e are ordinary floats
            const int e = amax > 0.f && amax < INFINITY ? min(max((int)(__float_as_uint(amax) >> 23) - 127, -96), 96) : 0;
            const float down = __uint_as_float(((uint32_t)(127 - e) << 23) | sign), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                q[n][i] = pack_half2(__uint_as_float(raw[n][i] << 16) * down, __uint_as_float(raw[n][i] & 0xFFFF0000u) * down);
            // the power of two of each head whose logits this lane holds
            if constexpr (NH == 4) {
                sl2[0] = bits * __shfl_sync(0xffffffffu, up, 8 * t);
            } else {
                sl2[2 * n] = bits * __shfl_sync(0xffffffffu, up, 8 * t);
                sl2[2 * n + 1] = bits * __shfl_sync(0xffffffffu, up, 8 * t + 4);
            }
        }
#pragma unroll
        for (int i = 0; i < HL; ++i) {
            if (sl2[i] < kLeastScale) sl2[i] = kLeastScale;
            m[i] = kNone;
            l[i] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][i][k] = 0.f;

        bool owed = false;  // the last page's buffer is refilled after the merge
        uint32_t last = 0;
        for (int p = it.p0 + warp; p < it.p1; p += kWarps) {
            if (!__all_sync(0xffffffffu, mbar_wait(&bar[st], phase, abort_sh, a.wait_ns))) {
                bad = true;
                break;
            }
            --in_ring;
            const uint32_t so = st * L::kStage;
            const int live = (dead >> st) & 1u ? 0 : key_end - p * kPage;  // live keys (64 or more: all)
            if (live > 0) {
                // ---- S^T = K q^T
                float c[NQ][KB][4];
#pragma unroll
                for (int blk = 0; blk < KB; ++blk) {
                    uint32_t w[2][D / 32], sc[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint8_t* src = kbase + so + (blk * 16 + 8 * i) * (D / 2);
                        const uint8_t* scl = kscale + so + (blk * 16 + 8 * i) * (D / 16);
                        if constexpr (D == 128) {
                            const uint4 v = *reinterpret_cast<const uint4*>(src);
                            w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
                            sc[i] = e4m3x2_to_half2(*reinterpret_cast<const uint16_t*>(scl));
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(src);
                            w[i][0] = v.x; w[i][1] = v.y;
                            sc[i] = e4m3x2_to_half2(*scl);
                        }
                    }
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const int wi = kk / 2, byte = (kk & 1) * 2;
                        auto scaled = [&](int row, int at) {  // words 2, 3 are of the second scale block
                            return wi < 2 ? mul2_by<false>(code_pair(w[row][wi], at), sc[row])
                                          : mul2_by<true>(code_pair(w[row][wi], at), sc[row]);
                        };
                        const uint32_t a0 = scaled(0, byte), a1 = scaled(1, byte);
                        const uint32_t a2 = scaled(0, byte + 1), a3 = scaled(1, byte + 1);
#pragma unroll
                        for (int n = 0; n < NQ; ++n) {
                            if (kk == 0) mma16816_first(c[n][blk], a0, a1, a2, a3, q[n][0], q[n][1]);
                            else mma16816(c[n][blk], a0, a1, a2, a3, q[n][2 * kk], q[n][2 * kk + 1]);
                        }
                    }
                }
                // products x[i][2 blk + r] of head slot i, row 16 blk + 8 r + g
                float x[HL][2 * KB];
#pragma unroll
                for (int i = 0; i < HL; ++i)
#pragma unroll
                    for (int k = 0; k < 2 * KB; ++k) x[i][k] = c[i >> 1][k >> 1][2 * (k & 1) + (NH == 4 ? 0 : i & 1)];
                const bool tail = live < kPage;
                if (tail) {
#pragma unroll
                    for (int k = 0; k < 2 * KB; ++k)
                        if (8 * k + krow >= live) {
#pragma unroll
                            for (int i = 0; i < HL; ++i) x[i][k] = -INFINITY;
                        }
                }
                // ---- running softmax: lanes share a maximum only when one of them finds it too low
                bool raise = false;
                float top[HL];
#pragma unroll
                for (int i = 0; i < HL; ++i) {
                    top[i] = x[i][0];
#pragma unroll
                    for (int k = 1; k < 2 * KB; ++k) top[i] = fmaxf(top[i], x[i][k]);
                    raise |= (top[i] - m[i]) * sl2[i] > kSlack;
                }
                if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                    for (int i = 0; i < HL; ++i) {
                        float v = top[i];
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        const float mn = fmaxf(m[i], v);
                        const float alpha = ex2((m[i] - mn) * sl2[i]);
                        m[i] = mn;
                        l[i] *= alpha;
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int k = 0; k < MT; ++k)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (NH == 4 || (n == i >> 1 && (e & 1) == (i & 1))) o[n][k][e] *= alpha;
                    }
                }
                if constexpr (HL == 1) {
#pragma unroll
                    for (int k = 0; k < 2 * KB; ++k) x[0][k] = ex2(fmaf(x[0][k] - m[0], sl2[0], kShift));
                } else {  // two heads at a time, as the products lie
#pragma unroll
                    for (int i = 0; i < HL; i += 2) {
                        const F2 from = f2(-m[i], -m[i + 1]), by = f2(sl2[i], sl2[i + 1]), shift = f2(kShift, kShift);
#pragma unroll
                        for (int k = 0; k < 2 * KB; ++k) {
                            const float2 e = split(fma2(f2(x[i][k], x[i + 1][k]) + from, by, shift));
                            x[i][k] = ex2(e.x);
                            x[i + 1][k] = ex2(e.y);
                        }
                    }
                }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int blk = 0; blk < KB; ++blk) {
#pragma unroll
                    for (int i = 0; i < HL; ++i) l[i] += x[i][2 * blk] + x[i][2 * blk + 1];
                    uint32_t w[4][D / 64], b[4];  // keys vkey0, vkey1, vkey0 + 8, vkey1 + 8 of the block
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = (i & 1 ? vkey1 : vkey0) + 8 * (i >> 1) + 16 * blk;
                        if constexpr (D == 128) {
                            const uint2 v = *reinterpret_cast<const uint2*>(vslab + so + key * 64 + g * 8);
                            w[i][0] = v.x;
                            w[i][1] = v.y;
                            b[i] = vslab[so + kPage * 64 + key * 8 + g];
                        } else {
                            w[i][0] = *reinterpret_cast<const uint32_t*>(vslab + so + key * 32 + g * 4);
                            b[i] = vslab[so + kPage * 32 + key * 4 + (g >> 1)];
                        }
                    }
                    if (tail) {  // a dead key's scale may be a NaN, which a zero P would not cancel
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if ((i & 1 ? vkey1 : vkey0) + 8 * (i >> 1) + 16 * blk >= live) b[i] = 0;
                    }
                    const uint32_t s01 = e4m3x2_to_half2(b[0] | (b[1] << 8)), s23 = e4m3x2_to_half2(b[2] | (b[3] << 8));
                    if constexpr (NH == 4) {
                        // 8 keys at a time: A = (key, parity of the dim), B = P at one parity
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int k = 2 * blk + hf;
                            const uint32_t y = transpose8x8(pack_half2(x[0][k], x[0][k]));
                            const uint32_t p0 = __byte_perm(y, 0, sel0), p1 = __byte_perm(y, 0, sel1);
                            const uint32_t sh = hf ? s23 : s01;
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                const uint32_t wa = w[2 * hf][mt / 2], wb = w[2 * hf + 1][mt / 2];
                                const int byte = (mt & 1) * 2;
                                const uint32_t a0 = mul2_by<false>(code_pair(wa, byte), sh);
                                const uint32_t a1 = mul2_by<false>(code_pair(wa, byte + 1), sh);
                                const uint32_t a2 = mul2_by<true>(code_pair(wb, byte), sh);
                                const uint32_t a3 = mul2_by<true>(code_pair(wb, byte + 1), sh);
                                mma16816(o[0][mt], a0, a1, a2, a3, p0, p1);
                            }
                        }
                    } else {
                        // codes of one dim of two keys side by side: even and odd dims of a pair of keys' words
                        uint32_t even[2][D / 64], odd[2][D / 64];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int k = 0; k < D / 64; ++k) {
                                const uint32_t wa = w[2 * i][k], wb = w[2 * i + 1][k];
                                even[i][k] = (wa & 0x0F0F0F0Fu) | ((wb << 4) & 0xF0F0F0F0u);
                                odd[i][k] = ((wa >> 4) & 0x0F0F0F0Fu) | (wb & 0xF0F0F0F0u);
                            }
                        uint32_t pb[NQ][2];
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                pb[n][r] = transpose8x8(pack_half2(x[2 * n][2 * blk + r], x[(2 * n + 1) % HL][2 * blk + r]));
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const uint32_t a0 = mul2(code_pair(even[0][mt / 4], mt & 3), s01);
                            const uint32_t a1 = mul2(code_pair(odd[0][mt / 4], mt & 3), s01);
                            const uint32_t a2 = mul2(code_pair(even[1][mt / 4], mt & 3), s23);
                            const uint32_t a3 = mul2(code_pair(odd[1][mt / 4], mt & 3), s23);
#pragma unroll
                            for (int n = 0; n < NQ; ++n) mma16816(o[n][mt], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                        }
                    }
                }
            }
            __syncwarp();  // every lane is done with the stage
            if (p + kWarps < it.p1) fill();
            else {
                owed = true;
                last = so;
            }
            if (++st == S) {
                st = 0;
                phase ^= 1;
            }
        }
        if (j + 1 < it_hi) load_q(j + 1);  // lands while the warps merge

        // ---- merge the four warps: [head][dim] in each one's last page buffer, a lane's groups of 4 dims rotated by
        // its t, so that no two lanes of a store meet in a bank
#pragma unroll
        for (int i = 0; i < HL; ++i) {
            const int h = NH == 4 ? t : 8 * (i >> 1) + 2 * t + (i & 1);
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
            if (g == 0) {
                red_m[warp][h] = m[i];
                red_l[warp][h] = l[i];
                red_scale[h] = sl2[i];
            }
            if (owed && h < G) {
#pragma unroll
                for (int k = 0; k < M4; ++k) {
                    float4 v;
                    if constexpr (NH == 4) v = make_float4(o[0][k][0], o[0][k][1], o[0][k][2], o[0][k][3]);
                    else
                        v = make_float4(o[i >> 1][2 * k % MT][i & 1], o[i >> 1][2 * k % MT][2 + (i & 1)],
                                        o[i >> 1][(2 * k + 1) % MT][i & 1], o[i >> 1][(2 * k + 1) % MT][2 + (i & 1)]);
                    *reinterpret_cast<float4*>(ring + last + (h * D + g * (D / 8) + 4 * ((k + t) & (M4 - 1))) * 4) = v;
                }
            }
        }
        if (lane == 0) scratch_at[warp] = (int)(ring - smem) + (int)last;
        if (__syncthreads_or(bad || *abort_sh != 0)) {
            bad = true;
            break;
        }
        const bool partial = it.nsplit > 1;
        const long long head0 = (long long)it.kvh * G;
        const long long orow = partial ? (long long)(it.split_base + it.s) * a.num_q_heads + head0
                                       : (long long)it.b * a.num_q_heads + head0;
        const float* from[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) from[w] = reinterpret_cast<const float*>(smem + scratch_at[w]);
#pragma unroll
        for (int i = 0; i < (NH * D / 4 + kThreads - 1) / kThreads; ++i) {  // 4 dims of a head per thread
            const int idx = threadIdx.x + i * kThreads;
            if (idx >= G * (D / 4)) break;
            const int h = idx / (D / 4), d = idx % (D / 4) * 4;
            const int ht = NH == 4 ? h : (h >> 1) & 3;  // the t of the lanes that held head h
            const int slot = h * D + d / (D / 8) * (D / 8) + 4 * ((d % (D / 8) / 4 + ht) & (M4 - 1));
            const float bits_of = red_scale[h];
            float mw[kWarps], lw[kWarps], mm = kNone, ll = 0.f;
            float4 v[kWarps], val = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                mw[w] = red_m[w][h];
                lw[w] = red_l[w][h];
                v[w] = *reinterpret_cast<const float4*>(from[w] + slot);
                mm = fmaxf(mm, mw[w]);
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const bool any = lw[w] != 0.f;                // else no live key, and the buffer holds anything;
                const float f = any ? ex2((mw[w] - mm) * bits_of) : 0.f;  // a NaN logit leaves a NaN sum, and so a NaN output
                ll = fmaf(f, lw[w], ll);
                val.x = fmaf(f, any ? v[w].x : 0.f, val.x);
                val.y = fmaf(f, any ? v[w].y : 0.f, val.y);
                val.z = fmaf(f, any ? v[w].z : 0.f, val.z);
                val.w = fmaf(f, any ? v[w].w : 0.f, val.w);
            }
            const float r = ll == 0.f ? 0.f : __fdividef(vs, ll);
            val = make_float4(val.x * r, val.y * r, val.z * r, val.w * r);
            if (partial) {
                *reinterpret_cast<float4*>(a.o_part + (orow + h) * D + d) = val;
            } else {
                *reinterpret_cast<uint2*>(a.out + (orow + h) * D + d) =
                    make_uint2((uint32_t)to_bf16(val.x) | ((uint32_t)to_bf16(val.y) << 16),
                               (uint32_t)to_bf16(val.z) | ((uint32_t)to_bf16(val.w) << 16));
            }
            if (d == 0) {
                const float lse = ll == 0.f ? -INFINITY : fmaf(mm, bits_of, log2f(ll) - kShift) * kLn2;
                if (partial) a.lse_part[orow + h] = lse;
                else if (a.lse) a.lse[orow + h] = lse;
            }
        }
        fence_proxy_async_smem();  // the buffers go back to the async copies
        __syncthreads();
        if (owed) fill();
    }
    if (bad && lane == 0) {
        *abort_sh = 1;
        record(a.status, PA_ERR_TIMEOUT);
        // every copy must land before the CTA may exit
        for (; in_ring > 0; --in_ring) {
            mbar_wait(&bar[st], phase, nullptr, a.wait_ns);
            if (++st == S) {
                st = 0;
                phase ^= 1;
            }
        }
    }
}

// Merges the splits of every sequence that has more than one:
//   lse = m + ln sum_s exp(lse_s - m),  out = sum_s exp(lse_s - lse) o_s
// A kernel of its own: merged by the last CTA to finish a split instead, the
// wait for the partials and two rounds of dependent loads fell into that CTA's
// stream of pages (64 sequences of up to 4096 keys: 70.7 us a call, 51.1 with
// the merge moved here).
//
// A CTA has kMergeWarps rows (sequence, query head), or one where that leaves
// SMs empty.  A warp takes a row of its own if it has up to kTogether splits,
// whose loads are then in flight together; the CTA's warps share those of a row
// that has more, or is alone, every kMergeWarps-th each.  The order of the sums
// depends on the number of splits and of rows only.  One sequence of 131072 keys
// in 57 splits, 32 heads: 4 us of a 33 us call, 12 of 41 with a warp a row.
constexpr int kMergeWarps = 4, kTogether = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) combine_fp4_kernel(const __grid_constant__ DecodeArgs a, int rows) {
    constexpr int E = D / 32;  // elements of a lane
    __shared__ float part[kMergeWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long all = (long long)a.batch * a.num_q_heads, row0 = (long long)blockIdx.x * rows;
    int splits = 0;  // lane r: of the CTA's row r
    long long base = 0;
    if (lane < rows && row0 + lane < all) {
        const int b = (int)((row0 + lane) / a.num_q_heads), h = (int)(row0 + lane - (long long)b * a.num_q_heads);
        splits = __ldg(&a.meta[kMetaHeader + b]);
        base = (long long)__ldg(&a.meta[kMetaHeader + a.batch + b]) * a.num_q_heads + h;
    }
    // Let in by the attention kernel: the metadata was complete before that one
    // did so, its partials are now.  Every warp waits, also one with nothing to
    // do: this kernel must not be complete before that one.  (Launched plainly:
    // everything before it was complete.)
    grid_dependency_wait();
    for (int r = 0; r < rows; ++r) {
        const int n = __shfl_sync(0xffffffffu, splits, r);
        const bool alone = rows > 1 && n <= kTogether;  // of a warp: its own row
        if (n <= 1 || (alone && r != warp)) continue;
        const long long at = __shfl_sync(0xffffffffu, base, r);
        const int s0 = alone ? 0 : warp, step = alone ? 1 : kMergeWarps;
        // lanes hold the splits' log-sum-exps (at most PA_MAX_SPLITS = 64)
        const float l0 = lane < n ? a.lse_part[at + (long long)lane * a.num_q_heads] : -INFINITY;
        const float l1 = lane + 32 < n ? a.lse_part[at + (long long)(lane + 32) * a.num_q_heads] : -INFINITY;
        float acc[E] = {}, o[kTogether][E];
        auto load = [&](int first) {
#pragma unroll
            for (int i = 0; i < kTogether; ++i) {
                const int s = first + i * step;
                if (s < n) {
                    const float* src = a.o_part + (at + (long long)s * a.num_q_heads) * D + lane * E;
                    if constexpr (D == 128) *reinterpret_cast<float4*>(o[i]) = *reinterpret_cast<const float4*>(src);
                    else *reinterpret_cast<float2*>(o[i]) = *reinterpret_cast<const float2*>(src);
                }
            }
        };
        load(s0);
        float mm = fmaxf(l0, l1);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
        // a split without keys weighs nothing; a NaN stays one
        const float w0 = l0 == -INFINITY ? 0.f : __expf(l0 - mm), w1 = l1 == -INFINITY ? 0.f : __expf(l1 - mm);
        float sum = w0 + w1;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        for (int first = s0;;) {
#pragma unroll
            for (int i = 0; i < kTogether; ++i) {
                const int s = first + i * step;
                const float ws = __shfl_sync(0xffffffffu, s < 32 ? w0 : w1, s & 31);
                if (s < n) {
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(ws, o[i][e], acc[e]);
                }
            }
            first += kTogether * step;
            if (first >= n) break;
            load(first);
        }
        if (!alone) {
            if (r > 0) __syncthreads();  // the row before is written
#pragma unroll
            for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
            __syncthreads();
            if (warp != 0) continue;
#pragma unroll
            for (int w = 1; w < kMergeWarps; ++w)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += part[w][lane * E + e];
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const long long row = row0 + r;
        uint32_t* out = reinterpret_cast<uint32_t*>(a.out + row * D + lane * E);
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            out[i] = (uint32_t)to_bf16(acc[2 * i] * inv) | ((uint32_t)to_bf16(acc[2 * i + 1] * inv) << 16);
        if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : mm + __logf(sum);
    }
}

template <int D, int NH>
cudaError_t launch_d(const DecodeArgs& a, int grid, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = ensure_dynamic_smem(decode_fp4_kernel<D, NH>, Layout<D, NH>::kBytes, done);
    if (e != cudaSuccess) return e;
    return launch_overlapped(decode_fp4_kernel<D, NH>, dim3((unsigned)grid), dim3(kThreads), Layout<D, NH>::kBytes, stream, a);
}

template <int D>
cudaError_t launch_heads(const DecodeArgs& a, int grid, cudaStream_t stream) {
    return a.group <= 4 ? launch_d<D, 4>(a, grid, stream) : a.group <= 8 ? launch_d<D, 8>(a, grid, stream)
                                                                         : launch_d<D, 16>(a, grid, stream);
}

}  // namespace

cudaError_t launch_decode_fp4(int head_dim, const DecodeArgs& a, int grid, cudaStream_t stream) {
    return head_dim == 128 ? launch_heads<128>(a, grid, stream) : launch_heads<64>(a, grid, stream);
}

cudaError_t launch_combine_fp4(int head_dim, const DecodeArgs& a, bool behind_attention, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t all = (int64_t)a.batch * a.num_q_heads;
    const int rows = all <= 8 * (int64_t)sms ? 1 : kMergeWarps;
    const dim3 grid((unsigned)((all + rows - 1) / rows)), block(kMergeWarps * 32);
    if (behind_attention)
        return head_dim == 128 ? launch_overlapped(combine_fp4_kernel<128>, grid, block, 0, stream, a, rows)
                               : launch_overlapped(combine_fp4_kernel<64>, grid, block, 0, stream, a, rows);
    if (head_dim == 128) combine_fp4_kernel<128><<<grid, block, 0, stream>>>(a, rows);
    else combine_fp4_kernel<64><<<grid, block, 0, stream>>>(a, rows);
    return cudaGetLastError();
}

}  // namespace pa
