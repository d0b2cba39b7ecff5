// cache4.cu -- writing 4-bit pages (pa_append_kv with PA_KV_FP4_E2M1) and
// reading the rows of pages of any type back (pa_gather_kv).
//
// Both are copies with a conversion, so HBM-bound: 2 bytes of a 16-bit row
// against 0.5625 (4-bit), 1 (e4m3) or 2 bytes of a page row per element.  A
// thread owns one 16-element piece of a row -- the block of the 4-bit type, so
// neither its largest magnitude nor its scale crosses threads.  A warp takes
// 32 / (D / 16) consecutive tokens, whose rows are neighbours in a page, of up
// to kHeads heads: what it touches of a slab is contiguous (at D = 128, 256
// bytes of codes and one 32-byte sector of scales), and the search for the
// tokens' sequence and page is paid once for all heads.  All loads of a batch
// of heads are issued before any store.
//
// Measured: 4-bit rows of 262k tokens, 8 heads of 128, read back in 238 us
// (1.59 GB, 6.7 TB/s, the memory's copy rate); 4096 tokens written and 37k
// read back, two launches, 38.7 us (215 MB); 64 written and 64 read back 6.0 us.
// Written alone, 32768 tokens of 8 heads take 32.2 us (172 MB, 5.3 TB/s).
#include "cache4.cuh"
#include "pa_launch.h"
#include "token_place.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
// Heads of a warp.  Writing has work to do between its loads and its stores, and wants more warps: 32768 tokens of 8
// heads 32.3 us with 2, 37.2 with 4, 34.4 with 1; 512 tokens 3.3, 4.4, 2.9.  Reading back: 29.1 with 4, as with 2 and 1,
// 262k rows 237.4, 238.3, 241.0.
constexpr int kAppendHeads = 2, kGatherHeads = 4;

// This thread's token and the first of its warp's heads.
// grid: x = groups of tokens, kWarps to a CTA; y = groups of kHeads heads
template <int D, int kHeads>
struct Share {
    static constexpr int kLanes = D / 16, kTokens = 32 / kLanes;
    int tok0, tok, piece, h0;  // tok0: the warp's first token
    __device__ __forceinline__ Share()
        : tok0((int)(blockIdx.x * kWarps + (threadIdx.x >> 5)) * kTokens),
          tok(tok0 + (int)(threadIdx.x & 31) / kLanes),
          piece((int)(threadIdx.x & 31) % kLanes),
          h0((int)blockIdx.y * kHeads) {}
    // that of this thread's token; the whole warp calls it
    __device__ __forceinline__ Sequence sequence(const int32_t* __restrict__ cu, const int32_t* __restrict__ start_pos,
                                                 int batch) const {
        return warp_sequences<kTokens>(tok0, tok - tok0, cu, start_pos, batch);
    }
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) append_fp4_kernel(const __grid_constant__ AppendArgs a) {
    grid_dependency_wait();
    allow_dependents_launch();
    constexpr int kHeads = kAppendHeads;
    const Share<D, kHeads> my;
    if (my.tok0 >= a.total_new) return;
    const int nh = min(kHeads, a.num_kv_heads - my.h0);
    // rows first: they do not depend on the token's place
    const bool wide = aligned32(a.k_new) && aligned32(a.v_new);
    Sector w[kHeads][2];
    const long long src = ((long long)my.tok * a.num_kv_heads + my.h0) * D + my.piece * 16;
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < nh && my.tok < a.total_new) {
            w[i][0] = load_sector(a.k_new + src + i * D, wide);
            w[i][1] = load_sector(a.v_new + src + i * D, wide);
        }
    const Sequence seq = my.sequence(a.cu_new, a.start_pos, a.batch);
    if (my.tok >= a.total_new) return;
    int page, row;
    long long pos;
    const Place at = token_place(my.tok, seq, a.block_table, a.batch, a.max_pages, a.num_pool_pages, page, row, pos);
    if (at != Place::kOk) {
        if (my.piece == 0 && at == Place::kOutOfRange) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
        return;
    }
    const long long slab = ((long long)page * a.num_kv_heads + my.h0) * fp4_slab_bytes(D);
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < nh) {
            const long long at_head = slab + (long long)i * fp4_slab_bytes(D);
            fp4_store_block<D>(static_cast<uint8_t*>(a.k_pool) + at_head, row, my.piece, w[i][0].lo, w[i][0].hi,
                               __ldg(&a.k_scale[my.h0 + i]));
            fp4_store_block<D>(static_cast<uint8_t*>(a.v_pool) + at_head, row, my.piece, w[i][1].lo, w[i][1].hi,
                               __ldg(&a.v_scale[my.h0 + i]));
        }
}

// 16 elements as they lie in a page, before conversion
template <int kType>
struct Piece {
    uint4 raw[kType == PA_KV_BF16 || kType == PA_KV_FP16 ? 2 : 1];  // 4-bit: codes in x, y; the scale byte in z
};

template <int D, int kType>
__device__ __forceinline__ Piece<kType> load_piece(const uint8_t* pool, long long slab_index, int row, int piece, bool wide) {
    Piece<kType> p;
    if constexpr (kType == PA_KV_FP4_E2M1) {
        const uint8_t* slab = pool + slab_index * fp4_slab_bytes(D);
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(slab + row * (D / 2)) + piece);
        p.raw[0] = make_uint4(c.x, c.y, __ldg(slab + kPage * (D / 2) + row * (D / 16) + piece), 0);
    } else if constexpr (kType == PA_KV_FP8_E4M3) {
        p.raw[0] = __ldg(reinterpret_cast<const uint4*>(pool + (slab_index * kPage + row) * D) + piece);
    } else {
        const Sector s = load_sector(pool + (slab_index * kPage + row) * (2 * D) + 32 * piece, wide);
        p.raw[0] = s.lo;
        p.raw[1] = s.hi;
    }
    return p;
}

// two fp16 values times `scale` in fp32, rounded once to bf16
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h2, float scale) {
    const __half2 h = *reinterpret_cast<const __half2*>(&h2);
    const __nv_bfloat162 b = __floats2bfloat162_rn(__low2float(h) * scale, __high2float(h) * scale);
    return *reinterpret_cast<const uint32_t*>(&b);
}

template <int kType>
__device__ __forceinline__ void store_piece(uint16_t* dst, const Piece<kType>& p, float head, bool wide) {
    uint4 out[2];
    if constexpr (kType == PA_KV_FP4_E2M1) {
        // block scale * head scale in fp32: a code has 2 significant bits, so
        // the product with it is within one fp32 rounding of the exact value
        const float s = e4m3_to_float(p.raw[0].z) * head;
        const uint32_t c[2] = {p.raw[0].x, p.raw[0].y};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            out[i] = make_uint4(scaled_bf16x2(e2m1x2_to_half2<0>(c[i]), s), scaled_bf16x2(e2m1x2_to_half2<1>(c[i]), s),
                                scaled_bf16x2(e2m1x2_to_half2<2>(c[i]), s), scaled_bf16x2(e2m1x2_to_half2<3>(c[i]), s));
    } else if constexpr (kType == PA_KV_FP8_E4M3) {
        const uint32_t c[4] = {p.raw[0].x, p.raw[0].y, p.raw[0].z, p.raw[0].w};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            out[i] = make_uint4(scaled_bf16x2(e4m3x2_to_half2(c[2 * i]), head),
                                scaled_bf16x2(e4m3x2_to_half2(c[2 * i] >> 16), head),
                                scaled_bf16x2(e4m3x2_to_half2(c[2 * i + 1]), head),
                                scaled_bf16x2(e4m3x2_to_half2(c[2 * i + 1] >> 16), head));
    } else {
        out[0] = p.raw[0];
        out[1] = p.raw[1];
    }
    store_sector(dst, Sector{out[0], out[1]}, wide);
}

// grid as for append_fp4_kernel
template <int D, int kType>
__global__ void __launch_bounds__(kWarps * 32) gather_kernel(const __grid_constant__ GatherArgs a) {
    grid_dependency_wait();
    allow_dependents_launch();
    constexpr int kHeads = kGatherHeads;
    const Share<D, kHeads> my;
    if (my.tok0 >= a.total) return;
    const Sequence seq = my.sequence(a.cu, a.start_pos, a.batch);
    if (my.tok >= a.total) return;
    int page, row;
    long long pos;
    const Place at = token_place(my.tok, seq, a.block_table, a.batch, a.max_pages, a.num_pool_pages, page, row, pos);
    if (at != Place::kOk) {
        if (my.piece == 0 && at == Place::kOutOfRange) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int nh = min(kHeads, a.num_kv_heads - my.h0);
    const long long slab = (long long)page * a.num_kv_heads + my.h0;
    const bool wide_in = aligned32(a.k_pool) && aligned32(a.v_pool), wide_out = aligned32(a.k_out) && aligned32(a.v_out);
    Piece<kType> k[kHeads], v[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < nh) {
            k[i] = load_piece<D, kType>(a.k_pool, slab + i, row, my.piece, wide_in);
            v[i] = load_piece<D, kType>(a.v_pool, slab + i, row, my.piece, wide_in);
        }
    const long long dst = ((long long)my.tok * a.num_kv_heads + my.h0) * D + my.piece * 16;
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < nh) {
            float ks = 1.f, vs = 1.f;
            if constexpr (kType == PA_KV_FP4_E2M1 || kType == PA_KV_FP8_E4M3) {
                ks = __ldg(&a.k_scale[my.h0 + i]);
                vs = __ldg(&a.v_scale[my.h0 + i]);
            }
            store_piece<kType>(a.k_out + dst + i * D, k[i], ks, wide_out);
            store_piece<kType>(a.v_out + dst + i * D, v[i], vs, wide_out);
        }
}

template <int D, int kHeads>
dim3 token_grid(int tokens, int heads) {
    constexpr int per_cta = kWarps * Share<D, kHeads>::kTokens;
    return dim3((unsigned)((tokens + per_cta - 1) / per_cta), (unsigned)((heads + kHeads - 1) / kHeads));
}

template <int D>
cudaError_t launch_gather_d(const GatherArgs& a, int kv_dtype, cudaStream_t stream) {
    const dim3 grid = token_grid<D, kGatherHeads>(a.total, a.num_kv_heads), block(kWarps * 32);
    switch (kv_dtype) {
        case PA_KV_FP4_E2M1: return launch_overlapped(gather_kernel<D, PA_KV_FP4_E2M1>, grid, block, 0, stream, a);
        case PA_KV_FP8_E4M3: return launch_overlapped(gather_kernel<D, PA_KV_FP8_E4M3>, grid, block, 0, stream, a);
        default: return launch_overlapped(gather_kernel<D, PA_KV_BF16>, grid, block, 0, stream, a);  // either 16-bit type
    }
}

}  // namespace

cudaError_t launch_append_fp4(const AppendArgs& a, cudaStream_t stream) {
    const dim3 block(kWarps * 32);
    return a.head_dim == 128
               ? launch_overlapped(append_fp4_kernel<128>, token_grid<128, kAppendHeads>(a.total_new, a.num_kv_heads), block, 0, stream, a)
               : launch_overlapped(append_fp4_kernel<64>, token_grid<64, kAppendHeads>(a.total_new, a.num_kv_heads), block, 0, stream, a);
}

cudaError_t launch_gather(const GatherArgs& a, int head_dim, int kv_dtype, cudaStream_t stream) {
    return head_dim == 128 ? launch_gather_d<128>(a, kv_dtype, stream) : launch_gather_d<64>(a, kv_dtype, stream);
}

}  // namespace pa
