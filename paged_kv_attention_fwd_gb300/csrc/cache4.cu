// cache4.cu -- writing 4-bit pages (pa_append_kv with PA_KV_FP4_E2M1) and
// reading the rows of pages of any type back (pa_gather_kv).
//
// Both are copies with a conversion, so HBM-bound: 2 bytes of a 16-bit row
// against 0.5625 (4-bit), 1 (e4m3) or 2 bytes of a page row per element.  A
// thread owns one 16-element piece -- the block of the 4-bit type, so neither
// its largest magnitude nor its scale crosses threads -- of the key row and
// of the value row of one head, and issues all its loads before any store.
#include "cache4.cuh"
#include "pa_launch.h"
#include "token_place.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;

// grid: x = tokens / kWarps (one warp each), y = groups of 32 / (D / 16) KV heads
template <int D>
__global__ void __launch_bounds__(kWarps * 32) append_fp4_kernel(const AppendArgs a) {
    allow_dependents_launch();
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
    const int tok = (int)(blockIdx.x * kWarps + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
    if (tok >= a.total_new) return;
    int page, row;
    long long pos;
    const Place at = token_place(tok, a.cu_new, a.start_pos, a.block_table, a.batch, a.max_pages, a.num_pool_pages,
                                 page, row, pos);
    if (at != Place::kOk) {
        if (lane == 0 && at == Place::kOutOfRange) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int h = (int)blockIdx.y * kHeads + lane / kLanes, piece = lane % kLanes;
    if (h >= a.num_kv_heads) return;
    const long long src = ((long long)tok * a.num_kv_heads + h) * D + piece * 16;
    const uint4* k = reinterpret_cast<const uint4*>(a.k_new + src);
    const uint4* v = reinterpret_cast<const uint4*>(a.v_new + src);
    const uint4 k0 = __ldg(k), k1 = __ldg(k + 1), v0 = __ldg(v), v1 = __ldg(v + 1);
    const float ks = __ldg(&a.k_scale[h]), vs = __ldg(&a.v_scale[h]);
    const long long slab = ((long long)page * a.num_kv_heads + h) * fp4_slab_bytes(D);
    fp4_store_block<D>(static_cast<uint8_t*>(a.k_pool) + slab, row, piece, k0, k1, ks);
    fp4_store_block<D>(static_cast<uint8_t*>(a.v_pool) + slab, row, piece, v0, v1, vs);
}

// 16 elements as they lie in a page, before conversion
template <int kType>
struct Piece {
    uint4 raw[kType == PA_KV_BF16 || kType == PA_KV_FP16 ? 2 : 1];  // 4-bit: codes in x, y; the scale byte in z
};

template <int D, int kType>
__device__ __forceinline__ Piece<kType> load_piece(const uint8_t* pool, long long slab_index, int row, int piece) {
    Piece<kType> p;
    if constexpr (kType == PA_KV_FP4_E2M1) {
        const uint8_t* slab = pool + slab_index * fp4_slab_bytes(D);
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(slab + row * (D / 2)) + piece);
        p.raw[0] = make_uint4(c.x, c.y, __ldg(slab + kPage * (D / 2) + row * (D / 16) + piece), 0);
    } else if constexpr (kType == PA_KV_FP8_E4M3) {
        p.raw[0] = __ldg(reinterpret_cast<const uint4*>(pool + (slab_index * kPage + row) * D) + piece);
    } else {
        const uint4* src = reinterpret_cast<const uint4*>(pool + (slab_index * kPage + row) * (2 * D)) + 2 * piece;
        p.raw[0] = __ldg(src);
        p.raw[1] = __ldg(src + 1);
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
__device__ __forceinline__ void store_piece(uint16_t* dst, const Piece<kType>& p, float head) {
    uint4* out = reinterpret_cast<uint4*>(dst);
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
}

// grid as for append_fp4_kernel
template <int D, int kType>
__global__ void __launch_bounds__(kWarps * 32) gather_kernel(const GatherArgs a) {
    allow_dependents_launch();
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
    const int tok = (int)(blockIdx.x * kWarps + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
    if (tok >= a.total) return;
    int page, row;
    long long pos;
    const Place at =
        token_place(tok, a.cu, a.start_pos, a.block_table, a.batch, a.max_pages, a.num_pool_pages, page, row, pos);
    if (at != Place::kOk) {
        if (lane == 0 && at == Place::kOutOfRange) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int h = (int)blockIdx.y * kHeads + lane / kLanes, piece = lane % kLanes;
    if (h >= a.num_kv_heads) return;
    const long long slab = (long long)page * a.num_kv_heads + h;
    const Piece<kType> k = load_piece<D, kType>(a.k_pool, slab, row, piece);
    const Piece<kType> v = load_piece<D, kType>(a.v_pool, slab, row, piece);
    float ks = 1.f, vs = 1.f;
    if constexpr (kType == PA_KV_FP4_E2M1 || kType == PA_KV_FP8_E4M3) {
        ks = __ldg(&a.k_scale[h]);
        vs = __ldg(&a.v_scale[h]);
    }
    const long long dst = ((long long)tok * a.num_kv_heads + h) * D + piece * 16;
    store_piece<kType>(a.k_out + dst, k, ks);
    store_piece<kType>(a.v_out + dst, v, vs);
}

template <int D>
dim3 token_grid(int tokens, int heads) {
    constexpr int kHeads = 32 / (D / 16);
    return dim3((unsigned)((tokens + kWarps - 1) / kWarps), (unsigned)((heads + kHeads - 1) / kHeads));
}

template <int D>
cudaError_t launch_gather_d(const GatherArgs& a, int kv_dtype, cudaStream_t stream) {
    const dim3 grid = token_grid<D>(a.total, a.num_kv_heads);
    switch (kv_dtype) {
        case PA_KV_FP4_E2M1: gather_kernel<D, PA_KV_FP4_E2M1><<<grid, kWarps * 32, 0, stream>>>(a); break;
        case PA_KV_FP8_E4M3: gather_kernel<D, PA_KV_FP8_E4M3><<<grid, kWarps * 32, 0, stream>>>(a); break;
        default: gather_kernel<D, PA_KV_BF16><<<grid, kWarps * 32, 0, stream>>>(a); break;  // either 16-bit type: a copy
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_fp4(const AppendArgs& a, cudaStream_t stream) {
    if (a.head_dim == 128)
        append_fp4_kernel<128><<<token_grid<128>(a.total_new, a.num_kv_heads), kWarps * 32, 0, stream>>>(a);
    else
        append_fp4_kernel<64><<<token_grid<64>(a.total_new, a.num_kv_heads), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_gather(const GatherArgs& a, int head_dim, int kv_dtype, cudaStream_t stream) {
    return head_dim == 128 ? launch_gather_d<128>(a, kv_dtype, stream) : launch_gather_d<64>(a, kv_dtype, stream);
}

}  // namespace pa
