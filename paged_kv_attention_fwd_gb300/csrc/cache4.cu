// cache4.cu -- writing 4-bit pages (pa_append_kv with PA_KV_FP4_E2M1) and
// reading the rows of pages of any type back (pa_gather_kv).
//
// Both are copies with a conversion, so HBM-bound: 2 bytes of a 16-bit row
// against 0.5625 (4-bit), 1 (e4m3) or 2 bytes of a page row per element.  A
// thread owns one 16-element piece of a row -- the block of the 4-bit type, so
// neither its largest magnitude nor its scale crosses threads.  A warp takes
// 32 / (D / 16) consecutive tokens, whose rows are neighbours in a page, of
// several heads: what it touches of a slab is contiguous (at D = 128, 256
// bytes of codes and one 32-byte sector of scales), and the search for the
// tokens' sequence and page is paid once for all its heads.
//
// Measured: 4-bit rows of 302k tokens, 8 heads of 128, read back in 238 us
// (1.59 GB, 6.7 TB/s, the memory's copy rate); 32768 tokens written in 28.5
// us (172 MB, 6.0 TB/s); 4096 written and 37k read back, two launches, 38 us
// (215 MB); 64 written and 64 read back 5.8 us.
#include "cache4.cuh"
#include "pa_launch.h"
#include "token_place.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kHeads = 4;  // heads of a warp that reads back (302k rows 237.4 us, with 2 238.3, with 1 241.0)

// This thread's token and piece of its rows.  grid: x = groups of tokens, kWarps to a CTA
template <int D>
struct Share {
    static constexpr int kLanes = D / 16, kTokens = 32 / kLanes;
    int tok0, tok, piece;  // tok0: the warp's first token
    __device__ __forceinline__ Share()
        : tok0((int)(blockIdx.x * kWarps + (threadIdx.x >> 5)) * kTokens),
          tok(tok0 + (int)(threadIdx.x & 31) / kLanes),
          piece((int)(threadIdx.x & 31) % kLanes) {}
    // that of this thread's token; the whole warp calls it
    __device__ __forceinline__ Sequence sequence(const int32_t* __restrict__ cu, const int32_t* __restrict__ start_pos,
                                                 int batch) const {
        return warp_sequences<kTokens>(tok0, tok - tok0, cu, start_pos, batch);
    }
};

// grid.y: a warp takes every gridDim.y-th head, the next one's rows on their way while this one's are quantised
template <int D>
__global__ void __launch_bounds__(kWarps * 32) append_fp4_kernel(const __grid_constant__ AppendArgs a) {
    grid_dependency_wait();
    allow_dependents_launch();
    const Share<D> my;
    if (my.tok0 >= a.total_new) return;
    const bool wide = aligned32(a.k_new) && aligned32(a.v_new), mine = my.tok < a.total_new;
    Sector k, v;
    auto load = [&](int h) {
        if (h < a.num_kv_heads && mine) {
            const long long src = ((long long)my.tok * a.num_kv_heads + h) * D + my.piece * 16;
            k = load_sector(a.k_new + src, wide);
            v = load_sector(a.v_new + src, wide);
        }
    };
    load((int)blockIdx.y);  // rows first: they do not depend on the token's place
    const Sequence seq = my.sequence(a.cu_new, a.start_pos, a.batch);
    if (!mine) return;
    int page, row;
    long long pos;
    const Place at = token_place(my.tok, seq, a.block_table, a.batch, a.max_pages, a.num_pool_pages, page, row, pos);
    if (at != Place::kOk) {
        if (my.piece == 0 && at == Place::kOutOfRange) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
        return;
    }
    for (int h = (int)blockIdx.y; h < a.num_kv_heads; h += (int)gridDim.y) {
        const Sector k_now = k, v_now = v;
        load(h + (int)gridDim.y);
        const long long slab = ((long long)page * a.num_kv_heads + h) * fp4_slab_bytes(D);
        fp4_store_block<D>(static_cast<uint8_t*>(a.k_pool) + slab, row, my.piece, k_now.lo, k_now.hi, __ldg(&a.k_scale[h]));
        fp4_store_block<D>(static_cast<uint8_t*>(a.v_pool) + slab, row, my.piece, v_now.lo, v_now.hi, __ldg(&a.v_scale[h]));
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

// grid.y: groups of kHeads heads
template <int D, int kType>
__global__ void __launch_bounds__(kWarps * 32) gather_kernel(const __grid_constant__ GatherArgs a) {
    grid_dependency_wait();
    allow_dependents_launch();
    const Share<D> my;
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
    const int h0 = (int)blockIdx.y * kHeads, nh = min(kHeads, a.num_kv_heads - h0);
    const long long slab = (long long)page * a.num_kv_heads + h0;
    const bool wide_in = aligned32(a.k_pool) && aligned32(a.v_pool), wide_out = aligned32(a.k_out) && aligned32(a.v_out);
    Piece<kType> k[kHeads], v[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < nh) {
            k[i] = load_piece<D, kType>(a.k_pool, slab + i, row, my.piece, wide_in);
            v[i] = load_piece<D, kType>(a.v_pool, slab + i, row, my.piece, wide_in);
        }
    const long long dst = ((long long)my.tok * a.num_kv_heads + h0) * D + my.piece * 16;
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < nh) {
            float ks = 1.f, vs = 1.f;
            if constexpr (kType == PA_KV_FP4_E2M1 || kType == PA_KV_FP8_E4M3) {
                ks = __ldg(&a.k_scale[h0 + i]);
                vs = __ldg(&a.v_scale[h0 + i]);
            }
            store_piece<kType>(a.k_out + dst + i * D, k[i], ks, wide_out);
            store_piece<kType>(a.v_out + dst + i * D, v[i], vs, wide_out);
        }
}

template <int D>
unsigned token_groups(int tokens) {
    constexpr int per_cta = kWarps * Share<D>::kTokens;
    return (unsigned)((tokens + per_cta - 1) / per_cta);
}

// A token's heads are dealt to as many warps as find room on the SMs together, 8 CTAs of them each: 32768 tokens of 8
// heads 28.5 us with all heads in one warp and 38 with one head each, 64 tokens 6.3 and 3.0.
template <int D>
cudaError_t launch_append_d(const AppendArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const unsigned groups = token_groups<D>(a.total_new), room = (unsigned)sms * 8 / groups;
    const unsigned heads = (unsigned)a.num_kv_heads, ways = room < 1 ? 1 : room < heads ? room : heads;
    const unsigned each = (heads + ways - 1) / ways;  // heads of a warp, and as few warps as take them
    return launch_overlapped(append_fp4_kernel<D>, dim3(groups, (heads + each - 1) / each), dim3(kWarps * 32), 0, stream, a);
}

template <int D>
cudaError_t launch_gather_d(const GatherArgs& a, int kv_dtype, cudaStream_t stream) {
    const dim3 grid(token_groups<D>(a.total), (unsigned)((a.num_kv_heads + kHeads - 1) / kHeads)), block(kWarps * 32);
    switch (kv_dtype) {
        case PA_KV_FP4_E2M1: return launch_overlapped(gather_kernel<D, PA_KV_FP4_E2M1>, grid, block, 0, stream, a);
        case PA_KV_FP8_E4M3: return launch_overlapped(gather_kernel<D, PA_KV_FP8_E4M3>, grid, block, 0, stream, a);
        default: return launch_overlapped(gather_kernel<D, PA_KV_BF16>, grid, block, 0, stream, a);  // either 16-bit type
    }
}

}  // namespace

cudaError_t launch_append_fp4(const AppendArgs& a, cudaStream_t stream) {
    return a.head_dim == 128 ? launch_append_d<128>(a, stream) : launch_append_d<64>(a, stream);
}

cudaError_t launch_gather(const GatherArgs& a, int head_dim, int kv_dtype, cudaStream_t stream) {
    return head_dim == 128 ? launch_gather_d<128>(a, kv_dtype, stream) : launch_gather_d<64>(a, kv_dtype, stream);
}

}  // namespace pa
