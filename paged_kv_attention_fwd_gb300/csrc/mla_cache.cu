// mla_cache.cu -- rows into a latent cache (pa_mla_append_kv: RMS norm of the
// 512 latent elements, rotation of the 64 rotary ones) and back out of it
// (pa_mla_gather_kv).
//
//   c = x / sqrt(mean(x^2) + eps) * weight            over the 512 elements
//   (a, b) -> (a cos - b sin, b cos + a sin)          for each of the 32 pairs
//
// Both move 2 bytes in and 2 out per element, so HBM-bound.  A warp takes 8
// consecutive tokens: a lane holds 32 bytes of every token's latent part and of
// one token's rotary part (4 lanes a token), so all its loads are in flight
// together and the tokens' places are found once for the warp.  Few new tokens
// are a chain of dependent steps, so there a warp takes 4 of them.
//
// Measured: 302k rows read back in 103 us (696 MB, 6.7 TB/s, the memory's copy
// rate); 16384 rows appended in 8.8 us (42 MB, 4.7 TB/s: a third of it is the
// launch), with 4 tokens a warp 9.6; 64 rows 2.9, with 8 tokens a warp 3.9 and with 2 3.0.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache4.cuh"
#include "pa_launch.h"
#include "pa_mla.h"
#include "token_place.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;

// the place of this lane's token (lane % kTokens of the warp's), as pool row or -1
struct Placed {
    long long row, pos;
    bool skip;
};
template <int kTokens>
__device__ __forceinline__ Placed place_of(const MlaCacheArgs& a, int tok0) {
    const int k = (int)(threadIdx.x & 31) % kTokens, tok = tok0 + k;
    const Sequence seq = warp_sequences<kTokens>(tok0, k, a.cu, a.start_pos, a.batch);
    int page = 0, row = 0;
    Placed p{-1, 0, true};
    if (tok >= a.total) return p;
    const Place at = token_place(tok, seq, a.block_table, a.batch, a.max_pages, a.num_pool_pages, page, row, p.pos);
    p.skip = at != Place::kOk;
    if (at == Place::kOutOfRange) p.row = -2;  // recorded unless it turns out to be padding
    if (at == Place::kOk) p.row = (long long)page * kPage + row;
    return p;
}

__device__ __forceinline__ float2 to_float2(uint32_t w, bool f16) {
    if (f16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t to_16x2(float x, float y, bool f16) {
    if (f16) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void unpack(const Sector& s, float (&x)[16], bool f16) {
    const uint32_t u[8] = {s.lo.x, s.lo.y, s.lo.z, s.lo.w, s.hi.x, s.hi.y, s.hi.z, s.hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = to_float2(u[i], f16);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
    }
}
__device__ __forceinline__ Sector pack(const float (&x)[16], bool f16) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = to_16x2(x[2 * i], x[2 * i + 1], f16);
    return Sector{make_uint4(u[0], u[1], u[2], u[3]), make_uint4(u[4], u[5], u[6], u[7])};
}

template <int kTokens, bool kF16, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32) mla_append_kernel(const __grid_constant__ MlaCacheArgs a) {
    grid_dependency_wait();
    allow_dependents_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tok0 = ((int)blockIdx.x * kWarps + warp) * kTokens;
    if (tok0 >= a.total) return;
    const int last = a.total - 1;
    const bool wide = aligned32(a.kv) && a.kv_stride % 16 == 0;
    Sector x[kTokens], r;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) x[i] = load_sector(a.kv + min(tok0 + i, last) * a.kv_stride + lane * 16, wide);
    // rotary part: lane j of 4 has pairs 8 j .. 8 j + 7 of token lane / 4
    const int rt = lane / 4 % kTokens, rj = lane % 4;
    const uint16_t* rsrc = a.kv + min(tok0 + rt, last) * a.kv_stride + kMlaLatent;
    const int ra = kInterleaved ? 16 * rj : 8 * rj, rb = kInterleaved ? 16 * rj + 8 : 32 + 8 * rj;
    r.lo = __ldg(reinterpret_cast<const uint4*>(rsrc + ra));
    r.hi = __ldg(reinterpret_cast<const uint4*>(rsrc + rb));
    Sector w{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (a.norm && a.weight != nullptr) {
        w.lo = __ldg(reinterpret_cast<const uint4*>(a.weight + lane * 16));
        w.hi = __ldg(reinterpret_cast<const uint4*>(a.weight + lane * 16 + 8));
    }
    // a lane's own token below is lane % kTokens
    Placed p = place_of<kTokens>(a, tok0);
    if (a.cos_sin != nullptr) {
        long long pos = p.pos;
        if (a.positions != nullptr) {
            pos = __ldg(&a.positions[min(tok0 + lane % kTokens, last)]);
            if (pos < 0) p.skip = true, p.row = -1;  // marked as padding
        }
        if (p.row != -1 && pos >= a.max_position) p.skip = true, p.row = -2;
        p.pos = pos;
    }
    if (p.row == -2 && lane < kTokens) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
    if (p.skip) p.row = -1;

    // the rotary part
    {
        const long long row = __shfl_sync(0xffffffffu, p.row, rt), pos = __shfl_sync(0xffffffffu, p.pos, rt);
        if (row >= 0 && lane < 4 * kTokens) {
            float v[16];
            unpack(r, v, kF16);
            if (a.cos_sin != nullptr) {
                float c[8], s[8];
                const float4* t = reinterpret_cast<const float4*>(a.cos_sin + pos * kMlaRope + 8 * rj);
                *reinterpret_cast<float4*>(&c[0]) = __ldg(t);
                *reinterpret_cast<float4*>(&c[4]) = __ldg(t + 1);
                *reinterpret_cast<float4*>(&s[0]) = __ldg(t + 8);
                *reinterpret_cast<float4*>(&s[4]) = __ldg(t + 9);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int f = kInterleaved ? 2 * i : i, g = kInterleaved ? 2 * i + 1 : 8 + i;
                    const float y = v[f] * c[i] - v[g] * s[i], z = v[g] * c[i] + v[f] * s[i];
                    v[f] = y;
                    v[g] = z;
                }
            }
            const Sector o = pack(v, kF16);
            uint16_t* dst = a.pool + row * kMlaRow + kMlaLatent;
            *reinterpret_cast<uint4*>(dst + ra) = o.lo;
            *reinterpret_cast<uint4*>(dst + rb) = o.hi;
        }
    }
    float wf[16];
    unpack(w, wf, kF16);
    if (!a.norm || a.weight == nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i) wf[i] = 1.f;
    }
    const bool wide_out = aligned32(a.pool);  // rows are 36 sectors
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const long long row = __shfl_sync(0xffffffffu, p.row, i);
        if (row < 0) continue;
        Sector o = x[i];
        if (a.norm) {
            float v[16];
            unpack(x[i], v, kF16);
            float sq = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) sq = fmaf(v[k], v[k], sq);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
            const float inv = rsqrtf(fmaf(sq, 1.f / kMlaLatent, a.eps));
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = v[k] * inv * wf[k];
            o = pack(v, kF16);
        }
        store_sector(a.pool + row * kMlaRow + lane * 16, o, wide_out);
    }
}

template <int kTokens>
__global__ void __launch_bounds__(kWarps * 32) mla_gather_kernel(const __grid_constant__ MlaCacheArgs a) {
    grid_dependency_wait();
    allow_dependents_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tok0 = ((int)blockIdx.x * kWarps + warp) * kTokens;
    if (tok0 >= a.total) return;
    const Placed p = place_of<kTokens>(a, tok0);
    if (p.row == -2 && lane < kTokens) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
    const bool wide_in = aligned32(a.pool), wide_out = aligned32(a.latent_out) && aligned32(a.rope_out);
    const long long my_row = p.skip ? -1 : p.row;
    Sector x[kTokens], r;
    static_assert(kTokens == 8, "4 lanes a token");
    const long long rrow = __shfl_sync(0xffffffffu, my_row, lane / 4);
    if (rrow >= 0) r = load_sector(a.pool + rrow * kMlaRow + kMlaLatent + lane % 4 * 16, wide_in);
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const long long row = __shfl_sync(0xffffffffu, my_row, i);
        if (row >= 0) x[i] = load_sector(a.pool + row * kMlaRow + lane * 16, wide_in);
    }
    if (rrow >= 0) store_sector(a.rope_out + (long long)(tok0 + lane / 4) * kMlaRope + lane % 4 * 16, r, wide_out);
#pragma unroll
    for (int i = 0; i < kTokens; ++i)
        if (__shfl_sync(0xffffffffu, my_row, i) >= 0)
            store_sector(a.latent_out + (long long)(tok0 + i) * kMlaLatent + lane * 16, x[i], wide_out);
}

template <int kTokens>
dim3 grid_of(int total) {
    return dim3((unsigned)((total + kWarps * kTokens - 1) / (kWarps * kTokens)));
}

template <int kTokens>
cudaError_t launch_append(const MlaCacheArgs& a, cudaStream_t stream) {
    const dim3 grid = grid_of<kTokens>(a.total), block(kWarps * 32);
    if (a.f16)
        return a.interleaved ? launch_overlapped(mla_append_kernel<kTokens, true, true>, grid, block, 0, stream, a)
                             : launch_overlapped(mla_append_kernel<kTokens, true, false>, grid, block, 0, stream, a);
    return a.interleaved ? launch_overlapped(mla_append_kernel<kTokens, false, true>, grid, block, 0, stream, a)
                         : launch_overlapped(mla_append_kernel<kTokens, false, false>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_mla_append(const MlaCacheArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // 8 tokens a warp once that gives every SM 8 warps
    return a.total >= 64 * sms ? launch_append<8>(a, stream) : launch_append<4>(a, stream);
}

cudaError_t launch_mla_gather(const MlaCacheArgs& a, cudaStream_t stream) {
    return launch_overlapped(mla_gather_kernel<8>, grid_of<8>(a.total), dim3(kWarps * 32), 0, stream, a);
}

}  // namespace pa
