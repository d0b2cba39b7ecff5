// norm_rope.cu -- RMS norm of every query and key head, then the rotary
// rotation, in one pass over the projections (pa_qk_norm_rope), optionally
// with the keys and values going straight into their cache pages
// (pa_norm_rope_append_kv).
//
//   y = x * rsqrt(mean_i x_i^2 + eps) * w             (fp32)
//   (a, b) -> (a cos - b sin, b cos + a sin)          (first rope_dim elements)
//
// with one rounding to 16 bits at the end.  HBM-bound: 2 bytes in, 2 out per
// element and a table row per token.  A head row is held by D / 8 lanes, 8
// elements each: two groups of 4 whose elements pair up with one another, so
// the rotation needs no shuffle in either pairing.  A warp takes
// kPasses * (32 / (D / 8)) rows of one token -- queries, keys, values in that
// order -- and loads all of them, and its angles once, before it computes.
#include "cache4.cuh"
#include "pa_launch.h"
#include "token_place.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4, kPasses = 4;

__device__ __forceinline__ float2 unpack16(uint32_t w, bool f16) {
    if (f16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool f16) {
    if (f16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// four e4m3 codes of x / scale, as pa_append_kv stores them
__device__ __forceinline__ uint32_t e4m3x4(uint2 w, float scale) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(__uint_as_float(w.x << 16), scale), __fdiv_rn(__uint_as_float(w.x & 0xFFFF0000u), scale)),
        __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(__uint_as_float(w.y << 16), scale), __fdiv_rn(__uint_as_float(w.y & 0xFFFF0000u), scale)),
        __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// The four cos and sin a lane needs: pairs pair0 .. pair0 + 3, whose positions
// may belong to different axes.
__device__ __forceinline__ void load_angles(const NormRopeArgs& a, const int (&pos)[3], int pair0, float (&c)[4],
                                            float (&s)[4]) {
    const int half = a.rope_dim / 2;
    const int e0 = a.sections[0], e1 = e0 + a.sections[1];
    auto axis = [&](int p) { return p < e0 ? pos[0] : p < e1 ? pos[1] : pos[2]; };
    const int first = axis(pair0), last = axis(pair0 + 3);
    if (first == last && axis(pair0 + 1) == first && axis(pair0 + 2) == first) {
        const float* t = a.cos_sin + (long long)first * a.rope_dim + pair0;
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(t)), s4 = __ldg(reinterpret_cast<const float4*>(t + half));
        c[0] = c4.x; c[1] = c4.y; c[2] = c4.z; c[3] = c4.w;
        s[0] = s4.x; s[1] = s4.y; s[2] = s4.z; s[3] = s4.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* t = a.cos_sin + (long long)axis(pair0 + i) * a.rope_dim + pair0 + i;
            c[i] = __ldg(t);
            s[i] = __ldg(t + half);
        }
    }
}

// kCache: -1 keys to k_out, else the page type they (and the values) go to
template <int D, bool kInterleaved, int kCache>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(const NormRopeArgs a) {
    allow_dependents_launch();
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    constexpr bool kAppend = kCache >= 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % kLanes;
    const int rows = a.num_q_heads + (kAppend ? 2 : 1) * a.num_kv_heads;
    const int chunks = (rows + kPasses * kRows - 1) / (kPasses * kRows);
    const long long id = (long long)blockIdx.x * kWarps + warp;
    const int tok = (int)(id / chunks), chunk = (int)(id % chunks);
    if (tok >= a.total_tokens) return;
    const bool f16 = a.f16;

    // where this lane's two groups of 4 elements lie in a row, and whether they turn
    const int half = a.rope_dim / 2;
    const bool turns = kInterleaved ? 8 * l < a.rope_dim : 4 * l < half;
    const int off0 = kInterleaved ? 8 * l : turns ? 4 * l : a.rope_dim + 8 * (l - half / 4);
    const int off1 = kInterleaved || !turns ? off0 + 4 : half + 4 * l;

    // rows of this warp: all loads first
    uint2 x[kPasses][2];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int r = (chunk * kPasses + p) * kRows + lane / kLanes;
        if (r < rows) {
            const uint16_t* src =
                r < a.num_q_heads ? a.q + tok * a.q_stride + (long long)r * D
                : r < a.num_q_heads + a.num_kv_heads ? a.k + tok * a.k_stride + (long long)(r - a.num_q_heads) * D
                                                     : a.v + tok * a.v_stride + (long long)(r - a.num_q_heads - a.num_kv_heads) * D;
            if constexpr (kInterleaved) {
                const uint4 w = *reinterpret_cast<const uint4*>(src + off0);
                x[p][0] = make_uint2(w.x, w.y);
                x[p][1] = make_uint2(w.z, w.w);
            } else {
                x[p][0] = *reinterpret_cast<const uint2*>(src + off0);
                x[p][1] = *reinterpret_cast<const uint2*>(src + off1);
            }
        }
    }

    // place in the cache, positions, angles
    int page = 0, prow = 0;
    long long cpos = 0;
    if constexpr (kAppend) {
        const Place at = token_place(tok, a.cu_new, a.start_pos, a.block_table, a.batch, a.max_pages,
                                     a.num_pool_pages, page, prow, cpos);
        if (at != Place::kOk) {
            if (lane == 0 && at == Place::kOutOfRange) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
            return;
        }
    }
    int pos[3] = {0, 0, 0};
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.rope_dim > 0) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < a.num_axes) {
                if (kAppend && a.positions == nullptr) pos[i] = (int)min(cpos, (long long)a.max_position);
                else pos[i] = __ldg(&a.positions[(long long)i * a.total_tokens + tok]);
                bad |= pos[i] < 0 || pos[i] >= a.max_position;
            }
        if (pos[0] < 0) return;  // a padding row
        if (bad) {
            if (lane == 0) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
            return;
        }
        if (turns) load_angles(a, pos, 4 * l, c, s);
    }

    __shared__ __align__(16) uint16_t stage[kCache == PA_KV_FP4_E2M1 ? kWarps : 1][kCache == PA_KV_FP4_E2M1 ? kRows * D : 8];

#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int r0 = (chunk * kPasses + p) * kRows;  // first row of the pass (warp-uniform)
        if (r0 >= rows) break;
        const int r = r0 + lane / kLanes;
        const bool is_q = r < a.num_q_heads, is_v = r >= a.num_q_heads + a.num_kv_heads;
        uint2 y0 = make_uint2(0, 0), y1 = make_uint2(0, 0);
        if (r < rows) {
            y0 = x[p][0];
            y1 = x[p][1];
        }
        float f[8];
        const float2 f01 = unpack16(y0.x, f16), f23 = unpack16(y0.y, f16), f45 = unpack16(y1.x, f16),
                     f67 = unpack16(y1.y, f16);
        f[0] = f01.x; f[1] = f01.y; f[2] = f23.x; f[3] = f23.y;
        f[4] = f45.x; f[5] = f45.y; f[6] = f67.x; f[7] = f67.y;
        if (a.norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = rsqrtf(ss * (1.f / D) + a.eps);
            const uint16_t* wp = is_q ? a.q_weight : a.k_weight;
            float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            if (wp != nullptr && !is_v) {
                const uint2 w0 = __ldg(reinterpret_cast<const uint2*>(wp + off0)),
                            w1 = __ldg(reinterpret_cast<const uint2*>(wp + off1));
                const float2 a01 = unpack16(w0.x, f16), a23 = unpack16(w0.y, f16), a45 = unpack16(w1.x, f16),
                             a67 = unpack16(w1.y, f16);
                w[0] = a01.x; w[1] = a01.y; w[2] = a23.x; w[3] = a23.y;
                w[4] = a45.x; w[5] = a45.y; w[6] = a67.x; w[7] = a67.y;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * w[i];
        }
        if (turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ia = kInterleaved ? 2 * i : i, ib = kInterleaved ? 2 * i + 1 : 4 + i;
                const float u = f[ia], v = f[ib];
                f[ia] = u * c[i] - v * s[i];
                f[ib] = v * c[i] + u * s[i];
            }
        }
        if (!is_v) {  // values pass through bit for bit
            y0 = make_uint2(pack16(f[0], f[1], f16), pack16(f[2], f[3], f16));
            y1 = make_uint2(pack16(f[4], f[5], f16), pack16(f[6], f[7], f16));
        }
        uint16_t* dst = nullptr;  // a 16-bit destination row
        if (r < rows) {
            if (is_q) dst = a.q_out + tok * a.q_out_stride + (long long)r * D;
            else if constexpr (!kAppend) dst = a.k_out + tok * a.k_out_stride + (long long)(r - a.num_q_heads) * D;
        }
        if constexpr (kAppend) {
            const int h = is_v ? r - a.num_q_heads - a.num_kv_heads : r - a.num_q_heads;
            const long long slab = (long long)page * a.num_kv_heads + h;
            uint8_t* pool = static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool);
            const float* scales = is_v ? a.v_scale : a.k_scale;
            if constexpr (kCache == PA_KV_BF16) {  // either 16-bit type
                if (r < rows && !is_q) dst = reinterpret_cast<uint16_t*>(pool) + (slab * kPage + prow) * D;
            } else if constexpr (kCache == PA_KV_FP8_E4M3) {
                if (r < rows && !is_q) {
                    uint8_t* out = pool + (slab * kPage + prow) * D;
                    const float scale = __ldg(&scales[h]);
                    *reinterpret_cast<uint32_t*>(out + off0) = e4m3x4(y0, scale);
                    *reinterpret_cast<uint32_t*>(out + off1) = e4m3x4(y1, scale);
                }
            } else if (r0 + kRows > a.num_q_heads) {  // the pass holds a cache row: through shared memory, so
                uint16_t* st = stage[warp];           // that one lane sees the 16 elements of a block
                *reinterpret_cast<uint2*>(st + (lane / kLanes) * D + off0) = y0;
                *reinterpret_cast<uint2*>(st + (lane / kLanes) * D + off1) = y1;
                __syncwarp();
                constexpr int kBlocks = D / 16;
                const int br = r0 + lane / kBlocks, piece = lane % kBlocks;
                if (lane < kRows * kBlocks && br >= a.num_q_heads && br < rows) {
                    const bool bv = br >= a.num_q_heads + a.num_kv_heads;
                    const int bh = br - a.num_q_heads - (bv ? a.num_kv_heads : 0);
                    const uint4* w = reinterpret_cast<const uint4*>(st + (lane / kBlocks) * D + piece * 16);
                    fp4_store_block<D>(static_cast<uint8_t*>(bv ? a.v_pool : a.k_pool) +
                                           ((long long)page * a.num_kv_heads + bh) * fp4_slab_bytes(D),
                                       prow, piece, w[0], w[1], __ldg(&(bv ? a.v_scale : a.k_scale)[bh]));
                }
                __syncwarp();
            }
        }
        if (dst != nullptr) {
            if constexpr (kInterleaved) {
                *reinterpret_cast<uint4*>(dst + off0) = make_uint4(y0.x, y0.y, y1.x, y1.y);
            } else {
                *reinterpret_cast<uint2*>(dst + off0) = y0;
                *reinterpret_cast<uint2*>(dst + off1) = y1;
            }
        }
    }
}

template <int D, bool kInterleaved, int kCache>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t stream) {
    constexpr int kRows = 32 / (D / 8) * kPasses;
    const int rows = a.num_q_heads + (kCache >= 0 ? 2 : 1) * a.num_kv_heads;
    const long long warps = (long long)a.total_tokens * ((rows + kRows - 1) / kRows);
    norm_rope_kernel<D, kInterleaved, kCache><<<(unsigned)((warps + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int D, int kCache>
cudaError_t launch_pairing(const NormRopeArgs& a, cudaStream_t stream) {
    return a.interleaved ? launch<D, true, kCache>(a, stream) : launch<D, false, kCache>(a, stream);
}

template <int D>
cudaError_t launch_cache(const NormRopeArgs& a, int kv_dtype, cudaStream_t stream) {
    switch (kv_dtype) {
        case PA_KV_FP4_E2M1: return launch_pairing<D, PA_KV_FP4_E2M1>(a, stream);
        case PA_KV_FP8_E4M3: return launch_pairing<D, PA_KV_FP8_E4M3>(a, stream);
        default: return launch_pairing<D, PA_KV_BF16>(a, stream);
    }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, cudaStream_t stream) {
    switch (head_dim) {
        case 64: return launch_pairing<64, -1>(a, stream);
        case 128: return launch_pairing<128, -1>(a, stream);
        default: return launch_pairing<256, -1>(a, stream);
    }
}

cudaError_t launch_norm_rope_append(const NormRopeArgs& a, int head_dim, int kv_dtype, cudaStream_t stream) {
    return head_dim == 64 ? launch_cache<64>(a, kv_dtype, stream) : launch_cache<128>(a, kv_dtype, stream);
}

}  // namespace pa
