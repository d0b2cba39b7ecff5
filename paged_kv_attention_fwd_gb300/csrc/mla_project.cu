// mla_project.cu -- the products with every head's own matrix that attention in
// the latent space needs before and after:
//
//   pa_mla_query   out[t, h, :512]  = q[t, h, :128] W_uk[h]     (128 x 512)
//                  out[t, h, 512:]  = q[t, h, 128:] turned by the token's angles
//   pa_mla_output  out[t, h]        = W_uv[h] o[t, h]           (128 x 512)
//
// With few tokens the weights are what is read, with many the activations; the
// products themselves stay far below the tensor cores' rate.  A CTA takes 128
// tokens (rows of the MMA) of one head, and of a query 256 of the 512 columns.
// W_uk lies with its columns contiguous (an MN-major operand), W_uv with the
// summed dimension contiguous, so both are read as they are loaded.
//
//   warp 0     loads (TMA) and MMAs, one thread
//   warps 1-4  the result, a token a thread; a query's rotary part meanwhile
#include "pa_launch.h"
#include "pa_mla.h"
#include "pa_ptx.cuh"
#include "prefill_common.cuh"

namespace pa {
namespace {

constexpr int kTokens = 128;
constexpr int kThreads = 160;

template <bool kQuery>
struct Layout {
    static constexpr int kSum = kQuery ? kMlaNope : kMlaLatent;  // summed over
    static constexpr int kSteps = kSum / 64;
    static constexpr int kCols = kQuery ? 256 : kMlaValue;  // of the result, per CTA
    static constexpr int kParts = kQuery ? kMlaLatent / kCols : 1;
    static constexpr int kABytes = kTokens * 128;  // 64 elements of 128 tokens
    static constexpr int kBBytes = kCols * 128;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = kQuery ? 2 : 3;
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    static constexpr int kOutRow = kQuery ? kMlaRow : kMlaValue;
};

// A query's rotary part of one token.
template <bool kF16, bool kInterleaved>
__device__ __forceinline__ void turn_row(const uint16_t* src, uint16_t* dst, const float* cs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 8 pairs each
        const int ra = kInterleaved ? 16 * i : 8 * i, rb = kInterleaved ? 16 * i + 8 : 32 + 8 * i;
        const uint4 lo = __ldg(reinterpret_cast<const uint4*>(src + ra)), hi = __ldg(reinterpret_cast<const uint4*>(src + rb));
        uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        if (cs != nullptr) {
            float v[16], c[8], s[8];
            const float4* t = reinterpret_cast<const float4*>(cs + 8 * i);
            *reinterpret_cast<float4*>(&c[0]) = __ldg(t);
            *reinterpret_cast<float4*>(&c[4]) = __ldg(t + 1);
            *reinterpret_cast<float4*>(&s[0]) = __ldg(t + 8);
            *reinterpret_cast<float4*>(&s[4]) = __ldg(t + 9);
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
        }
        *reinterpret_cast<uint4*>(dst + ra) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(dst + rb) = make_uint4(u[4], u[5], u[6], u[7]);
    }
}

template <bool kQuery, bool kF16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) mla_project_kernel(const __grid_constant__ MlaProjectArgs a,
                                                               const __grid_constant__ CUtensorMap map_in,
                                                               const __grid_constant__ CUtensorMap map_w) {
    using L = Layout<kQuery>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[L::kStages], empty[L::kStages], done;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_store;
    volatile int* abort_sh = &abort_store;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = (int)blockIdx.x % L::kParts, h = (int)blockIdx.x / L::kParts, tok0 = (int)blockIdx.y * kTokens;
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
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
        tmem_alloc(&tmem_base_sh, L::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = tmem_base_sh;

    if (warp == 0) {
        if (lane == 0) {
            auto load = [&](int step) {
                const int slot = step % L::kStages;
                uint8_t* at = sm + slot * L::kStageBytes;
                mbar_arrive_expect_tx(&full[slot], L::kStageBytes);
                if constexpr (kQuery) {
                    for (int c = 0; c < L::kCols / 64; ++c)
                        tma_load_3d(at + L::kABytes + c * 8192, &map_w, &full[slot], part * L::kCols + c * 64, step * 64, h);
                } else {
                    tma_load_3d(at + L::kABytes, &map_w, &full[slot], step * 64, 0, h);
                }
                tma_load_3d(at, &map_in, &full[slot], step * 64, h, tok0);
            };
            for (int step = 0; step < L::kStages && step < L::kSteps; ++step) load(step);
            constexpr uint32_t idesc = idesc_f16(kTokens, L::kCols, !kF16, false, kQuery);
            bool ok = true;
            int loaded = L::kStages < L::kSteps ? L::kStages : L::kSteps;
            for (int step = 0; step < L::kSteps && ok; ++step) {
                const int slot = step % L::kStages;
                ok = mbar_wait(&full[slot], (step / L::kStages) & 1, abort_sh, a.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = smem_u32(sm + slot * L::kStageBytes);
                const uint64_t ad = sdesc_sw128(at, 16, 1024);
                const uint64_t bd = sdesc_sw128(at + L::kABytes, kQuery ? 8192 : 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ss(tbase, ad + (uint64_t)(kk * 32 >> 4), bd + (uint64_t)((kQuery ? kk * 2048 : kk * 32) >> 4), idesc,
                           step > 0 || kk > 0);
                if (step + 1 == L::kSteps) {
                    mma_commit(&done);
                } else if (loaded < L::kSteps) {
                    mma_commit(&empty[slot]);
                    ok = mbar_wait(&empty[slot], (step / L::kStages) & 1, abort_sh, a.wait_ns);
                    if (ok) load(loaded++);
                }
            }
            if (!ok) {
                *abort_sh = 1;
                atomicCAS(a.status, 0, PA_ERR_TIMEOUT);
                // copies and MMAs in flight end before the CTA does
                for (int s = 0; s < L::kStages && s < loaded; ++s) {
                    const int last = loaded - 1 - (loaded - 1 - s) % L::kStages;
                    mbar_wait(&full[s], (last / L::kStages) & 1, nullptr, a.wait_ns);
                }
                mma_commit(&done);
                mbar_wait(&done, 0, nullptr, a.wait_ns);
            }
        }
    } else {
        const int q4 = warp & 3, row = q4 * 32 + lane, tok = tok0 + row;
        bool write = tok < a.total;
        uint16_t* dst = a.out + (write ? tok : 0) * a.out_stride + (long long)h * L::kOutRow;
        if constexpr (kQuery) {
            const float* cs = nullptr;
            if (a.cos_sin != nullptr && write) {
                const int pos = __ldg(&a.positions[tok]);
                if (pos >= a.max_position) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
                if (pos < 0 || pos >= a.max_position) write = false;
                else cs = a.cos_sin + (long long)pos * kMlaRope;
            }
            if (part == L::kParts - 1 && write)
                turn_row<kF16, kInterleaved>(a.in + tok * a.in_stride + (long long)h * (kMlaNope + kMlaRope) + kMlaNope,
                                             dst + kMlaLatent, cs);
        }
        dst += part * L::kCols;
        const bool ok = mbar_wait(&done, 0, abort_sh, a.wait_ns);
        if (__all_sync(0xffffffffu, ok) && __any_sync(0xffffffffu, write)) {
            tc_fence_after();
#pragma unroll 2
            for (int c = 0; c < L::kCols / 32; ++c) {
                uint32_t o[32];
                tmem_ld_x32(tbase + ((uint32_t)(q4 * 32) << 16) + c * 32, o);
                tmem_ld_wait();
                reg_fence(o);
                if (write) {
                    uint4* d4 = reinterpret_cast<uint4*>(dst + c * 32);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = pack16x2(__uint_as_float(o[8 * k + 2 * i]), __uint_as_float(o[8 * k + 2 * i + 1]), kF16);
                        d4[k] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tbase, L::kCols);
    }
}

template <bool kQuery, bool kF16, bool kInterleaved>
cudaError_t launch(const MlaProjectArgs& a, const CUtensorMap* map_in, const CUtensorMap* map_w, cudaStream_t stream) {
    using L = Layout<kQuery>;
    auto kernel = mla_project_kernel<kQuery, kF16, kInterleaved>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_dynamic_smem(kernel, L::kSmem, configured);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.heads * L::kParts), (unsigned)((a.total + kTokens - 1) / kTokens));
    return launch_overlapped(kernel, grid, dim3(kThreads), L::kSmem, stream, a, *map_in, *map_w);
}

}  // namespace

cudaError_t launch_mla_query(const MlaProjectArgs& a, const CUtensorMap* map_in, const CUtensorMap* map_w,
                             cudaStream_t stream) {
    if (a.f16)
        return a.interleaved ? launch<true, true, true>(a, map_in, map_w, stream) : launch<true, true, false>(a, map_in, map_w, stream);
    return a.interleaved ? launch<true, false, true>(a, map_in, map_w, stream) : launch<true, false, false>(a, map_in, map_w, stream);
}

cudaError_t launch_mla_output(const MlaProjectArgs& a, const CUtensorMap* map_in, const CUtensorMap* map_w,
                              cudaStream_t stream) {
    return a.f16 ? launch<false, true, false>(a, map_in, map_w, stream) : launch<false, false, false>(a, map_in, map_w, stream);
}

}  // namespace pa
