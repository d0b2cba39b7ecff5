// pa_step.h -- declarations of the serving step around a 4-bit cache, shared
// by the host API and its kernel files.
#pragma once

#include "pa_internal.h"

namespace pa {

// 4-bit pages (decode_fp4.cu): CTAs that fit on one SM, by query heads per KV head
__host__ __device__ constexpr int fp4_ctas_per_sm(int group) { return group > 8 ? 2 : 3; }
cudaError_t launch_decode_fp4(int head_dim, const DecodeArgs& a, int grid, cudaStream_t stream);
// Merges the splits that launch_decode_fp4 left in a.o_part and a.lse_part.
// behind_attention: that was the launch just before, so that the merge may be
// let in as its CTAs leave and read the metadata, which it waited for, at once.
// Else what came before may still be writing the metadata: a plain launch.
cudaError_t launch_combine_fp4(int head_dim, const DecodeArgs& a, bool behind_attention, cudaStream_t stream);

// 4-bit pages and the read-back (cache4.cu)
cudaError_t launch_append_fp4(const AppendArgs& a, cudaStream_t stream);

struct GatherArgs {
    const uint8_t* k_pool;
    const uint8_t* v_pool;
    const float* k_scale;
    const float* v_scale;
    const int32_t* cu;
    const int32_t* start_pos;
    const int32_t* block_table;
    uint16_t* k_out;  // [total, Hk, D], bf16 (fp16 for fp16 pools)
    uint16_t* v_out;
    int* status;
    int32_t batch, num_kv_heads, max_pages, num_pool_pages, total;
};

cudaError_t launch_gather(const GatherArgs& a, int head_dim, int kv_dtype, cudaStream_t stream);

// Head norms and the rotary rotation (norm_rope.cu)
struct NormRopeArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;  // append only
    const uint16_t* q_weight;
    const uint16_t* k_weight;
    const int32_t* positions;  // [num_axes, total_tokens]
    const float* cos_sin;      // [max_position, rope_dim]
    uint16_t* q_out;
    uint16_t* k_out;  // nullptr with append
    int* status;
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    int32_t total_tokens, num_q_heads, num_kv_heads, rope_dim, interleaved, num_axes, max_position, f16, norm;
    int32_t warps, share, longer;  // set by the launch
    int32_t sections[2];  // pairs of the first two axes (the third takes the rest)
    float eps;
    // append only
    const int32_t* cu_new;
    const int32_t* start_pos;
    const int32_t* block_table;
    void* k_pool;
    void* v_pool;
    const float* k_scale;
    const float* v_scale;
    int32_t batch, max_pages, num_pool_pages;
};

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, cudaStream_t stream);
cudaError_t launch_norm_rope_append(const NormRopeArgs& a, int head_dim, int kv_dtype, cudaStream_t stream);

}  // namespace pa
