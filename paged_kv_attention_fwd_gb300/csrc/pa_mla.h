// pa_mla.h -- declarations of the serving step around a latent cache, shared
// by the host API and its kernel files.
#pragma once

#include "pa_internal.h"

namespace pa {

constexpr int kMlaLatent = 512, kMlaRope = 64, kMlaRow = kMlaLatent + kMlaRope;  // elements of a cached row
constexpr int kMlaOutputGroup = 32;  // tokens that pa_mla_output loads by one copy
constexpr int kMlaNope = 128, kMlaValue = 128;                                     // of a head, before absorption

// Host helpers of pa_api.cu: a status with a message for pa_last_error(), a
// 16-bit tensor map with 128-byte swizzle, the time limit of device waits.
pa_status host_fail(pa_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
pa_status host_map_16(bool f16, CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                      const uint64_t* strides_bytes, const uint32_t* box);
uint64_t host_wait_limit_ns();

// Attention over latent pages (mla_decode.cu)
constexpr int kMlaBlockRows = 64;  // query rows (token, head) of a block at most, and those of a sequence's blocks
constexpr int mla_block_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : kMlaBlockRows; }
struct MlaMerge {
    int32_t b, blk, pieces, first;  // pieces of a split item, the first of them in range `first` (0: none)
};
struct MlaDecodeArgs {
    const uint8_t* pool;
    const int32_t* block_table;
    const int32_t* seq_lens;
    uint16_t* out;     // [batch * rows, 512]
    float* lse;        // [batch * rows] or nullptr
    float* o_part;     // fp32 [2 * ranges * blocks, 64, 512]
    float* ref_part;   // fp32 [2 * ranges * blocks, 64]
    float* sum_part;   // fp32 [2 * ranges * blocks, 4, 64]
    MlaMerge* merges;  // [ranges * blocks]: of the CTA's split item, or where few is set of (sequence, block)
    int* status;
    int32_t batch, rows, q_len, num_heads, max_pages, num_pool_pages;
    int32_t f16;
    int32_t ranges, few;  // set by the launch
    float scale_log2;
    uint64_t wait_ns;
};
// maps: rows of 576 elements as [9 chunks, rows, 64], so that a box's chunks lie one behind the other: the queries'
// (boxes of all chunks of mla_block_rows rows), the pool's (two chunks of a page, one chunk of a page)
cudaError_t launch_mla_decode(MlaDecodeArgs a, int sms, const CUtensorMap* maps, cudaStream_t stream);

// Rows into and out of latent pages (mla_cache.cu)
struct MlaCacheArgs {
    const uint16_t* kv;  // append: rows of 576, kv_stride elements apart
    const uint16_t* weight;
    const int32_t* positions;
    const float* cos_sin;
    const int32_t* cu;
    const int32_t* start_pos;
    const int32_t* block_table;
    uint16_t* pool;
    uint16_t* latent_out;  // gather
    uint16_t* rope_out;
    int* status;
    long long kv_stride;
    int32_t batch, max_pages, num_pool_pages, total, interleaved, max_position, f16, norm;
    float eps;
};
cudaError_t launch_mla_append(const MlaCacheArgs& a, cudaStream_t stream);
cudaError_t launch_mla_gather(const MlaCacheArgs& a, cudaStream_t stream);

// The products with every head's own matrix (mla_project.cu)
struct MlaProjectArgs {
    const uint16_t* in;
    const int32_t* positions;
    const float* cos_sin;  // query; nullptr: the rotary part is copied
    uint16_t* out;
    int* status;
    long long in_stride, out_stride;  // elements from one token to the next
    int32_t total, heads, interleaved, max_position, f16;
    uint64_t wait_ns;
};
// maps: the input as [tokens, heads, elements] in boxes of 64 elements of 128 tokens (query) or kMlaOutputGroup (output),
// the weights as [heads, 128, 512] in boxes of 64 elements of 128 rows, the query's output like its input
cudaError_t launch_mla_query(const MlaProjectArgs& a, const CUtensorMap* maps, cudaStream_t stream);
cudaError_t launch_mla_output(const MlaProjectArgs& a, const CUtensorMap* maps, cudaStream_t stream);

}  // namespace pa
