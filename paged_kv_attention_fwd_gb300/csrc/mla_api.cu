// mla_api.cu -- host side of the calls around a latent cache: argument checks,
// tensor maps and launches.  Nothing here allocates device memory or
// synchronises a stream.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "pa_mla.h"

namespace {

using pa::host_fail;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

pa_status launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? PA_OK : host_fail(PA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// What every call checks of the rows' sizes and type.
pa_status check_row(int32_t latent_dim, int32_t rope_dim, int32_t dtype) {
    if (latent_dim != pa::kMlaLatent || rope_dim != pa::kMlaRope)
        return host_fail(PA_ERR_UNSUPPORTED, "latent_dim must be 512 and rope_dim 64 (got %d, %d)", latent_dim, rope_dim);
    if (dtype == PA_KV_FP8_E4M3 || dtype == PA_KV_FP4_E2M1)
        return host_fail(PA_ERR_UNSUPPORTED, "latent pages are bf16 or fp16 (got type %d)", dtype);
    if (dtype != PA_KV_BF16 && dtype != PA_KV_FP16) return host_fail(PA_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    return PA_OK;
}

pa_status check_pages(int32_t page_size, int32_t max_pages_per_seq, int32_t num_pool_pages) {
    if (page_size != pa::kPage) return host_fail(PA_ERR_INVALID_ARG, "page_size must be 64 (got %d)", page_size);
    if (max_pages_per_seq <= 0 || num_pool_pages <= 0)
        return host_fail(PA_ERR_INVALID_ARG, "max_pages_per_seq and num_pool_pages must be positive");
    return PA_OK;
}

pa_status check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (!workspace) return host_fail(PA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned16(workspace)) return host_fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    if (bytes < need) return host_fail(PA_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, bytes);
    return PA_OK;
}

pa_status check_stride(int64_t stride, int64_t least, const char* name) {
    if (stride < least || stride % 8 != 0 || stride >= ((int64_t)1 << 38))
        return host_fail(PA_ERR_INVALID_ARG, "%s (%lld) must be a multiple of 8, at least %lld and below 2^38", name,
                         (long long)stride, (long long)least);
    return PA_OK;
}

// ------------------------------------------------------------ attention

// CTAs of a launch that may leave parts of items: the SMs' (a launch of more has one range a block, and no parts).
int decode_ctas(const pa_mla_decode_shapes* sh) { return sh->num_sms; }

size_t merges_offset() { return PA_STATUS_BYTES; }
size_t ref_offset(int ctas) { return merges_offset() + up256((size_t)ctas * sizeof(pa::MlaMerge)); }
size_t sum_offset(int ctas) { return ref_offset(ctas) + (size_t)2 * ctas * pa::kMlaBlockRows * 4; }
size_t part_offset(int ctas) { return sum_offset(ctas) + (size_t)2 * ctas * 4 * pa::kMlaBlockRows * 4; }

pa_status check_decode_shapes(const pa_mla_decode_shapes* sh) {
    if (!sh) return host_fail(PA_ERR_INVALID_ARG, "shapes must not be NULL");
    if (sh->batch < 0) return host_fail(PA_ERR_INVALID_ARG, "batch must be >= 0 (got %d)", sh->batch);
    if (sh->num_q_heads <= 0 || sh->q_len <= 0)
        return host_fail(PA_ERR_INVALID_ARG, "num_q_heads (%d) and q_len (%d) must be positive", sh->num_q_heads, sh->q_len);
    if ((int64_t)sh->num_q_heads * sh->q_len > 65536)
        return host_fail(PA_ERR_UNSUPPORTED, "num_q_heads * q_len above 65536");
    if ((int64_t)sh->batch * sh->num_q_heads * sh->q_len >= ((int64_t)1 << 31))
        return host_fail(PA_ERR_UNSUPPORTED, "batch * q_len * num_q_heads must be below 2^31");
    if (sh->num_sms <= 0 || sh->num_sms > 4096)
        return host_fail(PA_ERR_INVALID_ARG, "num_sms must be in [1, 4096] (got %d)", sh->num_sms);
    pa_status st = check_row(sh->latent_dim, sh->rope_dim, sh->dtype);
    if (st == PA_OK) st = check_pages(sh->page_size, sh->max_pages_per_seq, sh->num_pool_pages);
    if (st == PA_OK && (int64_t)sh->batch * ((int64_t)sh->max_pages_per_seq + 16) >= ((int64_t)1 << 31))
        return host_fail(PA_ERR_UNSUPPORTED, "batch * (max_pages_per_seq + 16) must be below 2^31");
    if (st == PA_OK && (int64_t)sh->num_pool_pages * pa::kPage >= ((int64_t)1 << 31))
        return host_fail(PA_ERR_UNSUPPORTED, "pool rows (pages * 64) must be below 2^31");
    return st;
}

// ------------------------------------------------------------ cache rows

pa_status fill_cache(const pa_mla_cache_shapes* sh, const int32_t* cu_seqlens, const int32_t* start_pos,
                     const int32_t* block_table, const void* pool, void* workspace, size_t workspace_bytes,
                     pa::MlaCacheArgs* a) {
    pa_status st = check_row(sh->latent_dim, sh->rope_dim, sh->dtype);
    if (st == PA_OK) st = check_pages(sh->page_size, sh->max_pages_per_seq, sh->num_pool_pages);
    if (st != PA_OK) return st;
    if (!cu_seqlens || !start_pos || !block_table || !pool) return host_fail(PA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned16(pool)) return host_fail(PA_ERR_INVALID_ARG, "the pool must be 16-byte aligned");
    st = check_workspace(workspace, workspace_bytes, PA_STATUS_BYTES);
    if (st != PA_OK) return st;
    std::memset(a, 0, sizeof *a);
    a->cu = cu_seqlens;
    a->start_pos = start_pos;
    a->block_table = block_table;
    a->pool = static_cast<uint16_t*>(const_cast<void*>(pool));
    a->status = static_cast<int*>(workspace);
    a->batch = sh->batch;
    a->max_pages = sh->max_pages_per_seq;
    a->num_pool_pages = sh->num_pool_pages;
    a->total = sh->total_new;
    a->f16 = sh->dtype == PA_KV_FP16;
    return PA_OK;
}

pa_status check_cache_sizes(const pa_mla_cache_shapes* sh) {
    if (!sh) return host_fail(PA_ERR_INVALID_ARG, "shapes must not be NULL");
    if (sh->batch < 0 || sh->total_new < 0) return host_fail(PA_ERR_INVALID_ARG, "batch and total_new must be >= 0");
    if (sh->total_new > 0x7FFFFFFF - 64) return host_fail(PA_ERR_UNSUPPORTED, "total_new above 2^31 - 65");
    return PA_OK;
}

// ------------------------------------------------------------ products

// Checks of both products; fills `a` and the maps of the input and the weights.
// in_row, out_row: a head's elements of the input and the output; in_tokens:
// loaded by one copy.
pa_status fill_project(const pa_mla_project_shapes* sh, int in_row, int out_row, uint32_t in_tokens, const void* in,
                       const void* w, void* out, void* workspace, size_t workspace_bytes, pa::MlaProjectArgs* a, CUtensorMap* maps) {
    pa_status st = check_row(sh->latent_dim, sh->rope_dim, sh->dtype);
    if (st != PA_OK) return st;
    if (sh->head_dim != pa::kMlaNope) return host_fail(PA_ERR_UNSUPPORTED, "head_dim must be 128 (got %d)", sh->head_dim);
    if (sh->num_heads <= 0 || sh->num_heads > 65535)
        return host_fail(PA_ERR_INVALID_ARG, "num_heads must be in [1, 65535] (got %d)", sh->num_heads);
    if ((int64_t)sh->num_heads * (((int64_t)sh->total_tokens + 127) / 128) >= ((int64_t)1 << 28))
        return host_fail(PA_ERR_UNSUPPORTED, "num_heads * total_tokens / 128 must be below 2^28");
    if (sh->total_tokens > 65535 * 128) return host_fail(PA_ERR_UNSUPPORTED, "total_tokens above 65535 * 128");
    st = check_stride(sh->in_stride, (int64_t)sh->num_heads * in_row, "in_stride");
    if (st == PA_OK) st = check_stride(sh->out_stride, (int64_t)sh->num_heads * out_row, "out_stride");
    if (st == PA_OK) st = check_stride(sh->w_stride, 128 * pa::kMlaLatent, "w_stride");
    if (st != PA_OK) return st;
    if (!in || !w || !out) return host_fail(PA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned16(in) || !aligned16(w) || !aligned16(out))
        return host_fail(PA_ERR_INVALID_ARG, "input, weights and output must be 16-byte aligned");
    st = check_workspace(workspace, workspace_bytes, PA_STATUS_BYTES);
    if (st != PA_OK) return st;
    std::memset(a, 0, sizeof *a);
    a->in = static_cast<const uint16_t*>(in);
    a->out = static_cast<uint16_t*>(out);
    a->status = static_cast<int*>(workspace);
    a->in_stride = sh->in_stride;
    a->out_stride = sh->out_stride;
    a->total = sh->total_tokens;
    a->heads = sh->num_heads;
    a->interleaved = sh->interleaved != 0;
    a->max_position = sh->max_position;
    a->f16 = sh->dtype == PA_KV_FP16;
    a->wait_ns = pa::host_wait_limit_ns();
    const uint64_t heads = (uint64_t)sh->num_heads;
    const uint64_t id[3] = {(uint64_t)in_row, heads, (uint64_t)sh->total_tokens};
    const uint64_t is[2] = {(uint64_t)in_row * 2, (uint64_t)sh->in_stride * 2};
    const uint32_t ib[3] = {64, 1, in_tokens};
    const uint64_t wd[3] = {(uint64_t)pa::kMlaLatent, 128, heads};
    const uint64_t ws[2] = {(uint64_t)pa::kMlaLatent * 2, (uint64_t)sh->w_stride * 2};
    const uint32_t wb[3] = {64, 128, 1};
    st = pa::host_map_16(a->f16, &maps[0], in, 3, id, is, ib);
    if (st == PA_OK) st = pa::host_map_16(a->f16, &maps[1], w, 3, wd, ws, wb);
    return st;
}

}  // namespace

extern "C" {

size_t pa_mla_decode_workspace_size(const pa_mla_decode_shapes* sh) {
    if (!sh || sh->num_sms <= 0) return PA_STATUS_BYTES;
    const int ctas = decode_ctas(sh);
    return part_offset(ctas) + (size_t)2 * ctas * pa::kMlaBlockRows * pa::kMlaLatent * 4;
}

pa_status pa_mla_decode(const pa_mla_decode_shapes* sh, const void* q, const void* pool, const int32_t* block_table,
                        const int32_t* seq_lens, float scale, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
    pa::NvtxRange nvtx_range("pa_mla_decode");
    pa_status st = check_decode_shapes(sh);
    if (st != PA_OK || sh->batch == 0) return st;
    if (!q || !pool || !block_table || !seq_lens || !out) return host_fail(PA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned16(q) || !aligned16(pool) || !aligned16(out))
        return host_fail(PA_ERR_INVALID_ARG, "q, the pool and out must be 16-byte aligned");
    if (!std::isfinite(scale)) return host_fail(PA_ERR_INVALID_ARG, "scale must be finite");
    st = check_workspace(workspace, workspace_bytes, pa_mla_decode_workspace_size(sh));
    if (st != PA_OK) return st;
    pa::MlaDecodeArgs a;
    std::memset(&a, 0, sizeof a);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int ctas = decode_ctas(sh);
    a.pool = static_cast<const uint8_t*>(pool);
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.merges = reinterpret_cast<pa::MlaMerge*>(ws + merges_offset());
    a.ref_part = reinterpret_cast<float*>(ws + ref_offset(ctas));
    a.sum_part = reinterpret_cast<float*>(ws + sum_offset(ctas));
    a.o_part = reinterpret_cast<float*>(ws + part_offset(ctas));
    a.status = static_cast<int*>(workspace);
    a.batch = sh->batch;
    a.q_len = sh->q_len;
    a.num_heads = sh->num_q_heads;
    a.rows = sh->q_len * sh->num_q_heads;
    a.max_pages = sh->max_pages_per_seq;
    a.num_pool_pages = sh->num_pool_pages;
    a.f16 = sh->dtype == PA_KV_FP16;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.wait_ns = pa::host_wait_limit_ns();
    CUtensorMap maps[3];
    const uint64_t strides[2] = {pa::kMlaRow * 2, 128};
    const uint64_t qd[3] = {64, (uint64_t)sh->batch * a.rows, pa::kMlaRow / 64};
    const uint64_t kd[3] = {64, (uint64_t)sh->num_pool_pages * pa::kPage, pa::kMlaRow / 64};
    const uint32_t qbox[3] = {64, (uint32_t)pa::mla_block_rows(a.rows), pa::kMlaRow / 64};
    const uint32_t latent[3] = {64, pa::kPage, 2}, rope[3] = {64, pa::kPage, 1};
    st = pa::host_map_16(a.f16, &maps[0], q, 3, qd, strides, qbox);
    if (st == PA_OK) st = pa::host_map_16(a.f16, &maps[1], pool, 3, kd, strides, latent);
    if (st == PA_OK) st = pa::host_map_16(a.f16, &maps[2], pool, 3, kd, strides, rope);
    if (st != PA_OK) return st;
    return launched(pa::launch_mla_decode(a, sh->num_sms, maps, stream), "latent decode launch");
}

pa_status pa_mla_append_kv(const pa_mla_cache_shapes* sh, const void* kv_new, const void* weight,
                           const int32_t* positions, const float* cos_sin, const int32_t* cu_seqlens_new,
                           const int32_t* start_pos, const int32_t* block_table, void* pool, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
    pa::NvtxRange nvtx_range("pa_mla_append_kv");
    pa_status st = check_cache_sizes(sh);
    if (st != PA_OK || sh->batch == 0 || sh->total_new == 0) return st;
    pa::MlaCacheArgs a;
    st = fill_cache(sh, cu_seqlens_new, start_pos, block_table, pool, workspace, workspace_bytes, &a);
    if (st == PA_OK) st = check_stride(sh->kv_stride, pa::kMlaRow, "kv_stride");
    if (st != PA_OK) return st;
    if (!kv_new) return host_fail(PA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned16(kv_new) || !aligned16(weight) || !aligned16(cos_sin))
        return host_fail(PA_ERR_INVALID_ARG, "kv_new, weight and cos_sin must be 16-byte aligned");
    if (sh->norm != 0 && sh->norm != 1) return host_fail(PA_ERR_INVALID_ARG, "norm must be 0 or 1 (got %d)", sh->norm);
    if (sh->norm && !(std::isfinite(sh->eps) && sh->eps >= 0.f))
        return host_fail(PA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (cos_sin && sh->max_position <= 0) return host_fail(PA_ERR_INVALID_ARG, "max_position must be positive");
    a.kv = static_cast<const uint16_t*>(kv_new);
    a.weight = static_cast<const uint16_t*>(weight);
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.kv_stride = sh->kv_stride;
    a.interleaved = sh->interleaved != 0;
    a.max_position = sh->max_position;
    a.norm = sh->norm;
    a.eps = sh->eps;
    return launched(pa::launch_mla_append(a, stream), "latent append launch");
}

pa_status pa_mla_gather_kv(const pa_mla_cache_shapes* sh, const void* pool, const int32_t* cu_seqlens,
                           const int32_t* start_pos, const int32_t* block_table, void* latent_out, void* rope_out,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    pa::NvtxRange nvtx_range("pa_mla_gather_kv");
    pa_status st = check_cache_sizes(sh);
    if (st != PA_OK || sh->batch == 0 || sh->total_new == 0) return st;
    pa::MlaCacheArgs a;
    st = fill_cache(sh, cu_seqlens, start_pos, block_table, pool, workspace, workspace_bytes, &a);
    if (st != PA_OK) return st;
    if (!latent_out || !rope_out) return host_fail(PA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned16(latent_out) || !aligned16(rope_out))
        return host_fail(PA_ERR_INVALID_ARG, "the outputs must be 16-byte aligned");
    a.latent_out = static_cast<uint16_t*>(latent_out);
    a.rope_out = static_cast<uint16_t*>(rope_out);
    return launched(pa::launch_mla_gather(a, stream), "latent gather launch");
}

pa_status pa_mla_query(const pa_mla_project_shapes* sh, const void* q, const void* w_uk, const int32_t* positions,
                       const float* cos_sin, void* q_out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    pa::NvtxRange nvtx_range("pa_mla_query");
    if (!sh) return host_fail(PA_ERR_INVALID_ARG, "shapes must not be NULL");
    if (sh->total_tokens < 0) return host_fail(PA_ERR_INVALID_ARG, "total_tokens must be >= 0");
    if (sh->total_tokens == 0) return PA_OK;
    if (cos_sin && !positions) return host_fail(PA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (cos_sin && sh->max_position <= 0) return host_fail(PA_ERR_INVALID_ARG, "max_position must be positive");
    if (!aligned16(cos_sin)) return host_fail(PA_ERR_INVALID_ARG, "cos_sin must be 16-byte aligned");
    pa::MlaProjectArgs a;
    CUtensorMap maps[3];
    pa_status st = fill_project(sh, pa::kMlaNope + pa::kMlaRope, pa::kMlaRow, 128, q, w_uk, q_out, workspace, workspace_bytes,
                                &a, maps);
    const uint64_t od[3] = {(uint64_t)pa::kMlaRow, (uint64_t)sh->num_heads, (uint64_t)sh->total_tokens};
    const uint64_t os[2] = {(uint64_t)pa::kMlaRow * 2, (uint64_t)sh->out_stride * 2};
    const uint32_t ob[3] = {64, 1, 128};
    if (st == PA_OK) st = pa::host_map_16(a.f16, &maps[2], q_out, 3, od, os, ob);
    if (st != PA_OK) return st;
    a.positions = positions;
    a.cos_sin = cos_sin;
    return launched(pa::launch_mla_query(a, maps, stream), "latent query launch");
}

pa_status pa_mla_output(const pa_mla_project_shapes* sh, const void* o, const void* w_uv, void* out, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
    pa::NvtxRange nvtx_range("pa_mla_output");
    if (!sh) return host_fail(PA_ERR_INVALID_ARG, "shapes must not be NULL");
    if (sh->total_tokens < 0) return host_fail(PA_ERR_INVALID_ARG, "total_tokens must be >= 0");
    if (sh->total_tokens == 0) return PA_OK;
    pa::MlaProjectArgs a;
    CUtensorMap maps[2];
    pa_status st = fill_project(sh, pa::kMlaLatent, pa::kMlaValue, pa::kMlaOutputGroup, o, w_uv, out, workspace, workspace_bytes, &a, maps);
    if (st != PA_OK) return st;
    return launched(pa::launch_mla_output(a, maps, stream), "latent output launch");
}

}  // extern "C"
