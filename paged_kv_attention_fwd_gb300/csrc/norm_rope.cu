// norm_rope.cu -- RMS norm of every query and key head, then the rotary
// rotation, in one pass over the projections (pa_qk_norm_rope), optionally
// with the keys and values going straight into their cache pages
// (pa_norm_rope_append_kv).
//
//   y = x * rsqrt(mean_i x_i^2 + eps) * w             (fp32)
//   (a, b) -> (a cos - b sin, b cos + a sin)          (first rope_dim elements)
//
// with one rounding to 16 bits at the end.  HBM-bound: 2 bytes in, 2 out per
// element and a table row per token; what it must not be is issue-bound.  So
// a head row is held by D / 8 lanes, 8 elements each, in two groups of 4 that
// pair up with one another (the rotation needs no shuffle in either pairing);
// a warp takes 32 / (D / 8) tokens and kPasses heads of one kind (queries, keys
// or values) at a time, with the weights multiplied into the cosines and sines,
//   a' = inv (a (w_a cos) - b (w_b sin)),  b' = inv (b (w_b cos) + a (w_a sin)),
// the arithmetic runs on pairs of fp32 (f32x2), and a warp goes on to the next
// such chunk with its elements and angles already on the way.  The warps are as
// many as the SMs hold, with equal shares: 4097 tokens, 16 + 4 heads of 64, 4.9
// us, where whole multiples of the largest share, in fewer warps, took 5.9.
//
// Several tokens, not more heads, fill the lanes: a kind may have one head only.
// One token at a time, 65536 tokens of 8 + 1 heads took 72 us (59 now), of 3 + 3
// heads of 64 68 us (22.5).
//
// Measured: 16384 tokens, 64 + 8 heads of 128 (613 MB), 96.7 us a call, 6.3
// TB/s; the append form, 8 x 512 tokens, 32 + 8 + 8 heads, 21.5 us with 16-bit
// pages (103 MB), 22.3 with e4m3 ones, 20.5 with 4-bit ones; one token 3 us, a
// launch.  Against 97 and 22 us, 3 CTAs an SM took 106 and 23.4, 5 104 and 26.7,
// 2 passes and 6 CTAs 114 and 25.8.  Rows through a ring of bulk copies in
// shared memory, 3 or 4 deep, were no faster: the loads in flight are not what
// bounds it.
#include "cache4.cuh"
#include "f32x2.cuh"
#include "pa_launch.h"
#include "token_place.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kCtas = 4;    // CTAs of an SM
constexpr int kPasses = 4;  // heads of a chunk: rows of a lane whose loads are in flight together

// Whether a warp goes from one chunk of its tokens to the next (else from some
// tokens to the next with the same chunk).  With a cache the kinds differ in
// work, keys and values that are quantised taking longest, and each warp needs
// its share of all: 8 x 512 tokens, 32 + 8 + 8 heads, 21.5 us against 21.7 with
// 16-bit pages, 22.3 against 31.4 with e4m3 ones, 20.5 against 25.7 with 4-bit
// ones.  Without, one chunk keeps its weights: 16384 tokens 96.7 us against 98.4.
constexpr bool walks_chunks(int cache) { return cache >= 0; }

__device__ __forceinline__ float2 unpack16(uint32_t w, bool f16) {
    if (f16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack16(F2 a, bool f16) {
    const float2 v = split(a);
    if (f16) {
        const __half2 h = __floats2half2_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight e4m3 codes of x / scale, the bits that pa_append_kv stores: fp32
// quotients (nearest even), then nearest even, saturating.  Away from the ends
// of fp32 the quotient is the correctly rounded reciprocal's with one residual
// step, as for 4-bit codes, q' = q + (x - q scale) r: the residual is exact for
// every quotient that does not round to code 0 either way.  It is taken of -q,
// whose steps leave a zero of x its sign.
__device__ __forceinline__ uint2 e4m3x8(uint2 w0, uint2 w1, float scale) {
    const uint32_t u[4] = {w0.x, w0.y, w1.x, w1.y};
    const uint32_t m2 = absmax_bf16x2(absmax_bf16x2(u[0], u[1]), absmax_bf16x2(u[2], u[3]));
    const float largest = __uint_as_float((absmax_bf16x2(m2, m2 >> 16) & 0x7FFFu) << 16);
    uint32_t c[4];
    if (largest < 1e15f && fabsf(scale) > 1e-15f && fabsf(scale) < 1e15f) {
        const float r1 = __frcp_rn(scale);
        const F2 minus_r = f2(-r1, -r1), s = f2(scale, scale);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 x = f2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u)), q = x * minus_r;
            c[i] = __nv_cvt_float2_to_fp8x2(split(fma2(fma2(q, s, x), minus_r, q)), __NV_SATFINITE, __NV_E4M3) ^ 0x8080u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(__uint_as_float(u[i] << 16), scale),
                                                        __fdiv_rn(__uint_as_float(u[i] & 0xFFFF0000u), scale)),
                                            __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The four cos and sin a lane needs: pairs pair0 .. pair0 + 3, whose positions
// may belong to different axes.
struct Angles {
    float c[4], s[4];
};
__device__ __forceinline__ void load_angles(const NormRopeArgs& a, const int (&pos)[3], int pair0, Angles& to) {
    const int half = a.rope_dim / 2;
    const int e0 = a.sections[0], e1 = e0 + a.sections[1];
    auto axis = [&](int p) { return p < e0 ? pos[0] : p < e1 ? pos[1] : pos[2]; };
    const int first = axis(pair0);
    if (a.num_axes == 1 || (axis(pair0 + 1) == first && axis(pair0 + 2) == first && axis(pair0 + 3) == first)) {
        const float* t = a.cos_sin + (long long)first * a.rope_dim + pair0;
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(t)), s4 = __ldg(reinterpret_cast<const float4*>(t + half));
        to.c[0] = c4.x; to.c[1] = c4.y; to.c[2] = c4.z; to.c[3] = c4.w;
        to.s[0] = s4.x; to.s[1] = s4.y; to.s[2] = s4.z; to.s[3] = s4.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* t = a.cos_sin + (long long)axis(pair0 + i) * a.rope_dim + pair0 + i;
            to.c[i] = __ldg(t);
            to.s[i] = __ldg(t + half);
        }
    }
}

// kCache: -1 keys to k_out, else the page type they (and the values) go to
template <int D, bool kInterleaved, int kCache, bool kF16>
__global__ void __launch_bounds__(kWarps * 32, kCtas) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
    grid_dependency_wait();
    allow_dependents_launch();
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    constexpr bool kAppend = kCache >= 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % kLanes;
    // The heads of one kind -- queries, keys, values -- come in chunks of kPasses, tokens in groups of kRows; lanes of one
    // sub hold the rows of one token
    const int sub = lane / kLanes, last_token = a.total_tokens - 1;
    const int qchunks = (a.num_q_heads + kPasses - 1) / kPasses, kchunks = (a.num_kv_heads + kPasses - 1) / kPasses;
    const int chunks = qchunks + (kAppend ? 2 : 1) * kchunks;
    // This warp's share: a.share (the first a.longer warps one more) of the chunks of all groups, or of the groups
    const int id = (int)blockIdx.x * kWarps + warp;
    if (id >= a.warps) return;
    const int nth = walks_chunks(kCache) ? id : id / chunks;
    const long long from = (long long)nth * a.share + min(nth, a.longer);
    const int share = a.share + (nth < a.longer);
    const int first = !walks_chunks(kCache) ? (int)from : from <= 0x7FFFFFFF ? (int)from / chunks : (int)(from / chunks);
    auto kind_of = [&](int c) { return c < qchunks ? 0 : c < qchunks + kchunks ? 1 : 2; };
    auto first_head_of = [&](int c) { return (c < qchunks ? c : c < qchunks + kchunks ? c - qchunks : c - qchunks - kchunks) * kPasses; };
    auto heads_of = [&](int c) { return c < qchunks ? a.num_q_heads : a.num_kv_heads; };

    // where this lane's two groups of 4 elements lie in a row, and whether they turn
    const int half = a.rope_dim / 2;
    const bool turns = kInterleaved ? 8 * l < a.rope_dim : 4 * l < half;
    const int off0 = kInterleaved ? 8 * l : 4 * l < half ? 4 * l : a.rope_dim + 8 * (l - half / 4);
    const int off1 = kInterleaved || 4 * l >= half ? off0 + 4 : half + 4 * l;

    struct Rows {
        uint2 x[kPasses][2];
    };
    // 4-bit pages: a row has kBlocks blocks of 16 elements, and the chunk's rows kPasses / 2 for every lane, of the token
    // block_sub and the heads block_head and that plus 2.  Values are loaded that way, keys get there through shared
    // memory.
    constexpr bool kFp4 = kCache == PA_KV_FP4_E2M1;
    constexpr int kBlocks = D / 16;
    static_assert(kPasses % 2 == 0, "a lane holds kPasses / 2 blocks");
    __shared__ __align__(16) uint16_t stage[kFp4 ? kWarps : 1][kFp4 ? kPasses * kRows * D : 8];
    const bool wide_v = kFp4 && aligned32(a.v) && a.v_stride % 16 == 0;
    const int block_sub = lane / kBlocks % kRows, block_head = lane / 16, piece = lane % kBlocks;
    auto load_rows = [&](Rows& to, int tok, int chunk) {
        const int kind = kind_of(chunk), first_head = first_head_of(chunk), last_head = heads_of(chunk) - 1;
        if constexpr (kFp4) {
            if (kind == 2) {
                const uint16_t* src = a.v + min(tok + block_sub, last_token) * a.v_stride + piece * 16;
#pragma unroll
                for (int p = 0; p < kPasses; p += 2) {
                    const Sector s = load_sector(src + min(first_head + p + block_head, last_head) * D, wide_v);
                    to.x[p][0] = make_uint2(s.lo.x, s.lo.y);
                    to.x[p][1] = make_uint2(s.lo.z, s.lo.w);
                    to.x[p + 1][0] = make_uint2(s.hi.x, s.hi.y);
                    to.x[p + 1][1] = make_uint2(s.hi.z, s.hi.w);
                }
                return;
            }
        }
        const int mine = min(tok + sub, last_token);  // past the last token or head: that one again
        const uint16_t* src = kind == 0 ? a.q + mine * a.q_stride : kind == 1 ? a.k + mine * a.k_stride : a.v + mine * a.v_stride;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const uint16_t* row = src + min(first_head + p, last_head) * D;
            if constexpr (kInterleaved) {
                const uint4 w = *reinterpret_cast<const uint4*>(row + off0);
                to.x[p][0] = make_uint2(w.x, w.y);
                to.x[p][1] = make_uint2(w.z, w.w);
            } else {
                to.x[p][0] = *reinterpret_cast<const uint2*>(row + off0);
                to.x[p][1] = *reinterpret_cast<const uint2*>(row + off1);
            }
        }
    };
    struct Pos {
        int at[3];
    };
    const bool by_place = kAppend && a.positions == nullptr;  // positions are those in the cache
    auto load_pos = [&](Pos& to, int tok) {
        if (a.rope_dim == 0 || by_place) return;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < a.num_axes) to.at[i] = __ldg(&a.positions[(long long)i * a.total_tokens + min(tok + sub, last_token)]);
    };
    struct Where {  // a token's place in the cache
        int page, row;
        Place place;
    };
    // Tokens come in order: the sequence is searched for where it changes, its block table read where the page does.
    Sequence seq{-1, 0, 0};
    int seq_end = 0;  // the first token that is not seq's
    auto find_place = [&](Where& to, Pos& pos, int tok) {
        const int mine = tok + sub;
        const bool search = __any_sync(0xffffffffu, mine >= seq_end);
        if (search) {
            seq = warp_sequences<kRows>(tok, sub, a.cu_new, a.start_pos, a.batch);
            seq_end = seq.b >= a.batch ? 0x7FFFFFFF : seq.b < 0 ? mine + 1 : __ldg(&a.cu_new[seq.b + 1]);
        }
        long long cpos = (long long)seq.start + (mine - seq.cu);
        if (search || to.place != Place::kOk || to.row + kRows >= kPage)
            to.place = token_place(mine, seq, a.block_table, a.batch, a.max_pages, a.num_pool_pages, to.page, to.row, cpos);
        else
            to.row += kRows;
        if (by_place) {
            const int p = to.place == Place::kOk ? (int)min(cpos, (long long)a.max_position) : 0;
            pos.at[0] = pos.at[1] = pos.at[2] = p;
        }
    };
    // angles of a token whose positions are known; false where one is outside the table
    auto start_angles = [&](Angles& to, const Pos& pos) {
        if (a.rope_dim == 0) return true;
        bool ok = true;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < a.num_axes) ok &= (unsigned)pos.at[i] < (unsigned)a.max_position;
        if (ok && turns) load_angles(a, pos.at, 4 * l, to);
        return ok;
    };

    Rows rows;
    Pos pos{{0, 0, 0}}, pos1{{0, 0, 0}};
    Angles ang{{1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}};
    Where where{0, 0, Place::kOk};
    int tok = first * kRows;  // the group's first token
    int chunk = walks_chunks(kCache) ? (int)(from - (long long)first * chunks) : id - nth * chunks;
    load_rows(rows, tok, chunk);
    load_pos(pos, tok);
    load_pos(pos1, tok + kRows);
    const uint32_t one = kF16 ? 0x3C003C00u : 0x3F803F80u;
    uint2 wq[2] = {{one, one}, {one, one}}, wk[2] = {{one, one}, {one, one}};
    auto load_weight = [&](uint2 (&to)[2], const uint16_t* from) {
        if (!a.norm || from == nullptr) return;
        to[0] = __ldg(reinterpret_cast<const uint2*>(from + off0));
        to[1] = __ldg(reinterpret_cast<const uint2*>(from + off1));
    };
    if (walks_chunks(kCache)) {
        load_weight(wq, a.q_weight);
        load_weight(wk, a.k_weight);
    } else {
        load_weight(wq, kind_of(chunk) == 0 ? a.q_weight : a.k_weight);
    }
    if constexpr (kAppend) {
        if (by_place) find_place(where, pos, tok);
    }
    bool in_table = start_angles(ang, pos);
    if constexpr (kAppend) {
        if (!by_place) find_place(where, pos, tok);
    }

#pragma unroll 1
    for (int left = share;; --left) {
        const int kind = kind_of(chunk), first_head = first_head_of(chunk), heads = heads_of(chunk);
        const int my_tok = tok + sub;
        // y = inv (x c1 + partner c2): elements 01, 23, 45, 67 of the lane
        F2 c1[4], c2[4];
        {
            const bool second = walks_chunks(kCache) && kind != 0;
            const uint2 w0 = second ? wk[0] : wq[0], w1 = second ? wk[1] : wq[1];
            const float2 p0 = unpack16(w0.x, kF16), p1 = unpack16(w0.y, kF16), p2 = unpack16(w1.x, kF16), p3 = unpack16(w1.y, kF16);
            const float w[8] = {p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kInterleaved) {
                    c1[i] = f2(w[2 * i] * ang.c[i], w[2 * i + 1] * ang.c[i]);
                    c2[i] = f2(-w[2 * i + 1] * ang.s[i], w[2 * i] * ang.s[i]);
                } else {
                    const int e = 2 * (i & 1), n = 2 * i, m = (n + 4) & 7;  // pairs e, e + 1; elements n, n + 1; partners m, m + 1
                    const float sg = i < 2 ? -1.f : 1.f;
                    c1[i] = f2(w[n] * ang.c[e], w[n + 1] * ang.c[e + 1]);
                    c2[i] = f2(sg * w[m] * ang.s[e], sg * w[m + 1] * ang.s[e + 1]);
                }
            }
        }
        // a padding token (a negative given position makes it one wherever it lies), or one that is out of range:
        // nothing is written
        const bool padding = my_tok > last_token || where.place == Place::kPadding || (a.rope_dim > 0 && pos.at[0] < 0);
        const bool skip = padding || where.place != Place::kOk || !in_table;
        if (skip && !padding && l == 0) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
        const int page = where.page, prow = where.row;
        const Rows now = rows;
        const bool new_tokens = !walks_chunks(kCache) || ++chunk == chunks;
        if (new_tokens) {
            if (walks_chunks(kCache)) chunk = 0;
            tok += kRows;
        }
        const bool more = left > 1;
        if (more) {  // the next chunk's loads
            load_rows(rows, tok, chunk);
            if (new_tokens) {
                pos = pos1;
                if constexpr (kAppend) find_place(where, pos, tok);
                in_table = start_angles(ang, pos);
                load_pos(pos1, tok + kRows);
            }
        }
        if (__all_sync(0xffffffffu, skip)) {
            if (!more) return;
            continue;
        }

        // all passes of a stage side by side: their chains of dependent steps overlap
        Rows out = now;
        if (kind != 2) {  // values pass through bit for bit
            F2 y[kPasses][4];
            float inv[kPasses];
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                const uint32_t u[4] = {now.x[p][0].x, now.x[p][0].y, now.x[p][1].x, now.x[p][1].y};
                F2 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = unpack16(u[i], kF16);
                    f[i] = f2(v.x, v.y);
                }
                const float2 sq = split(fma2(f[3], f[3], fma2(f[2], f[2], fma2(f[1], f[1], f[0] * f[0]))));
                inv[p] = sq.x + sq.y;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[p][i] = f[i] * c1[i];
                if (turns) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[p][i] = fma2(kInterleaved ? swapped(f[i]) : f[(i + 2) & 3], c2[i], y[p][i]);
                }
            }
            if (a.norm) {
#pragma unroll
                for (int o = kLanes / 2; o >= 1; o >>= 1)
#pragma unroll
                    for (int p = 0; p < kPasses; ++p) inv[p] += __shfl_xor_sync(0xffffffffu, inv[p], o);
#pragma unroll
                for (int p = 0; p < kPasses; ++p) {
                    asm("rsqrt.approx.f32 %0, %1;" : "=f"(inv[p]) : "f"(fmaf(inv[p], 1.f / D, a.eps)));
                    const F2 inv2 = f2(inv[p], inv[p]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[p][i] = y[p][i] * inv2;
                }
            }
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                out.x[p][0] = make_uint2(pack16(y[p][0], kF16), pack16(y[p][1], kF16));
                out.x[p][1] = make_uint2(pack16(y[p][2], kF16), pack16(y[p][3], kF16));
            }
        }
        if constexpr (kFp4) {
            if (kind != 0) {
                uint16_t* st = stage[warp];
                if (kind == 1) {
#pragma unroll
                    for (int p = 0; p < kPasses; ++p) {
                        uint16_t* row = st + (p * kRows + sub) * D;
                        *reinterpret_cast<uint2*>(row + off0) = out.x[p][0];
                        *reinterpret_cast<uint2*>(row + off1) = out.x[p][1];
                    }
                    __syncwarp();
                }
                uint8_t* pool = static_cast<uint8_t*>(kind == 2 ? a.v_pool : a.k_pool);
                const float* scales = kind == 2 ? a.v_scale : a.k_scale;
                const int block_page = __shfl_sync(0xffffffffu, skip ? -1 : page, block_sub * kLanes);
                const int block_row = __shfl_sync(0xffffffffu, prow, block_sub * kLanes);
#pragma unroll
                for (int p = 0; p < kPasses; p += 2) {
                    const int h = first_head + p + block_head;
                    uint4 lo = make_uint4(out.x[p][0].x, out.x[p][0].y, out.x[p][1].x, out.x[p][1].y);
                    uint4 hi = make_uint4(out.x[p + 1][0].x, out.x[p + 1][0].y, out.x[p + 1][1].x, out.x[p + 1][1].y);
                    if (kind == 1) {
                        const uint4* w = reinterpret_cast<const uint4*>(st + (16 * p + lane) * 16);
                        lo = w[0];
                        hi = w[1];
                    }
                    if (h < heads && block_page >= 0)
                        fp4_store_block<D>(pool + ((long long)block_page * a.num_kv_heads + h) * fp4_slab_bytes(D), block_row,
                                           piece, lo, hi, __ldg(&scales[h]));
                }
                __syncwarp();  // the stage is free again
                if (!more) return;
                continue;
            }
        }
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int r = first_head + p;
            const bool mine = r < heads && !skip;
            const uint2 y0 = out.x[p][0], y1 = out.x[p][1];
            uint16_t* dst = nullptr;  // a 16-bit destination row
            if (kind == 0) dst = a.q_out + my_tok * a.q_out_stride + (long long)r * D;
            else if constexpr (!kAppend) dst = a.k_out + my_tok * a.k_out_stride + (long long)r * D;
            if constexpr (kAppend && !kFp4) {
                if (kind != 0) {
                    const long long slab = (long long)page * a.num_kv_heads + r;
                    uint8_t* pool = static_cast<uint8_t*>(kind == 2 ? a.v_pool : a.k_pool);
                    if constexpr (kCache == PA_KV_BF16) {  // either 16-bit type
                        dst = reinterpret_cast<uint16_t*>(pool) + (slab * kPage + prow) * D;
                    } else if (mine) {
                        uint8_t* to = pool + (slab * kPage + prow) * D;
                        const uint2 codes = e4m3x8(y0, y1, __ldg(&(kind == 2 ? a.v_scale : a.k_scale)[r]));
                        *reinterpret_cast<uint32_t*>(to + off0) = codes.x;
                        *reinterpret_cast<uint32_t*>(to + off1) = codes.y;
                    }
                }
            }
            if (dst != nullptr && mine) {
                if constexpr (kInterleaved) {
                    *reinterpret_cast<uint4*>(dst + off0) = make_uint4(y0.x, y0.y, y1.x, y1.y);
                } else {
                    *reinterpret_cast<uint2*>(dst + off0) = y0;
                    *reinterpret_cast<uint2*>(dst + off1) = y1;
                }
            }
        }
        if (!more) return;
    }
}

template <int D, bool kInterleaved, int kCache, bool kF16>
cudaError_t launch(NormRopeArgs a, cudaStream_t stream) {
    constexpr int kRows = 32 / (D / 8);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long chunks = (a.num_q_heads + kPasses - 1) / kPasses + (kCache >= 0 ? 2 : 1) * ((a.num_kv_heads + kPasses - 1) / kPasses);
    const long long groups = (a.total_tokens - 1) / kRows + 1;
    // As many warps as stay on the SMs, their shares as equal as can be
    const long long resident = (long long)sms * kCtas * kWarps;
    const long long columns = walks_chunks(kCache) ? 1 : chunks, all = walks_chunks(kCache) ? groups * chunks : groups;
    const long long sharers = min(all, max(resident / columns, 1ll));
    a.warps = (int)(sharers * columns);
    a.share = (int)(all / sharers);
    a.longer = (int)(all % sharers);
    return launch_overlapped(norm_rope_kernel<D, kInterleaved, kCache, kF16>, dim3((unsigned)((a.warps + kWarps - 1) / kWarps)),
                             dim3(kWarps * 32), 0, stream, a);
}

template <int D, int kCache>
cudaError_t launch_pairing(const NormRopeArgs& a, cudaStream_t stream) {
    if constexpr (kCache <= PA_KV_BF16) {  // the other page types take bf16 tokens only
        if (a.f16) return a.interleaved ? launch<D, true, kCache, true>(a, stream) : launch<D, false, kCache, true>(a, stream);
    }
    return a.interleaved ? launch<D, true, kCache, false>(a, stream) : launch<D, false, kCache, false>(a, stream);
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
