// mla_decode.cu -- attention of one or a few new tokens a sequence over a paged
// cache of latent rows (pa_mla_decode):
//
//   s_j = scale <q, row_j>          over the row's 576 elements
//   out = sum_j softmax_j(s) row_j  over its first 512
//   lse = ln sum_j exp(s_j)
//
// Every head of a sequence reads the same rows, so a sequence's (token, head)
// pairs are the rows of one product, 128 at a time (a block), and both products
// run on the tensor cores with the heads in M.  A row of 128 x 512 fp32 would
// fill the tensor memory of an SM, and 128 query rows of 576 most of its shared
// memory, so a pair of CTAs shares a block (cta_group::2, M = 128: 64 rows in
// each CTA): S takes 64 columns of each CTA's tensor memory, O 256.  In that
// layout lanes 0-63 hold the first half of a product's columns and lanes 64-127
// the second, for the CTA's 64 rows.
//
//   warp 0     producer (both CTAs): queries, and per 128 keys (two pages) this
//              CTA's page for S = Q K^T and its half of the values' columns, of
//              both pages, for O += P V (from L2 the second time)
//   warp 1     rank 0: the MMA thread of the pair
//   warps 2-5  softmax (both CTAs): two threads a row, each on the 64 keys of
//              one page; P to shared memory, O rescaled when the maximum grows
//              by more than 2^8, output written
//
// The sequences' costs (tiles and a constant) are laid end to end and cut into
// as many equal ranges as there are pairs: a pair takes what lies in its range,
// at most two pieces of which are parts of an item.  Those go to the workspace
// in fp32 and are merged by a second kernel.  Lengths are read on the device
// only.
#include "pa_launch.h"
#include "pa_mla.h"
#include "pa_ptx.cuh"
#include "prefill_common.cuh"

namespace pa {
namespace {

constexpr int kChunks = kMlaRow / 64;      // 64-element chunks of a row: 9, the first 8 of them latent
constexpr int kChunkBytes = 64 * 128;      // 64 rows of a chunk
constexpr int kKStages = 3, kKChunks = 3;  // a K stage: 3 chunks of this CTA's page
constexpr int kKStageBytes = kKChunks * kChunkBytes;
constexpr int kVStages = 2;                // a V stage: 128 columns of both pages
constexpr int kVStageBytes = 4 * kChunkBytes;
constexpr int kQOff = 0;
constexpr int kPOff = kQOff + kChunks * kChunkBytes;
constexpr int kKOff = kPOff + 2 * kChunkBytes;
constexpr int kVOff = kKOff + kKStages * kKStageBytes;
constexpr int kSmem = kVOff + kVStages * kVStageBytes + 1024;
constexpr int kThreads = 192;
constexpr uint32_t kSCols = 64, kOCol = 256, kOCols = 128;
constexpr long long kFixed = 1;     // what an item costs besides its tiles, in tiles
constexpr long long kMinShare = 3;  // a pair's range is at least this long

enum : int {
    B_QF = 0,                   // rank 0: queries landed in both CTAs
    B_QE = 1,                   // both: queries used
    B_KF = 2,                   // [3] rank 0
    B_KE = B_KF + kKStages,     // [3] both
    B_VF = B_KE + kKStages,     // [2] rank 0
    B_VE = B_VF + kVStages,     // [2] both
    B_SF = B_VE + kVStages,     // [2] both: S ready
    B_PF = B_SF + 2,            // rank 0: P written in both CTAs
    B_OD = B_PF + 1,            // both: a tile's PV retired
    B_DONE = B_OD + 1,          // rank 0
    B_COUNT = B_DONE + 1
};

// One stretch of tiles [lo, hi) of item (b, blk) that a pair takes.
struct Piece {
    int b, blk, lo, hi, tiles, len;
    long long at;  // where the item's cost starts
};

__device__ __forceinline__ int clamped_len(const MlaDecodeArgs& a, int b, bool report) {
    const int len = __ldg(&a.seq_lens[b]);
    const long long most = min((long long)a.max_pages * kPage, 0x7FFFFF80ll);
    if (len >= 0 && len <= most) return len;
    if (report) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
    return len < 0 ? 0 : (int)most;
}

struct Walk {
    long long from, to, at;
    int b, blk, blocks;
    __device__ __forceinline__ bool next(const MlaDecodeArgs& a, Piece& p) {
        while (b < a.batch && at < to) {
            p.b = b;
            p.blk = blk;
            p.at = at;
            p.len = clamped_len(a, b, false);
            p.tiles = (p.len + 127) / 128;
            const long long t0 = at + kFixed;
            p.lo = (int)min((long long)p.tiles, max(0ll, from - t0));
            p.hi = (int)min((long long)p.tiles, max(0ll, to - t0));
            const bool mine = p.tiles == 0 ? at >= from : p.hi > p.lo;
            at = t0 + p.tiles;
            if (++blk == blocks) {
                blk = 0;
                ++b;
            }
            if (mine) return true;
        }
        return false;
    }
};

__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t nthreads, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)p), "r"(id), "r"(nthreads)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

template <bool kF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_decode_kernel(const __grid_constant__ MlaDecodeArgs a, const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_kv) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t bars[B_COUNT];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_store;
    __shared__ Walk start_sh;
    __shared__ long long sums[kThreads / 32];
    __shared__ float row_max[2][2][64];  // [tile parity][half of the keys][row]
    __shared__ float row_sum[2][64];
    volatile int* abort_sh = &abort_store;

    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pair = (int)blockIdx.x >> 1;
    auto lead = [&](int i) { return mapa_shared(smem_u32(&bars[i]), 0); };

    if (threadIdx.x == 0) {
        mbar_init(&bars[B_QF], 2);
        mbar_init(&bars[B_QE], 1);
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(&bars[B_KF + s], 2);
            mbar_init(&bars[B_KE + s], 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(&bars[B_VF + s], 2);
            mbar_init(&bars[B_VE + s], 1);
        }
        for (int s = 0; s < 2; ++s) mbar_init(&bars[B_SF + s], 1);
        mbar_init(&bars[B_PF], 8);
        mbar_init(&bars[B_OD], 1);
        mbar_init(&bars[B_DONE], 1);
        *abort_sh = 0;
        start_sh.b = a.batch;
        fence_barrier_init();
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_kv);
    }
    grid_dependency_wait();
    if (warp == 1) {
        tmem_alloc_pair(&tmem_base_sh, 512);
        tmem_relinquish_pair();
    }
    // ---- this pair's range: every thread sums the costs of a run of sequences
    const int blocks = (a.rows + kMlaBlockRows - 1) / kMlaBlockRows;
    {
        const int per = (a.batch + kThreads - 1) / kThreads;
        const int b0 = min((int)threadIdx.x * per, a.batch), b1 = min(b0 + per, a.batch);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += kFixed + (clamped_len(a, b, pair == 0) + 127) / 128;
        mine *= blocks;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        long long before = incl - mine, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += sums[w];
            total += sums[w];
        }
        const long long share = max((total + a.pairs - 1) / a.pairs, kMinShare);
        const long long from = pair * share;
        if (from >= before && from < before + mine) {
            Walk w;
            w.from = from;
            w.to = from + share;
            w.at = before;
            w.b = b0;
            w.blk = 0;
            w.blocks = blocks;
            for (;;) {
                const long long cost = kFixed + (clamped_len(a, w.b, false) + 127) / 128;
                if (from < w.at + cost * blocks) {
                    w.blk = (int)((from - w.at) / cost);
                    w.at += w.blk * cost;
                    break;
                }
                w.at += cost * blocks;
                ++w.b;
            }
            start_sh = w;
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers initialised and TMEM allocated
    tc_fence_after();
    const uint32_t tbase = tmem_base_sh;
    Walk walk = start_sh;
    Piece pc;

    if (warp == 0) {
        // ---------------------------------------------------------------- producer (both CTAs)
        bool ok = true;
        uint32_t items = 0, kst = 0, vst = 0;  // pieces with tiles, K and V stages issued
        while (ok && walk.next(a, pc)) {
            const int n = pc.hi - pc.lo;
            if (n == 0) continue;
            const int block_rows = min(kMlaBlockRows, a.rows - pc.blk * kMlaBlockRows), half = (block_rows + 1) / 2;
            if (items > 0) ok = mbar_wait(&bars[B_QE], (items - 1) & 1, abort_sh, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx_cl(lead(B_QF), kChunks * kChunkBytes);
                const int row = pc.b * a.rows + pc.blk * kMlaBlockRows + (int)rank * half;
                for (int c = 0; c < kChunks; ++c)
                    tma_load_2d_pair(sm + kQOff + c * kChunkBytes, &map_q, lead(B_QF), c * 64, row);
            }
            ++items;
            const int pages = (pc.len + kPage - 1) / kPage;
            int ids = 0;  // page ids of 16 tiles, a lane each
            auto page_rows = [&](int p) { return __shfl_sync(0xffffffffu, ids, (p - 2 * pc.lo) & 31) * kPage; };
            auto fetch_ids = [&](int t) {
                const int p = min(2 * t + lane, pages - 1);  // past the last: that one again, masked
                ids = __ldg(&a.block_table[(long long)pc.b * a.max_pages + p]);
                if ((unsigned)ids >= (unsigned)a.num_pool_pages) {
                    atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
                    ids = 0;
                }
            };
            int vp0 = 0, vp1 = 0;  // rows of the pages of the tile whose V comes next
            for (int t = pc.lo; t <= pc.hi && ok; ++t) {
                int p0 = 0, p1 = 0;
                if (t < pc.hi) {
                    if (((t - pc.lo) & 15) == 0) fetch_ids(t);
                    p0 = page_rows(2 * t);
                    p1 = page_rows(2 * t + 1);
                    for (int s = 0; s < kChunks / kKChunks && ok; ++s, ++kst) {
                        const int slot = kst % kKStages;
                        ok = mbar_wait(&bars[B_KE + slot], ((kst / kKStages) & 1) ^ 1, abort_sh, a.wait_ns);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (lane == 0) {
                            const uint32_t full = lead(B_KF + slot);
                            mbar_arrive_expect_tx_cl(full, kKStageBytes);
                            for (int c = 0; c < kKChunks; ++c)
                                tma_load_2d_pair(sm + kKOff + slot * kKStageBytes + c * kChunkBytes, &map_kv, full,
                                                 (s * kKChunks + c) * 64, leader ? p0 : p1);
                        }
                    }
                }
                if (t > pc.lo) {
                    for (int j = 0; j < 2 && ok; ++j, ++vst) {
                        const int slot = vst % kVStages;
                        ok = mbar_wait(&bars[B_VE + slot], ((vst / kVStages) & 1) ^ 1, abort_sh, a.wait_ns);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (lane == 0) {
                            const uint32_t full = lead(B_VF + slot);
                            mbar_arrive_expect_tx_cl(full, kVStageBytes);
                            for (int c = 0; c < 2; ++c)
                                for (int i = 0; i < 2; ++i)
                                    tma_load_2d_pair(sm + kVOff + slot * kVStageBytes + (2 * c + i) * kChunkBytes, &map_kv,
                                                     full, j * 256 + (int)rank * 128 + c * 64, i ? vp1 : vp0);
                        }
                    }
                }
                vp0 = p0;
                vp1 = p1;
            }
        }
        if (!ok && lane == 0) {
            *abort_sh = 1;
            atomicCAS(a.status, 0, PA_ERR_TIMEOUT);
        }
        // every copy issued lands before the pair may exit; rank 0's barriers count both CTAs'
        if (leader && lane == 0) {
            if (items > 0) mbar_wait(&bars[B_QF], (items - 1) & 1, nullptr, a.wait_ns);
            for (uint32_t s = 0; s < (uint32_t)kKStages && s < kst; ++s) {
                const uint32_t last = kst - 1 - ((kst - 1 - s) % kKStages);
                mbar_wait(&bars[B_KF + s], (last / kKStages) & 1, nullptr, a.wait_ns);
            }
            for (uint32_t s = 0; s < (uint32_t)kVStages && s < vst; ++s) {
                const uint32_t last = vst - 1 - ((vst - 1 - s) % kVStages);
                mbar_wait(&bars[B_VF + s], (last / kVStages) & 1, nullptr, a.wait_ns);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA thread (rank 0)
        if (leader && lane == 0) {
            constexpr uint32_t idesc_qk = idesc_f16(128, 128, !kF16, false, false);
            constexpr uint32_t idesc_pv = idesc_f16(128, 256, !kF16, false, true);
            const uint64_t qd = sdesc_sw128(smem_u32(sm + kQOff), 16, 1024), pd = sdesc_sw128(smem_u32(sm + kPOff), 16, 1024);
            const uint64_t kd = sdesc_sw128(smem_u32(sm + kKOff), 16, 1024);
            const uint64_t vd = sdesc_sw128(smem_u32(sm + kVOff), 2 * kChunkBytes, 1024);
            const uint32_t q_lo = (uint32_t)qd, p_lo = (uint32_t)pd, k_lo = (uint32_t)kd, v_lo = (uint32_t)vd;
            const uint32_t kmajor_hi = (uint32_t)(qd >> 32), v_hi = (uint32_t)(vd >> 32);
            bool ok = true;
            uint32_t items = 0, kst = 0, vst = 0, qk_tiles = 0, pv_tiles = 0;
            auto qk = [&](bool last) {
                const uint32_t dt = tbase + (qk_tiles & 1) * kSCols;
                for (int s = 0; s < kChunks / kKChunks; ++s, ++kst) {
                    const int slot = kst % kKStages;
                    if (!mbar_wait(&bars[B_KF + slot], (kst / kKStages) & 1, abort_sh, a.wait_ns)) return false;
                    tc_fence_after();
                    const uint32_t qw = q_lo + (uint32_t)((s * kKStageBytes) >> 4);
                    const uint32_t kw = k_lo + (uint32_t)((slot * kKStageBytes) >> 4);
                    if (s == 0) mma_pair_ss_w<0>(dt, qw, kmajor_hi, kw, kmajor_hi, idesc_qk);
                    else mma_pair_ss_w<1>(dt, qw, kmajor_hi, kw, kmajor_hi, idesc_qk);
#pragma unroll
                    for (int kk = 1; kk < 4 * kKChunks; ++kk) {
                        const uint32_t o = (uint32_t)(((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4);
                        mma_pair_ss_w<1>(dt, qw + o, kmajor_hi, kw + o, kmajor_hi, idesc_qk);
                    }
                    mma_commit_pair_mc(&bars[B_KE + slot], 3);
                }
                mma_commit_pair_mc(&bars[B_SF + (qk_tiles & 1)], 3);
                if (last) mma_commit_pair_mc(&bars[B_QE], 3);
                ++qk_tiles;
                return true;
            };
            auto pv = [&](bool first) {
                if (!mbar_wait_cl(&bars[B_PF], pv_tiles & 1, abort_sh, a.wait_ns)) return false;
                for (int j = 0; j < 2; ++j, ++vst) {
                    const int slot = vst % kVStages;
                    if (!mbar_wait(&bars[B_VF + slot], (vst / kVStages) & 1, abort_sh, a.wait_ns)) return false;
                    tc_fence_after();
                    const uint32_t dt = tbase + kOCol + j * kOCols;
                    const uint32_t vw = v_lo + (uint32_t)((slot * kVStageBytes) >> 4);
                    if (first) mma_pair_ss_w<0>(dt, p_lo, kmajor_hi, vw, v_hi, idesc_pv);
                    else mma_pair_ss_w<1>(dt, p_lo, kmajor_hi, vw, v_hi, idesc_pv);
#pragma unroll
                    for (int kk = 1; kk < 8; ++kk)
                        mma_pair_ss_w<1>(dt, p_lo + (uint32_t)(((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4), kmajor_hi,
                                         vw + (uint32_t)((kk * 2048) >> 4), v_hi, idesc_pv);
                    mma_commit_pair_mc(&bars[B_VE + slot], 3);
                }
                mma_commit_pair_mc(&bars[B_OD], 3);
                ++pv_tiles;
                return true;
            };
            while (ok && walk.next(a, pc)) {
                const int n = pc.hi - pc.lo;
                if (n == 0) continue;
                ok = mbar_wait(&bars[B_QF], items & 1, abort_sh, a.wait_ns);
                ++items;
                if (ok) ok = qk(n == 1);
                for (int t = 0; t < n && ok; ++t) {
                    if (t + 1 < n) ok = qk(t + 2 == n);
                    if (ok) ok = pv(t == 0);
                }
            }
            if (!ok) {
                *abort_sh = 1;
                atomicCAS(a.status, 0, PA_ERR_TIMEOUT);
            }
            mma_commit_pair_mc(&bars[B_DONE], 1);
            mbar_wait(&bars[B_DONE], 0, nullptr, a.wait_ns);
        }
    } else {
        // ---------------------------------------------------------------- softmax (both CTAs)
        const int q4 = warp & 3;                  // TMEM lanes 32 q4 .. 32 q4 + 31
        const int row = (q4 & 1) * 32 + lane;     // this CTA's query row
        const int kh = q4 >> 1;                   // page of the tile (keys 64 kh .. of S), columns 128 kh .. of O
        const int tid = (int)threadIdx.x - 64;    // of the CTA's softmax threads
        const uint32_t lane_addr = (uint32_t)(q4 * 32) << 16;
        const float sl2 = a.scale_log2;
        uint32_t g = 0;    // tiles done
        bool bad = false;  // a wait ran out; all softmax threads leave at the next barrier
        uint32_t vst = 0;
        MlaMerge merge{0, 0, 0, 0};
        while (walk.next(a, pc)) {
            const int n = pc.hi - pc.lo;
            const int block_rows = min(kMlaBlockRows, a.rows - pc.blk * kMlaBlockRows), half = (block_rows + 1) / 2;
            const int my_rows = leader ? half : block_rows - half;
            const bool live = (q4 & 1) * 32 < my_rows;  // the warp has rows
            const int in_block = (int)rank * half + row;
            const int in_seq = pc.blk * kMlaBlockRows + in_block;
            const bool write = row < my_rows;
            // keys that the row's token sees: all but those of the tokens after it
            const long long sees = (long long)pc.len - (a.q_len - 1 - min(in_seq / a.num_heads, a.q_len - 1));
            float m_run = -INFINITY, l_run = 0.f;
            for (int t = pc.lo; t < pc.hi; ++t, ++g, vst += 2) {
                if (!bad) bad = !mbar_wait(&bars[B_SF + (g & 1)], (g >> 1) & 1, abort_sh, a.wait_ns);
                uint32_t r[64];
                uint32_t (&ra)[32] = *reinterpret_cast<uint32_t (*)[32]>(&r[0]);
                uint32_t (&rb)[32] = *reinterpret_cast<uint32_t (*)[32]>(&r[32]);
                const int vis = (int)min(64ll, max(0ll, sees - (long long)t * 128 - kh * 64));
                bool full = false;
                float mt = -INFINITY;
                if (live && __all_sync(0xffffffffu, !bad)) {
                    tc_fence_after();
                    const uint32_t s_addr = tbase + lane_addr + (g & 1) * kSCols;
                    tmem_ld_x32(s_addr, ra);
                    tmem_ld_x32(s_addr + 32, rb);
                    tmem_ld_wait();
                    reg_fence(ra);
                    reg_fence(rb);
                    full = __all_sync(0xffffffffu, vis >= 64) && sl2 > 0.f;
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    if (full) {
#pragma unroll
                        for (int k = 0; k < 64; k += 2)
                            m4[(k >> 1) & 3] = fmax3(m4[(k >> 1) & 3], __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
                    } else {
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (k < vis) m4[k & 3] = fmaxf(m4[k & 3], __uint_as_float(r[k]) * sl2);
                    }
                    mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    if (full) mt *= sl2;
                    row_max[g & 1][kh][row] = mt;
                }
                bad = bar_or(1, 128, bad);
                if (bad) break;
                bool grow = false;
                float m_new = m_run;
                if (live) {
                    mt = fmaxf(mt, row_max[g & 1][kh ^ 1][row]);
                    grow = mt > m_run + kRescaleThreshold;
                    if (grow) m_new = mt;
                }
                // P and O are free once the tile before has been through PV
                if (g > 0) bad = !mbar_wait(&bars[B_OD], (g - 1) & 1, abort_sh, a.wait_ns);
                if (live && __all_sync(0xffffffffu, !bad)) {
                    const bool rescale = grow && t > pc.lo && m_run != -INFINITY;
                    const float alpha = rescale ? ex2(m_run - m_new) : 1.f;
                    if (__any_sync(0xffffffffu, rescale)) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o[32];
                            const uint32_t at = tbase + lane_addr + kOCol + c * 32;
                            tmem_ld_x32(at, o);
                            tmem_ld_wait();
                            reg_fence(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                            tmem_st_x32(at, o);
                        }
                        tmem_st_wait();
                    }
                    l_run *= alpha;
                    m_run = m_new;
                    const bool none = m_run == -INFINITY;
                    const bool fast = __all_sync(0xffffffffu, full && !none);
                    uint8_t* p_row = sm + kPOff + kh * kChunkBytes + row * 128;
                    uint64_t acc[2] = {f2_pack(0u, 0u), f2_pack(0u, 0u)};
                    float rsum = 0.f;
                    auto store8 = [&](int u, const uint32_t (&pw)[4]) {
                        *reinterpret_cast<uint4*>(p_row + ((u ^ (row & 7)) << 4)) = make_uint4(pw[0], pw[1], pw[2], pw[3]);
                    };
                    if (fast) {
                        const uint64_t sc2 = f2_pack(__float_as_uint(sl2), __float_as_uint(sl2));
                        const uint64_t nm2 = f2_pack(__float_as_uint(-m_run), __float_as_uint(-m_run));
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            uint32_t pw[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float x0, x1;
                                f2_unpack(f2_fma(f2_pack(r[u * 8 + 2 * k], r[u * 8 + 2 * k + 1]), sc2, nm2), x0, x1);
                                const float p0 = ex2(x0), p1 = ex2(x1);
                                acc[k & 1] = f2_add(acc[k & 1], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
                                pw[k] = pack16x2(p0, p1, kF16);
                            }
                            store8(u, pw);
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            uint32_t pw[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int e = u * 8 + 2 * k;
                                const float p0 = none || e >= vis ? 0.f : ex2(__uint_as_float(r[e]) * sl2 - m_run);
                                const float p1 = none || e + 1 >= vis ? 0.f : ex2(__uint_as_float(r[e + 1]) * sl2 - m_run);
                                rsum += p0 + p1;
                                pw[k] = pack16x2(p0, p1, kF16);
                            }
                            store8(u, pw);
                        }
                    }
                    float a0, a1, b0, b1;
                    f2_unpack(acc[0], a0, a1);
                    f2_unpack(acc[1], b0, b1);
                    l_run += (a0 + a1) + (b0 + b1) + rsum;
                }
                const int live_keys = pc.len - t * 128;  // of this tile
                if (leader && live_keys < 128 && !bad) {
                    // 0 * NaN would poison the product: rows of the V tile past the last key are zeroed in both CTAs
                    for (int j = 0; j < 2; ++j)
                        if (!bad)
                            bad = !mbar_wait(&bars[B_VF + (vst + j) % kVStages], ((vst + j) / kVStages) & 1, abort_sh, a.wait_ns);
                    if (!bad && tid >= live_keys) {
                        for (int j = 0; j < 2; ++j)
                            for (int c = 0; c < 2; ++c) {
                                uint8_t* v = sm + kVOff + ((vst + j) % kVStages) * kVStageBytes + 2 * c * kChunkBytes + tid * 128;
                                const uint32_t v1 = mapa_shared(smem_u32(v), 1);
#pragma unroll
                                for (int u = 0; u < 8; ++u) {
                                    *reinterpret_cast<uint4*>(v + u * 16) = make_uint4(0, 0, 0, 0);
                                    st_cl_v4(v1 + u * 16, make_uint4(0, 0, 0, 0));
                                }
                            }
                    }
                }
                // P lies in this CTA's shared memory and is read there by its own half of the pair's MMA: once the proxy
                // fence is through, the arrival itself has nothing left to order (a release at cluster scope takes 700
                // cycles, and the fence over the cluster 900).  Rows zeroed in the peer are released as a whole.
                const bool zeroed = leader && live_keys < 128;
                if (zeroed) fence_proxy_async_cluster();
                else fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (zeroed) mbar_arrive_cl(lead(B_PF));
                    else mbar_signal_cl(lead(B_PF));
                }
            }
            if (bad) break;
            // ---- output of the piece
            if (n > 0) {
                if (!bad) bad = !mbar_wait(&bars[B_OD], (g - 1) & 1, abort_sh, a.wait_ns);
                row_sum[kh][row] = l_run;
                bad = bar_or(1, 128, bad);
                if (bad) break;
            }
            const bool whole = n == pc.tiles;
            const float l = n > 0 ? l_run + row_sum[kh ^ 1][row] : 0.f;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const float lse2 = l > 0.f ? m_run + __log2f(l) : -INFINITY;
            const long long orow = (long long)pc.b * a.rows + in_seq;
            const int slot = 2 * pair + (pc.lo == 0);
            const long long prow = (long long)slot * kMlaBlockRows + in_block;
            if (live) {
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld_x32(tbase + lane_addr + kOCol + c * 32, o);
                        tmem_ld_wait();
                        reg_fence(o);
                    }
                    const int col = (c >> 2) * 256 + kh * 128 + (c & 3) * 32;
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = inv > 0.f ? __float_as_uint(__uint_as_float(o[k]) * inv) : 0u;
                    if (write) {
                        if (whole) {
                            uint32_t w[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                w[k] = pack16x2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]), kF16);
                            uint4* d4 = reinterpret_cast<uint4*>(a.out + orow * kMlaLatent + col);
#pragma unroll
                            for (int k = 0; k < 4; ++k) d4[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                        } else {
                            float* dst = a.o_part + prow * kMlaLatent + col;
#pragma unroll
                            for (int k = 0; k < 4; ++k) st_global_v8(dst + 8 * k, &o[8 * k]);
                        }
                    }
                }
                if (write && kh == 0) {
                    if (!whole) a.lse_part[prow] = lse2;
                    else if (a.lse) a.lse[orow] = lse2 * kLn2f;
                }
            }
            if (!whole && pc.lo == 0) {
                merge.b = pc.b;
                merge.blk = pc.blk;
                merge.first = pair;
                const long long share = walk.to - walk.from;
                merge.pieces = (int)((pc.at + kFixed + pc.tiles - 1) / share) - pair + 1;
            }
            tc_fence_before();  // (the next piece's row_sum is written after barriers of its tiles)
        }
        if (leader && tid == 0) a.merges[pair] = merge;
        if (bad) {
            *abort_sh = 1;
            atomicCAS(a.status, 0, PA_ERR_TIMEOUT);
        }
    }
    tc_fence_before();
    __syncthreads();
    allow_dependents_launch();
    cluster_sync_all();  // the pair's MMAs, copies and peer accesses are over
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tbase, 512);
    }
}

// Merge of split items: with m = max_s lse_s, lse = m + ln sum_s exp(lse_s - m),
// out = sum_s exp(lse_s - lse) o_s.  A warp takes 128 columns of a row.
constexpr int kMergeRows = 2;
template <bool kF16>
__global__ void __launch_bounds__(kMergeRows * 128) mla_merge_kernel(const __grid_constant__ MlaDecodeArgs a) {
    grid_dependency_wait();
    const MlaMerge m = a.merges[blockIdx.y];
    if (m.pieces == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int in_block = (int)blockIdx.x * kMergeRows + (warp >> 2);
    const int in_seq = m.blk * kMlaBlockRows + in_block;
    if (in_block >= kMlaBlockRows || in_seq >= a.rows) return;
    const int col = (warp & 3) * 128 + lane * 4;
    // slot of the s-th piece
    auto slot = [&](int s) { return (long long)(2 * (m.first + s) + (s == 0)) * kMlaBlockRows + in_block; };
    float top = -INFINITY;
    for (int s = lane; s < m.pieces; s += 32) top = fmaxf(top, a.lse_part[slot(s)]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    if (top != -INFINITY) {
#pragma unroll 4
        for (int s = 0; s < m.pieces; ++s) {
            const float w = ex2(a.lse_part[slot(s)] - top);
            const float4 v = *reinterpret_cast<const float4*>(a.o_part + slot(s) * kMlaLatent + col);
            sum += w;
            acc.x = fmaf(w, v.x, acc.x);
            acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z);
            acc.w = fmaf(w, v.w, acc.w);
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const long long orow = (long long)m.b * a.rows + in_seq;
    *reinterpret_cast<uint2*>(a.out + orow * kMlaLatent + col) =
        make_uint2(pack16x2(acc.x * inv, acc.y * inv, kF16), pack16x2(acc.z * inv, acc.w * inv, kF16));
    if (a.lse && (warp & 3) == 0 && lane == 0) a.lse[orow] = sum > 0.f ? (top + __log2f(sum)) * kLn2f : -INFINITY;
}

// Pairs of CTAs of the kernel that fit on the device at once (per device, cached).
template <typename K>
int pair_capacity(K* kernel) {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) {
        const int c = cached[dev].load(std::memory_order_acquire);
        if (c > 0) return c;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    if (dev >= 0 && dev < 64 && clusters > 0) cached[dev].store(clusters, std::memory_order_release);
    return clusters;
}

template <bool kF16>
cudaError_t launch(MlaDecodeArgs& a, int max_pairs, const CUtensorMap* mq, const CUtensorMap* mkv, cudaStream_t stream) {
    auto kernel = mla_decode_kernel<kF16>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_dynamic_smem(kernel, kSmem, configured);
    if (e != cudaSuccess) return e;
    const int fit = pair_capacity(kernel);
    if (fit <= 0) return cudaErrorNotSupported;
    // no more pairs than the longest lengths could give a range
    const long long blocks = (a.rows + kMlaBlockRows - 1) / kMlaBlockRows;
    const long long most = ((long long)a.batch * blocks * (kFixed + (a.max_pages + 1) / 2) + kMinShare - 1) / kMinShare;
    a.pairs = (int)min(min((long long)fit, (long long)max_pairs), most);
    e = launch_overlapped(kernel, dim3(2 * a.pairs), dim3(kThreads), kSmem, stream, a, *mq, *mkv);
    if (e != cudaSuccess || a.pairs == 1) return e;
    const int rows = min(a.rows, kMlaBlockRows);
    return launch_overlapped(mla_merge_kernel<kF16>, dim3((rows + kMergeRows - 1) / kMergeRows, a.pairs),
                             dim3(kMergeRows * 128), 0, stream, a);
}

}  // namespace

cudaError_t launch_mla_decode(MlaDecodeArgs a, int max_pairs, const CUtensorMap* mq, const CUtensorMap* mkv,
                              cudaStream_t stream) {
    return a.f16 ? launch<true>(a, max_pairs, mq, mkv, stream) : launch<false>(a, max_pairs, mq, mkv, stream);
}

}  // namespace pa
