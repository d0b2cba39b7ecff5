// mla_decode.cu -- attention of one or a few new tokens a sequence over a paged
// cache of latent rows (pa_mla_decode):
//
//   s_j = scale <q, row_j>          over the row's 576 elements
//   out = sum_j softmax_j(s) row_j  over its first 512
//   lse = ln sum_j exp(s_j)
//
// Every head of a sequence reads the same rows, so a sequence's (token, head)
// pairs are the columns of one product, N at a time (a block: 16, 32 or 64 of
// them), and a page's keys and latent elements its rows:
//
//   S^T[64 keys, N]      = K  Q^T        K: a page, 576 elements a row
//   O^T[512 elements, N] += V^T P^T      V: the same page's first 512 elements
//
// One page lies once in shared memory, for both products (K-major for the first,
// MN-major for the second): a page is read from memory once and from L2 once per
// block.  At 64 columns the queries take 72 KB of shared memory and leave room
// for two pages; O takes 4 N columns of tensor memory, so 128 columns would not
// fit one SM.  Two blocks of a sequence run side by side, on neighbouring CTAs
// that walk over the same pages.
//
//   warp 0     producer: queries, and pages through a ring (128 latent elements
//              of a page a stage, the 64 rotary ones in a ring of their own)
//   warp 1     the MMAs of S          warp 10   the MMAs of O
//   warps 2-9  softmax: 16 keys a warp (M = 64 fills as many lanes of four
//              groups of 32), half of the columns, a quarter a lane; P to shared
//              memory
//
// The softmax's reference is not each key's running maximum but one value a
// column, which changes only when a score exceeds it by more than 2^8.  P is
// written with the references as they are, and then the four warps of a column
// agree whether one was exceeded; if so, in an item's first page, and as long as a
// column has seen scores of -inf only or has a reference beyond 2^14, the columns'
// maxima over the page are found, the accumulators rescaled and P written again
// (with the vote before P a call took 61.2 us, with it after 60.0; with the first
// half of every sequence at -inf one of 64 sequences and 128 heads takes 66.7
// against 59.1, one of 16 heads 39.2 as without).
//
// The sequences' costs (pages and a constant) are laid end to end and cut into
// equal ranges, as many as there are CTAs a block: a CTA takes what lies in its
// range, at most two pieces of which are parts of an item.  Those go to the
// workspace in fp32, with their references and sums, and are merged by a second
// kernel.  Lengths are read on the device only.
//
// P is rounded to the rows' type, as an operand of the second product has to be;
// its sum is taken before, in fp32.  That is half a step of bf16, 2^-8 of a weight,
// or of fp16, 2^-11 of one.  fp16 has few exponents: there P is 2^7 times the weight
// beside the reference, so that a weight keeps all its bits down to 2^-21 of the
// reference's, half a step is 2^-32 of that below, and what is less than 2^-32 of it
// vanishes (without the factor 2^-14 and 2^-25: 131072 keys at 2^-25 of one lost
// their 0.4% of the output).
//
// What bounds it.  A byte of a row meets 2 x heads x 1.9 operations: with 128
// heads more than the memory's rate asks of the tensor cores at N = 64, where an
// MMA reads 6 KB of shared memory for 34 cycles of products (48 at 128 B a
// cycle): 1920 cycles a page and block, against 1640 for the memory's share of an
// SM (73.7 KB for two of them, at the 1.96 GHz that they run at).  Measured, 64
// sequences of 1-4096 keys, 128 heads, bf16: 58.8 us.  A page takes about 2400
// cycles (shared memory has room for two, and two take 4800: load 1150, S, softmax
// 1000, O), so an SM's 28 pages take 67 thousand of the 107 thousand cycles of this
// kernel, 34 us of 54; the other 20 are the start (6: launch, dealing, first page),
// the outputs of pieces and the wait for the last CTA, and then there is the merge.
// 32 sequences of 64-16384 keys, 16 heads, two tokens each: 59 us (287 MB, 4.9 TB/s;
// 6.6, the memory's copy rate, while pages stream).  One sequence of 777 keys, 128
// heads: 11.8 us.
#include "pa_launch.h"
#include "pa_mla.h"
#include "pa_ptx.cuh"
#include "prefill_common.cuh"

namespace pa {
namespace {

constexpr int kChunks = kMlaRow / 64;  // 64-element chunks of a row: 8 latent ones and the rotary one
constexpr int kBox = 64 * 128;         // a chunk of a page's rows
constexpr int kPageStages = 4;         // latent stages of a page, two chunks each
constexpr int kRopeStages = 2, kMaxStages = 11;
constexpr int kSoftmaxWarps = 8;
constexpr int kListed = 16;  // sequences of a CTA's range whose pieces are found at its start
constexpr int kThreads = 96 + 32 * kSoftmaxWarps;
// What an item costs besides its pages, in pages (64 sequences of 1-4096 keys: 58.7 us a call with 3, 58.3 with 4, 59.5
// with 5; one of 777: 11.8, 13.1 and 11.8), and the shortest range (one sequence of 777 keys: 17.1 us with 6, 14.0 with 3,
// 13.0 with 2, 13.3 with 1, of which the output and the merge took one more than now).  All at 64 columns; narrower
// blocks, whose items cost less besides their pages, share both.
constexpr int kFixed = 3;
constexpr int kMinShare = 2;
// fp16 weights are held as 2^7 times those beside the reference: at most 2^15, and whole steps of fp16 down to 2^-21 of it.
constexpr float kShiftF16 = 7.f;
// From here on (in bits) a column's weights are made of its products with the scale as they are rounded, page by page: up
// to here the rounding is 2^-11 of a weight at most.
constexpr float kFarReference = 16384.f;

template <int N>
struct Layout {
    static constexpr int kHalf = N / 2;           // columns of a softmax warp
    static constexpr int kQuarter = N / 4;        // and of a lane
    static constexpr int kQChunk = N * 128;       // 64 elements of the queries
    static constexpr int kPBuffers = N > 32 ? 1 : 2;  // side by side in the 128-byte rows of P, a key each
    static constexpr int kStages = N > 32 ? 8 : N > 16 ? 10 : 11;  // latent stages that shared memory has room for
    static constexpr int kQOff = 0;
    static constexpr int kPOff = kChunks * kQChunk;
    static constexpr int kRopeOff = kPOff + kBox;
    static constexpr int kRingOff = kRopeOff + kRopeStages * kBox;
    static constexpr int kEnd = kRingOff + kStages * 2 * kBox;
    static constexpr uint32_t kOCol = 2 * N, kCols = N > 32 ? 512 : N > 16 ? 256 : 128;  // tensor memory: two S, O
    static_assert(kStages <= kMaxStages, "barriers of the ring");
};

enum : int {
    B_QF = 0,                    // queries landed
    B_QE = 1,                    // queries used
    B_RF = 2,                    // [kRopeStages] rotary chunk landed
    B_RE = B_RF + kRopeStages,   // [kRopeStages] and used
    B_LF = B_RE + kRopeStages,   // [kMaxStages] latent chunks landed
    B_LE = B_LF + kMaxStages,    // [kMaxStages] and used
    B_SF = B_LE + kMaxStages,    // [2] S ready
    B_PF = B_SF + 2,             // [2] P written (by turns: the MMA warps wait for it a page apart)
    B_OD = B_PF + 2,             // [2] a page's MMAs of O retired (by turns: waited for one page behind or two)
    B_DONE = B_OD + 2,           // [2] every MMA of S, of O retired
    B_COUNT = B_DONE + 2
};

// A stretch of pages [lo, hi) of sequence b that a CTA takes.
struct Piece {
    int b, lo, hi, pages, len;
    int at;  // where the item's cost starts
};

__device__ __forceinline__ int clamped_len(const MlaDecodeArgs& a, int b, bool report) {
    const int len = __ldg(&a.seq_lens[b]);
    const long long most = min((long long)a.max_pages * kPage, 0x7FFFFF80ll);
    if (len >= 0 && len <= most) return len;
    if (report) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
    return len < 0 ? 0 : (int)most;
}

// The pieces of a range [from, to) of costs, from sequence b on, whose cost starts at `at`.
struct Walk {
    int from, to, at;
    int b;
    __device__ __forceinline__ bool take(const MlaDecodeArgs& a, int len, Piece& p) {
        p.b = b++;
        p.at = at;
        p.len = len;
        p.pages = (len + kPage - 1) / kPage;
        const int t0 = at + kFixed;
        p.lo = min(p.pages, max(0, from - t0));
        p.hi = min(p.pages, max(0, to - t0));
        at = t0 + p.pages;
        return p.pages == 0 ? p.at >= from : p.hi > p.lo;
    }
    __device__ __noinline__ bool next(const MlaDecodeArgs& a, Piece& p) {
        while (b < a.batch && at < to)
            if (take(a, clamped_len(a, b, false), p)) return true;
        return false;
    }
};

// The kernel's waits, bounded like mbar_wait: fewer instructions, as they stand in many places, and asked without a
// suspend hint first (60 cycles against 95 where the phase is complete).
struct Waiter {
    const volatile int* abort;
    uint64_t limit_ns;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        if (mbar_test(bar, parity)) return true;
        const uint64_t until = globaltimer_ns() + limit_ns;
#pragma unroll 1
        while (!mbar_try_wait(bar, parity))
            if (*abort || globaltimer_ns() > until) return false;
        return true;
    }
};

// Joins every column's values over 16 lanes, n columns (4, 8 or 16): at each step a lane hands over the columns that its
// partner keeps.  In the end v[0] is that of column lane % n.
template <int n, typename Op>
__device__ __forceinline__ void join_columns(float (&v)[n], Op op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = n / 2; o >= 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int c = 0; c < o; ++c) {
            const float give = up ? v[c] : v[c + o], keep = up ? v[c + o] : v[c];
            v[c] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
#pragma unroll
    for (int o = n; o < 16; o <<= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
}

template <int N, bool kF16>
__global__ void __launch_bounds__(kThreads, 1)
    mla_decode_kernel(const __grid_constant__ MlaDecodeArgs a, const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_latent, const __grid_constant__ CUtensorMap map_rope) {
    using L = Layout<N>;
    constexpr int kHalf = L::kHalf, kQuarter = L::kQuarter, kStages = L::kStages;
    constexpr float kShift = kF16 ? kShiftF16 : 0.f;
    struct Small {
        uint64_t bars[B_COUNT];
        Walk start;            // where the walk goes on behind the pieces listed here
        Piece pieces[kListed];
        int count, share;
        int sums[kThreads / 32];
        uint32_t tmem_base;
        int abort;
        alignas(16) float part[4][N];  // the 4 parts of a column's reduction
        alignas(16) float minus_ref[N];  // read by four: -reference (0 while it is -inf)
        alignas(16) float factor[N];  // of the last change, or of the output
        alignas(16) int sees[N];  // read by four: keys that the column's token sees
    };
    static_assert(L::kEnd + sizeof(Small) <= 232448, "shared memory of a CTA");
    extern __shared__ __align__(1024) uint8_t sm[];
    Small& sh = *reinterpret_cast<Small*>(sm + L::kEnd);
    uint64_t* const bars = sh.bars;
    volatile int* const abort_sh = &sh.abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = (a.rows + N - 1) / N;
    const int blk = (int)blockIdx.x % blocks, range = (int)blockIdx.x / blocks;

    if (threadIdx.x == 0) {
        mbar_init(&bars[B_QF], 1);
        mbar_init(&bars[B_QE], 1);
        for (int s = 0; s < kRopeStages; ++s) {
            mbar_init(&bars[B_RF + s], 1);
            mbar_init(&bars[B_RE + s], 1);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars[B_LF + s], 1);
            mbar_init(&bars[B_LE + s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars[B_SF + s], 1);
            mbar_init(&bars[B_PF + s], kSoftmaxWarps);
            mbar_init(&bars[B_OD + s], 1);
            mbar_init(&bars[B_DONE + s], 1);
        }
        *abort_sh = 0;
        sh.start.b = a.batch;
        sh.start.at = sh.start.from = sh.start.to = 0;
        fence_barrier_init();
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_latent);
        tma_prefetch_map(&map_rope);
    }
    grid_dependency_wait();
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, L::kCols);
        tmem_relinquish();
    }
    // ---- this CTA's range: every thread sums the costs of a run of sequences
    {
        const int per = (a.batch + kThreads - 1) / kThreads;
        const int b0 = min((int)threadIdx.x * per, a.batch), b1 = min(b0 + per, a.batch);
        int mine = 0;
        for (int b = b0; b < b1; ++b) mine += kFixed + (clamped_len(a, b, blockIdx.x == 0) + kPage - 1) / kPage;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) sh.sums[warp] = incl;
        __syncthreads();
        int before = incl - mine, total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int sum = sh.sums[w];
            if (w < warp) before += sum;
            total += sum;
        }
        // (as many ranges as are at least that long, and all alike; the launch sees to sums below 2^31)
        const int ranges = max(1, min(a.ranges, total / kMinShare));
        const int share = (total + ranges - 1) / ranges;
        const int from = range < ranges ? range * share : total;
        if (from >= before && from < before + mine) {
            Walk w;
            w.from = from;
            w.to = min(from + share, total);
            w.at = before;
            w.b = b0;
            for (;;) {
                const int cost = kFixed + (clamped_len(a, w.b, false) + kPage - 1) / kPage;
                if (from < w.at + cost) break;
                w.at += cost;
                ++w.b;
            }
            sh.start = w;
            sh.share = share;
        }
    }
    __syncthreads();
    if (warp == 2) {
        // the pieces among the next kListed sequences, their lengths fetched at once: a role that asked for one at an item's
        // end would wait for the load behind all the stores of the output
        Walk w = sh.start;
        const int b = w.b + lane;
        const bool in = lane < kListed && b < a.batch;
        const int len = in ? clamped_len(a, b, false) : 0;
        const int cost = in ? kFixed + (len + kPage - 1) / kPage : 0;
        int incl = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        Walk mine = w;
        mine.b = b;
        mine.at = w.at + incl - cost;
        Piece p;
        const bool take = in && mine.at < w.to && mine.take(a, len, p);
        const unsigned taken = __ballot_sync(0xffffffffu, take);
        if (take) sh.pieces[__popc(taken & ((1u << lane) - 1))] = p;
        if (lane == 31) {
            sh.count = __popc(taken);
            w.b = min(w.b + kListed, a.batch);
            w.at += incl;
            sh.start = w;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sh.tmem_base;
    Walk walk = sh.start;
    Piece pc;
    int listed = 0;
    auto next_piece = [&]() {
        if (listed < sh.count) {
            pc = sh.pieces[listed++];
            return true;
        }
        return walk.next(a, pc);
    };
    const Waiter wait{abort_sh, a.wait_ns};
    bool ok = true;

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        if (elect_one()) {
            uint32_t items = 0, pages = 0;  // pieces with pages, pages issued
            uint32_t slot = 0, phase = 1;   // of the ring's next stage
            while (ok && next_piece()) {
                if (pc.hi == pc.lo) continue;
                if (items > 0) ok = wait(&bars[B_QE], (items - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&bars[B_QF], kChunks * L::kQChunk);
                tma_load_3d(sm + L::kQOff, &map_q, &bars[B_QF], 0, pc.b * a.rows + blk * N, 0);
                ++items;
                const int32_t* table = a.block_table + (long long)pc.b * a.max_pages;
                auto row_of = [&](int p) {  // first row of page p (past the last one: that one's)
                    const int id = __ldg(&table[min(p, pc.hi - 1)]);
                    const bool in = (unsigned)id < (unsigned)a.num_pool_pages;
                    if (!in) atomicCAS(a.status, 0, PA_ERR_DEVICE_BOUNDS);
                    return in ? id * kPage : 0;
                };
                int y = row_of(pc.lo), next = row_of(pc.lo + 1);
#pragma unroll 1
                for (int p = pc.lo; p < pc.hi && ok; ++p, ++pages) {
                    // the page behind is asked for in L2: with two pages in shared memory its loads are issued too late to
                    // hide the memory's latency (64 sequences, 128 heads: 79 us a call without, 72 with, 73 two pages ahead)
                    if (blk == 0 && p + 1 < pc.hi) prefetch_l2(a.pool + (long long)next * (kMlaRow * 2), kPage * kMlaRow * 2);
                    const uint32_t r = pages % kRopeStages;
                    ok = wait(&bars[B_RE + r], ((pages / kRopeStages) & 1) ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bars[B_RF + r], kBox);
                    tma_load_3d(sm + L::kRopeOff + r * kBox, &map_rope, &bars[B_RF + r], 0, y, kChunks - 1);
#pragma unroll 1
                    for (int i = 0; i < kPageStages; ++i) {
                        ok = wait(&bars[B_LE + slot], phase);
                        if (!ok) break;
                        uint8_t* at = sm + L::kRingOff + slot * (2 * kBox);
                        mbar_arrive_expect_tx(&bars[B_LF + slot], 2 * kBox);
                        tma_load_3d(at, &map_latent, &bars[B_LF + slot], 0, y, 2 * i);
                        if (++slot == kStages) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
                    y = next;
                    next = row_of(p + 2);
                }
            }
            // every copy issued lands before the CTA may exit (after a timeout the last page may be short of some)
            if (items > 0) mbar_wait(&bars[B_QF], (items - 1) & 1, nullptr, a.wait_ns);
#pragma unroll 1
            for (uint32_t s = 0; s < (uint32_t)kRopeStages && s < pages; ++s)
                mbar_wait(&bars[B_RF + s], ((pages - 1 - (pages - 1 - s) % kRopeStages) / kRopeStages) & 1, nullptr, a.wait_ns);
            const uint32_t issued = pages * kPageStages;
#pragma unroll 1
            for (uint32_t s = 0; s < (uint32_t)kStages && s < issued; ++s)
                mbar_wait(&bars[B_LF + s], ((issued - 1 - (issued - 1 - s) % kStages) / kStages) & 1, nullptr, a.wait_ns);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMAs of S: keys x columns
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_f16(64, N, !kF16, false, false);
            const uint64_t qd = sdesc_sw128(smem_u32(sm + L::kQOff), 16, 1024);
            const uint64_t rd = sdesc_sw128(smem_u32(sm + L::kRopeOff), 16, 1024), kd = sdesc_sw128(smem_u32(sm + L::kRingOff), 16, 1024);
            const uint32_t q_lo = (uint32_t)qd, r_lo = (uint32_t)rd, k_lo = (uint32_t)kd, hi = (uint32_t)(qd >> 32);
            uint32_t items = 0, g = 0, slot = 0, phase = 0;  // pieces, pages, the ring's next stage
            while (ok && next_piece()) {
                if (pc.hi == pc.lo) continue;
                ok = wait(&bars[B_QF], items & 1);
                ++items;
#pragma unroll 1
                for (int p = pc.lo; p < pc.hi && ok; ++p, ++g) {
                    // the scores that lay here are P by now
                    if (g >= 2) ok = wait(&bars[B_PF + (g & 1)], ((g >> 1) & 1) ^ 1);
                    const uint32_t r = g % kRopeStages, dt = tbase + (g & 1) * N;
                    if (ok) ok = wait(&bars[B_RF + r], (g / kRopeStages) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t rw = r_lo + r * (kBox >> 4), qr = q_lo + (uint32_t)(((kChunks - 1) * L::kQChunk) >> 4);
                    mma_ss_w<0>(dt, rw, hi, qr, hi, idesc);
#pragma unroll
                    for (int i = 1; i < 4; ++i) mma_ss_w<1>(dt, rw + 2 * i, hi, qr + 2 * i, hi, idesc);
                    mma_commit(&bars[B_RE + r]);
                    uint32_t q = q_lo;
#pragma unroll 1
                    for (int i = 0; i < kPageStages; ++i, q += (2 * L::kQChunk) >> 4) {
                        ok = wait(&bars[B_LF + slot], phase);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t k = k_lo + slot * ((2 * kBox) >> 4);
#pragma unroll
                        for (int m = 0; m < 8; ++m)
                            mma_ss_w<1>(dt, k + (uint32_t)((m / 4 * kBox) >> 4) + (m & 3) * 2, hi,
                                        q + (uint32_t)((m / 4 * L::kQChunk) >> 4) + (m & 3) * 2, hi, idesc);
                        if (++slot == kStages) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
                    if (!ok) break;
                    mma_commit(&bars[B_SF + (g & 1)]);
                    if (p + 1 == pc.hi) mma_commit(&bars[B_QE]);
                }
            }
            mma_commit(&bars[B_DONE]);
            mbar_wait(&bars[B_DONE], 0, nullptr, a.wait_ns);
        }
    } else if (warp == 2 + kSoftmaxWarps) {
        // ---------------------------------------------------------------- MMAs of O: elements x columns
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_f16(128, N, !kF16, true, true);
            const uint64_t pd = sdesc_sw128(smem_u32(sm + L::kPOff), 16, 1024), vd = sdesc_sw128(smem_u32(sm + L::kRingOff), kBox, 1024);
            const uint32_t p_lo = (uint32_t)pd, v_lo = (uint32_t)vd, p_hi = (uint32_t)(pd >> 32), v_hi = (uint32_t)(vd >> 32);
            auto desc = [](uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; };
            uint32_t g = 0, slot = 0;
            while (ok && next_piece()) {
#pragma unroll 1
                for (int p = pc.lo; p < pc.hi; ++p, ++g) {
                    ok = wait(&bars[B_PF + (g & 1)], (g >> 1) & 1);  // (its S was made of the page: that has landed)
                    if (!ok) break;
                    tc_fence_after();
                    const int groups = (min(kPage, pc.len - p * kPage) + 15) / 16;  // of 16 keys
                    const uint32_t w = p_lo + (uint32_t)((g % L::kPBuffers * N * 2) >> 4);
#pragma unroll 1
                    for (int i = 0; i < kPageStages; ++i) {
                        const uint32_t dt = tbase + L::kOCol + i * N, v = v_lo + slot * ((2 * kBox) >> 4);
                        mma_ss(dt, desc(v, v_hi), desc(w, p_hi), idesc, p > pc.lo);
#pragma unroll
                        for (int k = 1; k < 4; ++k)
                            if (k < groups) mma_ss_w<1>(dt, v + 128 * k, v_hi, w + 128 * k, p_hi, idesc);
                        mma_commit(&bars[B_LE + slot]);
                        if (++slot == kStages) slot = 0;
                    }
                    mma_commit(&bars[B_OD + (g & 1)]);
                }
            }
            mma_commit(&bars[B_DONE + 1]);
            mbar_wait(&bars[B_DONE + 1], 0, nullptr, a.wait_ns);
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const int q4 = warp & 3;                          // TMEM lanes 32 q4 .. 32 q4 + 31
        const int half = (warp - 2) >> 2;                 // of the columns
        const int tid = ((int)threadIdx.x - 64) & 127;    // of the half's threads: column half * kHalf + tid is its to keep
        const int key = q4 * 16 + (lane & 15);            // of the page
        const int first = half * kHalf + (lane >> 4) * kQuarter;  // of this lane's columns
        const int joined = half * kHalf + (lane >> 4) * kQuarter + lane % kQuarter;  // the one it has of joined columns
        const uint32_t bar_id = 1 + half, lane_addr = (uint32_t)(q4 * 32) << 16;
        const float sl2 = a.scale_log2;
        const int block_rows = min(N, a.rows - blk * N);
        const int columns = max(0, min(kHalf, block_rows - half * kHalf));  // of this half that are used
        const int column = half * kHalf + tid;
        const float4* ref4 = reinterpret_cast<const float4*>(&sh.minus_ref[first]);
        const int4* sees4 = reinterpret_cast<const int4*>(&sh.sees[first]);
        uint32_t g = 0;       // pages done
        bool bad = false;     // a wait ran out: the half's threads leave together at their next barrier
        MlaMerge merge{0, 0, 0, 0};
        uint64_t l2[kQuarter / 2];  // the key's sums of weights, of two columns each
        float s[kQuarter];          // and its scores, in units of ln 2

        while (next_piece()) {
            const int n = pc.hi - pc.lo;
            float ref = -INFINITY;  // of the column to keep: what its weights are in units of (2^kShift below the maximum it was set by)
            bool open = false;      // a column of the half has no reference yet (its scores so far were all -inf), or a far one
            if (n > 0) {
                if (tid < kHalf) {
                    const int tok = min(blk * N + column, a.rows - 1) / a.num_heads;
                    sh.sees[column] = pc.len - (a.q_len - 1 - tok);
                }
                bad = bar_or(bar_id, 128, bad);
                if (bad) break;
            }
            const int all_see = pc.len - (a.q_len - 1);
#pragma unroll
            for (int c = 0; c < kQuarter / 2; ++c) l2[c] = f2_pack(0u, 0u);
#pragma unroll 1
            for (int p = pc.lo; p < pc.hi; ++p, ++g) {
                const int k0 = p * kPage + key;  // the key
                const bool edge = (p + 1) * kPage > all_see;
                const int live = pc.len - p * kPage;
                if (!bad) bad = !wait(&bars[B_SF + (g & 1)], (g >> 1) & 1);
                if (live < kPage && (live & 15) != 0 && !bad) {
                    // 0 * NaN would poison the product: in the last group of 16 keys the rows past the last key are zeroed
                    // (the page has landed and S is made of it)
                    for (int w = (int)threadIdx.x - 64; w < (16 - (live & 15)) * 64; w += 32 * kSoftmaxWarps) {
                        const int box = (w >> 3) & 7, i = w & 7;  // 16 bytes of a row of a box
                        const uint32_t stage = (g * kPageStages + box / 2) % kStages;
                        *reinterpret_cast<uint4*>(sm + L::kRingOff + stage * (2 * kBox) + (box & 1) * kBox +
                                                  (live + (w >> 6)) * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                auto load_scores = [&]() {
                    tc_fence_after();
                    uint32_t (&r)[kQuarter] = reinterpret_cast<uint32_t (&)[kQuarter]>(s);
                    tmem_ld_halves<kQuarter, kQuarter>(tbase + lane_addr + (g & 1) * N + half * kHalf, r);
                    tmem_ld_wait();
                    reg_fence(r);
                };
                auto mask = [&]() {
                    if (!edge) return;
#pragma unroll
                    for (int c = 0; c < kQuarter; c += 4) {
                        const int4 see = sees4[c / 4];
                        s[c] = k0 < see.x ? s[c] : -INFINITY;
                        s[c + 1] = k0 < see.y ? s[c + 1] : -INFINITY;
                        s[c + 2] = k0 < see.z ? s[c + 2] : -INFINITY;
                        s[c + 3] = k0 < see.w ? s[c + 3] : -INFINITY;
                    }
                };
                // P where the page that its buffer was used for has been through O's MMAs; s becomes the weights
                auto write_p = [&]() {
                    uint8_t* const p_row = sm + L::kPOff + key * 128;
                    uint32_t w[kQuarter / 2];
#pragma unroll
                    for (int c = 0; c < kQuarter; ++c) s[c] = ex2(s[c]);
#pragma unroll
                    for (int c = 0; c < kQuarter / 2; ++c) w[c] = pack16x2(s[2 * c], s[2 * c + 1], kF16);
                    const int at = (int)(g % L::kPBuffers) * (N * 2) + first * 2;  // byte of the row, 16-byte groups swizzled
                    if constexpr (kQuarter == 4) {
                        *reinterpret_cast<uint2*>(p_row + ((((at >> 4) ^ (key & 7)) << 4) | (at & 15))) = make_uint2(w[0], w[1]);
                    } else {
#pragma unroll
                        for (int u = 0; u < kQuarter / 8; ++u)
                            *reinterpret_cast<uint4*>(p_row + ((((at >> 4) + u) ^ (key & 7)) << 4)) =
                                make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
                    }
                };
                auto passed = [&](uint32_t behind) {  // O's MMAs of the page that many before this one
                    return g < behind || wait(&bars[B_OD + ((g - behind) & 1)], ((g - behind) >> 1) & 1);
                };
                // ---- P with the references as they are, and then: did a score exceed its own?  With a column that has none,
                // any score above -inf does: the page's maxima are looked at without asking.  With a far one too, as a
                // product with the scale that is not rounded differs from its reference, one that was, by up to 2^-24 of
                // it: nothing near 0, and more than all that weights depend on where masks add the type's lowest value.
                bool change = p == pc.lo || open;
                if (!change) {
                    float top = -INFINITY;
                    if (columns > 0 && __all_sync(0xffffffffu, !bad)) {
                        load_scores();
#pragma unroll
                        for (int c = 0; c < kQuarter; c += 4) {
                            const float4 m = ref4[c / 4];
                            s[c] = fmaf(s[c], sl2, m.x);
                            s[c + 1] = fmaf(s[c + 1], sl2, m.y);
                            s[c + 2] = fmaf(s[c + 2], sl2, m.z);
                            s[c + 3] = fmaf(s[c + 3], sl2, m.w);
                        }
                        mask();
#pragma unroll
                        for (int c = 0; c < kQuarter; c += 2) top = fmax3(top, s[c], s[c + 1]);
                    }
                    if (!bad) bad = !passed(L::kPBuffers);
                    if (columns > 0 && __all_sync(0xffffffffu, !bad)) write_p();
                    fence_proxy_async_smem();
                    tc_fence_before();
                    change = bar_or(bar_id, 128, bad || top > kRescaleThreshold + kShift);
                }
                if (change) {
                    // ---- the columns' maxima over the page, new references, O rescaled, P with those
                    if (columns > 0 && __all_sync(0xffffffffu, !bad)) {
                        load_scores();
#pragma unroll
                        for (int c = 0; c < kQuarter; ++c) s[c] = __fmul_rn(s[c], sl2);
                        mask();
                        float v[kQuarter];
#pragma unroll
                        for (int c = 0; c < kQuarter; ++c) v[c] = s[c];
                        join_columns(v, [](float x, float y) { return fmaxf(x, y); });
                        sh.part[q4][joined] = v[0];  // (lanes of the same column have the same value)
                    }
                    bad = bar_or(bar_id, 128, bad);
                    if (bad) break;
                    if (tid < kHalf) {
                        const float most = fmaxf(fmaxf(sh.part[0][column], sh.part[1][column]),
                                                 fmaxf(sh.part[2][column], sh.part[3][column]));
                        float factor = 1.f;
                        if (most - ref > kRescaleThreshold + kShift) {  // (not where both are infinite)
                            if (ref != -INFINITY) factor = ex2(ref - (most - kShift));
                            ref = most - kShift;
                        }
                        sh.minus_ref[column] = ref == -INFINITY ? 0.f : -ref;
                        sh.factor[column] = factor;
                    }
                    open = bar_or(bar_id, 128, tid < columns && !(fabsf(ref) < kFarReference));
                    const bool rescale = p > pc.lo;
                    bad = !passed(rescale ? 1 : L::kPBuffers);
                    if (columns > 0 && __all_sync(0xffffffffu, !bad)) {
                        if (rescale) {
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < kQuarter / 2; ++c) {
                                const float2 f = *reinterpret_cast<const float2*>(&sh.factor[first + 2 * c]);
                                float x, y;
                                f2_unpack(l2[c], x, y);
                                l2[c] = f2_pack(__float_as_uint(x * f.x), __float_as_uint(y * f.y));
                            }
#pragma unroll 1
                            for (int i = 0; i < kPageStages; ++i) {
                                uint32_t o[kHalf];
                                const uint32_t at = tbase + lane_addr + L::kOCol + i * N + half * kHalf;
                                tmem_ld_cols<kHalf>(at, o);
                                tmem_ld_wait();
                                reg_fence(o);
#pragma unroll
                                for (int c = 0; c < kHalf; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * sh.factor[half * kHalf + c]);
                                tmem_st_cols<kHalf>(at, o);
                            }
                            tmem_st_wait();
                        }
#pragma unroll
                        for (int c = 0; c < kQuarter; c += 4) {
                            const float4 m = ref4[c / 4];
                            s[c] += m.x;
                            s[c + 1] += m.y;
                            s[c + 2] += m.z;
                            s[c + 3] += m.w;
                        }
                        write_p();
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&bars[B_PF + (g & 1)]);
                // (the sums while O's MMAs run)
                if (columns > 0)
#pragma unroll
                    for (int c = 0; c < kQuarter / 2; ++c)
                        l2[c] = f2_add(l2[c], f2_pack(__float_as_uint(s[2 * c]), __float_as_uint(s[2 * c + 1])));
            }
            if (n > 0) bad = bar_or(bar_id, 128, bad);
            if (bad) break;
            // ---- output of the piece: of a whole item normalised, of a part as it is, with its references and sums
            const bool whole = n == pc.pages;
            const long long slot = (long long)(2 * range + (pc.lo == 0)) * blocks + blk;
            const long long row0 = (long long)pc.b * a.rows + blk * N;  // of the block's first column
            if (n > 0) {
                float v[kQuarter];
#pragma unroll
                for (int c = 0; c < kQuarter / 2; ++c) f2_unpack(l2[c], v[2 * c], v[2 * c + 1]);
                join_columns(v, [](float x, float y) { return x + y; });
                if (whole) {
                    sh.part[q4][joined] = v[0];
                    bar_or(bar_id, 128, false);
                    if (tid < kHalf) {
                        const float l = (sh.part[0][column] + sh.part[1][column]) + (sh.part[2][column] + sh.part[3][column]);
                        sh.factor[column] = l == 0.f ? 0.f : 1.f / l;  // (a NaN stays one)
                        if (tid < columns && a.lse) a.lse[row0 + column] = l == 0.f ? -INFINITY : (ref + __log2f(l)) * kLn2f;
                    }
                    bar_or(bar_id, 128, false);
                } else {
                    if ((lane & 15) < kQuarter) a.sum_part[(slot * 4 + q4) * kMlaBlockRows + joined] = v[0];
                    if (tid < kHalf) a.ref_part[slot * kMlaBlockRows + column] = ref;
                }
                bad = !wait(&bars[B_OD + ((g - 1) & 1)], ((g - 1) >> 1) & 1);
                tc_fence_after();
            } else if (tid < columns && a.lse) {
                a.lse[row0 + column] = -INFINITY;
            }
            if (columns > 0 && __all_sync(0xffffffffu, !bad)) {
                const int element = q4 * 32 + lane;
                uint16_t* out = a.out + (row0 + half * kHalf) * kMlaLatent + element;
                float* part = a.o_part + (slot * kMlaBlockRows + half * kHalf) * kMlaLatent + element;
                const float* by = &sh.factor[half * kHalf];
                bool plain = n > 0 && columns == kHalf;
                if (whole && plain) plain = __all_sync(0xffffffffu, lane >= kHalf || by[lane % kHalf] != 0.f);
                if (plain) {
#pragma unroll
                    for (int i = 0; i < kPageStages; ++i) {
                        uint32_t o[kHalf];
                        tmem_ld_cols<kHalf>(tbase + lane_addr + L::kOCol + i * N + half * kHalf, o);
                        tmem_ld_wait();
                        reg_fence(o);
                        if (whole) {
#pragma unroll
                            for (int c = 0; c < kHalf; ++c)
                                out[c * kMlaLatent + i * 128] = (uint16_t)pack16x2(__uint_as_float(o[c]) * by[c], 0.f, kF16);
                        } else {
#pragma unroll
                            for (int c = 0; c < kHalf; ++c) part[c * kMlaLatent + i * 128] = __uint_as_float(o[c]);
                        }
                    }
                } else {  // columns that are not there, or see nothing (whatever the rows hold)
#pragma unroll 1
                    for (int i = 0; i < kPageStages; ++i) {
                        uint32_t o[kHalf];
                        if (n > 0) {
                            tmem_ld_cols<kHalf>(tbase + lane_addr + L::kOCol + i * N + half * kHalf, o);
                            tmem_ld_wait();
                            reg_fence(o);
                        }
#pragma unroll
                        for (int c = 0; c < kHalf; ++c) {
                            if (c >= columns) continue;
                            if (whole) {
                                const float y = n == 0 || by[c] == 0.f ? 0.f : __uint_as_float(o[c]) * by[c];
                                out[c * kMlaLatent + i * 128] = (uint16_t)pack16x2(y, 0.f, kF16);
                            } else {
                                part[c * kMlaLatent + i * 128] = __uint_as_float(o[c]);
                            }
                        }
                    }
                }
            }
            if (pc.lo == 0) {  // (at most one piece of a CTA is the first of several)
                const MlaMerge m{pc.b, blk, whole ? 0 : (pc.at + kFixed + pc.pages - 1) / sh.share - range + 1, range};
                if (a.few && threadIdx.x == 64) a.merges[pc.b * blocks + blk] = m;
                if (!whole) merge = m;
            }
            tc_fence_before();
        }
        if (threadIdx.x == 64 && a.ranges > 1 && !a.few) a.merges[blockIdx.x] = merge;
        ok = !bad;
    }
    if (!ok) {
        *abort_sh = 1;
        atomicCAS(a.status, 0, PA_ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    allow_dependents_launch();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, L::kCols);
    }
}

// Merge of split items: with a piece's references r_s, sums l_s and accumulators o_s (in units of 2^r_s),
//   out = sum_s 2^(r_s - m) o_s / sum_s 2^(r_s - m) l_s,  lse = m ln 2 + ln of that sum,  m = max_s r_s.
// Bound by the partials, 2 KB a row and piece out of L2, and by its launch: 40 MB in 6 us for 64 sequences and 128 heads.
// A warp takes a row, a CTA four; blockIdx.y is the attention kernel's CTA.  Where sequences are few (kFew) their pieces
// are many: the CTA's warps share the pieces of a quarter of a row, and blockIdx.y is (sequence, block).  One sequence of
// 131072 keys, 16 heads, is 152 pieces a row: a call takes 40 us, with a warp a quarter of a row 58.  64 sequences take
// 65 us that way against 60, with four pieces ahead instead of two 60.8.
constexpr int kMergeWarps = 4;
template <int N, bool kF16, bool kFew>
__global__ void __launch_bounds__(kMergeWarps * 32) mla_merge_kernel(const __grid_constant__ MlaDecodeArgs a) {
    constexpr int kVecs = kFew ? 1 : kMlaLatent / 128;  // of 4 columns a lane
    constexpr int kAhead = kFew ? 8 : N > 32 ? 2 : 4;  // pieces whose accumulators are on their way
    __shared__ float top_sh[kMergeWarps], sum_sh[kMergeWarps];
    __shared__ __align__(16) float acc_sh[kMergeWarps][128];
    grid_dependency_wait();
    allow_dependents_launch();
    const MlaMerge m = a.merges[blockIdx.y];
    const int blocks = (a.rows + N - 1) / N;
    // (after a call that ended at its wait limit an entry may be another call's)
    if (m.pieces <= 0 || m.first < 0 || m.pieces > a.ranges - m.first || (unsigned)m.blk >= (unsigned)blocks ||
        (unsigned)m.b >= (unsigned)a.batch)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int in_block = kFew ? (int)blockIdx.x : (int)blockIdx.x * kMergeWarps + warp;
    const int in_seq = m.blk * N + in_block;
    if (in_block >= N || in_seq >= a.rows) return;  // (all of a CTA's warps, or with kFew 0 none that others wait for)
    const int per = kFew ? (m.pieces + kMergeWarps - 1) / kMergeWarps : m.pieces;
    const int from = kFew ? min(warp * per, m.pieces) : 0, to = min(from + per, m.pieces);
    auto slot = [&](int s) { return (long long)(2 * (m.first + s) + (s == 0)) * blocks + m.blk; };  // of the s-th piece
    auto ref_of = [&](int s) { return a.ref_part[slot(s) * kMlaBlockRows + in_block]; };
    const int column = lane * 4 + (kFew ? (int)blockIdx.z * 128 : 0);
    const float* part = a.o_part + (long long)in_block * kMlaLatent + column;
    // the first pieces' accumulators on their way while their weights are found
    float4 v[kAhead][kVecs];
    auto load = [&](float4 (&to_v)[kVecs], int s) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            to_v[i] = *reinterpret_cast<const float4*>(part + slot(s) * (kMlaBlockRows * kMlaLatent) + i * 128);
    };
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
        if (from + s < to) load(v[s], from + s);
    float top = -INFINITY;
    for (int s = from + lane; s < to; s += 32) top = fmaxf(top, ref_of(s));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if constexpr (kFew) {
        if (lane == 0) top_sh[warp] = top;
        __syncthreads();
        top = fmaxf(fmaxf(top_sh[0], top_sh[1]), fmaxf(top_sh[2], top_sh[3]));
    }
    const float minus_top = top == -INFINITY ? 0.f : -top;
    float sum = 0.f;
    float4 acc[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = from; s0 < to; s0 += 32) {
        float weight = 0.f;  // of piece s0 + lane
        if (s0 + lane < to) {
            weight = ex2(ref_of(s0 + lane) + minus_top);
            float l = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) l += a.sum_part[(slot(s0 + lane) * 4 + i) * kMlaBlockRows + in_block];
            sum = fmaf(weight, l, sum);
        }
        const int count = min(32, to - s0);
        for (int s = 0; s < count; s += kAhead) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (s + j >= count) break;
                const float w = __shfl_sync(0xffffffffu, weight, s + j);
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    acc[i].x = fmaf(w, v[j][i].x, acc[i].x);
                    acc[i].y = fmaf(w, v[j][i].y, acc[i].y);
                    acc[i].z = fmaf(w, v[j][i].z, acc[i].z);
                    acc[i].w = fmaf(w, v[j][i].w, acc[i].w);
                }
                if (s0 + s + j + kAhead < to) load(v[j], s0 + s + j + kAhead);
            }
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const long long orow = (long long)m.b * a.rows + in_seq;
    if constexpr (kFew) {
        if (lane == 0) sum_sh[warp] = sum;
        *reinterpret_cast<float4*>(&acc_sh[warp][lane * 4]) = acc[0];
        __syncthreads();
        if (warp != 0) return;
        sum = (sum_sh[0] + sum_sh[1]) + (sum_sh[2] + sum_sh[3]);
#pragma unroll
        for (int w = 1; w < kMergeWarps; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(&acc_sh[w][lane * 4]);
            acc[0] = make_float4(acc[0].x + x.x, acc[0].y + x.y, acc[0].z + x.z, acc[0].w + x.w);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* out = a.out + orow * kMlaLatent + column;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        *reinterpret_cast<uint2*>(out + i * 128) =
            sum == 0.f ? make_uint2(0u, 0u) : make_uint2(pack16x2(acc[i].x * inv, acc[i].y * inv, kF16),
                                                         pack16x2(acc[i].z * inv, acc[i].w * inv, kF16));
    if (a.lse && blockIdx.z == 0 && lane == 0) a.lse[orow] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2f;
}

template <int N, bool kF16>
cudaError_t launch(MlaDecodeArgs& a, int sms, const CUtensorMap* maps, cudaStream_t stream) {
    auto kernel = mla_decode_kernel<N, kF16>;
    constexpr int smem = 232448;  // all of an SM's: one CTA each
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = ensure_dynamic_smem(kernel, smem, configured);
    if (e != cudaSuccess) return e;
    const long long blocks = (a.rows + N - 1) / N;
    // as many ranges as there are SMs for them, and no more than the longest lengths could give one each
    const long long most = ((long long)a.batch * (kFixed + a.max_pages) + kMinShare - 1) / kMinShare;
    a.ranges = (int)max(1ll, min((long long)sms / blocks, most));
    // (The choice of the merge knows the batch and not the lengths.  Up to here entries by sequence fit into the list, and
    // pieces may be more than 8 on average.  A long sequence among more short ones pays for it: one of 131072 keys and 18
    // of 100, 16 heads, take 41.1 us, with a nineteenth of 100 52.2.)
    a.few = 8ll * a.batch <= a.ranges;
    const unsigned ctas = (unsigned)(a.ranges * blocks);
    e = launch_overlapped(kernel, dim3(ctas), dim3(kThreads), smem, stream, a, maps[0], maps[1], maps[2]);
    if (e != cudaSuccess || a.ranges == 1) return e;
    const unsigned rows = (unsigned)min(a.rows, N);
    const dim3 block(kMergeWarps * 32);
    if (a.few)
        return launch_overlapped(mla_merge_kernel<N, kF16, true>, dim3(rows, (unsigned)(a.batch * blocks), kMlaLatent / 128), block, 0, stream, a);
    return launch_overlapped(mla_merge_kernel<N, kF16, false>, dim3((rows + kMergeWarps - 1) / kMergeWarps, ctas), block, 0, stream, a);
}

template <bool kF16>
cudaError_t launch_block(MlaDecodeArgs& a, int sms, const CUtensorMap* maps, cudaStream_t stream) {
    switch (mla_block_rows(a.rows)) {
        case 16: return launch<16, kF16>(a, sms, maps, stream);
        case 32: return launch<32, kF16>(a, sms, maps, stream);
        default: return launch<64, kF16>(a, sms, maps, stream);
    }
}

}  // namespace

cudaError_t launch_mla_decode(MlaDecodeArgs a, int sms, const CUtensorMap* maps, cudaStream_t stream) {
    return a.f16 ? launch_block<true>(a, sms, maps, stream) : launch_block<false>(a, sms, maps, stream);
}

}  // namespace pa
