// paged_mla.cu -- dense causal absorbed MLA of new tokens over a paged latent
// cache on tcgen05 tensor cores (dsa_paged_mla's fast path).
//
// For token t at position pos, head h, and rows s = 0..pos of its sequence:
//   l_s = scale * (q_lat[t,h] . c_s + q_rope[t,h] . r_s)
//   out[t,h] = sum_s softmax(l)_s c_s,  lse[t,h] = log sum_s exp(l_s)
//
// Rows and tiles.  The (token, head) pairs of a sequence are the rows of one
// attention over its cache rows: all heads share a cache row.  A row tile is
// floor(128 / heads) whole tokens (at most 128 rows, the M of a full-rate
// tcgen05.mma); a key tile is 128 cache rows.  One unit of work is a row tile
// against a key tile.
//
// Why two CTAs work on one row tile.  128 rows x 512 output dims in float32 are
// the whole tensor memory of an SM, so the CTA that accumulates the output has no
// room for the logits, and queries (144 KB) with cache rows of both products do
// not fit one SM's shared memory.  A cluster of two splits the two products:
//   score CTA (rank 0)  holds the 128 x 576 query tile; streams key blocks (128
//            rows x 64 dims, 16 KB) through a ring of five; S = Q K^T (N = 128)
//            into one of four TMEM buffers; eight softmax warps (a row's 128
//            logits over two threads) keep the running maximum and sum and write
//            P (bf16) straight into the value CTA's shared memory.
//   value CTA (rank 1)  streams value blocks (64 rows x 256 dims, 32 KB) through
//            a ring of five and accumulates O += P V (N = 256) in all 512 TMEM
//            columns; its eight other warps rescale O when the score CTA raised a
//            row's maximum by more than 2^8 (rare), and write the result.
// Both products have full-rate shapes: 36 x 64 cycles for S and 16 x 128 for O per
// unit, so the pair is bound by the score CTA at 94% of the two SMs' peak.
//
// Split.  The units of the whole batch, in order, are cut into one equal range
// per cluster, wherever the cuts fall: a batch of short and long sequences, or a
// single long one, fills the GPU evenly.  A row tile that a cut divides leaves
// float32 partials (O, maximum, sum) in the workspace, merged by a second kernel.
// The ranges follow from the lengths alone, which every cluster sums for itself
// (the units of a sequence's row tiles are a sum of floors, in closed form).
#include <cfloat>
#include <climits>

#include <cuda_bf16.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "tma_encode.cuh"

namespace dsa {
namespace {

constexpr int kRows = 128;                       // rows of a row tile
constexpr int kKeys = 128;                       // cache rows of a key tile
constexpr int kBlk = 64 * 128;                   // 64 rows x 64 dims, bf16: 8 KB
constexpr int kNB = kRow / 64;                   // 9 blocks of 64 dims
constexpr int kQTmem = 7;                        // query blocks held in tensor memory
constexpr int kQBytes = (kNB - kQTmem) * 2 * kBlk;  // the others
constexpr int kKStage = 2 * kBlk;                // 128 keys (or query rows) x 64 dims
constexpr int kKStages = 8;
constexpr int kVStage = 4 * kBlk;                // 64 keys x 256 dims
constexpr int kVStages = 5;
constexpr int kPSlot = 4 * kBlk;                 // 128 rows x 128 keys
constexpr int kBig = kQBytes + 2 * kPSlot + kKStages * kKStage;
static_assert(kBig == 2 * kPSlot + kVStages * kVStage, "both CTAs fill the same space");
constexpr int kSmemMax = 232448;                 // 227 KB
constexpr int kThreads = 320;                    // 8 softmax / output warps, producer, MMA
constexpr int kSBufs = 2;
constexpr int kQCol = kSBufs * kKeys;            // TMEM column of the query blocks, 32 columns each
static_assert(kQCol + 32 * kQTmem <= 512, "tensor memory");
constexpr float kRescale = 8.0f;                 // log2: P stays below 2^8
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kIdescS128 = idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdescS64 = idesc_bf16(128, 64, false, false);
constexpr uint32_t kIdescO = idesc_bf16(128, 256, false, true);

enum { kCmdRescale = 0, kCmdFinish = 1, kCmdExit = 2 };

// Same layout in both CTAs of a cluster: remote addresses are a CTA's own ones,
// mapped to the other rank.
struct Small {
    // score CTA
    uint64_t q_full, q_free, k_full[kKStages], k_free[kKStages], s_full[kSBufs], s_free[kSBufs];
    uint64_t x_bar[4];        // the two warps of a quadrant exchange their maxima
    uint64_t p_free[2];       // P V of the slot's tile has completed (from the value CTA)
    uint64_t stat_free;       // the value CTA has read the row statistics
    // value CTA
    uint64_t p_full[2], v_full[kVStages], v_free[kVStages], cmd_full, cmd_done, stat_full;
    uint64_t fin;
    uint32_t tmem_base;
    int abort;
    int plan_b, plan_rt, plan_k0, plan_active;
    long long plan_units, plan_end, plan_total, plan_sum[kThreads / 32];
    int cmd;
    int flags[2][4];          // value CTA: [slot][quadrant] some row's O must be rescaled
    uint32_t key_ok[kSBufs];  // score CTA: [S buffer] bit i: keys 8i..8i+7 are in the pool
    union {
        float xmax[2][2][kRows];  // score CTA: [parity][half][row]
        struct {
            float alpha[2][kRows];  // value CTA: [slot][row]
            float m[kRows], l[kRows];
        } v;
    };
};
static_assert(kBig + sizeof(Small) <= kSmemMax, "shared memory");

struct Meta {  // a row tile whose first part ends its cluster's range
    int parts, row0, rows, pad;
};

struct TcArgs {
    PagedMlaArgs p;
    int clusters;
    int tok_tile;       // tokens per row tile
    int page_pitch;     // rows from one page to the next in the pool's row space
    int box;            // rows per TMA box (divides page_rows, 8..64)
    int oob_row;        // a row coordinate past the pool: TMA fills zeros
    Meta *meta;         // [clusters]
    float *part_ml;     // [2 * clusters][128][2] maximum (log2), sum
    float *part_o;      // [2 * clusters][128][512]
};

// ------------------------------------------------------------------ cluster PTX
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_remote(uint32_t a, uint32_t x) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ void arrive_expect_remote(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// Copy of own shared memory into the other CTA's, counted on a barrier there.
__device__ __forceinline__ void copy_remote(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// 128 rows x 32 bytes of a K-major tile into 8 TMEM columns.
__device__ __forceinline__ void tmem_copy(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// umma_bf16 with A in tensor memory (row m in lane m, two values per column).
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on the barrier of the same address in the CTAs of `mask` when this
// thread's earlier MMAs have completed.
__device__ __forceinline__ void umma_commit_to(uint64_t *bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(mask)
        : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// mbar_wait for a barrier that the other CTA arrives on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, uint32_t *status,
                                                  volatile int *abort_flag) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort_flag) return false;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                report_status(status, DSA_ERR_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
        }
    }
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// ------------------------------------------------------------------ the units of a sequence
struct Seq {
    int n, len, q0, tiles;
};

__device__ __forceinline__ Seq make_seq(const TcArgs &a, int q0, int q1, int len, bool &bad) {
    Seq s;
    s.q0 = q0;
    s.n = q1 - q0;
    s.len = len;
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.p.n_tok && len >= s.n &&
                    len <= static_cast<long long>(a.p.max_pages) * a.p.page_rows;
    if (!ok) {
        bad = true;
        s.n = 0;
    }
    s.tiles = (s.n + a.tok_tile - 1) / a.tok_tile;
    return s;
}

// Visible cache rows of row tile rt (those of its last token), and its key tiles.
__device__ __forceinline__ int tile_seen(const Seq &s, int tt, int rt) { return s.len - s.n + min(s.n, tt * (rt + 1)); }
__device__ __forceinline__ int tile_keys(const Seq &s, int tt, int rt) {
    return (tile_seen(s, tt, rt) + kKeys - 1) / kKeys;
}

// sum_{i < n} floor((a i + b) / m), in O(log m) steps (a, b >= 0).
__device__ __forceinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
    long long r = 0;
    while (n > 0) {
        r += n * (n - 1) / 2 * (a / m) + n * (b / m);
        a %= m;
        b %= m;
        const long long y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const long long t = a;
        a = m;
        m = t;
    }
    return r;
}

// Units of the sequence's first x row tiles.  The units of tile i < tiles - 1 are
// ceil((len - n + tt (i + 1)) / 128).
__device__ __forceinline__ long long units_before(const Seq &s, int tt, int x) {
    if (x <= 0 || s.tiles == 0) return 0;
    const int full = min(x, s.tiles - 1);
    long long r = full > 0 ? floor_sum(full, kKeys, tt, static_cast<long long>(s.len) - s.n + tt + kKeys - 1) : 0;
    if (x >= s.tiles) r += (s.len + kKeys - 1) / kKeys;
    return r;
}

// This cluster's range of units, by all threads of the CTA: each sums the units of
// its share of the sequences, a scan places them, and the thread whose share holds
// the range's start finds sequence, row tile and key tile.
__device__ void make_plan(const TcArgs &a, Small *sm, int cluster, bool report) {
    long long *wsum = sm->plan_sum;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_seq = a.p.n_seq, per = (n_seq + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, n_seq), b1 = min(b0 + per, n_seq);
    long long mine = 0;
    bool bad = false;
    if (b0 < b1) {
        int q = a.p.q_begin[b0];
        for (int b = b0; b < b1; ++b) {
            const int q1 = a.p.q_begin[b + 1];
            const Seq s = make_seq(a, q, q1, a.p.seq_len[b], bad);
            mine += units_before(s, a.tok_tile, s.tiles);
            q = q1;
        }
    }
    if (bad && report) report_status(a.p.status, DSA_ERR_INVALID);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    long long before = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
    }
    const int active = static_cast<int>(min(total, static_cast<long long>(a.clusters)));
    const long long start = cluster < active ? total * cluster / active : 0;
    const long long end = cluster < active ? total * (cluster + 1) / active : 0;
    if (tid == 0) {
        sm->plan_active = active;
        sm->plan_total = total;
        sm->plan_end = end;
        sm->plan_units = end - start;
    }
    if (cluster < active && start >= before && start < before + mine) {
        long long at = before;
        int q = a.p.q_begin[b0];
        for (int b = b0; b < b1; ++b) {
            const int q1 = a.p.q_begin[b + 1];
            const Seq s = make_seq(a, q, q1, a.p.seq_len[b], bad);
            const long long u = units_before(s, a.tok_tile, s.tiles);
            if (start < at + u) {
                int lo = 0, hi = s.tiles;  // last row tile whose first unit is not past the start
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (at + units_before(s, a.tok_tile, mid) <= start)
                        lo = mid;
                    else
                        hi = mid;
                }
                sm->plan_b = b;
                sm->plan_rt = lo;
                sm->plan_k0 = static_cast<int>(start - at - units_before(s, a.tok_tile, lo));
                break;
            }
            at += u;
            q = q1;
        }
    }
    __syncthreads();
}

// Every role walks the cluster's range by itself: piece after piece, a piece being
// a run of key tiles k0..k1-1 of one row tile.  The next sequence's lengths are
// loaded while the current one is worked on.
struct Walk {
    const TcArgs &a;
    int b, rt, k0, k1, nk, next_q1, next_len;
    long long left;
    Seq s;
    __device__ Walk(const TcArgs &args, const Small *sm) : a(args), left(sm->plan_units) {
        if (left <= 0) return;
        b = sm->plan_b;
        rt = sm->plan_rt;
        k0 = sm->plan_k0;
        bool bad = false;
        s = make_seq(a, a.p.q_begin[b], a.p.q_begin[b + 1], a.p.seq_len[b], bad);
        prefetch();
        piece();
    }
    __device__ void prefetch() {
        if (b + 1 < a.p.n_seq) {
            next_q1 = a.p.q_begin[b + 2];
            next_len = a.p.seq_len[b + 1];
        }
    }
    __device__ void piece() {
        nk = tile_keys(s, a.tok_tile, rt);
        k1 = static_cast<int>(min(static_cast<long long>(nk), k0 + left));
    }
    __device__ bool valid() const { return left > 0; }
    __device__ void next() {
        left -= k1 - k0;
        if (left <= 0) return;
        k0 = 0;
        ++rt;
        while (rt >= s.tiles) {  // (units are left, so a sequence with tiles follows)
            if (++b >= a.p.n_seq) {
                left = 0;
                return;
            }
            bool bad = false;
            // an out-of-order q_begin keeps its own pair of borders
            s = make_seq(a, a.p.q_begin[b], next_q1, next_len, bad);
            rt = 0;
            prefetch();
        }
        piece();
    }
    __device__ int tokens() const { return min(a.tok_tile, s.n - rt * a.tok_tile); }
    __device__ int rows() const { return tokens() * a.p.heads; }
    __device__ int seen() const { return tile_seen(s, a.tok_tile, rt); }
    __device__ int64_t row0() const { return static_cast<int64_t>(s.q0 + rt * a.tok_tile) * a.p.heads; }
    // cache rows of key tile kt that some row of the tile sees, 1..128
    __device__ int keys(int kt) const { return min(kKeys, seen() - kt * kKeys); }
};

// Row coordinate, in the pool's row space, of the cache rows s..s+box-1 (one page
// holds them); past the sequence or outside the pool: a coordinate that fills zeros.
__device__ __forceinline__ int box_row(const TcArgs &a, const Walk &w, int s, bool &missing) {
    missing = false;
    if (s >= w.s.len) return a.oob_row;
    const int pi = s / a.p.page_rows;
    const int page = __ldg(a.p.block_table + w.b * a.p.table_stride + pi);
    if (page < 0 || page >= a.p.n_pages) {
        missing = true;
        return a.oob_row;
    }
    return page * a.page_pitch + (s - pi * a.p.page_rows);
}

// ------------------------------------------------------------------ score CTA
__device__ void score_producer(const TcArgs &a, Small *sm, uint8_t *q_sm, uint8_t *k_sm, const CUtensorMap *mq,
                               const CUtensorMap *mkv) {
    const int lane = threadIdx.x & 31;
    const int boxes = kKeys / a.box;  // per block, 2..16: one lane each
    uint32_t it = 0, tile = 0, piece = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next(), ++piece) {
        // the query tile: seven blocks through the ring (the MMA thread moves them on to
        // tensor memory), the last two into their own space once the previous piece's
        // products have read it
        const int halves = w.rows() > 64 ? 2 : 1;
        const int qrow = static_cast<int>(w.row0());
        for (int kb = 0; kb < kQTmem; ++kb, ++it) {
            const int st = it % kKStages;
            if (it >= kKStages && !mbar_wait(&sm->k_free[st], (it / kKStages - 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&sm->k_full[st], halves * kBlk);
            __syncwarp();
            if (lane < halves)
                tma_load_2d(k_sm + st * kKStage + lane * kBlk, mq, &sm->k_full[st], 64 * kb, qrow + 64 * lane);
        }
        if (!ok || (piece > 0 && !mbar_wait(&sm->q_free, (piece - 1) & 1, a.p.status, &sm->abort))) break;
        if (lane == 0) mbar_arrive_expect_tx(&sm->q_full, halves * (kNB - kQTmem) * kBlk);
        __syncwarp();
        if (lane < (kNB - kQTmem) * halves) {
            const int kb = lane >> (halves - 1), hf = lane & (halves - 1);
            tma_load_2d(q_sm + kb * 2 * kBlk + hf * kBlk, mq, &sm->q_full, 64 * (kQTmem + kb), qrow + 64 * hf);
        }
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++tile) {
            const int need = w.keys(kt) > 64 ? kKeys : 64;
            bool missing = false;
            int row = a.oob_row;
            if (lane < boxes) row = box_row(a, w, kt * kKeys + lane * a.box, missing);
            const unsigned miss = __ballot_sync(0xffffffffu, missing);
            uint32_t okbits = 0xFFFFu;
            if (miss) {
                okbits = 0;
                for (int i = 0; i < 16; ++i)
                    if (!((miss >> (i * 8 / a.box)) & 1)) okbits |= 1u << i;
                if (lane == 0) report_status(a.p.status, DSA_ERR_INVALID);
            }
            for (int kb = 0; kb < kNB; ++kb, ++it) {
                const int st = it % kKStages;
                if (it >= kKStages && !mbar_wait(&sm->k_free[st], (it / kKStages - 1) & 1, a.p.status, &sm->abort)) {
                    ok = false;
                    break;
                }
                if (kb == 0) {
                    // (the S buffer of this tile is free: its s_free came before the MMA of the
                    // tile four back could be overtaken; checked here for key_ok's sake)
                    if (tile >= kSBufs &&
                        !mbar_wait(&sm->s_free[tile % kSBufs], (tile / kSBufs - 1) & 1, a.p.status, &sm->abort)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) sm->key_ok[tile % kSBufs] = okbits;
                }
                if (lane == 0) mbar_arrive_expect_tx(&sm->k_full[st], need * 128);
                __syncwarp();
                if (lane * a.box < need)
                    tma_load_2d(k_sm + st * kKStage + lane * a.box * 128, mkv, &sm->k_full[st], 64 * kb, row);
            }
        }
    }
    // every copy has landed before the CTA may exit
    __syncwarp();
    for (uint32_t i = it > kKStages ? it - kKStages : 0; i < it; ++i)
        mbar_wait(&sm->k_full[i % kKStages], (i / kKStages) & 1, a.p.status, nullptr);
    if (piece > 0) mbar_wait(&sm->q_full, (piece - 1) & 1, a.p.status, nullptr);
}

__device__ void score_mma(const TcArgs &a, Small *sm, uint8_t *q_sm, uint8_t *k_sm) {
    const uint32_t tb = sm->tmem_base;
    const uint64_t qd = sdesc_sw128(smem_u32(q_sm), 16, 1024);
    const uint64_t kd = sdesc_sw128(smem_u32(k_sm), 16, 1024);
    uint32_t it = 0, tile = 0, piece = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next(), ++piece) {
        // query blocks to tensor memory, after the previous piece's products
        if (piece > 0 && !mbar_wait(&sm->q_free, (piece - 1) & 1, a.p.status, &sm->abort)) break;
        for (int kb = 0; kb < kQTmem; ++kb, ++it) {
            const int st = it % kKStages;
            if (!mbar_wait(&sm->k_full[st], (it / kKStages) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
                tmem_copy(tb + kQCol + 32 * kb + 8 * k, kd + static_cast<uint64_t>((st * kKStage + k * 32) >> 4));
            umma_commit(&sm->k_free[st]);
        }
        if (!ok || !mbar_wait(&sm->q_full, piece & 1, a.p.status, &sm->abort)) break;
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++tile) {
            const uint32_t buf = tile % kSBufs;
            const uint32_t idesc = w.keys(kt) > 64 ? kIdescS128 : kIdescS64;
            if (tile >= kSBufs && !mbar_wait(&sm->s_free[buf], (tile / kSBufs - 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            for (int kb = 0; kb < kNB; ++kb, ++it) {
                const int st = it % kKStages;
                if (!mbar_wait(&sm->k_full[st], (it / kKStages) & 1, a.p.status, &sm->abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t bd = kd + static_cast<uint64_t>((st * kKStage) >> 4);
                if (kb < kQTmem) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16_ta(tb + kKeys * buf, tb + kQCol + 32 * kb + 8 * k, bd + 2 * k, idesc, kb + k > 0 ? 1u : 0u);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16(tb + kKeys * buf, qd + (((kb - kQTmem) * 2 * kBlk + k * 32) >> 4), bd + 2 * k, idesc, 1u);
                }
                umma_commit(&sm->k_free[st]);
            }
            if (ok) umma_commit(&sm->s_full[buf]);
        }
        if (ok) umma_commit(&sm->q_free);
    }
    umma_commit(&sm->fin);
    mbar_wait(&sm->fin, 0, a.p.status, nullptr);
}

// Warp w: rows 32 (w & 3) + lane, keys 64 (w >> 2) .. + 63 of every tile.
__device__ void score_softmax(const TcArgs &a, Small *sm, uint8_t *p_stage, uint32_t p_remote) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = warp & 3, half = warp >> 2;
    const int r = 32 * quad + lane;
    const uint32_t tb = sm->tmem_base + (static_cast<uint32_t>(32 * quad) << 16) + 64 * half;
    const float c2 = a.p.scale * kLog2e;
    const uint32_t r_alpha = map_rank(smem_u32(&sm->v.alpha[0][0]), 1), r_flags = map_rank(smem_u32(&sm->flags[0][0]), 1);
    const uint32_t r_pfull = map_rank(smem_u32(&sm->p_full[0]), 1), r_stat = map_rank(smem_u32(&sm->stat_full), 1);
    const uint32_t r_m = map_rank(smem_u32(&sm->v.m[0]), 1), r_l = map_rank(smem_u32(&sm->v.l[0]), 1);
    uint32_t tile = 0, piece = 0, xphase = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next(), ++piece) {
        const int rows = w.rows();
        const bool live = 32 * quad < rows;  // some row of the warp belongs to the tile
        // last cache row this thread's token sees
        const int tok = w.rt * a.tok_tile + min(r, rows - 1) / a.p.heads;
        const int pos = w.s.len - w.s.n + tok;
        const int pos0 = w.s.len - w.s.n + w.rt * a.tok_tile;  // the tile's first token
        float m = -INFINITY, l = 0.f;
        for (int kt = w.k0; kt < w.k1; ++kt, ++tile) {
            const uint32_t buf = tile % kSBufs, slot = tile & 1;
            if (!mbar_wait(&sm->s_full[buf], (tile / kSBufs) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t okbits = *reinterpret_cast<volatile uint32_t *>(&sm->key_ok[buf]);
            const bool used = 64 * half < w.keys(kt);  // (with up to 64 keys the upper half was not computed)
            uint32_t x[64];
            if (live && used) {
                tmem_ld32(tb + kKeys * buf, reinterpret_cast<uint32_t(&)[32]>(x[0]));
                tmem_ld32(tb + kKeys * buf + 32, reinterpret_cast<uint32_t(&)[32]>(x[32]));
                tmem_ld_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->s_free[buf]);
            float mx = -INFINITY;
            if (live && used) {
                const int s0 = kt * kKeys + 64 * half;
                if (s0 + 63 > pos0 || okbits != 0xFFFFu) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (s0 + i > pos || !((okbits >> (8 * half + i / 8)) & 1)) x[i] = 0xFF800000u;
                }
#pragma unroll
                for (int i = 0; i < 64; ++i) mx = fmaxf(mx, u2f(x[i]));
                mx *= c2;  // (scale > 0)
            }
            float al = 1.f;
            if (live) {
                sm->xmax[tile & 1][half][r] = mx;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->x_bar[quad]);
                if (!mbar_wait(&sm->x_bar[quad], xphase, a.p.status, &sm->abort)) {
                    ok = false;
                    break;
                }
                xphase ^= 1;
                mx = fmaxf(mx, sm->xmax[tile & 1][half ^ 1][r]);
                if (m == -INFINITY) {
                    m = mx;  // nothing accumulated for the row yet
                } else if (r < rows && mx > m + kRescale) {
                    al = ex2(m - mx);
                    m = mx;
                    l *= al;
                }
            }
            const bool flag = __any_sync(0xffffffffu, al != 1.f);
            if (tile >= 2 && !mbar_wait_cluster(&sm->p_free[slot], (tile / 2 - 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            if (live) {
                const float mu = m == -INFINITY ? 0.f : m;
                uint8_t *pl = p_stage + slot * kPSlot + half * 2 * kBlk;
                if (used) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float p[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            p[i] = ex2(fmaf(u2f(x[8 * c + i]), c2, -mu));
                            l += p[i];
                        }
                        // bf16 weights for the MMA; the sum keeps the float32 values, so the
                        // roundings (half a step, 2^-8 relative) average out in the output
                        *reinterpret_cast<uint4 *>(pl + sw128_offset(r, c)) =
                            make_uint4(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]),
                                       pack_bf16(p[6], p[7]));
                    }
                }
            }
            if (half == 0) {
                if (flag) {
                    st_remote(r_alpha + (slot * kRows + r) * 4, __float_as_uint(al));
                    fence_cluster();
                }
                if (lane == 0) st_remote(r_flags + (slot * 4 + quad) * 4, flag ? 1u : 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                // the warp's 32 rows x 64 keys are 4 KB in a row of the staged tile
                const uint32_t off = slot * kPSlot + half * 2 * kBlk + quad * 4096;
                const bool send = live && used;
                arrive_expect_remote(r_pfull + slot * 8, send ? 4096 : 0);
                if (send) copy_remote(p_remote + off, smem_u32(p_stage) + off, 4096, r_pfull + slot * 8);
            }
        }
        if (!ok) break;
        // row statistics to the value CTA: both halves' sums joined
        if (piece > 0 && !mbar_wait_cluster(&sm->stat_free, (piece - 1) & 1, a.p.status, &sm->abort)) break;
        if (live) {
            // (every read of this parity's maxima is past: the other parity's barrier followed)
            sm->xmax[tile & 1][half][r] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->x_bar[quad]);
            if (!mbar_wait(&sm->x_bar[quad], xphase, a.p.status, &sm->abort)) break;
            xphase ^= 1;
            if (half == 0) {
                l += sm->xmax[tile & 1][1][r];
                st_remote(r_m + r * 4, __float_as_uint(m));
                st_remote(r_l + r * 4, __float_as_uint(l));
            }
            // the partner has read before the next tile writes this parity again
            if (half == 0) __syncwarp();
            if (lane == 0) mbar_arrive(&sm->x_bar[quad]);
            if (!mbar_wait(&sm->x_bar[quad], xphase, a.p.status, &sm->abort)) break;
            xphase ^= 1;
        }
        if (half == 0) {
            __syncwarp();
            if (lane == 0) arrive_remote(r_stat);
        }
    }
}

// ------------------------------------------------------------------ value CTA
__device__ void value_producer(const TcArgs &a, Small *sm, uint8_t *v_sm, const CUtensorMap *mkv) {
    const int lane = threadIdx.x & 31;
    const int boxes = 64 / a.box;  // of 64 rows x 64 dims, 1..8
    uint32_t it = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next()) {
        for (int kt = w.k0; ok && kt < w.k1; ++kt) {
            const int khs = w.keys(kt) > 64 ? 2 : 1;
            // lane i looks up box i of the tile
            bool missing = false;
            int row = a.oob_row;
            if (lane < 2 * boxes) row = box_row(a, w, kt * kKeys + lane * a.box, missing);
            for (int g = 0; g < 2 * khs; ++g, ++it) {
                const int d = g / khs, kh = g % khs, st = it % kVStages;  // dims 256 d .., keys 64 kh ..
                if (it >= kVStages && !mbar_wait(&sm->v_free[st], (it / kVStages - 1) & 1, a.p.status, &sm->abort)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&sm->v_full[st], kVStage);
                __syncwarp();
                // 4 dim blocks x boxes, one per lane (4..32)
                const int bx = lane >> 2, db = lane & 3;
                const int y = __shfl_sync(0xffffffffu, row, kh * boxes + min(bx, boxes - 1));
                if (bx < boxes)
                    tma_load_2d(v_sm + st * kVStage + db * kBlk + bx * a.box * 128, mkv, &sm->v_full[st], 256 * d + 64 * db,
                                y);
            }
        }
    }
    __syncwarp();
    for (uint32_t i = it > kVStages ? it - kVStages : 0; i < it; ++i)
        mbar_wait(&sm->v_full[i % kVStages], (i / kVStages) & 1, a.p.status, nullptr);
}

// Posts a command to the output warps; they start once this thread's MMAs have
// completed (the commit) and it has written the command (its own arrival).
__device__ __forceinline__ bool post_command(const TcArgs &a, Small *sm, int cmd, uint32_t &phase, bool wait) {
    sm->cmd = cmd;
    mbar_arrive(&sm->cmd_full);
    umma_commit(&sm->cmd_full);
    const uint32_t ph = phase;
    phase ^= 1;
    return !wait || mbar_wait(&sm->cmd_done, ph, a.p.status, &sm->abort);
}

__device__ void value_mma(const TcArgs &a, Small *sm, uint8_t *p_sm, uint8_t *v_sm) {
    const int lane = threadIdx.x & 31;
    const uint32_t tb = sm->tmem_base;
    const uint64_t pd = sdesc_sw128(smem_u32(p_sm), 16, 1024);
    const uint64_t vd = sdesc_sw128(smem_u32(v_sm), kBlk, 1024);
    uint32_t it = 0, tile = 0, cphase = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next()) {
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++tile) {
            const uint32_t slot = tile & 1;
            const int khs = w.keys(kt) > 64 ? 2 : 1;
            if (!mbar_wait_cluster(&sm->p_full[slot], (tile >> 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const volatile int *fl = sm->flags[slot];
            if (fl[0] | fl[1] | fl[2] | fl[3]) {
                uint32_t good = 1;
                if (lane == 0) good = post_command(a, sm, kCmdRescale + (slot << 8), cphase, true) ? 1u : 0u;
                good = __shfl_sync(0xffffffffu, good, 0);
                cphase = __shfl_sync(0xffffffffu, cphase, 0);
                if (!good) {
                    ok = false;
                    break;
                }
                tc_fence_after();
            }
            for (int g = 0; g < 2 * khs; ++g, ++it) {
                const int d = g / khs, kh = g % khs, st = it % kVStages;
                if (!mbar_wait(&sm->v_full[st], (it / kVStages) & 1, a.p.status, &sm->abort)) {
                    ok = false;
                    break;
                }
                // rows at or past the sequence's end may hold anything, and 0 x NaN is NaN
                const int z0 = w.s.len - kt * kKeys - 64 * kh;
                if (z0 < 64) {
                    uint8_t *v = v_sm + st * kVStage;
                    for (int i = lane; i < 4 * (64 - z0) * 8; i += 32) {
                        const int db = i & 3, rest = i >> 2;
                        *reinterpret_cast<uint4 *>(v + db * kBlk + z0 * 128 + rest * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16(tb + 256 * d, pd + static_cast<uint64_t>((slot * kPSlot + kh * 2 * kBlk + k * 32) >> 4),
                                  vd + static_cast<uint64_t>((st * kVStage + k * 2048) >> 4), kIdescO,
                                  (kt > w.k0 || kh + k > 0) ? 1u : 0u);
                    umma_commit(&sm->v_free[st]);
                }
                __syncwarp();
            }
            if (ok && lane == 0) umma_commit_to(&sm->p_free[slot], 1);
        }
        if (!ok) break;
        uint32_t good = 1;
        if (lane == 0) good = post_command(a, sm, kCmdFinish, cphase, true) ? 1u : 0u;
        good = __shfl_sync(0xffffffffu, good, 0);
        cphase = __shfl_sync(0xffffffffu, cphase, 0);
        if (!good) break;
        tc_fence_after();
    }
    if (lane == 0) {
        post_command(a, sm, kCmdExit, cphase, false);
        umma_commit(&sm->fin);
        mbar_wait(&sm->fin, 0, a.p.status, nullptr);
    }
    __syncwarp();
}

// Warp w: rows 32 (w & 3) + lane, output dims 256 (w >> 2) .. + 255.
__device__ void value_output(const TcArgs &a, Small *sm, int cluster) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = warp & 3, half = warp >> 2;
    const int r = 32 * quad + lane;
    const uint32_t tb = sm->tmem_base + (static_cast<uint32_t>(32 * quad) << 16) + 256 * half;
    const uint32_t r_free = map_rank(smem_u32(&sm->stat_free), 0);
    uint32_t cphase = 0, piece = 0;
    Walk w(a, sm);
    while (true) {
        if (!mbar_wait(&sm->cmd_full, cphase, a.p.status, &sm->abort)) break;
        cphase ^= 1;
        tc_fence_after();
        const int cmd = *reinterpret_cast<volatile int *>(&sm->cmd);
        if ((cmd & 255) == kCmdExit) break;
        if ((cmd & 255) == kCmdRescale) {
            const int slot = cmd >> 8;
            if (*reinterpret_cast<volatile int *>(&sm->flags[slot][quad])) {
                const float al = sm->v.alpha[slot][r];
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(tb + c, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(u2f(x[i]) * al);
                    tmem_st32(tb + c, x);
                }
                tmem_st_wait();
            }
        } else {
            if (!mbar_wait_cluster(&sm->stat_full, piece & 1, a.p.status, &sm->abort)) break;
            const int rows = w.rows();
            const bool live = r < rows;
            const float l = sm->v.l[r], m = sm->v.m[r];
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const bool whole = w.k0 == 0 && w.k1 == w.nk;
            const int64_t row = w.row0() + r;
            const int64_t pslot = 2 * cluster + (w.k0 == 0 ? 1 : 0);
            if (32 * quad < rows) {
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.p.out) + row * kLatent + 256 * half;
                float *po = a.part_o + (pslot * kRows + r) * kLatent + 256 * half;
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(tb + c, x);
                    tmem_ld_wait();
                    if (live && whole) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4 *>(o + c + i) =
                                make_uint4(pack_bf16(u2f(x[i]) * inv, u2f(x[i + 1]) * inv),
                                           pack_bf16(u2f(x[i + 2]) * inv, u2f(x[i + 3]) * inv),
                                           pack_bf16(u2f(x[i + 4]) * inv, u2f(x[i + 5]) * inv),
                                           pack_bf16(u2f(x[i + 6]) * inv, u2f(x[i + 7]) * inv));
                    } else if (live) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<uint4 *>(po + c + i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                    }
                }
            }
            if (live && half == 0) {
                if (!whole) {
                    a.part_ml[(pslot * kRows + r) * 2] = m;
                    a.part_ml[(pslot * kRows + r) * 2 + 1] = l;
                } else if (a.p.lse) {
                    a.p.lse[row] = l > 0.f ? m * kLn2 + logf(l) : -INFINITY;
                }
            }
            if (tid == 0 && w.k0 == 0 && w.k1 < w.nk) {
                // the row tile goes on in the next clusters' ranges
                const long long last = sm->plan_end - w.k1 + w.nk - 1;
                const int end = static_cast<int>(((last + 1) * sm->plan_active - 1) / sm->plan_total);
                a.meta[cluster] = Meta{end - cluster + 1, static_cast<int>(w.row0()), rows, 0};
            }
            __syncwarp();
            if (lane == 0) arrive_remote(r_free);
            ++piece;
            w.next();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->cmd_done);
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_mla_tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkv) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Small *sm = reinterpret_cast<Small *>(smem + kBig);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = blockIdx.x >> 1, rank = blockIdx.x & 1;
    if (tid == 0) {
        mbar_init(&sm->q_full, 1);
        mbar_init(&sm->q_free, 1);
        for (int i = 0; i < kKStages; ++i) {
            mbar_init(&sm->k_full[i], 1);
            mbar_init(&sm->k_free[i], 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&sm->v_full[i], 1);
            mbar_init(&sm->v_free[i], 1);
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(&sm->s_full[i], 1);
            mbar_init(&sm->s_free[i], 8);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&sm->x_bar[i], 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->p_free[i], 1);
            mbar_init(&sm->p_full[i], 8);
        }
        mbar_init(&sm->stat_free, 8);
        mbar_init(&sm->stat_full, 4);
        mbar_init(&sm->cmd_full, 2);
        mbar_init(&sm->cmd_done, 8);
        mbar_init(&sm->fin, 1);
        sm->abort = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(&sm->tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&mq);
        tma_prefetch_desc(&mkv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    make_plan(a, sm, cluster, rank == 0 && cluster == 0);
    if (tid == 0 && rank == 1) a.meta[cluster].parts = 0;
    cluster_sync_all();  // both CTAs' barriers are set up before either signals the other
    if (rank == 0) {
        if (warp < 8)
            score_softmax(a, sm, smem + kQBytes, map_rank(smem_u32(smem), 1));
        else if (warp == 8)
            score_producer(a, sm, smem, smem + kQBytes + 2 * kPSlot, &mq, &mkv);
        else if (lane == 0)
            score_mma(a, sm, smem, smem + kQBytes + 2 * kPSlot);
    } else {
        if (warp < 8)
            value_output(a, sm, cluster);
        else if (warp == 8)
            value_producer(a, sm, smem + 2 * kPSlot, &mkv);
        else
            value_mma(a, sm, smem, smem + 2 * kPSlot);
    }
    __syncwarp();
    griddep_launch_dependents();
    tc_fence_before();
    cluster_sync_all();  // neither CTA leaves while the other may still write to it
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(sm->tmem_base, 512);
    }
}

// Merge of the row tiles that a cut divided: o = sum_i 2^(m_i - M) o_i / sum_i
// 2^(m_i - M) l_i over the parts, the first in its cluster's second slot, the
// others in the next clusters' first slots.  One CTA per (cluster, 4 rows); most
// find nothing to do.
constexpr int kMergeRows = 4;

__global__ void __launch_bounds__(256) paged_mla_merge_kernel(const TcArgs a) {
    griddep_wait();
    const int c = blockIdx.x;
    const Meta me = a.meta[c];
    if (me.parts == 0) return;
    const int d = (threadIdx.x & 127) * 4;
#pragma unroll 1
    for (int k = 0; k < kMergeRows / 2; ++k) {
        const int r = blockIdx.y * kMergeRows + 2 * k + (threadIdx.x >> 7);
        if (r >= me.rows) continue;
        auto slot = [&](int i) { return static_cast<int64_t>(2 * (c + i) + (i == 0 ? 1 : 0)) * kRows + r; };
        float M = -INFINITY;
        for (int i = 0; i < me.parts; ++i) M = fmaxf(M, a.part_ml[slot(i) * 2]);
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (M != -INFINITY)
            for (int i = 0; i < me.parts; ++i) {
                const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + slot(i) * 2);
                if (ml.x == -INFINITY) continue;
                const float wt = exp2f(ml.x - M);
                const float4 x = *reinterpret_cast<const float4 *>(a.part_o + slot(i) * kLatent + d);
                L += wt * ml.y;
                acc.x += wt * x.x, acc.y += wt * x.y, acc.z += wt * x.z, acc.w += wt * x.w;
            }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int64_t row = static_cast<int64_t>(me.row0) + r;
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.p.out) + row * kLatent + d) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (d == 0 && a.p.lse) a.p.lse[row] = L > 0.f ? M * kLn2 + logf(L) : -INFINITY;
    }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

bool paged_mla_tc_shape(const PagedMlaArgs &a) {
    // (the softmax takes the maximum before it scales: a positive scale)
    if (!a.is_bf16 || a.kv_fp8 || !(a.scale > 0.f) || a.scale > FLT_MAX || a.heads > kRows || a.d_lat != kLatent || a.d_rope != kRope) return false;
    if (a.page_rows % 8 != 0 || a.kv_row_stride % 8 != 0 || a.kv_row_stride < kRow) return false;
    if (a.kv_page_stride % a.kv_row_stride != 0) return false;
    const int64_t pitch = a.kv_page_stride / a.kv_row_stride;
    const auto mis = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.kv) | reinterpret_cast<uintptr_t>(a.out);
    return (mis & 15u) == 0 && (a.n_pages - 1) * pitch + a.page_rows < INT32_MAX &&
           static_cast<int64_t>(a.n_tok) * a.heads < INT32_MAX;
}

size_t paged_mla_tc_scratch(int num_sms) {
    const size_t c = num_sms / 2;
    return align256(c * sizeof(Meta)) + align256(2 * c * kRows * 2 * sizeof(float)) + 2 * c * kRows * kLatent * sizeof(float);
}

cudaError_t launch_paged_mla_tc(const PagedMlaArgs &p, void *scratch, int num_sms, cudaStream_t st) {
    EncodeTiledFn enc = tma_encode_fn();
    if (!enc) return cudaErrorNotSupported;
    TcArgs a;
    a.p = p;
    a.clusters = num_sms / 2;
    a.tok_tile = kRows / p.heads;
    a.page_pitch = static_cast<int>(p.kv_page_stride / p.kv_row_stride);
    a.box = 64;
    while (p.page_rows % a.box != 0) a.box >>= 1;
    const int64_t rows = static_cast<int64_t>(p.n_pages - 1) * a.page_pitch + p.page_rows;
    a.oob_row = static_cast<int>(rows);
    uint8_t *s = static_cast<uint8_t *>(scratch);
    a.meta = reinterpret_cast<Meta *>(s);
    s += align256(a.clusters * sizeof(Meta));
    a.part_ml = reinterpret_cast<float *>(s);
    s += align256(static_cast<size_t>(2) * a.clusters * kRows * 2 * sizeof(float));
    a.part_o = reinterpret_cast<float *>(s);
    CUtensorMap mq, mkv;
    const cuuint32_t es[2] = {1, 1};
    const cuuint64_t qd[2] = {static_cast<cuuint64_t>(kRow), static_cast<cuuint64_t>(p.n_tok) * p.heads};
    const cuuint64_t qs[1] = {static_cast<cuuint64_t>(kRow) * 2};
    const cuuint32_t qb[2] = {64, 64};
    if (enc(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p.q), qd, qs, qb, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const cuuint64_t kd[2] = {static_cast<cuuint64_t>(kRow), static_cast<cuuint64_t>(rows)};
    const cuuint64_t ks[1] = {static_cast<cuuint64_t>(p.kv_row_stride) * 2};
    const cuuint32_t kb[2] = {64, static_cast<cuuint32_t>(a.box)};
    if (enc(&mkv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p.kv), kd, ks, kb, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    cudaError_t e = set_max_dynamic_smem(paged_mla_tc_kernel, kBig + static_cast<int>(sizeof(Small)));
    if (e != cudaSuccess) return e;
    e = launch_pdl(paged_mla_tc_kernel, dim3(2 * a.clusters), dim3(kThreads), kBig + sizeof(Small), st, a, mq, mkv);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_mla_merge_kernel, dim3(a.clusters, kRows / kMergeRows), dim3(256), 0, st, a);
}

}  // namespace dsa
