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
//   score CTA (rank 0)  holds the query tile (latent part in tensor memory, RoPE
//            part in shared memory); streams keys (128 rows x 192 dims, 48 KB)
//            through a ring of three; S = Q K^T (N = 128) into one of two TMEM
//            buffers; eight softmax warps (a row's 128 logits over two threads)
//            keep the running maximum and sum, stage P (bf16) and copy it into the
//            value CTA's shared memory.
//   value CTA (rank 1)  streams values (64 rows x 256 dims, 32 KB) through a ring
//            of five and accumulates O += P V (N = 256) in all 512 TMEM columns;
//            its eight other warps rescale O when the score CTA raised a row's
//            reference maximum (rare), and write the result.
// Both products have full-rate shapes: 36 x 64 cycles for S and 16 x 128 for O per
// unit, which would bound the pair at 94% of the two SMs' peak.
//
// Measured (one B200, calls back to back over inputs that are not in the caches, all
// launches included).  2048 tokens behind 16384 rows, 64 heads, bf16: 4.5 ms (1.1
// PFLOP/s; the power limit lowers the clock, single calls with pauses take 4.05); a unit
// takes some 3000 cycles, and what exceeds 2304 is the keys' copies, which have one
// tile's time to arrive from L2 in, and the MMA thread's waits.  One token at 777 rows:
// 22 us, the fixed part of every call: plan, query, the first tile's way through the
// pipeline, partials and their merge.  Eight tokens at 32768 rows: 99 us, 303 MB at 4
// TB/s behind that part.  32 tokens at up to 24000 packed FP8 rows: 163 us (215 MB): with
// one S buffer the MMAs, the softmax and the widening, 3000 to 4000 cycles a tile each,
// wait for one another.
//
// Split.  The units of the whole batch, in order, are cut into one equal range
// per cluster, wherever the cuts fall: a batch of short and long sequences, or a
// single long one, fills the GPU evenly.  A row tile that a cut divides leaves
// float32 partials (O, maximum, sum) in the workspace, merged by a second kernel.
// The ranges follow from the lengths alone, which every cluster sums for itself
// (the units of a sequence's row tiles are a sum of floors, in closed form).
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cstddef>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "tma_encode.cuh"

namespace dsa {
namespace {

constexpr int kRows = 128;                       // rows of a row tile
constexpr int kKeys = 128;                       // cache rows of a key tile
constexpr int kBlk = 64 * 128;                   // 64 rows x 64 dims, bf16: 8 KB
constexpr int kNB = kRow / 64;                   // 9 blocks of 64 dims
constexpr int kQTmem = 8;                        // query blocks held in tensor memory (the latent ones)
constexpr int kQBytes = (kNB - kQTmem) * 2 * kBlk;  // the RoPE block, in shared memory
constexpr int kKBlocks = 3;                      // 64-dim blocks per stage
constexpr int kKStage = kKBlocks * 2 * kBlk;     // 128 keys (or query rows) x 192 dims
constexpr int kKStages = kNB / kKBlocks;
constexpr int kVStage = 4 * kBlk;                // 64 keys x 256 dims
constexpr int kVStages = 5;
constexpr int kPSlot = 4 * kBlk;                 // 128 rows x 128 keys
constexpr int kBig = kQBytes + 2 * kPSlot + kKStages * kKStage;
static_assert(kBig == 2 * kPSlot + kVStages * kVStage, "both CTAs fill the same space");
// Packed FP8 rows, score CTA: two tiles of codes (128 keys x 512 bytes), one of RoPE
// keys; value CTA: units of 32 keys, codes as they come and widened to fp16.  (Whole
// 656-byte rows copied as they lie and laid out for the MMA by two warps: 210 us where
// this takes 205, the layout having no second buffer to work ahead in.)
constexpr int kCodes = 8 * kBlk;
constexpr int kRawStage = 2 * kBlk, kRawStages = 4;
constexpr int kHStage = 4 * kBlk, kHStages = 3;
static_assert(kBig == kQBytes + 2 * kPSlot + 2 * kCodes + 2 * kBlk, "shared memory, FP8 score CTA");
static_assert(kBig == 2 * kPSlot + kRawStages * kRawStage + kHStages * kHStage, "shared memory, FP8 value CTA");
constexpr int kSmemMax = 232448;                 // 227 KB
constexpr int kThreads = 384;                    // 8 softmax / output warps, producer, MMA; FP8: row scales; idle
constexpr int kSBufs = 2;
constexpr int kQCol = kSBufs * kKeys;            // TMEM column of the query blocks, 32 columns each
static_assert(kQCol + 32 * kQTmem <= 512, "tensor memory");
// A row's reference maximum is raised only when it grew by more than 2^32 (each time
// costs the pair a stop): weights below 2^32 over 2^20 rows stay far inside float32
// and bf16, whose precision does not depend on the scale.
constexpr float kRescale = 32.0f;
// Packed FP8 rows: a weight times its row's scale goes to the MMA as fp16, 2^4 at the
// reference maximum, which is of that product over the rows that a token sees: below
// 2^15 (with a scale's mantissa) until the reference is raised, and rounded to fp16's
// smallest step only 2^-28 under it.  Where the scales of a tile's rows lie within 2^8
// of one another, the largest one stands for all of them, seen or not: the reference is
// then up to 2^8 above the product, and the smallest step 2^-20 under it.
constexpr float kRescaleFp8 = 10.0f;
constexpr float kShiftFp8 = 4.0f;
constexpr uint32_t kSpreadFp8 = 8u << 23;  // of a float's bits
// A row's weight alone, in the same unit, is its product over its scale: scales below
// 2^-60, or 2^-100 of the tile's largest, count as that much in the reference (log2),
// which keeps the weights and their sum finite in float32.
constexpr float kLowScaleFp8 = -60.0f, kLowInTileFp8 = -100.0f;
constexpr uint32_t kNoRow = 0x80000000u;         // scale of a row nobody sees
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kIdescS = idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdescO = idesc_bf16(128, 256, false, true);
constexpr uint32_t kIdescS8 = idesc_e4m3(128, 128);
constexpr uint32_t kIdescO16 = idesc_f16(128, 256, false, true);

enum { kCmdRescale = 0, kCmdFinish = 1, kCmdExit = 2 };

struct Seq {  // one sequence's new tokens, rows, first query row, row tiles
    int n, len, q0, tiles;
};
struct Box {  // a TMA copy of cache rows: page and 8-row group in it
    int page, group;
    bool missing;
};

// Same layout in both CTAs of a cluster: remote addresses are a CTA's own ones,
// mapped to the other rank.
struct Small {
    // score CTA
    uint64_t q_full, q_free, k_full[kKStages], k_free[kKStages], s_full[kSBufs], s_free[kSBufs];
    uint64_t x_bar[4];        // the two warps of a quadrant have written their maxima
    uint64_t p_free[2];       // P V of the slot's tile has completed (from the value CTA)
    uint64_t p_got[2];        // the slot's tile has arrived there
    uint64_t out_done;        // the value CTA has written a piece's result (its P slots are free)
    // value CTA
    uint64_t p_full[2], v_full[kVStages], v_free[kVStages], cmd_full, cmd_done, stat_full;
    uint64_t fin;
    // packed FP8 rows
    uint64_t sig_full[2], sig_free[2];                // score CTA: row scales of the tiles of either parity
    int sig_exp[2], sig_gap[2];                       // .. their power of two; 1: some key of the tile has none, 2: far apart
    uint64_t h_full[kHStages], h_free[kHStages];      // value CTA: widened units
    uint32_t tmem_base;
    int abort;
    int plan_b, plan_rt, plan_k0, plan_active;
    Seq plan_seq;
    int plan_q1;              // q_begin[plan_b + 1]
    Box plan_box[16];         // of the first key tile
    long long plan_units, plan_end, plan_total, plan_first, plan_sum[kThreads / 32];
    int cmd;
    int flags[2][4];          // value CTA: [slot][quadrant] 1: some row's O must be rescaled; 2: clean the values
    uint32_t key_ok[kSBufs];  // score CTA: [S buffer] bit i: keys 8i..8i+7 are in the pool
    union {
        struct alignas(16) {  // (the scales are read 16 bytes at a time)
            float sigma[2][kKeys];      // score CTA: [tile parity] row scales
            uint16_t xmax[2][2][kRows];  // [tile parity][half][row] maxima, bf16
            int nf[2][4];               // [tile parity][quadrant] the upper half has a logit that is not finite
        } q;
        struct {
            float alpha[2][kRows];  // value CTA: [slot][row]
            float factor[kRows];    // .. what a piece's O is multiplied by
        } v;
    };
};
static_assert(kBig + sizeof(Small) <= kSmemMax, "shared memory");
static_assert(offsetof(Small, q.sigma) % 16 == 0, "row scales");

struct Meta {  // a row tile whose first part ends its cluster's range
    int parts, row0, rows, pad;
};

struct TcArgs {
    PagedMlaArgs p;
    int clusters;
    int tok_tile;       // tokens per row tile
    int max_len;        // rows of a block-table row; 1025 short of int32's end, for the sums of positions
    int box;            // rows per TMA copy (divides page_rows, 8..64)
    Meta *meta;         // [clusters]
    float *part_ml;     // [2 * clusters][2][128] maximum (log2), sum
    float *part_o;      // [2 * clusters][512][128]
    const uint8_t *q8;  // packed FP8 rows: the queries' latent part as two E4M3 terms [rows][2][512]
    const float *q8_scale;  // [rows] their power-of-two scale
};

// ------------------------------------------------------------------ cluster PTX
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// A store to the other CTA's shared memory, counted (4 bytes) on a barrier there.
__device__ __forceinline__ void st_remote(uint32_t a, uint32_t x, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(a), "r"(x), "r"(bar)
                 : "memory");
}
// (relaxed: what the barrier announces comes by copies and stores that it counts
// itself; a release at cluster scope waits 2000 cycles for earlier stores)
__device__ __forceinline__ void arrive_expect_remote(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
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
// The same with 8-bit E4M3 operands (four values per column).
__device__ __forceinline__ void umma_e4m3_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// For what ordinary reads and writes of this CTA precede.
__device__ __forceinline__ void arrive_remote_release(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
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
// mbar_wait in fewer instructions: the roles' loops wait in some thirty places, and
// together they have to stay in the instruction cache.  Acquires at cluster scope, for
// the barriers that the other CTA arrives on.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, uint32_t *status, volatile int *abort_flag) {
    uint32_t it = 0;
    uint64_t t0 = 0;
#pragma unroll 1
    while (!mbar_try_wait_cluster(bar, parity)) {
        if ((++it & 255u) == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (abort_flag && *abort_flag) return false;
            if (now - t0 > kWaitLimitNs) {
                report_status(status, DSA_ERR_TIMEOUT);
                if (abort_flag) *abort_flag = 1;
                return false;
            }
        }
    }
    return true;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 8 TMEM columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two float32 operations in one instruction, on pairs in 64-bit registers (packed FP8
// decode 169 us where single ones took 188: fewer instructions to fetch, no spills).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// Two E4M3 codes as two fp16 (exact).
__device__ __forceinline__ uint32_t widen2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// ------------------------------------------------------------------ the units of a sequence
__device__ __forceinline__ Seq make_seq(const TcArgs &a, int q0, int q1, int len, bool &bad) {
    Seq s;
    s.q0 = q0;
    s.n = q1 - q0;
    s.len = len;
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.p.n_tok && len >= s.n && len <= a.max_len;
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

// sum_{i < n} floor((a i + b) / 128): points under a line, by the Euclidean reduction that
// swaps its axes (slope and divisor as in a gcd), in O(log 128) steps (a <= 128, n < 2^24:
// a n stays in 32 bits).
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t a, uint32_t b) {
    long long r = static_cast<long long>(n) * (b >> 7);
    b &= 127;
    uint32_t m = 128;
    while (true) {
        if (a >= m) {
            r += static_cast<long long>(n) * (n - 1) / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            r += static_cast<long long>(n) * (b / m);
            b %= m;
        }
        const uint32_t y = a * n + b;
        if (y < m) return r;
        n = y / m;
        b = y % m;
        const uint32_t t = a;
        a = m;
        m = t;
    }
}

// Units of the sequence's first x row tiles.  The units of tile i < tiles - 1 are
// ceil((len - n + tt (i + 1)) / 128).
__device__ __forceinline__ long long units_before(const Seq &s, int tt, int x) {
    if (x <= 0 || s.tiles == 0) return 0;
    const int full = min(x, s.tiles - 1);
    long long r = full > 0 ? floor_sum(full, tt, static_cast<uint32_t>(s.len - s.n) + tt + kKeys - 1) : 0;
    if (x >= s.tiles) r += (s.len + kKeys - 1) / kKeys;
    return r;
}

// The page of cache rows s..s+box-1 (one page holds them) as a TMA coordinate, and
// their 8-row group in it; past the sequence or outside the pool: page n_pages, for
// which TMA fills zeros.
__device__ __forceinline__ Box find_box(const TcArgs &a, const Seq &q, int b, int s) {
    Box x = {a.p.n_pages, 0, false};
    if (s >= q.len) return x;
    const int pi = s / a.p.page_rows;
    const int page = __ldg(a.p.block_table + b * a.p.table_stride + pi);
    if (page < 0 || page >= a.p.n_pages) {
        x.missing = true;
        return x;
    }
    x.page = page;
    x.group = (s - pi * a.p.page_rows) >> 3;
    return x;
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
                sm->plan_b = b;
                sm->plan_first = start - at;  // unit of the sequence
                break;
            }
            at += u;
            q = q1;
        }
    }
    __syncthreads();
    // the last row tile whose first unit is not past it: every thread tries one of
    // kThreads places, twice for long chunks
    if (sm->plan_units > 0) {
        const int b = sm->plan_b;
        const long long unit = sm->plan_first;
        const Seq s = make_seq(a, a.p.q_begin[b], a.p.q_begin[b + 1], a.p.seq_len[b], bad);
        int lo = 0, span = s.tiles;  // the tile is in lo .. lo + span - 1
        if (tid == 0) sm->plan_rt = 0;
        while (true) {
            const int step = (span + kThreads - 1) / kThreads;
            const int x = lo + tid * step;
            __syncthreads();
            if (tid * step < span) {
                const long long u0 = units_before(s, a.tok_tile, x);
                const long long u1 = units_before(s, a.tok_tile, min(x + step, lo + span));
                if (u0 <= unit && unit < u1) {
                    sm->plan_rt = x;
                    sm->plan_k0 = static_cast<int>(unit - u0);
                }
            }
            __syncthreads();
            if (step == 1) break;  // (uniform)
            span = min(step, lo + span - sm->plan_rt);
            lo = sm->plan_rt;
        }
        // what every role reads first: looked up here, before the copies load the memory
        if (tid == 0) {
            sm->plan_seq = s;
            sm->plan_q1 = a.p.q_begin[b + 1];
        }
        if (tid < kKeys / a.box) sm->plan_box[tid] = find_box(a, s, b, sm->plan_k0 * kKeys + tid * a.box);
    }
}

// Every role walks the cluster's range by itself: piece after piece, a piece being
// a run of key tiles k0..k1-1 of one row tile.  The next sequence's lengths are
// loaded while the current one is worked on.
struct Walk {
    const TcArgs &a;
    int b, rt, k0, k1, nk, q1, next_q1, next_len;  // q1: q_begin[b + 1]
    long long left;
    Seq s;
    __device__ Walk(const TcArgs &args, const Small *sm) : a(args), left(sm->plan_units) {
        if (left <= 0) return;
        b = sm->plan_b;
        rt = sm->plan_rt;
        k0 = sm->plan_k0;
        s = sm->plan_seq;
        next_q1 = sm->plan_q1;
        prefetch();
        piece();
    }
    __device__ void prefetch() {
        q1 = next_q1;
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
            s = make_seq(a, q1, next_q1, next_len, bad);
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

// Copies of cache rows land as [8-row group][64-dim block][8 rows][128 bytes], a
// swizzle atom per (group, block): a run of blocks of a whole page comes with one
// instruction (each costs the issuing warp some 300 cycles), and both products'
// descriptors take the strides between groups and blocks.
__device__ __forceinline__ void tma_load_rows(void *dst, const CUtensorMap *map, uint64_t *bar, int block, const Box &x) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(0), "r"(block), "r"(x.group), "r"(x.page)
        : "memory");
}

// The RoPE keys of packed FP8 rows: [8-row group][8 rows][128 bytes].
__device__ __forceinline__ void tma_load_rope(void *dst, const CUtensorMap *map, uint64_t *bar, const Box &x) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(0), "r"(x.group), "r"(x.page)
        : "memory");
}

// ------------------------------------------------------------------ score CTA
// Stage i of the ring holds blocks 3i..3i+2 of the key tiles, and of the query tile
// before them: constant addresses let the MMA thread issue at full rate.
__device__ void score_producer(const TcArgs &a, Small *sm, uint8_t *q_sm, uint8_t *p_stage, uint8_t *k_sm, const CUtensorMap *mq,
                               const CUtensorMap *mk) {
    const int lane = threadIdx.x & 31;
    const int boxes = kKeys / a.box;  // per stage, 2..16: one lane each
    uint32_t fills = 0, tile = 0, q_use = 0;  // fills of each stage so far
    bool ok = true;
    auto stage_free = [&](int i) {
        return fills == 0 || wait_bar(&sm->k_free[i], (fills - 1) & 1, a.p.status, &sm->abort);
    };
    uint32_t piece = 0, part = 0;  // part: stages filled of the current round
    for (Walk w(a, sm); ok && w.valid(); w.next(), ++piece) {
        Box x = {a.p.n_pages, 0, false};
        if (lane < boxes) x = piece == 0 ? sm->plan_box[lane] : find_box(a, w.s, w.b, w.k0 * kKeys + lane * a.box);
        const bool small = w.rows() <= 64;
        const int qrow = static_cast<int>(w.row0());
        // More than 64 rows: the latent blocks of the query tile come through the ring, and
        // the MMA thread moves them on to tensor memory; up to 64 rows they fit the space
        // where P is staged, and the key blocks need not wait for them.
        if (!small) {
            for (int i = 0; ok && i < kKStages; ++i) {
                const int nb = i < kKStages - 1 ? kKBlocks : kQTmem - kKBlocks * (kKStages - 1);
                if (!stage_free(i)) {
                    ok = false;
                    break;
                }
                part = i + 1;
                if (lane == 0) mbar_arrive_expect_tx(&sm->k_full[i], 2 * nb * kBlk);
                __syncwarp();
                if (lane < nb * 2)
                    tma_load_2d(k_sm + i * kKStage + lane * kBlk, mq, &sm->k_full[i], 64 * (kKBlocks * i + (lane >> 1)),
                                qrow + 64 * (lane & 1));
            }
            if (!ok) break;
            ++fills;
            part = 0;
        }
        auto load_query = [&]() {
            if (piece > 0 && !wait_bar(&sm->q_free, (piece - 1) & 1, a.p.status, &sm->abort)) return false;
            if (small)  // the staged P of the last two tiles has left
                for (uint32_t t = tile > 2 ? tile - 2 : 0; t < tile; ++t)
                    if (!wait_bar(&sm->p_got[t & 1], (t >> 1) & 1, a.p.status, &sm->abort)) return false;
            ++q_use;
            if (lane == 0) mbar_arrive_expect_tx(&sm->q_full, (small ? kNB : 2) * kBlk);
            __syncwarp();
            if (small) {
                if (lane < kNB)
                    tma_load_2d(lane < kQTmem ? p_stage + lane * kBlk : q_sm, mq, &sm->q_full, 64 * lane, qrow);
            } else if (lane < 2) {
                tma_load_2d(q_sm + lane * kBlk, mq, &sm->q_full, 64 * kQTmem, qrow + 64 * lane);
            }
            return true;
        };
        if (piece == 0 || !small) ok = load_query();
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++tile) {
            const int need = w.keys(kt) > 64 ? kKeys : 64;
            const unsigned miss = __ballot_sync(0xffffffffu, x.missing);
            uint32_t okbits = 0xFFFFu;
            if (miss) {
                okbits = 0;
                for (int i = 0; i < 16; ++i)
                    if (!((miss >> (i * 8 / a.box)) & 1)) okbits |= 1u << i;
                if (lane == 0) report_status(a.p.status, DSA_ERR_INVALID);
            }
            // key_ok of this tile's S buffer: its previous tile has been read
            if (tile >= kSBufs && !wait_bar(&sm->s_free[tile % kSBufs], (tile / kSBufs - 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            if (lane == 0) sm->key_ok[tile % kSBufs] = okbits;
            for (int i = 0; i < kKStages; ++i) {
                if (!stage_free(i)) {
                    ok = false;
                    break;
                }
                part = i + 1;
                if (lane == 0) mbar_arrive_expect_tx(&sm->k_full[i], need * kKBlocks * 128);
                __syncwarp();
                if (lane * a.box < need)
                    tma_load_rows(k_sm + i * kKStage + lane * a.box * kKBlocks * 128, mk, &sm->k_full[i], kKBlocks * i, x);
            }
            if (!ok) break;
            ++fills;
            part = 0;
            // (a later piece's first key blocks are on their way before its query tile)
            if (kt == w.k0 && piece > 0 && small && !load_query()) {
                ok = false;
                break;
            }
            // the next tile's pages are looked up while this one's copies run
            if (kt + 1 < w.k1 && lane < boxes) x = find_box(a, w.s, w.b, (kt + 1) * kKeys + lane * a.box);
        }
    }
    // every copy has landed before the CTA may exit
    __syncwarp();
    for (uint32_t i = 0; i < kKStages; ++i) {
        const uint32_t n = fills + (i < part ? 1 : 0);
        if (n > 0) wait_bar(&sm->k_full[i], (n - 1) & 1, a.p.status, nullptr);
    }
    if (q_use > 0) wait_bar(&sm->q_full, (q_use - 1) & 1, a.p.status, nullptr);
}

// One unit's 36 MMAs into S buffer buf.  Tensor memory is allocated whole, so its
// base is 0 and the query's columns and the stages' descriptors follow from one base
// each; only the S buffer's column changes from tile to tile.  One body for both
// buffers: with a copy of it for each, the MMAs waited for instructions (an MMA of this
// shape takes 64 cycles and its issue some 60).
// A tile of 64 keys or fewer multiplies what an earlier tile left in the upper
// half too; those columns are not read.
__device__ __forceinline__ bool score_tile(const TcArgs &a, Small *sm, uint32_t q_addr, uint32_t k_addr, uint32_t parity,
                                           uint32_t buf) {
    const uint32_t d = kKeys * buf;
#pragma unroll
    for (int i = 0; i < kKStages; ++i) {
        if (!wait_bar(&sm->k_full[i], parity, a.p.status, &sm->abort)) return false;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < kKBlocks; ++j) {
            const int kb = i * kKBlocks + j;
            const uint64_t bd = sdesc_sw128(k_addr + i * kKStage + j * 1024, 16, kKBlocks * 1024);
            if (kb < kQTmem) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_bf16_ta(d, kQCol + 32 * kb + 8 * k, bd + 2 * k, kIdescS, kb + k > 0 ? 1u : 0u);
            } else {
                const uint64_t ad = sdesc_sw128(q_addr, 16, 1024);
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_bf16(d, ad + 2 * k, bd + 2 * k, kIdescS, 1u);
            }
        }
        umma_commit(&sm->k_free[i]);
    }
    umma_commit(&sm->s_full[buf]);
    return true;
}

__device__ void score_mma(const TcArgs &a, Small *sm, uint8_t *q_sm, uint8_t *p_stage, uint8_t *k_sm) {
    const uint32_t q_addr = smem_u32(q_sm), k_addr = smem_u32(k_sm), p_addr = smem_u32(p_stage);
    uint32_t tile = 0, piece = 0, fills = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next(), ++piece) {
        // query blocks to tensor memory, after the previous piece's products
        if (piece > 0 && !wait_bar(&sm->q_free, (piece - 1) & 1, a.p.status, &sm->abort)) break;
        if (w.rows() > 64) {
#pragma unroll
            for (int i = 0; i < kKStages; ++i) {
                if (!ok || !wait_bar(&sm->k_full[i], fills & 1, a.p.status, &sm->abort)) {
                    ok = false;
                    continue;
                }
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < kKBlocks; ++j) {
                    const int kb = i * kKBlocks + j;
                    if (kb >= kQTmem) continue;
                    const uint64_t kd = sdesc_sw128(k_addr + i * kKStage + j * 2 * kBlk, 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_copy(kQCol + 32 * kb + 8 * k, kd + 2 * k);
                }
                umma_commit(&sm->k_free[i]);
            }
            ++fills;
            if (!ok) break;
        }
        if (!wait_bar(&sm->q_full, piece & 1, a.p.status, &sm->abort)) break;
        if (w.rows() <= 64) {
            // (rows 64..127 take what follows in shared memory: rows of no token)
            tc_fence_after();
#pragma unroll
            for (int kb = 0; kb < kQTmem; ++kb)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tmem_copy(kQCol + 32 * kb + 8 * k, sdesc_sw128(p_addr + kb * kBlk, 16, 1024) + 2 * k);
        }
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++tile, ++fills) {
            const uint32_t buf = tile % kSBufs;
            if (tile >= kSBufs && !wait_bar(&sm->s_free[buf], (tile / kSBufs - 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            ok = score_tile(a, sm, q_addr, k_addr, fills & 1, buf);
        }
        if (ok) umma_commit(&sm->q_free);
    }
    umma_commit(&sm->fin);
    wait_bar(&sm->fin, 0, a.p.status, nullptr);
}

// Packed FP8 rows, score CTA.  q = s (q1 + q2) with q1, q2 in E4M3 and s a power of
// two: a bf16 value's eight significant bits are two terms of four, so the latent
// logits come from the codes as they are, two 8-bit MMAs (K = 32, 64 cycles) in the
// place of two 16-bit ones, and nothing is widened here.  The RoPE part has its own
// accumulator (the row scale applies to the latent part alone), which leaves room
// for one S buffer.  Barriers 0 and 1 of the ring: codes of the tiles of either
// parity; 2: RoPE keys.
__device__ void score_producer_fp8(const TcArgs &a, Small *sm, uint8_t *q_sm, uint8_t *p_stage, uint8_t *c_sm, uint8_t *r_sm,
                                   const CUtensorMap *mq, const CUtensorMap *mq8, const CUtensorMap *mk,
                                   const CUtensorMap *mr) {
    const int lane = threadIdx.x & 31;
    const int boxes = kKeys / a.box;
    uint32_t fills[3] = {0, 0, 0};
    uint32_t tile = 0, piece = 0, q_use = 0;
    bool ok = true;
    auto stage_free = [&](int i) {
        return fills[i] == 0 || wait_bar(&sm->k_free[i], (fills[i] - 1) & 1, a.p.status, &sm->abort);
    };
    for (Walk w(a, sm); ok && w.valid(); w.next(), ++piece) {
        Box x = {a.p.n_pages, 0, false};
        if (lane < boxes) x = piece == 0 ? sm->plan_box[lane] : find_box(a, w.s, w.b, w.k0 * kKeys + lane * a.box);
        const bool small = w.rows() <= 64;
        const int qrow = static_cast<int>(w.row0());
        // more than 64 rows: q1 through one code stage, q2 through the other; else both
        // through the space where P is staged
        if (!small) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!ok || !stage_free(i)) {
                    ok = false;
                    continue;
                }
                ++fills[i];
                if (lane == 0) mbar_arrive_expect_tx(&sm->k_full[i], kCodes);
                __syncwarp();
                if (lane < 8)
                    tma_load_2d(c_sm + i * kCodes + lane * kBlk, mq8, &sm->k_full[i], 512 * i + 128 * (lane >> 1),
                                qrow + 64 * (lane & 1));
            }
            if (!ok) break;
        }
        auto load_query = [&]() {
            if (piece > 0 && !wait_bar(&sm->q_free, (piece - 1) & 1, a.p.status, &sm->abort)) return false;
            if (small)  // the staged P of the last two tiles has left
                for (uint32_t t = tile > 2 ? tile - 2 : 0; t < tile; ++t)
                    if (!wait_bar(&sm->p_got[t & 1], (t >> 1) & 1, a.p.status, &sm->abort)) return false;
            ++q_use;
            if (lane == 0) mbar_arrive_expect_tx(&sm->q_full, (small ? 9 : 2) * kBlk);
            __syncwarp();
            if (small && lane < 8) tma_load_2d(p_stage + lane * kBlk, mq8, &sm->q_full, 128 * lane, qrow);
            if (lane >= 8 && lane < (small ? 9 : 10))
                tma_load_2d(q_sm + (lane - 8) * kBlk, mq, &sm->q_full, kLatent, qrow + 64 * (lane - 8));
            return true;
        };
        if (piece == 0 || !small) ok = load_query();
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++tile) {
            const int need = w.keys(kt) > 64 ? kKeys : 64;
            if (__any_sync(0xffffffffu, x.missing) && lane == 0) report_status(a.p.status, DSA_ERR_INVALID);
            const int st = tile & 1;
            if (!(st ? stage_free(1) : stage_free(0))) {
                ok = false;
                break;
            }
            if (st)
                ++fills[1];
            else
                ++fills[0];
            if (lane == 0) mbar_arrive_expect_tx(&sm->k_full[st], need * 512);
            __syncwarp();
            if (lane * a.box < need) tma_load_rows(c_sm + st * kCodes + lane * a.box * 512, mk, &sm->k_full[st], 0, x);
            if (!stage_free(2)) {
                ok = false;
                break;
            }
            ++fills[2];
            if (lane == 0) mbar_arrive_expect_tx(&sm->k_full[2], need * 128);
            __syncwarp();
            if (lane * a.box < need) tma_load_rope(r_sm + lane * a.box * 128, mr, &sm->k_full[2], x);
            if (kt == w.k0 && piece > 0 && small && !load_query()) {
                ok = false;
                break;
            }
            if (kt + 1 < w.k1 && lane < boxes) x = find_box(a, w.s, w.b, (kt + 1) * kKeys + lane * a.box);
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (fills[i] > 0) wait_bar(&sm->k_full[i], (fills[i] - 1) & 1, a.p.status, nullptr);
    if (q_use > 0) wait_bar(&sm->q_full, (q_use - 1) & 1, a.p.status, nullptr);
}

// Row scales of every key tile to shared memory, divided by the tile's largest power
// of two; -0 for a row nobody sees (a visible row may well have scale 0: its latent
// part is zero, its RoPE part still counts).
__device__ void score_scales_fp8(const TcArgs &a, Small *sm) {
    const int lane = threadIdx.x & 31;
    uint32_t tile = 0;
    const uint8_t *kv = static_cast<const uint8_t *>(a.p.kv) + kFp8ScaleOff;
    for (Walk w(a, sm); w.valid(); w.next())
        for (int kt = w.k0; kt < w.k1; ++kt, ++tile) {
            const int s0 = kt * kKeys + 4 * lane;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            int seen = 0;
            const Box x = find_box(a, w.s, w.b, s0);  // (four rows of one 8-row group)
            if (x.page < a.p.n_pages) {
                const uint8_t *row = kv + x.page * a.p.kv_page_stride + (8 * x.group + (s0 & 7)) * a.p.kv_row_stride;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (s0 + i < w.s.len) {
                        v[i] = __ldg(reinterpret_cast<const float *>(row + i * a.p.kv_row_stride));
                        ++seen;
                    }
            }
            // the largest of the finite ones (a token need not see the others), as bits
            uint32_t mx = 0, mn = 0x7FFFFFFFu;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFFu;
                mx = max(mx, u < 0x7F800000u ? u : 0u);
                mn = i < seen ? min(mn, u) : mn;
            }
            mx = __reduce_max_sync(0xffffffffu, mx);
            const bool spread = mn + kSpreadFp8 <= max(mx, kSpreadFp8);
            const uint32_t flags = __reduce_or_sync(0xffffffffu, (seen < 4 ? 1u : 0u) | (spread ? 2u : 0u));
            // (2^-e multiplies a row's sum, which has to stay finite: no less than -80)
            const int e = mx > 0 ? min(max(static_cast<int>(mx >> 23) - 127, -80), 120) : 0;
            const float down = u2f(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = i < seen ? v[i] * down + 0.f : -0.f;
            if (tile >= 2 && !wait_bar(&sm->sig_free[tile & 1], (tile / 2 - 1) & 1, a.p.status, &sm->abort)) return;
            *reinterpret_cast<float4 *>(&sm->q.sigma[tile & 1][4 * lane]) =
                make_float4(v[0], v[1], v[2], v[3]);
            if (lane == 0) {
                sm->sig_exp[tile & 1] = e;
                sm->sig_gap[tile & 1] = static_cast<int>(flags);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->sig_full[tile & 1]);
        }
}

__device__ __forceinline__ bool score_tile_fp8(const TcArgs &a, Small *sm, uint32_t q_addr, uint32_t c_addr, uint32_t r_addr,
                                               int st, uint32_t parity, uint32_t parity_rope) {
    if (!wait_bar(&sm->k_full[st], parity, a.p.status, &sm->abort)) return false;
    tc_fence_after();
    uint64_t bd = sdesc_sw128(c_addr + st * kCodes, 16, 4096);
    uint32_t at = kQCol;
#pragma unroll 1
    for (int j = 0; j < 4; ++j, bd += 1024 >> 4, at += 32)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            umma_e4m3_ta(0, at + 8 * k, bd + 2 * k, kIdescS8, j + k > 0 ? 1u : 0u);
            umma_e4m3_ta(0, at + 128 + 8 * k, bd + 2 * k, kIdescS8, 1u);
        }
    umma_commit(&sm->k_free[st]);
    if (!wait_bar(&sm->k_full[2], parity_rope, a.p.status, &sm->abort)) return false;
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < 4; ++k)
        umma_bf16(kKeys, sdesc_sw128(q_addr, 16, 1024) + 2 * k, sdesc_sw128(r_addr, 16, 1024) + 2 * k, kIdescS, k > 0 ? 1u : 0u);
    umma_commit(&sm->k_free[2]);
    umma_commit(&sm->s_full[st]);
    return true;
}

__device__ void score_mma_fp8(const TcArgs &a, Small *sm, uint8_t *q_sm, uint8_t *p_stage, uint8_t *c_sm, uint8_t *r_sm) {
    const uint32_t q_addr = smem_u32(q_sm), c_addr = smem_u32(c_sm), r_addr = smem_u32(r_sm), p_addr = smem_u32(p_stage);
    uint32_t tile = 0, piece = 0, fill0 = 0, fill1 = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next(), ++piece) {
        if (piece > 0 && !wait_bar(&sm->q_free, (piece - 1) & 1, a.p.status, &sm->abort)) break;
        if (w.rows() > 64) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!ok || !wait_bar(&sm->k_full[i], (i ? fill1 : fill0) & 1, a.p.status, &sm->abort)) {
                    ok = false;
                    continue;
                }
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    tmem_copy(kQCol + 128 * i + 8 * k,
                              sdesc_sw128(c_addr + i * kCodes + (k >> 2) * 2 * kBlk, 16, 1024) + 2 * (k & 3));
                umma_commit(&sm->k_free[i]);
            }
            ++fill0;
            ++fill1;
            if (!ok) break;
        }
        if (!wait_bar(&sm->q_full, piece & 1, a.p.status, &sm->abort)) break;
        if (w.rows() <= 64) {
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 32; ++k)
                tmem_copy(kQCol + 8 * k, sdesc_sw128(p_addr + (k >> 2) * kBlk, 16, 1024) + 2 * (k & 3));
        }
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++tile) {
            if (tile >= 1 && !wait_bar(&sm->s_free[0], (tile - 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int st = tile & 1;
            ok = score_tile_fp8(a, sm, q_addr, c_addr, r_addr, st, (st ? fill1 : fill0) & 1, st);
            if (st)
                ++fill1;
            else
                ++fill0;
        }
        if (ok) umma_commit(&sm->q_free);
    }
    umma_commit(&sm->fin);
    wait_bar(&sm->fin, 0, a.p.status, nullptr);
}

// Softmax.  Warp w: rows 32 (w & 3) + lane, keys 64 (w >> 2) .. + 63 of every tile;
// the two warps of a quadrant exchange their maxima (as bf16, rounded up: any
// reference not far below the maximum will do, as long as both take the same).  A
// loop body that fits the instruction cache matters more than anything else here: a
// thread per row with 128 logits in registers, its loops unrolled, waited for
// instructions more often than it issued one.
__device__ __forceinline__ float bf16_up(float x) {
    // the next bf16 at or above x (x finite or -infinity)
    const uint32_t b = __float_as_uint(x);
    const uint32_t t = b & 0xFFFF0000u;
    return u2f((b & 0xFFFFu) && !(b >> 31) ? t + 0x10000u : t);
}

// Scales far apart: the maximum over 64 keys, those up to `last`, of the weight times its
// own row's scale (log2).  The logits are read from tensor memory again, eight at a time
// in a rolled loop: the scales of a sound cache hardly ever lie that far apart, and the
// same unrolled in the loop over tiles took 173 us of decode where this takes 169.
__device__ __forceinline__ float spread_max(uint32_t taddr, const float *sig, int last, float qs, float c2, float low) {
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 64; c += 8) {
        uint32_t x[8], y[8];
        tmem_ld8(taddr + c, x);
        tmem_ld8(taddr + kKeys + c, y);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float g = sig[c + i];
            const float z = fmaf(u2f(x[i]) * g, qs, u2f(y[i]));
            if (c + i <= last && __float_as_uint(g) != kNoRow) mx = fmaxf(mx, fmaf(z, c2, fmaxf(lg2(fabsf(g)), low)));
        }
    }
    return mx;
}

template <bool kFp8>
__device__ void score_softmax(const TcArgs &a, Small *sm, uint8_t *p_stage, uint32_t p_remote, int cluster) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = warp & 3, half = warp >> 2;
    const int r = 32 * quad + lane;
    const uint32_t tb = (static_cast<uint32_t>(32 * quad) << 16) + 64 * half;
    const float c2 = a.p.scale * kLog2e;
    const uint32_t r_alpha = map_rank(smem_u32(&sm->v.alpha[0][0]), 1), r_flags = map_rank(smem_u32(&sm->flags[0][0]), 1);
    const uint32_t r_pfull = map_rank(smem_u32(&sm->p_full[0]), 1), r_stat = map_rank(smem_u32(&sm->stat_full), 1);
    const uint32_t r_factor = map_rank(smem_u32(&sm->v.factor[0]), 1);
    uint32_t tile = 0, piece = 0, xphase = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next(), ++piece) {
        const int rows = w.rows();
        const bool live = 32 * quad < rows;  // some row of the warp belongs to the tile
        // last cache row this thread's token sees
        const int tok = w.rt * a.tok_tile + min(r, rows - 1) / a.p.heads;
        const int pos = w.s.len - w.s.n + tok;
        const int pos0 = w.s.len - w.s.n + w.rt * a.tok_tile;  // the tile's first token
        const float q8s = kFp8 ? a.q8_scale[w.row0() + min(r, rows - 1)] : 0.f;
        float m = -INFINITY, l = 0.f, lp = 0.f;  // lp: of the rounded weights
        for (int kt = w.k0; kt < w.k1; ++kt, ++tile) {
            const uint32_t slot = tile & 1;  // of P, and of bf16's S buffers
            const uint32_t sbuf = kFp8 ? 0 : slot;
            if (kFp8 && !wait_bar(&sm->sig_full[slot], (tile >> 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            // packed FP8 rows: the tile's row scales are 2^sig_exp times what is in sig (read
            // before the wait for S: what comes after it is on the way to the next MMA)
            const float te = kFp8 ? static_cast<float>(*reinterpret_cast<volatile int *>(&sm->sig_exp[slot])) : 0.f;
            const int sgap = kFp8 ? *reinterpret_cast<volatile int *>(&sm->sig_gap[slot]) : 0;
            if (!wait_bar(&sm->s_full[slot], (tile >> 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int nk = w.keys(kt);
            const bool used = live && 64 * half < nk;
            const float *sig = &sm->q.sigma[slot][64 * half];
            const uint32_t okbits =
                kFp8 ? 0xFFu : *reinterpret_cast<volatile uint32_t *>(&sm->key_ok[slot]) >> (8 * half) & 0xFFu;
            const bool gap = kFp8 ? sgap != 0 : okbits != 0xFFu;
            uint32_t x[64];
            float mspread = INFINITY;  // (scales far apart)
            if (used) {
                if constexpr (!kFp8) {
                    tmem_ld32(tb + kKeys * slot, reinterpret_cast<uint32_t(&)[32]>(x[0]));
                    tmem_ld32(tb + kKeys * slot + 32, reinterpret_cast<uint32_t(&)[32]>(x[32]));
                    tmem_ld_wait();
                } else {
                    // logit over the scale: s sigma S_lat + S_rope
                    const float qs = q8s * ex2(te);
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t y[32];
                        tmem_ld32(tb + c, reinterpret_cast<uint32_t(&)[32]>(x[c]));
                        tmem_ld32(tb + kKeys + c, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 g4 = *reinterpret_cast<const float4 *>(sig + c + i);
                            const uint64_t g[2] = {pair(g4.x, g4.y), pair(g4.z, g4.w)};
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int e = c + i + 2 * k;
                                const float2 z =
                                    unpair(fma2(mul2(pair(u2f(x[e]), u2f(x[e + 1])), g[k]), pair(qs, qs),
                                                pair(u2f(y[i + 2 * k]), u2f(y[i + 2 * k + 1]))));
                                x[e] = __float_as_uint(z.x);
                                x[e + 1] = __float_as_uint(z.y);
                            }
                        }
                    }
                }
            }
            auto free_s = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->s_free[sbuf]);
            };
            if (!kFp8) free_s();
            float mx = -INFINITY;
            // some logit is not finite, in a tile of tokens that do not see the same rows: the
            // row's values may be NaN, and 0 x NaN is NaN for those that do not see it (see
            // clean_stage)
            bool nf = false;
            const int s0 = kt * kKeys + 64 * half;
            if (used && (s0 + 63 > pos0 || gap)) {
                if (kFp8 && (sgap & 2))  // (reads S, so S is free only behind it)
                    mspread = spread_max(tb, sig, pos - s0, q8s * ex2(te), c2,
                                         fmaxf(kLowInTileFp8, kLowScaleFp8 - te)) + te;
                float z4[4] = {0.f, 0.f, 0.f, 0.f};  // NaN where a logit is not finite
                if (kFp8 && pos0 < w.s.len - 1) {    // (in the loop below it would spill)
#pragma unroll
                    for (int i = 0; i < 64; ++i) z4[i & 3] = fmaf(u2f(x[i]), 0.f, z4[i & 3]);
                }
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    if (!kFp8) z4[i & 3] = fmaf(u2f(x[i]), 0.f, z4[i & 3]);
                    if (s0 + i > pos || (kFp8 ? __float_as_uint(sig[i]) == kNoRow : !((okbits >> (i / 8)) & 1)))
                        x[i] = 0xFF800000u;
                }
                nf = __any_sync(0xffffffffu, r < rows && pos0 < w.s.len - 1 && !((z4[0] + z4[1]) + (z4[2] + z4[3]) == 0.f));
            }
            if (kFp8) free_s();
            if (used) {
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 64; i += 4)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], u2f(x[i + k]));
                // (scale > 0; packed FP8 rows: the weight times the tile's power of two)
                mx = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), c2, te);
                if (kFp8) mx = fminf(mx, mspread);
                mx = bf16_up(mx);
            }
            float al = 1.f;
            if (live) {
                sm->q.xmax[slot][half][r] = static_cast<uint16_t>(__float_as_uint(mx) >> 16);
                if (half == 1 && lane == 0) sm->q.nf[slot][quad] = nf;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->x_bar[quad]);
                if (!wait_bar(&sm->x_bar[quad], xphase, a.p.status, &sm->abort)) {
                    ok = false;
                    break;
                }
                xphase ^= 1;
                if (half == 0) nf |= sm->q.nf[slot][quad] != 0;
                mx = fmaxf(mx, u2f(static_cast<uint32_t>(sm->q.xmax[slot][half ^ 1][r]) << 16));
                if (m == -INFINITY) {
                    m = mx;  // nothing accumulated for the row yet
                } else if (r < rows && mx > m + (kFp8 ? kRescaleFp8 : kRescale)) {
                    al = ex2(m - mx);
                    m = mx;
                    l *= al;
                    lp *= al;
                }
            }
            const bool flag = __any_sync(0xffffffffu, al != 1.f);
            // the staged tile two back has left
            if (tile >= 2 && !wait_bar(&sm->p_got[slot], (tile / 2 - 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            if (used) {
                const float mu = (m == -INFINITY ? 0.f : m) - (kFp8 ? kShiftFp8 + te : 0.f);
                const uint64_t c22 = pair(c2, c2), mu2 = pair(-mu, -mu);
                uint64_t l2[2] = {0, 0}, lp2[2] = {0, 0};
                uint8_t *pl = p_stage + slot * kPSlot + half * 2 * kBlk;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float p[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 z = unpair(fma2(pair(u2f(x[8 * c + i]), u2f(x[8 * c + i + 1])), c22, mu2));
                        p[i] = ex2(z.x);
                        p[i + 1] = ex2(z.y);
                        l2[(i / 2) & 1] = add2(l2[(i / 2) & 1], pair(p[i], p[i + 1]));
                    }
                    if constexpr (kFp8) {
                        const float4 ga = *reinterpret_cast<const float4 *>(sig + 8 * c);
                        const float4 gb = *reinterpret_cast<const float4 *>(sig + 8 * c + 4);
                        const uint64_t g[4] = {pair(ga.x, ga.y), pair(ga.z, ga.w), pair(gb.x, gb.y), pair(gb.z, gb.w)};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 z = unpair(mul2(pair(p[2 * i], p[2 * i + 1]), g[i]));
                            p[2 * i] = z.x;
                            p[2 * i + 1] = z.y;
                        }
                    }
                    // bf16 (fp16) weights for the MMA, off by at most half a step, 2^-8 (2^-11) of a
                    // weight.  bf16: O is divided by the sum of the rounded weights, so that an
                    // error that few rows with all the weight share cancels (one such row is
                    // returned as it is); error of the output 0.0017 (float32 weights 0.00165)
                    // where the sum of the float32 weights gave 0.0023, for 2 to 3% of the time.
                    // That sum is for the lse.
                    uint4 pk;
                    uint32_t *pw = reinterpret_cast<uint32_t *>(&pk);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        pw[i] = kFp8 ? pack_f16(p[2 * i], p[2 * i + 1]) : pack_bf16(p[2 * i], p[2 * i + 1]);
                        if (!kFp8) lp2[i & 1] = add2(lp2[i & 1], pair(u2f(pw[i] << 16), u2f(pw[i] & 0xFFFF0000u)));
                    }
                    *reinterpret_cast<uint4 *>(pl + sw128_offset(r, c)) = pk;
                }
                const float2 lps = unpair(add2(lp2[0], lp2[1]));
                if (!kFp8) lp += lps.x + lps.y;
                const float2 ls = unpair(add2(l2[0], l2[1]));
                const float lt = ls.x + ls.y;
                l += kFp8 ? lt * ex2(-te) : lt;
                if (kFp8 && nf) {  // (a scale that is not finite)
#pragma unroll 1
                    for (int i = 0; i < 64; ++i)
                        if (s0 + i > pos || __float_as_uint(sig[i]) == kNoRow)
                            *reinterpret_cast<uint16_t *>(pl + sw128_offset(r, i >> 3) + 2 * (i & 7)) = 0;
                }
            }
            fence_proxy_async_smem();
            if (kFp8) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->sig_free[slot]);
            }
            // (the value CTA stages a piece's result in the P slots)
            if (kt < w.k0 + 2 && piece > 0 && !wait_bar(&sm->out_done, (piece - 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            if (tile >= 2 && !wait_bar(&sm->p_free[slot], (tile / 2 - 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            if (half == 0) {
                if (flag) st_remote(r_alpha + (slot * kRows + r) * 4, __float_as_uint(al), r_pfull + slot * 8);
                if (lane == 0)
                    st_remote(r_flags + (slot * 4 + quad) * 4, (flag ? 1u : 0u) | (nf ? 2u : 0u), r_pfull + slot * 8);
            }
            __syncwarp();
            if (lane == 0) {
                // the warp's 32 rows x 64 keys are 4 KB in a row of the staged tile
                const uint32_t off = slot * kPSlot + half * 2 * kBlk + quad * 4096;
                arrive_expect_remote(r_pfull + slot * 8, (used ? 4096 : 0) + (half ? 0 : flag ? 132 : 4));
                if (used) copy_remote(p_remote + off, smem_u32(p_stage) + off, 4096, r_pfull + slot * 8);
            }
        }
        if (!ok) break;
        // row statistics to the value CTA: both halves' sums joined, through the maxima's
        // place of the next tile's parity (a piece's result is out before the next
        // piece's first P: see out_done).  A row's sum goes in two halves to the places of
        // its own two maxima: x_bar orders a quadrant's two warps and nothing else, so the
        // exchange has to stay in the quadrant's own bytes.
        if (live) {
            uint16_t(*lx)[kRows] = sm->q.xmax[tile & 1];
#pragma unroll 1
            for (int i = 0; i < (kFp8 ? 1 : 2); ++i) {
                const float sum = i == 0 ? l : lp;
                if (half == 1) {
                    lx[0][r] = static_cast<uint16_t>(__float_as_uint(sum));
                    lx[1][r] = static_cast<uint16_t>(__float_as_uint(sum) >> 16);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->x_bar[quad]);
                ok = ok && wait_bar(&sm->x_bar[quad], xphase, a.p.status, &sm->abort);
                xphase ^= 1;
                const float other = u2f(static_cast<uint32_t>(lx[0][r]) | static_cast<uint32_t>(lx[1][r]) << 16);
                if (half == 0 && i == 0) l += other;
                if (half == 0 && i == 1) lp += other;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->x_bar[quad]);  // read, before the place is written again
                ok = ok && wait_bar(&sm->x_bar[quad], xphase, a.p.status, &sm->abort);
                xphase ^= 1;
            }
            if (!ok) break;
        }
        if (half == 0) {
            if (piece > 0 && !wait_bar(&sm->out_done, (piece - 1) & 1, a.p.status, &sm->abort)) break;
            if (live) {
                // a whole piece is divided by its sum and done; a partial one keeps l as its sum
                const bool whole = w.k0 == 0 && w.k1 == w.nk;
                const float d = kFp8 ? l : lp, mr = kFp8 ? m - kShiftFp8 : m;
                const float factor = d != 0.f ? (whole ? 1.f : l) / d : 0.f;
                if (r < rows) {
                    const int64_t pslot = 2 * cluster + (w.k0 == 0 ? 1 : 0);
                    if (!whole) {
                        a.part_ml[pslot * 2 * kRows + r] = mr;
                        a.part_ml[(pslot * 2 + 1) * kRows + r] = l;
                    } else if (a.p.lse) {
                        a.p.lse[w.row0() + r] = l != 0.f ? mr * kLn2 + logf(l) : -INFINITY;
                    }
                }
                st_remote(r_factor + r * 4, __float_as_uint(factor), r_stat);
            }
            __syncwarp();
            if (lane == 0) arrive_expect_remote(r_stat, live ? 128 : 0);
        }
    }
}

// ------------------------------------------------------------------ value CTA
__device__ void value_producer(const TcArgs &a, Small *sm, uint8_t *v_sm, const CUtensorMap *mv) {
    const int lane = threadIdx.x & 31;
    const int boxes = 64 / a.box;  // per stage, 1..8: one lane each
    uint32_t it = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next()) {
        // lane i looks up box i of the tile's 128 rows, a tile ahead
        Box x = {a.p.n_pages, 0, false};
        if (lane < 2 * boxes) x = it == 0 ? sm->plan_box[lane] : find_box(a, w.s, w.b, w.k0 * kKeys + lane * a.box);
        for (int kt = w.k0; ok && kt < w.k1; ++kt) {
            const int khs = w.keys(kt) > 64 ? 2 : 1;
            for (int g = 0; g < 2 * khs; ++g, ++it) {
                const int d = g / khs, kh = g % khs, st = it % kVStages;  // dims 256 d .., keys 64 kh ..
                if (it >= kVStages && !wait_bar(&sm->v_free[st], (it / kVStages - 1) & 1, a.p.status, &sm->abort)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&sm->v_full[st], kVStage);
                __syncwarp();
                const int i = lane - kh * boxes;
                if (i >= 0 && i < boxes)
                    tma_load_rows(v_sm + st * kVStage + i * a.box * 4 * 128, mv, &sm->v_full[st], 4 * d, x);
            }
            if (kt + 1 < w.k1 && lane < 2 * boxes) x = find_box(a, w.s, w.b, (kt + 1) * kKeys + lane * a.box);
        }
    }
    __syncwarp();
    for (uint32_t i = it > kVStages ? it - kVStages : 0; i < it; ++i)
        wait_bar(&sm->v_full[i % kVStages], (i / kVStages) & 1, a.p.status, nullptr);
}

// Packed FP8 rows: units of 32 keys x 512 codes.
__device__ void value_producer_fp8(const TcArgs &a, Small *sm, uint8_t *raw_sm, const CUtensorMap *mv) {
    const int lane = threadIdx.x & 31;
    const int box = min(a.box, 32), boxes = 32 / box;  // per unit, 1..4
    uint32_t it = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next()) {
        Box x = {a.p.n_pages, 0, false};
        if (lane < 4 * boxes) x = find_box(a, w.s, w.b, w.k0 * kKeys + lane * box);
        for (int kt = w.k0; ok && kt < w.k1; ++kt) {
            const int units = (w.keys(kt) + 31) / 32;
            for (int u = 0; u < units; ++u, ++it) {
                const int st = it % kRawStages;
                if (it >= kRawStages && !wait_bar(&sm->v_free[st], (it / kRawStages - 1) & 1, a.p.status, &sm->abort)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&sm->v_full[st], kRawStage);
                __syncwarp();
                const int i = lane - u * boxes;
                if (i >= 0 && i < boxes) tma_load_rows(raw_sm + st * kRawStage + i * box * 512, mv, &sm->v_full[st], 0, x);
            }
            if (kt + 1 < w.k1 && lane < 4 * boxes) x = find_box(a, w.s, w.b, (kt + 1) * kKeys + lane * box);
        }
    }
    __syncwarp();
    for (uint32_t i = it > kRawStages ? it - kRawStages : 0; i < it; ++i)
        wait_bar(&sm->v_full[i % kRawStages], (i / kRawStages) & 1, a.p.status, nullptr);
}

// One unit's codes to fp16 (exact), this warp's quarter (of four): raw [4 groups of 8 keys][4 x
// 128 dims][8 keys][128 bytes], widened [4][8 x 64 dims][8][128], both 128-byte
// swizzled.  Eight lanes take the eight keys of a group, so neither side conflicts.
// Rows from `live` on are past the sequence and may hold anything: zeros.
__device__ __forceinline__ void widen_unit(const uint8_t *raw, uint8_t *h, int warp, int lane, int live) {
    const int k = lane & 7;
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
        const int q = (i & 1) * 16 + warp * 4 + (lane >> 3), c = q & 7, j = q >> 3, g = i >> 1;
        uint4 v = *reinterpret_cast<const uint4 *>(raw + g * 4096 + j * 1024 + k * 128 + ((c ^ k) << 4));
        if (8 * g + k >= live) v = make_uint4(0, 0, 0, 0);
        uint8_t *d = h + g * 8192 + (2 * j + (c >> 2)) * 1024 + k * 128;
        const int p = 2 * (c & 3);
        *reinterpret_cast<uint4 *>(d + ((p ^ k) << 4)) =
            make_uint4(widen2(v.x & 0xffffu), widen2(v.x >> 16), widen2(v.y & 0xffffu), widen2(v.y >> 16));
        *reinterpret_cast<uint4 *>(d + (((p + 1) ^ k) << 4)) =
            make_uint4(widen2(v.z & 0xffffu), widen2(v.z >> 16), widen2(v.w & 0xffffu), widen2(v.w >> 16));
    }
}

// Posts a command to the output warps; they start once this thread's MMAs have
// completed (the commit) and it has written the command (its own arrival).
__device__ __forceinline__ bool post_command(const TcArgs &a, Small *sm, int cmd, uint32_t &phase, bool wait) {
    sm->cmd = cmd;
    mbar_arrive(&sm->cmd_full);
    umma_commit(&sm->cmd_full);
    const uint32_t ph = phase;
    phase ^= 1;
    return !wait || wait_bar(&sm->cmd_done, ph, a.p.status, &sm->abort);
}

// A stage's values that are not finite (an exponent of all ones) become zeros.  For
// the tiles in which some token does not see such a row: the tokens that do see it
// have NaN weights there, from a logit that is NaN or +infinity as well (with -infinity
// the row has no weight and, cleaned, adds nothing).  One warp, some
// 5 us a tile: the rows of a sound cache never come here.
__device__ __forceinline__ void clean_stage(uint8_t *v, int lane, uint32_t expo) {
#pragma unroll 1
    for (int i = lane; i < 4 * kBlk / 16; i += 32) {
        uint4 x = reinterpret_cast<uint4 *>(v)[i];
        uint32_t *w = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t e = w[k] & expo;
            if ((e & 0xFFFFu) == (expo & 0xFFFFu)) w[k] &= 0xFFFF0000u;
            if ((e >> 16) == (expo >> 16)) w[k] &= 0x0000FFFFu;
        }
        reinterpret_cast<uint4 *>(v)[i] = x;
    }
    fence_proxy_async_smem();
    __syncwarp();
}

template <bool kFp8>
__device__ void value_mma(const TcArgs &a, Small *sm, uint8_t *p_sm, uint8_t *v_sm) {
    const int lane = threadIdx.x & 31;
    const uint32_t tb = sm->tmem_base;
    const uint64_t pd = sdesc_sw128(smem_u32(p_sm), 16, 1024);
    const uint64_t vd = sdesc_sw128(smem_u32(v_sm), 1024, 4096);
    uint32_t it = 0, tile = 0, cphase = 0;
    bool ok = true;
    for (Walk w(a, sm); ok && w.valid(); w.next()) {
        for (int kt = w.k0; ok && kt < w.k1; ++kt, ++tile) {
            const uint32_t slot = tile & 1;
            const int khs = w.keys(kt) > 64 ? 2 : 1;
            if (!wait_bar(&sm->p_full[slot], (tile >> 1) & 1, a.p.status, &sm->abort)) {
                ok = false;
                break;
            }
            if (lane == 0) arrive_remote(map_rank(smem_u32(&sm->p_got[slot]), 0));
            tc_fence_after();
            const volatile int *fl = sm->flags[slot];
            const int todo = fl[0] | fl[1] | fl[2] | fl[3];
            if (todo & 1) {
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
            if (kFp8) {
                const int units = (w.keys(kt) + 31) / 32;
                for (int u = 0; u < units; ++u, ++it) {
                    const int st = it % kHStages;
                    if (!wait_bar(&sm->h_full[st], (it / kHStages) & 1, a.p.status, &sm->abort)) {
                        ok = false;
                        break;
                    }
                    if (todo & 2) clean_stage(v_sm + st * kHStage, lane, 0x7C007C00u);
                    if (lane == 0) {
                        tc_fence_after();
                        const uint64_t hd = sdesc_sw128(smem_u32(v_sm), 1024, 8192);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int d = e >> 1, k = e & 1;  // dims 256 d .., keys 16 k ..
                            umma_bf16(tb + 256 * d,
                                      pd + static_cast<uint64_t>((slot * kPSlot + (u >> 1) * 2 * kBlk + (u & 1) * 64 + k * 32) >> 4),
                                      hd + static_cast<uint64_t>((st * kHStage + d * 4096 + k * 16384) >> 4), kIdescO16,
                                      (kt > w.k0 || u + k > 0) ? 1u : 0u);
                        }
                        umma_commit(&sm->h_free[st]);
                    }
                    __syncwarp();
                }
            }
            for (int g = 0; !kFp8 && g < 2 * khs; ++g, ++it) {
                const int d = g / khs, kh = g % khs, st = it % kVStages;
                if (!wait_bar(&sm->v_full[st], (it / kVStages) & 1, a.p.status, &sm->abort)) {
                    ok = false;
                    break;
                }
                // rows at or past the sequence's end may hold anything, and 0 x NaN is NaN
                const int z0 = w.s.len - kt * kKeys - 64 * kh;
                if (z0 < 64) {
                    uint8_t *v = v_sm + st * kVStage;
                    for (int i = lane; i < 32 * (64 - z0); i += 32) {
                        const int row = z0 + (i >> 5), db = (i >> 3) & 3;
                        *reinterpret_cast<uint4 *>(v + (row >> 3) * 4096 + db * 1024 + (row & 7) * 128 + (i & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (todo & 2) clean_stage(v_sm + st * kVStage, lane, 0x7F807F80u);
                if (lane == 0) {
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16(tb + 256 * d, pd + static_cast<uint64_t>((slot * kPSlot + kh * 2 * kBlk + k * 32) >> 4),
                                  vd + static_cast<uint64_t>((st * kVStage + k * 8192) >> 4), kIdescO,
                                  (kt > w.k0 || kh + k > 0) ? 1u : 0u);
                    umma_commit(&sm->v_free[st]);
                }
                __syncwarp();
            }
            if (ok && lane == 0) umma_commit_to(&sm->p_free[slot], 1);
        }
        if (!ok) break;
        uint32_t good = 1;
        if (lane == 0) {
            good = post_command(a, sm, kCmdFinish, cphase, true) ? 1u : 0u;
            // The output warps have arrived on cmd_done: their reads and writes of the P slots
            // and of the row statistics, which the score CTA's copies overwrite next, come
            // before this one arrival at cluster scope (their own would each wait for their
            // stores to memory).
            if (good) arrive_remote_release(map_rank(smem_u32(&sm->out_done), 0));
        }
        good = __shfl_sync(0xffffffffu, good, 0);
        cphase = __shfl_sync(0xffffffffu, cphase, 0);
        if (!good) break;
        tc_fence_after();
    }
    if (lane == 0) {
        post_command(a, sm, kCmdExit, cphase, false);
        umma_commit(&sm->fin);
        wait_bar(&sm->fin, 0, a.p.status, nullptr);
    }
    __syncwarp();
}

// 32 staged rows of 256 bytes (16-byte piece p of row i at p ^ (i & 15)) to memory,
// two rows per instruction.
__device__ __forceinline__ void put_rows(uint8_t *dst, int pitch, const uint8_t *st, int lane, int n_live) {
    const int c = lane & 15;
#pragma unroll
    for (int b = 0; b < 32; b += 16) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = b + 2 * k + (lane >> 4);
            v[k] = *reinterpret_cast<const uint4 *>(st + i * 256 + ((c ^ (i & 15)) << 4));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = b + 2 * k + (lane >> 4);
            if (i < n_live) *reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(i) * pitch + c * 16) = v[k];
        }
    }
}

// Warp w: rows 32 (w & 3) + lane, output dims 256 (w >> 2) .. + 255.
// Packed FP8 rows: between commands the warps widen the codes.
template <bool kFp8>
__device__ void value_output(const TcArgs &a, Small *sm, uint8_t *stage, const uint8_t *raw_sm, uint8_t *h_sm, int cluster) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = warp & 3, half = warp >> 2;
    const int r = 32 * quad + lane;
    const uint32_t tb = sm->tmem_base + (static_cast<uint32_t>(32 * quad) << 16) + 256 * half;
    uint32_t cphase = 0, piece = 0;
    Walk w(a, sm);
    Walk cw(a, sm);  // the units being widened
    int ckt = cw.k0, cu = 0;
    uint32_t cit = 0, idle = 0;
    uint64_t t_idle = 0;
    while (true) {
        if (kFp8) {
            // whichever is ready: a unit to widen, or a command; neither waits for the other
            // (a finished piece's output comes while the next one's units already wait)
            bool can = cw.valid();
            if (can) {
                // warps 0-3 take the even units, 4-7 the odd ones
                const uint32_t rs = cit % kRawStages, hs = cit % kHStages;
                const bool mine = (cit & 1) == static_cast<uint32_t>(half);
                can = !mine || ((cit < kHStages || mbar_test_wait(&sm->h_free[hs], (cit / kHStages - 1) & 1)) &&
                       mbar_test_wait(&sm->v_full[rs], (cit / kRawStages) & 1));
                if (__all_sync(0xffffffffu, can)) {
                    if (mine) {
                        widen_unit(raw_sm + rs * kRawStage, h_sm + hs * kHStage, quad, lane, cw.s.len - ckt * kKeys - 32 * cu);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sm->v_free[rs]);
                            mbar_arrive(&sm->h_full[hs]);
                        }
                    }
                    ++cit;
                    if (++cu == (cw.keys(ckt) + 31) / 32) {
                        cu = 0;
                        if (++ckt == cw.k1) {
                            cw.next();
                            ckt = cw.k0;
                        }
                    }
                    idle = 0;
                    continue;
                }
            }
            if (!__all_sync(0xffffffffu, mbar_test_wait(&sm->cmd_full, cphase))) {
                if ((++idle & 255u) == 0) {
                    if (*reinterpret_cast<volatile int *>(&sm->abort)) break;
                    const uint64_t now = global_timer_ns();
                    if (idle == 256) t_idle = now;
                    if (now - t_idle > kWaitLimitNs) {
                        report_status(a.p.status, DSA_ERR_TIMEOUT);
                        sm->abort = 1;
                        break;
                    }
                }
                continue;
            }
            idle = 0;
        } else if (!wait_bar(&sm->cmd_full, cphase, a.p.status, &sm->abort)) {
            break;
        }
        cphase ^= 1;
        tc_fence_after();
        const int cmd = *reinterpret_cast<volatile int *>(&sm->cmd);
        if ((cmd & 255) == kCmdExit) break;
        if ((cmd & 255) == kCmdRescale) {
            const int slot = cmd >> 8;
            if (*reinterpret_cast<volatile int *>(&sm->flags[slot][quad]) & 1) {
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
            if (!wait_bar(&sm->stat_full, piece & 1, a.p.status, &sm->abort)) break;
            const int rows = w.rows();
            const float factor = sm->v.factor[r];
            const bool whole = w.k0 == 0 && w.k1 == w.nk;
            const int64_t row = w.row0() + r;
            const int64_t pslot = 2 * cluster + (w.k0 == 0 ? 1 : 0);
            if (32 * quad < rows && whole) {
                // 128 columns at a time through the warp's 8 KB of the P slots (16-byte pieces
                // exchanged by row, so that neither side conflicts), then whole rows to memory:
                // a lane's own 16-byte stores, 1 KB apart, took four times as long
                uint8_t *st = stage + warp * 8192;
                const int n_live = min(32, rows - 32 * quad);
                uint8_t *o = static_cast<uint8_t *>(a.p.out) + ((row - lane) * kLatent + 256 * half) * 2;
#pragma unroll 1
                for (int c = 0; c < 256; c += 128) {
#pragma unroll 1
                    for (int g = 0; g < 4; ++g) {
                        uint32_t x[32];
                        tmem_ld32(tb + c + 32 * g, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4 *>(st + lane * 256 + (((4 * g + i / 8) ^ (lane & 15)) << 4)) =
                                make_uint4(pack_bf16(u2f(x[i]) * factor, u2f(x[i + 1]) * factor),
                                           pack_bf16(u2f(x[i + 2]) * factor, u2f(x[i + 3]) * factor),
                                           pack_bf16(u2f(x[i + 4]) * factor, u2f(x[i + 5]) * factor),
                                           pack_bf16(u2f(x[i + 6]) * factor, u2f(x[i + 7]) * factor));
                    }
                    if (c == 128) fence_proxy_async_smem();  // (the slots are next written by a copy)
                    __syncwarp();
                    put_rows(o + 2 * c, kLatent * 2, st, lane, n_live);
                    __syncwarp();
                }
            } else if (32 * quad < rows) {
                // partials [column][row]: a warp's 32 rows are one line, as they come
                float *po = a.part_o + (pslot * kLatent + 256 * half) * kRows + r;
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(tb + c, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) po[(c + i) * kRows] = u2f(x[i]) * factor;
                }
            }
            if (tid == 0 && w.k0 == 0 && w.k1 < w.nk) {
                // the row tile goes on in the next clusters' ranges
                const long long last = sm->plan_end - w.k1 + w.nk - 1;
                const int end = static_cast<int>(((last + 1) * sm->plan_active - 1) / sm->plan_total);
                a.meta[cluster] = Meta{end - cluster + 1, static_cast<int>(w.row0()), rows, 0};
            }
            ++piece;
            w.next();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->cmd_done);
    }
}

struct TcMaps {
    CUtensorMap q, k, v;  // queries; cache rows for either product
    CUtensorMap q8, r;    // packed FP8 rows: the queries' two terms, the RoPE keys
};

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_mla_tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ TcMaps maps) {
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
            mbar_init(&sm->v_free[i], kFp8 ? 4 : 1);
        }
        for (int i = 0; i < kHStages; ++i) {
            mbar_init(&sm->h_full[i], 4);
            mbar_init(&sm->h_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->sig_full[i], 1);
            mbar_init(&sm->sig_free[i], 8);
        }
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(&sm->s_full[i], 1);
            mbar_init(&sm->s_free[i], 8);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm->x_bar[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->p_free[i], 1);
            mbar_init(&sm->p_got[i], 1);
            mbar_init(&sm->p_full[i], 8);
        }
        mbar_init(&sm->out_done, 1);
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
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        if (kFp8) {
            tma_prefetch_desc(&maps.q8);
            tma_prefetch_desc(&maps.r);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sm->tmem_base != 0) {  // (the whole of it: its base is 0)
        report_status(a.p.status, DSA_ERR_CUDA);
        sm->abort = 1;
    }
    griddep_wait();
    make_plan(a, sm, cluster, rank == 0 && cluster == 0);
    if (tid == 0 && rank == 1) a.meta[cluster].parts = 0;
    cluster_sync_all();  // both CTAs' barriers are set up before either signals the other
    // registers from the producer's and MMA thread's warps to the others (168 each at
    // launch: 2 x 200 + 96 of 3 x 168)
    if (warp < 8)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (rank == 0) {
        uint8_t *stage = smem + kQBytes, *ring = stage + 2 * kPSlot;
        if (warp < 8) {
            score_softmax<kFp8>(a, sm, stage, map_rank(smem_u32(smem), 1), cluster);
        } else if (kFp8) {
            if (warp == 8)
                score_producer_fp8(a, sm, smem, stage, ring, ring + 2 * kCodes, &maps.q, &maps.q8, &maps.k, &maps.r);
            else if (warp == 9 && lane == 0)
                score_mma_fp8(a, sm, smem, stage, ring, ring + 2 * kCodes);
            else if (warp == 10)
                score_scales_fp8(a, sm);
        } else if (warp == 8) {
            score_producer(a, sm, smem, stage, ring, &maps.q, &maps.k);
        } else if (warp == 9 && lane == 0) {
            score_mma(a, sm, smem, stage, ring);
        }
    } else {
        uint8_t *v_sm = smem + 2 * kPSlot, *h_sm = v_sm + kRawStages * kRawStage;
        if (warp < 8)
            value_output<kFp8>(a, sm, smem, v_sm, h_sm, cluster);
        else if (warp == 8 && kFp8)
            value_producer_fp8(a, sm, v_sm, &maps.v);
        else if (warp == 8)
            value_producer(a, sm, v_sm, &maps.v);
        else if (warp == 9)
            value_mma<kFp8>(a, sm, smem, kFp8 ? h_sm : v_sm);
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

// The latent part of each query row (token, head) as s (q1 + q2): s a power of two
// that brings the row's largest value under E4M3's 448, q1 the nearest E4M3 value, q2
// the nearest to what is left (exact but below 2^-18 of the row's largest value).  A
// row with an infinity gets NaN for s: as codes it would be finite, and its logits with it.
// One warp per row, 16 dims per lane; bound by launch latency at decode sizes.
__global__ void __launch_bounds__(256) split_queries_kernel(const __nv_bfloat16 *q, uint8_t *q8, float *scale, int64_t rows) {
    griddep_wait();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(q + row * kRow + 16 * lane);
    const uint4 in[2] = {src[0], src[1]};
    float v[16];
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t two = reinterpret_cast<const uint32_t *>(in)[i];
        v[2 * i] = u2f(two << 16);
        v[2 * i + 1] = u2f(two & 0xFFFF0000u);
        mx = fmaxf(mx, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 2^k with mx 2^-k in (224, 448] (k kept where both powers are normal numbers)
    const uint32_t bits = __float_as_uint(mx);
    int k = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    k = mx > 0.f ? min(max(k, -120), 120) : 0;
    const float down = u2f(static_cast<uint32_t>(127 - k) << 23);
    uint32_t t1[4], t2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t1[i] = t2[i] = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 x = make_float2(v[4 * i + 2 * h] * down, v[4 * i + 2 * h + 1] * down);
            const uint32_t c1 = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
            const uint32_t w = widen2(c1);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
            const uint32_t c2 = __nv_cvt_float2_to_fp8x2(make_float2(x.x - f.x, x.y - f.y), __NV_SATFINITE, __NV_E4M3);
            t1[i] |= c1 << (16 * h);
            t2[i] |= c2 << (16 * h);
        }
    }
    uint4 *dst = reinterpret_cast<uint4 *>(q8 + row * 2 * kLatent + 16 * lane);
    dst[0] = make_uint4(t1[0], t1[1], t1[2], t1[3]);
    dst[kLatent / 16] = make_uint4(t2[0], t2[1], t2[2], t2[3]);
    if (lane == 0) scale[row] = u2f(mx <= FLT_MAX ? static_cast<uint32_t>(127 + k) << 23 : 0x7FC00000u);
}

// Merge of the row tiles that a cut divided: o = sum_i 2^(m_i - M) o_i / sum_i
// 2^(m_i - M) l_i over the parts, the first in its cluster's second slot, the
// others in the next clusters' first slots.  One CTA per (cluster, 32 rows, 64
// columns); most find nothing to do.  Bound by latency: two round trips to L2.
constexpr int kMergeCols = 64;  // columns and rows of a CTA
constexpr int kMergeRows = 32;
constexpr int kMaxParts = 96;  // clusters at most (74 on 148 SMs)

__global__ void __launch_bounds__(256) paged_mla_merge_kernel(const TcArgs a) {
    __shared__ float wt[kMaxParts][kMergeRows];
    __shared__ float tr[kMergeCols][kMergeRows + 1];
    griddep_wait();
    const int c = blockIdx.x, r0 = blockIdx.y * kMergeRows, c0 = blockIdx.z * kMergeCols;
    const Meta me = a.meta[c];
    if (r0 >= me.rows || me.parts == 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = r0 + lane;
    auto slot = [&](int i) { return static_cast<int64_t>(2 * (c + i) + (i == 0 ? 1 : 0)); };  // the first part is a head
    // a row per lane, eight columns per warp; the first two parts' values are on their
    // way while the weights are found
    const float *po = a.part_o + static_cast<int64_t>(c0 + 8 * warp) * kRows + r;
    auto fetch = [&](float (&x)[8], int i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = i < me.parts ? po[(slot(i) * kLatent + k) * kRows] : 0.f;
    };
    float x[2][8];
    fetch(x[0], 0);
    fetch(x[1], 1);
    // weights: warp w takes parts w, w + 8, ..
    float M = -INFINITY;
    for (int i = 0; i < me.parts; ++i) M = fmaxf(M, a.part_ml[(slot(i) * 2) * kRows + r]);
    float L = 0.f;
    for (int i = 0; i < me.parts; ++i) {
        const float m = a.part_ml[(slot(i) * 2) * kRows + r], l = a.part_ml[(slot(i) * 2 + 1) * kRows + r];
        const float w = m == -INFINITY ? 0.f : exp2f(m - M);
        if ((i & 7) == warp) wt[i][lane] = w;
        L += w * l;
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    if (warp == 0 && blockIdx.z == 0 && r < me.rows && a.p.lse)
        a.p.lse[static_cast<int64_t>(me.row0) + r] = L != 0.f ? M * kLn2 + logf(L) : -INFINITY;
    __syncthreads();
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int i = 0; i < me.parts; i += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // (a part without weight may have left anything, and 0 x NaN is NaN)
            const float w = i + h < me.parts ? wt[i + h][lane] : 0.f;
            if (w != 0.f)
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] += w * x[h][k];
            fetch(x[h], i + h + 2);
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) tr[8 * warp + k][lane] = acc[k] * inv;
    __syncthreads();
    // 64 columns of a row are 128 bytes of the output
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int row = r0 + 4 * warp + k;
        if (row < me.rows)
            reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.p.out) +
                                         (static_cast<int64_t>(me.row0) + row) * kLatent + c0)[lane] =
                pack_bf16(tr[2 * lane][4 * warp + k], tr[2 * lane + 1][4 * warp + k]);
    }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

bool paged_mla_tc_shape(const PagedMlaArgs &a) {
    // (the softmax takes the maximum before it scales: a positive scale)
    if (!a.is_bf16 || !(a.scale > 0.f) || a.scale > FLT_MAX || a.heads > kRows || a.d_lat != kLatent || a.d_rope != kRope)
        return false;
    const int64_t unit = a.kv_fp8 ? 16 : 8, row = a.kv_fp8 ? kFp8Row : kRow;
    if (a.page_rows % 8 != 0 || a.kv_row_stride % unit != 0 || a.kv_row_stride < row) return false;
    if (a.kv_page_stride % unit != 0 || a.kv_page_stride < 1) return false;
    const auto mis = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.kv) | reinterpret_cast<uintptr_t>(a.out);
    return (mis & 15u) == 0 && static_cast<int64_t>(a.n_tok) * a.heads < INT32_MAX;
}

static int tc_clusters(int num_sms) { return std::min(num_sms / 2, kMaxParts); }

size_t paged_mla_tc_scratch(const PagedMlaArgs &p, int num_sms) {
    const size_t c = tc_clusters(num_sms), rows = p.kv_fp8 ? static_cast<size_t>(p.n_tok) * p.heads : 0;
    return align256(c * sizeof(Meta)) + align256(2 * c * kRows * 2 * sizeof(float)) +
           2 * c * kRows * kLatent * sizeof(float) + rows * 2 * kLatent + rows * sizeof(float);
}

cudaError_t launch_paged_mla_tc(const PagedMlaArgs &p, void *scratch, int num_sms, cudaStream_t st) {
    EncodeTiledFn enc = tma_encode_fn();
    if (!enc) return cudaErrorNotSupported;
    TcArgs a = {};
    a.p = p;
    a.clusters = tc_clusters(num_sms);
    a.tok_tile = kRows / p.heads;
    a.max_len = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(p.max_pages) * p.page_rows, INT_MAX - 1025));
    a.box = 64;
    while (p.page_rows % a.box != 0) a.box >>= 1;
    const int64_t rows = static_cast<int64_t>(p.n_tok) * p.heads;
    uint8_t *s = static_cast<uint8_t *>(scratch);
    a.meta = reinterpret_cast<Meta *>(s);
    s += align256(a.clusters * sizeof(Meta));
    a.part_ml = reinterpret_cast<float *>(s);
    s += align256(static_cast<size_t>(2) * a.clusters * kRows * 2 * sizeof(float));
    a.part_o = reinterpret_cast<float *>(s);
    s += static_cast<size_t>(2) * a.clusters * kRows * kLatent * sizeof(float);
    uint8_t *q8 = s;
    float *q8_scale = reinterpret_cast<float *>(s + rows * 2 * kLatent);
    a.q8 = q8;
    a.q8_scale = q8_scale;
    TcMaps m = {};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    auto encode = [&](CUtensorMap *map, CUtensorMapDataType dt, cuuint32_t rank, const void *base, const cuuint64_t *dims,
                      const cuuint64_t *strides, const cuuint32_t *box) {
        return enc(map, dt, rank, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
               CUDA_SUCCESS;
    };
    const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const cuuint64_t qd[2] = {static_cast<cuuint64_t>(kRow), static_cast<cuuint64_t>(rows)};
    const cuuint64_t qs[1] = {static_cast<cuuint64_t>(kRow) * 2};
    const cuuint32_t qb[2] = {64, 64};
    bool ok = encode(&m.q, bf, 2, p.q, qd, qs, qb);
    const cuuint64_t groups = static_cast<cuuint64_t>(p.page_rows / 8), pages = static_cast<cuuint64_t>(p.n_pages);
    const cuuint32_t g64 = static_cast<cuuint32_t>(a.box / 8), g32 = std::min<cuuint32_t>(g64, 4);
    if (!p.kv_fp8) {
        // cache rows: {64 dims, 8 rows, 9 blocks, groups of a page, pages}
        const cuuint64_t rs = static_cast<cuuint64_t>(p.kv_row_stride) * 2;
        const cuuint64_t kd[5] = {64, 8, kNB, groups, pages};
        const cuuint64_t ks[4] = {rs, 128, 8 * rs, static_cast<cuuint64_t>(p.kv_page_stride) * 2};
        const cuuint32_t kb[5] = {64, 8, kKBlocks, g64, 1}, vb[5] = {64, 8, 4, g64, 1};
        ok = ok && encode(&m.k, bf, 5, p.kv, kd, ks, kb) && encode(&m.v, bf, 5, p.kv, kd, ks, vb);
    } else {
        // codes: {128 dims, 8 rows, 4 blocks, groups, pages}; RoPE keys: {64 dims, 8 rows, groups, pages}
        const cuuint64_t rs = static_cast<cuuint64_t>(p.kv_row_stride), ps = static_cast<cuuint64_t>(p.kv_page_stride);
        const cuuint64_t kd[5] = {128, 8, 4, groups, pages}, ks[4] = {rs, 128, 8 * rs, ps};
        const cuuint32_t kb[5] = {128, 8, 4, g64, 1}, vb[5] = {128, 8, 4, g32, 1};
        const cuuint64_t rd[4] = {64, 8, groups, pages}, rst[3] = {rs, 8 * rs, ps};
        const cuuint32_t rb[4] = {64, 8, g64, 1};
        const cuuint64_t q8d[2] = {2 * kLatent, static_cast<cuuint64_t>(rows)}, q8s[1] = {2 * kLatent};
        const cuuint32_t q8b[2] = {128, 64};
        ok = ok && encode(&m.k, u8, 5, p.kv, kd, ks, kb) && encode(&m.v, u8, 5, p.kv, kd, ks, vb) &&
             encode(&m.r, bf, 4, static_cast<const uint8_t *>(p.kv) + kFp8RopeOff, rd, rst, rb) &&
             encode(&m.q8, u8, 2, q8, q8d, q8s, q8b);
    }
    if (!ok) return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    if (p.kv_fp8) {
        e = launch_pdl(split_queries_kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, st,
                       static_cast<const __nv_bfloat16 *>(p.q), q8, q8_scale, rows);
        if (e != cudaSuccess) return e;
    }
    auto kernel = p.kv_fp8 ? paged_mla_tc_kernel<true> : paged_mla_tc_kernel<false>;
    const int smem = kBig + static_cast<int>(sizeof(Small));
    e = set_max_dynamic_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(2 * a.clusters), dim3(kThreads), smem, st, a, m);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_mla_merge_kernel, dim3(a.clusters, kRows / kMergeRows, kLatent / kMergeCols), dim3(256), 0, st, a);
}

}  // namespace dsa
