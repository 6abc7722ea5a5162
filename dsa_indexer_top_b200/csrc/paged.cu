// paged.cu -- paged caches: block tables and slot maps from request lengths
// (dsa_page_tables) and the entry point of attention over a paged latent cache
// (dsa_paged_mla: argument checks, choice of path, the CUDA-core kernel).
//
// Tables: sequence b needs need_b = max(held_b, ceil((ctx_b + new_b) / P)) pages;
// fresh_b = need_b - held_b come from the free list at the exclusive prefix sum
// of fresh, tokens stand at the exclusive prefix sum of new, and token j of
// sequence b has position ctx_b + j and slot table[b][pos / P] * P + pos % P.
// Bound by latency: the bytes are 12 per sequence and 12 per token (0.4 MB for
// 32K tokens).  So one launch, and no CTA waits for another: each scans every
// sequence's lengths itself (a few KB from L2) and fills its own range of tokens
// and every gridDim-th new page; a token whose page is new reads the free list,
// not the table entry another CTA may be writing.  Measured (one B200): 64 requests of
// one token 5.7 us, 700 requests with 0 to 160 tokens each in pages of 16 rows 8.7 us.
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <nvtx3/nvToolsExt.h>

#include "abi_checks.cuh"
#include "dsa.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tma_encode.cuh"

namespace dsa {
namespace {

// ------------------------------------------------------------------ page tables
constexpr int kTabThreads = 256;
constexpr int kTabPer = 4;                         // sequences per thread and step
constexpr int kTabStep = kTabThreads * kTabPer;

// Block-wide exclusive scan of two 64-bit sums (tokens, pages).
__device__ __forceinline__ void scan2(long long &x, long long &y, long long &tx, long long &ty, long long (*buf)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ax = __shfl_up_sync(0xffffffffu, ix, o), ay = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) ix += ax, iy += ay;
    }
    __syncthreads();  // buf and the previous step's arrays are free
    if (lane == 31) buf[warp][0] = ix, buf[warp][1] = iy;
    __syncthreads();
    long long px = 0, py = 0;
    tx = ty = 0;
#pragma unroll
    for (int w = 0; w < kTabThreads / 32; ++w) {
        if (w < warp) px += buf[w][0], py += buf[w][1];
        tx += buf[w][0], ty += buf[w][1];
    }
    x = px + ix - x;
    y = py + iy - y;
}

// Largest i in [0, n) with a[i] <= v (a[0] <= v, not decreasing).
__device__ __forceinline__ int last_le(const long long *a, int n, long long v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(const PageTablesArgs a) {
    __shared__ long long buf[kTabThreads / 32][2];
    __shared__ long long tok0[kTabStep], pg0[kTabStep];  // first token / first new page of each sequence of the step
    __shared__ int ctx_s[kTabStep], held_s[kTabStep];
    const dsa_page_plan &p = a.p;
    const int tid = threadIdx.x;
    griddep_wait();
    const long long head = p.free_begin ? *p.free_begin : 0;
    bool bad = head < 0 || head > p.n_free;
    const long long avail = bad ? 0 : p.n_free - head;
    // this CTA's tokens
    const long long per = (p.n_tok + gridDim.x - 1) / gridDim.x;
    const long long my0 = per * blockIdx.x, my1 = min(my0 + per, static_cast<long long>(p.n_tok));
    // page id of new page e (in hand-out order), or -1
    auto new_page = [&](long long e) -> int {
        if (e >= avail) return -1;
        const int id = p.free_pages[head + e];
        return id >= 0 && id < p.n_pages ? id : -1;
    };
    long long tok_base = 0, pg_base = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += kTabStep) {
        int ctx[kTabPer], nw[kTabPer], held[kTabPer];
        long long st = 0, sp = 0;
        long long lt[kTabPer], lp[kTabPer];
#pragma unroll
        for (int k = 0; k < kTabPer; ++k) {
            const int b = s0 + tid * kTabPer + k;
            ctx[k] = nw[k] = held[k] = 0;
            if (b < p.n_seq) ctx[k] = p.ctx_len[b], nw[k] = p.new_len[b], held[k] = p.held[b];
        }
#pragma unroll
        for (int k = 0; k < kTabPer; ++k) {
            const int b = s0 + tid * kTabPer + k;
            if (ctx[k] < 0 || nw[k] < 0 || held[k] < 0 || held[k] > p.max_pages ||
                static_cast<long long>(ctx[k]) + nw[k] > INT_MAX)
                bad = true;
            ctx[k] = max(ctx[k], 0);
            nw[k] = max(nw[k], 0);
            if (static_cast<long long>(ctx[k]) + nw[k] > INT_MAX) nw[k] = INT_MAX - ctx[k];
            held[k] = min(max(held[k], 0), p.max_pages);
            const long long total = static_cast<long long>(ctx[k]) + nw[k];
            long long need = (total + p.page_rows - 1) / p.page_rows;
            if (need > p.max_pages) {
                bad = true;
                need = p.max_pages;
            }
            need = max(need, static_cast<long long>(held[k]));
            lt[k] = st;
            lp[k] = sp;
            st += nw[k];
            sp += need - held[k];
            if (b < p.n_seq && blockIdx.x == (b / kTabStep) % gridDim.x) {
                p.seq_len[b] = static_cast<int>(total);
                p.held_out[b] = static_cast<int>(need);
            }
        }
        long long xt = st, xp = sp, tt, tp;
        scan2(xt, xp, tt, tp, buf);
#pragma unroll
        for (int k = 0; k < kTabPer; ++k) {
            const int i = tid * kTabPer + k, b = s0 + i;
            tok0[i] = tok_base + xt + lt[k];
            pg0[i] = pg_base + xp + lp[k];
            ctx_s[i] = ctx[k];
            held_s[i] = held[k];
            if (b < p.n_seq && blockIdx.x == (b / kTabStep) % gridDim.x)
                p.q_begin[b] = static_cast<int>(min(tok0[i], static_cast<long long>(p.n_tok)));
        }
        __syncthreads();
        const int n = min(kTabStep, p.n_seq - s0);
        // new table entries, dealt to the CTAs' threads in turn
        for (long long e = pg_base + blockIdx.x * kTabThreads + tid; e < pg_base + tp;
             e += static_cast<long long>(gridDim.x) * kTabThreads) {
            const int i = last_le(pg0, n, e);
            const int id = new_page(e);
            if (id < 0) bad = true;
            p.block_table[(s0 + i) * p.table_stride + held_s[i] + (e - pg0[i])] = id;
        }
        // this CTA's tokens of this step's sequences
        for (long long t = max(my0, tok_base) + tid; t < min(my1, tok_base + tt); t += kTabThreads) {
            const int i = last_le(tok0, n, t), b = s0 + i;
            const long long pos = ctx_s[i] + (t - tok0[i]);
            const long long page = pos / p.page_rows;
            int id = -1;
            if (page < held_s[i]) {
                id = p.block_table[b * p.table_stride + page];
                if (id < 0 || id >= p.n_pages) {
                    id = -1;
                    bad = true;
                }
            } else if (page < p.max_pages) {
                id = new_page(pg0[i] + (page - held_s[i]));
            }
            p.q_seq[t] = b;
            p.q_pos[t] = static_cast<int>(pos);
            p.slot_map[t] = id < 0 ? -1 : static_cast<int>(static_cast<long long>(id) * p.page_rows + pos % p.page_rows);
        }
        tok_base += tt;
        pg_base += tp;
    }
    // tokens past the last sequence's
    for (long long t = max(my0, tok_base) + tid; t < my1; t += kTabThreads) {
        p.q_seq[t] = 0;
        p.q_pos[t] = 0;
        p.slot_map[t] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.q_begin[p.n_seq] = static_cast<int>(min(tok_base, static_cast<long long>(p.n_tok)));
        *p.free_used = static_cast<int>(min(pg_base, avail));
        if (tok_base > p.n_tok) bad = true;
    }
    if (bad) report_status(a.status, DSA_ERR_INVALID);
}

// ------------------------------------------------------------------ CUDA-core attention
// One CTA per (token, head): the rows it sees in blocks of 128, one dot product
// per thread, with the running maximum and sum of an online softmax; each thread
// then adds the block's weighted values for its output dims.  The path of float32
// caches and of shapes the tensor cores' tiles do not fit: right for every shape,
// not tuned (every head reads the cache again, a strided row per thread: 8 tokens of 64
// heads over 32768 bf16 rows 59 ms, where the tensor cores take 0.1).
constexpr int kGenThreads = 128;

// One cache row as floats: kKind 0 float32, 1 bf16, 2 packed FP8.
template <int kKind>
struct GenRow {
    const uint8_t *p;
    float sigma;
    __device__ GenRow(const uint8_t *row, int d_lat, int d_rope) : p(row), sigma(1.f) {
        if (kKind == 2) sigma = *reinterpret_cast<const float *>(row + d_lat + 2 * d_rope);
    }
    __device__ float at(int d, int d_lat) const {
        if (kKind == 0) return reinterpret_cast<const float *>(p)[d];
        if (kKind == 1) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[d]);
        if (d >= d_lat) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p + d_lat)[d - d_lat]);
        const __half_raw h = __nv_cvt_fp8_to_halfraw(p[d], __NV_E4M3);
        return sigma * __half2float(*reinterpret_cast<const __half *>(&h));
    }
};

__device__ __forceinline__ float gen_reduce(float v, float *buf, bool is_max) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, v, o);
        v = is_max ? fmaxf(v, y) : v + y;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = buf[0];
#pragma unroll
    for (int w = 1; w < kGenThreads / 32; ++w) r = is_max ? fmaxf(r, buf[w]) : r + buf[w];
    return r;
}

template <int kKind>
__global__ void __launch_bounds__(kGenThreads) paged_mla_generic_kernel(const PagedMlaArgs a) {
    extern __shared__ float sh[];  // query (d_lat + d_rope), accumulated output (d_lat)
    __shared__ float pw[kGenThreads];
    __shared__ int64_t off[kGenThreads];
    __shared__ float red[kGenThreads / 32];
    griddep_wait();
    const int i = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int dk = a.d_lat + a.d_rope;
    if (i < a.q_begin[0] || i >= a.q_begin[a.n_seq]) return;
    int lo = 0, hi = a.n_seq;  // last b with q_begin[b] <= i
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_begin[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    const int b = lo, n = a.q_begin[b + 1] - a.q_begin[b], j = i - a.q_begin[b], len = a.seq_len[b];
    if (j < 0 || j >= n || len < n || len >= INT_MAX - 1024 ||
        len > static_cast<int64_t>(a.max_pages) * a.page_rows) {
        if (tid == 0 && h == 0) report_status(a.status, DSA_ERR_INVALID);
        return;
    }
    float *qs = sh, *acc = sh + dk;
    const int64_t qo = (static_cast<int64_t>(i) * a.heads + h) * dk;
    for (int d = tid; d < dk; d += kGenThreads)
        qs[d] = kKind == 0 ? static_cast<const float *>(a.q)[qo + d]
                           : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[qo + d]);
    for (int d = tid; d < a.d_lat; d += kGenThreads) acc[d] = 0.f;
    const uint8_t *kv = static_cast<const uint8_t *>(a.kv);
    constexpr int kElem = kKind == 0 ? 4 : kKind == 1 ? 2 : 1;
    const int seen = len - n + j + 1;
    float m = -INFINITY, l = 0.f;
    for (int s0 = 0; s0 < seen; s0 += kGenThreads) {
        __syncthreads();  // the query is in; pw and off are free
        const int s = s0 + tid;
        float x = -INFINITY;
        int64_t o = -1;
        if (s < seen) {
            const int page = a.block_table[b * a.table_stride + s / a.page_rows];
            if (page >= 0 && page < a.n_pages) {
                o = (page * a.kv_page_stride + (s % a.page_rows) * a.kv_row_stride) * kElem;
                const GenRow<kKind> row(kv + o, a.d_lat, a.d_rope);
                x = 0.f;
                for (int d = 0; d < dk; ++d) x = fmaf(qs[d], row.at(d, a.d_lat), x);
                x *= a.scale;
            } else if (h == 0) {
                report_status(a.status, DSA_ERR_INVALID);
            }
        }
        const float mc = fmaxf(m, gen_reduce(x, red, true));
        // (a logit of -infinity has no weight, also where the block has no other)
        const float al = mc == -INFINITY ? 1.f : expf(m - mc);
        const float pr = o < 0 || x == -INFINITY ? 0.f : expf(x - mc);
        l = l * al + gen_reduce(pr, red, false);
        m = mc;
        pw[tid] = pr;
        off[tid] = o;
        __syncthreads();
        const int cnt = min(kGenThreads, seen - s0);
        for (int d = tid; d < a.d_lat; d += kGenThreads) {
            float v = acc[d] * al;
            for (int k = 0; k < cnt; ++k)
                if (off[k] >= 0) v = fmaf(pw[k], GenRow<kKind>(kv + off[k], a.d_lat, a.d_rope).at(d, a.d_lat), v);
            acc[d] = v;
        }
    }
    const int64_t oo = (static_cast<int64_t>(i) * a.heads + h) * a.d_lat;
    const float inv = l != 0.f ? 1.f / l : 0.f;
    for (int d = tid; d < a.d_lat; d += kGenThreads) {
        if (kKind == 0)
            static_cast<float *>(a.out)[oo + d] = acc[d] * inv;
        else
            static_cast<__nv_bfloat16 *>(a.out)[oo + d] = __float2bfloat16_rn(acc[d] * inv);
    }
    if (tid == 0 && a.lse) a.lse[static_cast<int64_t>(i) * a.heads + h] = l != 0.f ? m + logf(l) : -INFINITY;
}

constexpr int kGenMaxDims = 8192;  // d_lat + d_rope of the CUDA-core kernel: shared memory of the launch

template <int kKind>
cudaError_t launch_generic_t(const PagedMlaArgs &a, cudaStream_t st) {
    const int smem = static_cast<int>(sizeof(float)) * (2 * a.d_lat + a.d_rope);
    cudaError_t e = set_max_dynamic_smem(paged_mla_generic_kernel<kKind>, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_mla_generic_kernel<kKind>, dim3(a.n_tok, a.heads), dim3(kGenThreads), smem, st, a);
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesArgs &a, int num_sms, cudaStream_t st) {
    const long long work = (static_cast<long long>(a.p.n_tok) + kTabStep - 1) / kTabStep;
    const int grid = static_cast<int>(work < 1 ? 1 : work > num_sms ? num_sms : work);
    return launch_pdl(page_tables_kernel, dim3(grid), dim3(kTabThreads), 0, st, a);
}

cudaError_t launch_paged_mla_generic(const PagedMlaArgs &a, cudaStream_t st) {
    if (a.kv_fp8) return launch_generic_t<2>(a, st);
    return a.is_bf16 ? launch_generic_t<1>(a, st) : launch_generic_t<0>(a, st);
}

}  // namespace dsa

using namespace dsa;

namespace {

constexpr size_t kStatus = 256;

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

bool ws_ok(void *ws, size_t ws_bytes, size_t need) {
    return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && ws_bytes >= need;
}

// Pools on the slots' int32 range.
bool pool_ok(int32_t n_pages, int32_t page_rows) {
    return n_pages >= 1 && page_rows >= 1 && static_cast<int64_t>(n_pages) * page_rows <= INT32_MAX;
}

dsa_status check_batch(const dsa_paged_batch *b) {
    if (!b || b->n_seq < 0 || b->n_tok < 0 || b->max_pages < 1 || !pool_ok(b->n_pages, b->page_rows))
        return DSA_ERR_INVALID;
    if ((b->n_seq > 1 && b->table_stride < b->max_pages) || !b->q_begin) return DSA_ERR_INVALID;
    if (b->n_seq > 0 && (!b->block_table || !b->seq_len)) return DSA_ERR_INVALID;
    return DSA_OK;
}

PagedMlaArgs paged_args(const dsa_paged_batch *batch, const dsa_mla *mla, void *ws) {
    PagedMlaArgs a = {};
    a.q = mla->q;
    a.kv = mla->kv;
    a.out = mla->out;
    a.lse = mla->lse;
    a.kv_page_stride = mla->kv_seq_stride;
    a.kv_row_stride = mla->kv_row_stride;
    a.block_table = batch->block_table;
    a.table_stride = batch->table_stride;
    a.q_begin = batch->q_begin;
    a.seq_len = batch->seq_len;
    a.n_seq = batch->n_seq;
    a.n_tok = batch->n_tok;
    a.n_pages = batch->n_pages;
    a.page_rows = batch->page_rows;
    a.max_pages = batch->max_pages;
    a.heads = mla->heads;
    a.d_lat = mla->d_latent;
    a.d_rope = mla->d_rope;
    a.scale = mla->scale;
    a.is_bf16 = mla->dtype == DSA_BF16;
    a.kv_fp8 = mla_kv_fp8(mla);
    a.status = static_cast<uint32_t *>(ws);
    return a;
}

}  // namespace

extern "C" {

dsa_status dsa_page_tables(const dsa_page_plan *p, void *ws, size_t ws_bytes, void *stream) {
    NvtxRange range("dsa_page_tables");
    if (!p || p->n_seq < 0 || p->n_tok < 0 || p->n_free < 0 || p->max_pages < 1 || !pool_ok(p->n_pages, p->page_rows))
        return DSA_ERR_INVALID;
    if ((p->n_seq > 1 && p->table_stride < p->max_pages) || !p->q_begin || !p->free_used) return DSA_ERR_INVALID;
    if (p->n_seq > 0 && (!p->ctx_len || !p->new_len || !p->held || !p->block_table || !p->seq_len || !p->held_out))
        return DSA_ERR_INVALID;
    if (p->n_tok > 0 && (!p->q_seq || !p->q_pos || !p->slot_map)) return DSA_ERR_INVALID;
    if (p->n_free > 0 && !p->free_pages) return DSA_ERR_INVALID;
    const void *in[] = {p->ctx_len, p->new_len, p->held, p->free_pages, p->free_begin};
    const void *out[] = {p->block_table, p->q_begin, p->seq_len, p->q_seq, p->q_pos, p->slot_map, p->held_out,
                         p->free_used};
    for (int o = 0; o < 8; ++o) {
        for (const void *x : in)
            if (out[o] && out[o] == x) return DSA_ERR_INVALID;
        for (int q = 0; q < o; ++q)
            if (out[o] && out[o] == out[q]) return DSA_ERR_INVALID;
    }
    if (!ws_ok(ws, ws_bytes, kStatus)) return DSA_ERR_WORKSPACE;
    PageTablesArgs a;
    a.p = *p;
    a.status = static_cast<uint32_t *>(ws);
    return launch_page_tables(a, sm_count(), static_cast<cudaStream_t>(stream)) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

size_t dsa_paged_mla_workspace_bytes(const dsa_paged_batch *batch, const dsa_mla *mla) {
    if (check_batch(batch) != DSA_OK || check_mla_layers(mla, 1) != DSA_OK) return 0;
    const PagedMlaArgs a = paged_args(batch, mla, nullptr);
    return kStatus + (paged_mla_tc_shape(a) ? paged_mla_tc_scratch(a, sm_count()) : 0);
}

dsa_status dsa_paged_mla(const dsa_paged_batch *batch, const dsa_mla *mla, void *ws, size_t ws_bytes, void *stream) {
    NvtxRange range("dsa_paged_mla");
    dsa_status s = check_batch(batch);
    if (s != DSA_OK) return s;
    s = check_mla_layers(mla, 1);
    if (s != DSA_OK) return s;
    if (!ws_ok(ws, ws_bytes, dsa_paged_mla_workspace_bytes(batch, mla))) return DSA_ERR_WORKSPACE;
    if (batch->n_seq == 0 || batch->n_tok == 0) return DSA_OK;
    const bool fp8 = mla_kv_fp8(mla);
    if (fp8 && (mla->dtype != DSA_BF16 || mla->d_latent != kLatent || mla->d_rope != kRope ||
                mla->kv_row_stride % 16 != 0 || mla->kv_seq_stride % 16 != 0 || !aligned16(mla->kv)))
        return DSA_ERR_UNSUPPORTED;
    if (mla->heads > 65535 || mla->d_latent + mla->d_rope > kGenMaxDims) return DSA_ERR_UNSUPPORTED;
    const PagedMlaArgs a = paged_args(batch, mla, ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = paged_mla_tc_shape(a)
                              ? launch_paged_mla_tc(a, static_cast<uint8_t *>(ws) + kStatus, sm_count(), st)
                              : launch_paged_mla_generic(a, st);
    return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
