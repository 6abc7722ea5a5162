// verify.cu -- verification of drafted tokens (dsa_verify_drafts).
//
// Draft x_i stands while u_i q_i(x_i) < p_i(x_i) (float64: the product of two
// float32 values is exact there).  At the first rejection i the next token is the
// lowest j with sum_{k<=j} w_k > u sum_k w_k, w = max(p_i - q_i, 0); with every
// draft accepted w = p_n.  The weights are summed in float64, so that neither the
// order of summation nor a float32 rounding decides the token.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <utility>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <nvtx3/nvToolsExt.h>

#include "dsa.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

// A cluster of CTAs per request.  One pass over the one row pair that decides the
// token: each warp sums a contiguous segment of the vocabulary; the segments' sums go
// to every CTA of the cluster, the one whose segment crosses the target reads that
// segment (an eighth of its share, still in L2) once more and finds the token by a scan of
// per-thread runs.  Bound by memory: 4 or 2 bytes per entry and row, and by latency
// (three dependent round trips) for few requests.  Measured (one B200): 96 requests, up
// to 4 drafts, vocabulary 131071 in float32 33 us (66 MB: the draft's row is read where a
// draft is rejected, some 30 of 96; 2.0 TB/s; float64 conversions and sums share the
// issue slots); one CTA per request 252 us; 512 threads, two CTAs per SM 43 us.  5
// requests, 32000 in bf16: 9.9 us (one CTA per request 34).
constexpr int kVerThreads = 256;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerPerSm = 4;  // CTAs per SM (they fit with up to 64 registers a thread)
constexpr int kVerMaxCluster = 8;
constexpr int kVerUnroll = 8;  // loads of a row in flight per thread

// A probability as float64; negative, NaN and infinite values count as 0.
__device__ __forceinline__ double prob(float x) { return x > 0.f && x <= FLT_MAX ? static_cast<double>(x) : 0.0; }
__device__ __forceinline__ float ld_p(const float *p, int64_t i) { return __ldg(p + i); }
__device__ __forceinline__ float ld_p(const __nv_bfloat16 *p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short *>(p) + i)) << 16);
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads) verify_kernel(const VerifyArgs a) {
    namespace cg = cooperative_groups;
    __shared__ double seg[kVerMaxCluster * kVerWarps];
    __shared__ int last_s[kVerMaxCluster * kVerWarps];
    __shared__ double run[kVerWarps];
    __shared__ int acc_s, first_s, chosen_s;
    cg::cluster_group cluster = cg::this_cluster();
    const dsa_verify &v = a.v;
    const int CL = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int r = blockIdx.x / CL, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Shared memory of another CTA may be written once that CTA has begun: this arrival
    // and the wait before the first such write say so (the pass over the row lies
    // between the two, so the wait costs nothing).
    auto begun = cluster.barrier_arrive();
    griddep_wait();
    const int D = v.n_draft, V = v.vocab;
    const T *pt = static_cast<const T *>(v.target) + r * v.t_req_stride;
    const T *qt = v.draft ? static_cast<const T *>(v.draft) + r * v.d_req_stride : nullptr;
    const int32_t *x = v.draft_tokens + static_cast<int64_t>(r) * D;
    int n = v.draft_len ? v.draft_len[r] : D;
    bool bad = n < 0 || n > D;
    n = min(max(n, 0), D);
    if (warp == 0) {
        int acc = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            bool ok = false;
            if (i < n) {
                const int t = x[i];
                if (t >= 0 && t < V) {
                    const double p = prob(ld_p(pt, i * v.t_row_stride + t));
                    const double q = qt ? prob(ld_p(qt, i * v.d_row_stride + t)) : 1.0;
                    ok = static_cast<double>(v.accept_u[static_cast<int64_t>(r) * D + i]) * q < p;
                }
            }
            const unsigned fail = ~__ballot_sync(0xffffffffu, ok);
            acc = i0 + (fail ? __ffs(fail) - 1 : 32);
            if (fail) break;
        }
        acc = min(acc, n);
        if (lane == 0) acc_s = acc;
    }
    if (tid == 0) chosen_s = -1, first_s = kVerThreads;
    __syncthreads();
    const int acc = acc_s;
    const bool rejected = acc < n;
    const T *prow = pt + acc * v.t_row_stride;
    const T *qrow = qt && rejected ? qt + acc * v.d_row_stride : nullptr;
    int gone = -1;  // greedy drafts: the rejected token itself
    if (rejected) {
        const int t = x[acc];
        if (t < 0 || t >= V)
            bad = true;
        else if (!qt)
            gone = t;
    }
    const float u = v.sample_u[r];
    const int nw = CL * kVerWarps;
    const int per = ((V + nw - 1) / nw + 31) / 32 * 32;  // a warp's segment
    const int gw = rank * kVerWarps + warp;
    const int j0 = static_cast<int>(min(static_cast<int64_t>(gw) * per, static_cast<int64_t>(V)));
    const int j1 = min(j0 + per, V);
    bool writer = false;
    for (int pass = 0; pass < 2; ++pass) {
        // the second pass only where the residual has no weight: the target's own row
        const T *qr = pass == 0 ? qrow : nullptr;
        const int skip = pass == 0 ? gone : -1;
        auto weight = [&](float p, float q, int j) -> double {
            const double w = prob(p) - (qr ? prob(q) : 0.0);
            return w > 0.0 && j != skip ? w : 0.0;
        };
        double s = 0.0;
        int last = -1;
        for (int b = j0 + lane; b < j1; b += 32 * kVerUnroll) {
            float p[kVerUnroll], q[kVerUnroll];
#pragma unroll
            for (int k = 0; k < kVerUnroll; ++k) {
                const int j = b + 32 * k;
                p[k] = j < j1 ? ld_p(prow, j) : 0.f;
                q[k] = qr && j < j1 ? ld_p(qr, j) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kVerUnroll; ++k) {
                const double w = weight(p[k], q[k], b + 32 * k);
                s += w;
                if (w > 0.0) last = b + 32 * k;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
        }
        if (pass == 0)
            cluster.barrier_wait(std::move(begun));  // every CTA has begun
        else
            cluster.sync();  // every CTA has read the first pass's sums
        if (lane < CL) {
            *cluster.map_shared_rank(&seg[gw], lane) = s;
            *cluster.map_shared_rank(&last_s[gw], lane) = last;
        }
        cluster.sync();
        // every warp alike: total weight, then the segment that crosses the target
        double total = 0.0;
        int any = -1;
        for (int w = 0; w < nw; ++w) {
            total += seg[w];
            any = max(any, last_s[w]);
        }
        if (any < 0 && pass == 0) continue;  // no weight at all (the same in every CTA)
        if (any < 0) {
            writer = rank == 0;
            break;
        }
        const double target = (u > 0.f ? static_cast<double>(u) : 0.0) * total;
        double before = 0.0;
        int sg = 0;
        for (; sg < nw - 1 && !(before + seg[sg] > target); ++sg) before += seg[sg];
        writer = sg / kVerWarps == rank;
        if (!writer) break;
        // a run of entries per thread, a scan of the runs' sums
        const int k0 = static_cast<int>(min(static_cast<int64_t>(sg) * per, static_cast<int64_t>(V)));
        const int k1 = min(k0 + per, V);
        const int len = (per + kVerThreads - 1) / kVerThreads;
        const int a0 = min(k0 + tid * len, k1), a1 = min(a0 + len, k1);
        double c = 0.0;
        for (int j = a0; j < a1; ++j) c += weight(ld_p(prow, j), qr ? ld_p(qr, j) : 0.f, j);
        double inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        // a run starts at the very sum its predecessor ends with, so that no target falls
        // between two runs
        const double prev = __shfl_up_sync(0xffffffffu, inc, 1);
        if (lane == 31) run[warp] = inc;
        __syncthreads();
        for (int w = 0; w < warp; ++w) before += run[w];
        const unsigned past = __ballot_sync(0xffffffffu, c > 0.0 && before + inc > target);
        if (lane == 0 && past) atomicMin(&first_s, 32 * warp + __ffs(past) - 1);
        __syncthreads();
        if (tid == first_s) {
            // this run crosses: its first entry past the target (its last with weight
            // where rounding leaves none)
            double t = lane > 0 ? before + prev : before;
            int pick = -1;
            for (int j = a0; j < a1; ++j) {
                const double w = weight(ld_p(prow, j), qr ? ld_p(qr, j) : 0.f, j);
                t += w;
                if (w > 0.0) {
                    pick = j;
                    if (t > target) break;
                }
            }
            chosen_s = pick;
        } else if (tid == 0 && first_s == kVerThreads) {
            // No run crosses: the segment's sum, added in another order than the runs',
            // rounds past the target and theirs do not (its last entry with weight), or the
            // target is at or past the total (u >= 1, rounding: the last of all).
            chosen_s = last_s[sg] >= 0 ? last_s[sg] : any;
        }
        __syncthreads();
        break;
    }
    cluster.sync();  // no CTA leaves while another may write to it
    if (!writer) return;
    const int chosen = chosen_s;
    if (chosen < 0) bad = true;
    for (int i = tid; i <= D; i += kVerThreads)
        v.tokens[static_cast<int64_t>(r) * (D + 1) + i] = i < acc ? x[i] : i == acc ? chosen : -1;
    if (tid == 0) {
        v.n_accept[r] = acc;
        if (bad) report_status(a.status, DSA_ERR_INVALID);
    }
}

template <typename T>
cudaError_t launch_verify_t(const VerifyArgs &a, int num_sms, cudaStream_t st) {
    // as many CTAs per request as are all resident at once
    const int64_t slots = static_cast<int64_t>(kVerPerSm) * num_sms;
    const int cl = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kVerMaxCluster, slots / a.v.n_req)));
    if (static_cast<int64_t>(a.v.n_req) * cl > INT_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.v.n_req) * cl);
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cl;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, int num_sms, cudaStream_t st) {
    return a.v.dtype == DSA_BF16 ? launch_verify_t<__nv_bfloat16>(a, num_sms, st) : launch_verify_t<float>(a, num_sms, st);
}

}  // namespace dsa

extern "C" dsa_status dsa_verify_drafts(const dsa_verify *v, void *ws, size_t ws_bytes, void *stream) {
    nvtxRangePushA("dsa_verify_drafts");
    struct Pop {
        ~Pop() { nvtxRangePop(); }
    } pop;
    if (!v || v->n_req < 0 || v->n_draft < 0 || v->n_draft >= INT32_MAX || v->vocab < 1) return DSA_ERR_INVALID;
    if (v->vocab > (1 << 30)) return DSA_ERR_UNSUPPORTED;
    if (v->dtype != DSA_BF16 && v->dtype != DSA_F32)
        return v->dtype == DSA_FP8_E4M3 ? DSA_ERR_UNSUPPORTED : DSA_ERR_INVALID;
    if (v->t_req_stride < 0 || v->t_row_stride < 0 || v->d_req_stride < 0 || v->d_row_stride < 0)
        return DSA_ERR_INVALID;
    if (v->n_req > 0 && (!v->target || !v->sample_u || !v->tokens || !v->n_accept)) return DSA_ERR_INVALID;
    if (v->n_req > 0 && v->n_draft > 0 && (!v->draft_tokens || !v->accept_u)) return DSA_ERR_INVALID;
    const uintptr_t el = v->dtype == DSA_F32 ? 3 : 1;
    if ((reinterpret_cast<uintptr_t>(v->target) & el) || (reinterpret_cast<uintptr_t>(v->draft) & el))
        return DSA_ERR_INVALID;
    const bool any = v->n_draft > 0;  // (empty arrays may stand anywhere)
    const void *in[] = {v->target,   v->sample_u, v->draft_len, any ? v->draft : nullptr, any ? v->draft_tokens : nullptr,
                        any ? v->accept_u : nullptr};
    for (const void *x : in)
        if (x && v->n_req > 0 && (x == v->tokens || x == v->n_accept)) return DSA_ERR_INVALID;
    if (v->n_req > 0 && static_cast<const void *>(v->tokens) == v->n_accept) return DSA_ERR_INVALID;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return DSA_ERR_WORKSPACE;
    if (v->n_req == 0) return DSA_OK;
    dsa::VerifyArgs a;
    a.v = *v;
    a.status = static_cast<uint32_t *>(ws);
    return dsa::launch_verify(a, dsa::sm_count(), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DSA_OK
               : DSA_ERR_CUDA;
}
