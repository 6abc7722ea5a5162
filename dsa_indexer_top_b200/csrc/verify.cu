// verify.cu -- verification of drafted tokens (dsa_verify_drafts).
//
// Draft x_i stands while u_i q_i(x_i) < p_i(x_i) (float64: the product of two
// float32 values is exact there).  At the first rejection i the next token is the
// lowest j with sum_{k<=j} w_k > u sum_k w_k, w = max(p_i - q_i, 0); with every
// draft accepted w = p_n.  The weights are summed in float64, so that neither the
// order of summation nor a float32 rounding decides the token.
#include <cfloat>
#include <climits>

#include <cuda_bf16.h>
#include <nvtx3/nvToolsExt.h>

#include "dsa.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;

// A probability as float64; negative, NaN and infinite values count as 0.
__device__ __forceinline__ double prob(float x) { return x > 0.f && x <= FLT_MAX ? static_cast<double>(x) : 0.0; }
__device__ __forceinline__ float ld_p(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ld_p(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }

// One CTA per request; each warp holds a contiguous segment of the vocabulary.
template <typename T>
__global__ void __launch_bounds__(kVerThreads) verify_kernel(const VerifyArgs a) {
    __shared__ double seg[kVerWarps];
    __shared__ int last_s[kVerWarps];
    __shared__ int acc_s;
    const dsa_verify &v = a.v;
    const int r = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    const int per = ((V + kVerWarps - 1) / kVerWarps + 31) / 32 * 32;
    const int j0 = min(warp * per, V), j1 = min(j0 + per, V);
    int chosen = -1;
    for (int pass = 0; pass < 2 && chosen < 0; ++pass) {
        // pass 1 only where the residual has no weight: the target's own row
        const T *qr = pass == 0 ? qrow : nullptr;
        const int skip = pass == 0 ? gone : -1;
        auto weight = [&](int j) -> double {
            if (j == skip) return 0.0;
            const double p = prob(ld_p(prow, j));
            return qr ? fmax(p - prob(ld_p(qr, j)), 0.0) : p;
        };
        double s = 0.0;
        int last = -1;
        for (int j = j0 + lane; j < j1; j += 32) {
            const double w = weight(j);
            s += w;
            if (w > 0.0) last = j;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
        }
        __syncthreads();
        if (lane == 0) seg[warp] = s, last_s[warp] = last;
        __syncthreads();
        double total = 0.0;
        int any = -1;
        for (int w = 0; w < kVerWarps; ++w) {
            total += seg[w];
            any = max(any, last_s[w]);
        }
        if (any < 0) continue;  // no weight at all
        const float u = v.sample_u[r];
        const double target = (u > 0.f ? static_cast<double>(u) : 0.0) * total;
        // the segment that crosses the target, scanned by every warp alike
        double before = 0.0;
        int sg = 0;
        for (; sg < kVerWarps - 1 && !(before + seg[sg] > target); ++sg) before += seg[sg];
        const int k0 = min(sg * per, V), k1 = min(k0 + per, V);
        for (int b = k0; b < k1 && chosen < 0; b += 32) {
            double c = b + lane < k1 ? weight(b + lane) : 0.0;
            const bool some = c > 0.0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) c += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, some && before + c > target);
            if (hit) chosen = b + __ffs(hit) - 1;
            before += __shfl_sync(0xffffffffu, c, 31);
        }
        // (a sum rounded past the total, or u >= 1: the last token with weight)
        if (chosen < 0 || chosen > any) chosen = any;
    }
    if (chosen < 0) bad = true;
    for (int i = threadIdx.x; i <= D; i += kVerThreads)
        v.tokens[static_cast<int64_t>(r) * (D + 1) + i] = i < acc ? x[i] : i == acc ? chosen : -1;
    if (threadIdx.x == 0) {
        v.n_accept[r] = acc;
        if (bad) report_status(a.status, DSA_ERR_INVALID);
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, int num_sms, cudaStream_t st) {
    (void)num_sms;
    if (a.v.dtype == DSA_BF16)
        return launch_pdl(verify_kernel<__nv_bfloat16>, dim3(a.v.n_req), dim3(kVerThreads), 0, st, a);
    return launch_pdl(verify_kernel<float>, dim3(a.v.n_req), dim3(kVerThreads), 0, st, a);
}

}  // namespace dsa

extern "C" dsa_status dsa_verify_drafts(const dsa_verify *v, void *ws, size_t ws_bytes, void *stream) {
    nvtxRangePushA("dsa_verify_drafts");
    struct Pop {
        ~Pop() { nvtxRangePop(); }
    } pop;
    if (!v || v->n_req < 0 || v->n_draft < 0 || v->n_draft >= INT32_MAX || v->vocab < 1) return DSA_ERR_INVALID;
    if (v->dtype != DSA_BF16 && v->dtype != DSA_F32)
        return v->dtype == DSA_FP8_E4M3 ? DSA_ERR_UNSUPPORTED : DSA_ERR_INVALID;
    if (v->t_req_stride < 0 || v->t_row_stride < 0 || v->d_req_stride < 0 || v->d_row_stride < 0)
        return DSA_ERR_INVALID;
    if (v->n_req > 0 && (!v->target || !v->sample_u || !v->tokens || !v->n_accept)) return DSA_ERR_INVALID;
    if (v->n_req > 0 && v->n_draft > 0 && (!v->draft_tokens || !v->accept_u)) return DSA_ERR_INVALID;
    const uintptr_t el = v->dtype == DSA_F32 ? 3 : 1;
    if ((reinterpret_cast<uintptr_t>(v->target) & el) || (reinterpret_cast<uintptr_t>(v->draft) & el))
        return DSA_ERR_INVALID;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < 256) return DSA_ERR_WORKSPACE;
    if (v->n_req == 0) return DSA_OK;
    dsa::VerifyArgs a;
    a.v = *v;
    a.status = static_cast<uint32_t *>(ws);
    return dsa::launch_verify(a, dsa::sm_count_current(), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DSA_OK
               : DSA_ERR_CUDA;
}
