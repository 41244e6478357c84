// logprobs.cu -- log probabilities of given tokens, with their ranks, the entropy
// of each row and its top alternatives.
//
// Row x of V logits, temperature T, token t:
//     logp = x_t / T - ln sum_i e^(x_i / T)
//     entropy = -sum_i p_i ln p_i = ln S - ln2 A / S, from the shifted sums
//         S = sum 2^(y - m), A = sum 2^(y - m) (y - m), y = x log2(e) / T
//     rank = number of tokens before t in the order (larger logit, then smaller id)
//     alternatives: the first `top` tokens of that order
#include <climits>

#include "common.cuh"
#include "launch.h"

namespace medusa {

namespace {

constexpr int kLpThreads = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LogprobArgs {
    const void *logits;
    long long stride;
    const int32_t *tokens;
    int V, top;
    float inv_T, y_scale;  // 1 / T, log2(e) / T
    float *logp, *entropy;
    int32_t *rank;
    int32_t *top_ids;
    float *top_logp;
    int *status;
};

template <typename F>
__device__ __forceinline__ float block_fold(float v, float *s, F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (lane == 0) s[warp] = v;
    __syncthreads();
    v = s[0];
    for (int w = 1; w < kLpThreads / 32; ++w) v = f(v, s[w]);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_kernel(LogprobArgs a) {
    pdl_enter();
    __shared__ float s_f[kLpThreads / 32];
    __shared__ int s_i[kLpThreads / 32];
    const int row = blockIdx.x, tid = threadIdx.x;
    const T *x = static_cast<const T *>(a.logits) + (long long)row * a.stride;
    auto add = [](float p, float q) { return p + q; };
    auto larger = [](float p, float q) { return fmaxf(p, q); };
    int tok = a.tokens[row];
    if (tok >= a.V || tok < -1) {
        if (tid == 0) set_status(a.status, MEDUSA_DEV_BAD_TOKEN);
        tok = -1;
    }
    const float xt = tok >= 0 ? Vec16<T>::load1(x + tok) : NAN;
    float m = -INFINITY, nan = 0.f;
    for (int i = tid; i < a.V; i += kLpThreads) {
        const float f = Vec16<T>::load1(x + i);
        m = fmaxf(m, f);
        if (!(f < INFINITY)) nan = 1.f;
    }
    m = block_fold(m, s_f, larger);
    const bool bad = block_fold(nan, s_f, larger) != 0.f;  // +inf or NaN in the row
    float S = 0.f, A = 0.f, before = 0.f;
    for (int i = tid; i < a.V; i += kLpThreads) {
        const float f = Vec16<T>::load1(x + i);
        const float t = fmaxf((f - m) * a.y_scale, -127.f), p = ex2_approx(t);
        S += p;
        A = fmaf(p, t, A);
        if (f > xt || (f == xt && i < tok)) before += 1.f;
    }
    S = block_fold(S, s_f, add);
    A = block_fold(A, s_f, add);
    before = block_fold(before, s_f, add);
    const bool none = m == -INFINITY;  // nothing is possible
    const float ls = log2f(S);
    auto logp_of = [&](float f) {
        return bad ? NAN : none ? -INFINITY : ((f - m) * a.inv_T - ls * kLn2);
    };
    if (tid == 0) {
        a.logp[row] = tok < 0 ? 0.f : logp_of(xt);
        a.rank[row] = tok < 0 || isnan(xt) ? -1 : (int)before;
        a.entropy[row] = bad ? NAN : none ? 0.f : fmaxf(kLn2 * (ls - A / S), 0.f);
    }
    float lv = INFINITY;  // the alternative before
    int li = -1;
    bool any = true;
    for (int k = 0; k < a.top; ++k) {
        float bv = -INFINITY;
        int bi = INT_MAX;
        if (any)
            for (int i = tid; i < a.V; i += kLpThreads) {
                const float f = Vec16<T>::load1(x + i);
                if (!isnan(f) && (k == 0 || better(lv, li, f, i)) && (bi == INT_MAX || better(f, i, bv, bi))) {
                    bv = f;
                    bi = i;
                }
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
            if (better(ov, oi, bv, bi)) bv = ov, bi = oi;
        }
        __syncthreads();
        if ((tid & 31) == 0) s_f[tid >> 5] = bv, s_i[tid >> 5] = bi;
        __syncthreads();
        for (int w = 0; w < kLpThreads / 32; ++w)
            if (better(s_f[w], s_i[w], bv, bi)) bv = s_f[w], bi = s_i[w];
        any = bi != INT_MAX;
        if (tid == 0) {
            a.top_ids[(size_t)row * a.top + k] = any ? bi : -1;
            a.top_logp[(size_t)row * a.top + k] = any ? logp_of(bv) : NAN;
        }
        lv = bv;
        li = bi;
    }
}

}  // namespace

cudaError_t launch_token_logprobs(medusa_dtype dtype, const void *logits, long long stride,
                                  const int32_t *tokens, int N, int V, int top, float temperature,
                                  float *logp, float *entropy, int32_t *rank, int32_t *top_ids,
                                  float *top_logp, void *ws, cudaStream_t stream) {
    LogprobArgs a;
    a.logits = logits;
    a.stride = stride;
    a.tokens = tokens;
    a.V = V;
    a.top = top;
    a.inv_T = 1.f / temperature;
    a.y_scale = kLog2e / temperature;
    a.logp = logp;
    a.entropy = entropy;
    a.rank = rank;
    a.top_ids = top_ids;
    a.top_logp = top_logp;
    a.status = static_cast<int *>(ws);
    auto kern = dtype == MEDUSA_F32 ? token_logprobs_kernel<float> : token_logprobs_kernel<bf16>;
    cudaError_t e = launch_pdl(kern, dim3(N), dim3(kLpThreads), 0, stream, a);
    note_launch();
    return e;
}

}  // namespace medusa
