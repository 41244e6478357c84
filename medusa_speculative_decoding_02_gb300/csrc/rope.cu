// rope.cu -- norms of queries and keys and the position rotation, one pass.
//
// For every head vector x of a row at position p:
//     y = x / sqrt(mean(x^2) + eps) * w                      (with norms)
//     (y_a, y_b) -> (y_a cos t - y_b sin t, y_a sin t + y_b cos t),
//     t = p * inv_freq[j],  j = 0 .. rot/2 - 1,
// the pair (a, b) being (j, j + rot/2) or, interleaved, (2j, 2j+1); elements
// from rot on stay.  K goes to k_out or straight into its cache slot, where V
// is copied as well.
//
// Each vector is held by dh/8 lanes with eight elements each: one or two
// 16-byte loads a lane, the sum of squares by shuffles inside the group, the
// partner half of a pair by one shuffle per element.  The row's angles are
// computed once per CTA: p * inv_freq reaches 10^5 turns at far positions,
// where fp32 has no fraction left, so the product and its reduction to a
// fraction of a turn are taken in fp64 (rot/2 of them per CTA, next to
// thousands of elements) and the sine and cosine in fp32 on [-1/2, 1/2] turn.
// A lane meets the same eight angles in every vector of the row and keeps
// their sines and cosines in registers.  Bound by the bytes of q, K and V read
// and written once; the loads are issued before the angles are computed.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace medusa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxRot = 128;

struct RopeArgs {
    const void *q, *k, *v;  // v: only with caches
    long long q_stride, k_stride, v_stride;
    const void *qw, *kw;    // [dh] or null (ones)
    float eps;
    int norm, interleaved;
    const int32_t *pos;
    const float *inv_freq;
    int rot;
    const int32_t *n_rows;
    int R, H, Hkv;
    void *q_out, *k_out;
    void *const *kc;        // null: K to k_out
    void *const *vc;
    const int32_t *prefix_len;
    int P_max;
    int *status;
};

template <typename T>
__device__ __forceinline__ void widen8(const uint4 (&w)[8 / Vec16<T>::N], float (&x)[8]) {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int u = 0; u < 8 / N; ++u) {
        float f[N];
        Vec16<T>::widen(w[u], f);
#pragma unroll
        for (int e = 0; e < N; ++e) x[u * N + e] = f[e];
    }
}

__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(bf16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * u], x[2 * u + 1]);
        w[u] = *reinterpret_cast<const uint32_t *>(&t);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// grid (B * R rows, vector groups); a CTA takes NP * 256 / (dh/8) vectors of
// its row: H queries, then Hkv keys, then (with caches) Hkv values
template <typename T, int DH, int NP>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(RopeArgs a) {
    pdl_enter();
    constexpr int LPV = DH / 8;                  // lanes per vector
    constexpr int VPP = kRopeThreads / LPV;      // vectors per pass
    __shared__ float2 cs[kMaxRot / 2];           // (cos, sin)
    const int tid = threadIdx.x, sub = tid % LPV, e0 = sub * 8;
    const long long row = blockIdx.x;
    const int b = (int)(row / a.R), i = (int)(row - (long long)b * a.R);
    if (a.n_rows && i >= a.n_rows[b]) return;    // uniform over the CTA
    T *krow = nullptr, *vrow = nullptr;
    if (a.kc) {
        T *kc = static_cast<T *>(a.kc[b]), *vc = static_cast<T *>(a.vc[b]);
        const int P = a.prefix_len[b];
        const bool bad_ptr =
            !kc || !vc ||
            ((reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) & 15u);
        if (bad_ptr || P < 0 || P > a.P_max) {   // the sequence is left untouched
            if (tid == 0) set_status(a.status, bad_ptr ? MEDUSA_DEV_BAD_CACHE : MEDUSA_DEV_BAD_PREFIX);
            return;
        }
        krow = kc + (size_t)(P + i) * a.Hkv * DH;
        vrow = vc + (size_t)(P + i) * a.Hkv * DH;
    } else {
        krow = static_cast<T *>(a.k_out) + row * a.Hkv * DH;
    }
    const int nv = a.H + a.Hkv + (a.kc ? a.Hkv : 0);
    const int v0 = blockIdx.y * (VPP * NP) + tid / LPV;
    constexpr int W = 8 / Vec16<T>::N;           // 16-byte words of a lane's elements
    uint4 raw[NP][W];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int v = v0 + n * VPP;
        const T *src = v < a.H           ? static_cast<const T *>(a.q) + row * a.q_stride + v * DH
                       : v < a.H + a.Hkv ? static_cast<const T *>(a.k) + row * a.k_stride + (v - a.H) * DH
                       : v < nv ? static_cast<const T *>(a.v) + row * a.v_stride + (v - a.H - a.Hkv) * DH
                                : nullptr;
#pragma unroll
        for (int c = 0; c < W; ++c)
            raw[n][c] = src ? ld_stream16(src + e0 + c * Vec16<T>::N) : make_uint4(0, 0, 0, 0);
    }
    const int half = a.rot / 2;
    if (tid < half) {
        const double turns =
            (double)a.pos[row] * ((double)a.inv_freq[tid] * 0.15915494309189533577);  // 1/(2 pi)
        const float frac = (float)(turns - rint(turns));  // of a turn, in [-1/2, 1/2]
        float s, c;
        sincospif(2.f * frac, &s, &c);
        cs[tid] = make_float2(c, s);
    }
    __syncthreads();
    // this lane's angles: pair index of element e
    float2 t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int el = e0 + e;
        const int j = a.interleaved ? el / 2 : el < half ? el : el - half;
        t[e] = el < a.rot ? cs[j] : make_float2(1.f, 0.f);
    }
    const int lane = tid & 31;
    const bool turned = e0 < a.rot;  // rot is a multiple of 16: the same for all eight
    const int partner = e0 < half ? lane + half / 8 : e0 < a.rot ? lane - half / 8 : lane;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int v = v0 + n * VPP;
        float x[8];
        widen8<T>(raw[n], x);
        if (a.norm) {  // uniform: the shuffles below run in every lane
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LPV / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const T *w = static_cast<const T *>(v < a.H ? a.qw : a.kw);
            if (v < a.H + a.Hkv) {
                const float inv = 1.f / sqrtf(ss / DH + a.eps);
                float wf[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
                if (w) {
                    uint4 ww[W];
#pragma unroll
                    for (int c = 0; c < W; ++c)
                        ww[c] = *reinterpret_cast<const uint4 *>(w + e0 + c * Vec16<T>::N);
                    widen8<T>(ww, wf);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * wf[e];
            }
        }
        float y[8];
        if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                y[e] = turned ? x[e] * t[e].x - x[e + 1] * t[e].y : x[e];
                y[e + 1] = turned ? x[e] * t[e].y + x[e + 1] * t[e].x : x[e + 1];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float o = __shfl_sync(0xffffffffu, x[e], partner);
                // lower half: a cos - b sin; upper half: b cos + a sin
                y[e] = turned ? x[e] * t[e].x + (e0 < half ? -o : o) * t[e].y : x[e];
            }
        }
        if (v < a.H)
            store8(static_cast<T *>(a.q_out) + (row * a.H + v) * DH + e0, y);
        else if (v < a.H + a.Hkv)
            store8(krow + (v - a.H) * DH + e0, y);
        else if (v < nv)
            store8(vrow + (v - a.H - a.Hkv) * DH + e0, x);
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(medusa_dtype dtype, const void *q, const void *k, const void *v,
                                long long q_stride, long long k_stride, long long v_stride,
                                const void *q_weight, const void *k_weight, float eps, int norm,
                                const int32_t *pos, const float *inv_freq, int rot,
                                int interleaved, const int32_t *n_rows, void *const *k_cache,
                                void *const *v_cache, const int32_t *prefix_len, int P_max, int B,
                                int R, int H, int Hkv, int dh, void *q_out, void *k_out, void *ws,
                                cudaStream_t stream) {
    RopeArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.qw = q_weight;
    a.kw = k_weight;
    a.eps = eps;
    a.norm = norm;
    a.interleaved = interleaved;
    a.pos = pos;
    a.inv_freq = inv_freq;
    a.rot = rot;
    a.n_rows = n_rows;
    a.R = R;
    a.H = H;
    a.Hkv = Hkv;
    a.q_out = q_out;
    a.k_out = k_out;
    a.kc = k_cache;
    a.vc = v_cache;
    a.prefix_len = prefix_len;
    a.P_max = P_max;
    a.status = static_cast<int *>(ws);
    const int nv = H + Hkv + (k_cache ? Hkv : 0);
    const long long rows = (long long)B * R;
    const int vpp = kRopeThreads / (dh / 8);
    // With few rows one pass per CTA puts more CTAs to work; with enough of them
    // four passes share a row's angles and keep four loads a lane in flight.
    const int passes = (nv + vpp - 1) / vpp;
    const bool many = rows * passes >= 16LL * device_sm_count();
    auto pick = [&](auto one, auto four) { return many ? four : one; };
    auto kern =
        dtype == MEDUSA_F32
            ? (dh == 128 ? pick(qk_norm_rope_kernel<float, 128, 1>, qk_norm_rope_kernel<float, 128, 4>)
                         : pick(qk_norm_rope_kernel<float, 64, 1>, qk_norm_rope_kernel<float, 64, 4>))
            : (dh == 128 ? pick(qk_norm_rope_kernel<bf16, 128, 1>, qk_norm_rope_kernel<bf16, 128, 4>)
                         : pick(qk_norm_rope_kernel<bf16, 64, 1>, qk_norm_rope_kernel<bf16, 64, 4>));
    const int per_cta = many ? 4 : 1;
    cudaError_t e = launch_pdl(kern, dim3((unsigned)rows, (passes + per_cta - 1) / per_cta),
                               dim3(kRopeThreads), 0, stream, a);
    note_launch();
    return e;
}

}  // namespace medusa
