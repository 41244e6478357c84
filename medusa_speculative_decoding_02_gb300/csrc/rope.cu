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
// partner half of a pair by one shuffle per element.
//
// Angles: p * inv_freq reaches 10^5 turns at far positions, where fp32 has no
// fraction left.  inv_freq becomes a 64-bit fixed-point number of turns per
// position, modulo one (turns_per_position); p times that, modulo 2^64, is the
// fraction of a turn to 2^-33 at every p.  Integers throughout: this GPU does
// two fp64 products a cycle and SM, and the same in fp64 cost 2.4 us at 65
// rows.  Sine and cosine are taken in fp32 on [-1/2, 1/2] turn.  A lane meets
// the same eight angles in every vector of the row and keeps their sines and
// cosines in registers.
//
// Bound by the bytes of q, K and V read and written once; the loads of a row
// are issued before its angles are computed.
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

// f / (2 pi) modulo one in units of 2^-64, for finite f: with f = m 2^e (m a
// 24-bit integer), 128 bits of 2^e / (2 pi) modulo one times m, its top half.
// w0 .. w3 are the first 256 bits of 1 / (2 pi) after the point.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
    constexpr uint64_t w0 = 0x28be60db9391054aull, w1 = 0x7f09d5f47d4d3770ull,
                       w2 = 0x36d8a5664f10e410ull, w3 = 0x7f9458eaf7aef158ull;
    const uint32_t u = __float_as_uint(f) & 0x7fffffffu;
    const int ex = (int)(u >> 23);
    const uint64_t m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int e = max(ex, 1) - 150;
    uint64_t hi, lo;
    if (e >= 0) {  // at most 104
        const int r = e & 63;
        const uint64_t a = e < 64 ? w0 : w1, b = e < 64 ? w1 : w2, c = e < 64 ? w2 : w3;
        hi = r ? (a << r) | (b >> (64 - r)) : a;
        lo = r ? (b << r) | (c >> (64 - r)) : b;
    } else {       // at least -149
        const int r = -e;
        hi = r < 64 ? w0 >> r : 0;
        lo = r < 64 ? (w1 >> r) | (w0 << (64 - r)) : r < 128 ? w0 >> (r - 64) : 0;
    }
    const uint64_t step = m * hi + __umul64hi(m, lo);
    return f < 0.f ? 0 - step : step;
}

// grid (R, vector groups, B); a CTA takes NP * 256 / (dh/8) vectors of its row: H queries, then Hkv keys, then (with caches) Hkv values
template <typename T, int DH, int NP>
__global__ void __launch_bounds__(kRopeThreads, NP == 1 ? 1 : sizeof(T) == 2 ? 4 : 2) qk_norm_rope_kernel(RopeArgs a) {
    pdl_enter();
    constexpr int LPV = DH / 8;                  // lanes per vector
    constexpr int VPP = kRopeThreads / LPV;      // vectors per pass
    // (cos, sin) of pair j at cs_at(j): the lanes of a vector then read
    // consecutive words
    __shared__ float2 cs[kMaxRot / 2];
    auto cs_at = [](int j) { return (j & 7) * (kMaxRot / 16) + (j >> 3); };
    const int tid = threadIdx.x, sub = tid % LPV, e0 = sub * 8;
    const int b = blockIdx.z, i = blockIdx.x;
    const long long row = (long long)b * a.R + i;
    const int half = a.rot / 2;
    constexpr int W = 8 / Vec16<T>::N;           // 16-byte words of a lane's elements
    // everything the row's loads and angles depend on, in one round of loads
    const int n_rows = a.n_rows ? a.n_rows[b] : a.R;
    T *const kc = a.kc ? static_cast<T *>(a.kc[b]) : nullptr;
    T *const vc = a.kc ? static_cast<T *>(a.vc[b]) : nullptr;
    const int P = a.kc ? a.prefix_len[b] : 0;
    const int pos = a.pos[row];
    const float freq = tid < half ? a.inv_freq[tid] : 0.f;
    uint4 wraw[2][W];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const T *w = static_cast<const T *>(k ? a.kw : a.qw);
#pragma unroll
        for (int c = 0; c < W; ++c)
            wraw[k][c] = w ? *reinterpret_cast<const uint4 *>(w + e0 + c * Vec16<T>::N) : make_uint4(0, 0, 0, 0);
    }
    if (i >= n_rows) return;                     // uniform over the CTA
    T *krow, *vrow = nullptr;
    if (a.kc) {
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
    const int nq = a.H, nqk = a.H + a.Hkv, nv = nqk + (a.kc ? a.Hkv : 0);
    const int v0 = blockIdx.y * (VPP * NP) + tid / LPV;
    // the row's vectors, as if each kind went on from the one before
    const T *const qrow = static_cast<const T *>(a.q) + row * a.q_stride + e0;
    const T *const kin = static_cast<const T *>(a.k) + row * a.k_stride - (long long)nq * DH + e0;
    const T *const vin = static_cast<const T *>(a.v) + row * a.v_stride - (long long)nqk * DH + e0;
    uint4 raw[NP][W];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int v = v0 + n * VPP;
        const T *src = (v < nq ? qrow : v < nqk ? kin : vin) + v * DH;
#pragma unroll
        for (int c = 0; c < W; ++c)
            raw[n][c] = v < nv ? ld_stream16(src + c * Vec16<T>::N) : make_uint4(0, 0, 0, 0);
    }
    if (tid < half) {
        // fraction of a turn, in [-1/2, 1/2)
        const int64_t frac = (int64_t)((uint64_t)(int64_t)pos * turns_per_position(freq));
        float s, c;
        sincospif((float)frac * 0x1p-63f, &s, &c);
        if (!(fabsf(freq) < INFINITY)) s = c = NAN;
        cs[cs_at(tid)] = make_float2(c, s);
    }
    __syncthreads();
    // this lane's cosines and sines, by pairs of elements; y = x cos + o sin, o
    // the partner element, so the first of a pair takes -sin
    const bool turned = e0 < a.rot;  // rot is a multiple of 16: the same for all eight
    const int lane = tid & 31;
    const int partner = e0 < half ? lane + half / 8 : turned ? lane - half / 8 : lane;
    float2 c2[4], s2[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        c2[e] = make_float2(1.f, 1.f);
        s2[e] = make_float2(0.f, 0.f);
        if (turned && a.interleaved) {
            const float2 t = cs[cs_at(e0 / 2 + e)];
            c2[e] = make_float2(t.x, t.x);
            s2[e] = make_float2(-t.y, t.y);
        } else if (turned) {
            const int j = (e0 < half ? e0 : e0 - half) + 2 * e;
            const float2 t = cs[cs_at(j)], u = cs[cs_at(j + 1)];
            c2[e] = make_float2(t.x, u.x);
            s2[e] = e0 < half ? make_float2(-t.y, -u.y) : make_float2(t.y, u.y);
        }
    }
    T *const qout = static_cast<T *>(a.q_out) + row * nq * DH + e0;
    T *const kout = krow - (long long)nq * DH + e0;
    T *const vout = vrow - (long long)nqk * DH + e0;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int v = v0 + n * VPP;
        T *dst = (v < nq ? qout : v < nqk ? kout : vout) + v * DH;
        if (__all_sync(0xffffffffu, v >= nqk)) {  // values (or past the end): copied
            if (v < nv)
#pragma unroll
                for (int c = 0; c < W; ++c)
                    *reinterpret_cast<uint4 *>(dst + c * Vec16<T>::N) = raw[n][c];
            continue;
        }
        float x[8];
        widen8<T>(raw[n], x);
        float2 x2[4], o2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x2[e] = make_float2(x[2 * e], x[2 * e + 1]);
        if (a.norm) {  // uniform: the shuffles run in every lane
            float2 q2 = __fmul2_rn(x2[0], x2[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) q2 = __ffma2_rn(x2[e], x2[e], q2);
            float ss = q2.x + q2.y;
#pragma unroll
            for (int o = LPV / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = rsqrtf(fmaf(ss, 1.f / DH, a.eps));  // within 2 units in the last place
            const float2 i2 = make_float2(inv, inv);
            const bool is_q = v < nq;
            if (is_q ? a.qw : a.kw) {
                uint4 ww[W];
                float wf[8];
#pragma unroll
                for (int c = 0; c < W; ++c) ww[c] = is_q ? wraw[0][c] : wraw[1][c];
                widen8<T>(ww, wf);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x2[e] = __fmul2_rn(x2[e], __fmul2_rn(i2, make_float2(wf[2 * e], wf[2 * e + 1])));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x2[e] = __fmul2_rn(x2[e], i2);
            }
        }
        if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o2[e] = make_float2(x2[e].y, x2[e].x);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o2[e] = make_float2(__shfl_sync(0xffffffffu, x2[e].x, partner),
                                    __shfl_sync(0xffffffffu, x2[e].y, partner));
        }
        if (a.rot < DH && !turned) {  // unchanged, whatever they hold (inf * 0 is not 0)
#pragma unroll
            for (int e = 0; e < 4; ++e) o2[e] = make_float2(0.f, 0.f);
        }
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 t = __ffma2_rn(o2[e], s2[e], __fmul2_rn(x2[e], c2[e]));
            y[2 * e] = t.x;
            y[2 * e + 1] = t.y;
        }
        if (v < nqk)
            store8(dst, y);
        else if (v < nv)  // a warp with a key and a value
#pragma unroll
            for (int c = 0; c < W; ++c)
                *reinterpret_cast<uint4 *>(dst + c * Vec16<T>::N) = raw[n][c];
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
    cudaError_t e = launch_pdl(kern, dim3(R, (passes + per_cta - 1) / per_cta, B),
                               dim3(kRopeThreads), 0, stream, a);
    note_launch();
    return e;
}

}  // namespace medusa
