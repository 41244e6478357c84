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
// Each vector is held by dh/8 lanes with four pairs each, both members of a pair
// in one lane: two pieces of four elements, rot/2 apart or, interleaved, next to
// each other.  A lane thus needs four angles and no exchange but the sum of
// squares (with 16-byte loads, eight shuffles fetched the partners and a lane kept
// eight sines and cosines: 38.5 against 31.3 us at the prompt below).
//
// Angles: p * inv_freq reaches 10^5 turns at far positions, where fp32 has no
// fraction left.  inv_freq becomes a 64-bit fixed-point number of turns per
// position, modulo one (turns_per_position, the argument reduction of Payne and
// Hanek: only those bits of 1/(2 pi) are multiplied that reach the fraction); p
// times that, modulo 2^64, is the fraction of a turn to 2^-33 at every p.
// Integers throughout: this GPU does two fp64 products a cycle and SM, and the
// same in fp64 cost 2.4 us at 65 rows.  Sine and cosine are taken in fp32 on
// [-1/2, 1/2] turn.
//
// Squares are summed in fp32, which holds for elements up to 2^60.  Taking vectors
// beyond it again, scaled by a power of two, was measured and not kept: the test in
// every pass, on a kernel bound by issue, took the prompt below from 31.6 us to
// 32.8-34.8.
//
// Bound by issue and, close behind, by the bytes of q, K and V read and written
// once; the loads of a row are issued before its angles are computed.  6481 rows
// of 32 + 8 + 8 vectors of 128 (159 MB) take 32.9 us, 4.8 TB/s (31.5 us back to
// back; fp32, 319 MB, 55.4 us, 5.8 TB/s); one row a CTA took 41.2 (40.7 M
// instructions a launch where four rows a CTA had 29.8 M).  65 rows of 32 + 32 +
// 32 vectors take 2.9 us, eight rows of 32 + 8 1.9 us: the latency of two rounds
// of loads.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace medusa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxRot = 128;
constexpr int kManyRows = 4, kManyPasses = 3;  // rows and passes of a CTA where there are many

struct RopeArgs {
    const void *q, *k, *v;  // v: only with caches
    long long q_stride, k_stride, v_stride;
    const void *qw, *kw;    // [dh] or null (ones)
    float eps;
    int norm;
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

// Four elements of a vector, the unit of a lane's loads and stores.
template <typename T>
using Piece = typename std::conditional<sizeof(T) == 2, uint2, uint4>::type;

// Plain loads that leave no line in L1: outputs may be the inputs (q_out = q), and
// the read-only path is for data that nothing writes during the kernel.  Every
// piece is read by the lane that overwrites it, before it does.
__device__ __forceinline__ uint2 ld_piece(const bf16 *p) {
    uint2 r;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ uint4 ld_piece(const float *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// element i of the lane's eight (lo: the first four, hi: the others)
__device__ __forceinline__ void widen(const uint2 &lo, const uint2 &hi, float (&x)[8]) {
    x[0] = bf_lo(lo.x), x[1] = bf_hi(lo.x), x[2] = bf_lo(lo.y), x[3] = bf_hi(lo.y);
    x[4] = bf_lo(hi.x), x[5] = bf_hi(hi.x), x[6] = bf_lo(hi.y), x[7] = bf_hi(hi.y);
}
__device__ __forceinline__ void widen(const uint4 &lo, const uint4 &hi, float (&x)[8]) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
}

__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(bf16 *p, float a, float b, float c, float d) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b), u = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&t), *reinterpret_cast<const uint32_t *>(&u));
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

// grid (row groups, vector groups, B).  A CTA takes NP * 256 / (dh/8) vectors (H
// queries, then Hkv keys, then, with caches, Hkv values) of each of NR rows: what
// comes before the first vector, some 300 instructions a warp, is then done once
// for the four rows, and the angles of all of them by all warps at once.  IL:
// interleaved pairs.
template <typename T, int DH, int NP, int NR, bool IL>
__global__ void __launch_bounds__(kRopeThreads, NP == 1 ? 1 : sizeof(T) == 2 ? 4 : 2) qk_norm_rope_kernel(RopeArgs a) {
    pdl_enter();
    constexpr int LPV = DH / 8;                  // lanes per vector
    constexpr int VPP = kRopeThreads / LPV;      // vectors per pass
    __shared__ __align__(16) float cosine[NR][kMaxRot / 2], sine[NR][kMaxRot / 2];
    const int tid = threadIdx.x, sub = tid % LPV;
    const int b = blockIdx.z, i0 = blockIdx.x * NR;
    const int half = a.rot / 2;
    // The lane's pairs are 4 sub .. 4 sub + 3, if there are as many: its pieces
    // begin at elements e_lo and e_hi (rot is a multiple of 16).
    const bool turned = 4 * sub < half;
    const int e_lo = IL || !turned ? 8 * sub : 4 * sub, e_hi = IL || !turned ? 8 * sub + 4 : 4 * sub + half;
    // the angle a thread computes: pair j of row i0 + jr
    constexpr int TPR = NR == 1 ? kRopeThreads : kMaxRot / 2;
    const int j = tid % TPR, jr = NR == 1 ? 0 : tid / TPR;
    // everything the rows' loads and angles depend on, in one round of loads
    const int n_rows = a.n_rows ? a.n_rows[b] : a.R;
    T *const kc = a.kc ? static_cast<T *>(a.kc[b]) : nullptr;
    T *const vc = a.kc ? static_cast<T *>(a.vc[b]) : nullptr;
    const int P = a.kc ? a.prefix_len[b] : 0;
    const bool angle = j < half && jr < NR && i0 + jr < a.R;
    const int pos = angle ? a.pos[(long long)b * a.R + i0 + jr] : 0;
    const float freq = angle ? a.inv_freq[j] : 0.f;
    Piece<T> wraw[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const T *w = static_cast<const T *>(k ? a.kw : a.qw);
        wraw[k][0] = w ? *reinterpret_cast<const Piece<T> *>(w + e_lo) : Piece<T>{};
        wraw[k][1] = w ? *reinterpret_cast<const Piece<T> *>(w + e_hi) : Piece<T>{};
    }
    const int rows = min(NR, min(n_rows, a.R) - i0);
    if (rows <= 0) return;                       // uniform over the CTA
    T *krow, *vrow = nullptr;
    if (a.kc) {
        const bool bad_ptr =
            !kc || !vc ||
            ((reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) & 15u);
        if (bad_ptr || P < 0 || P > a.P_max) {   // the sequence is left untouched
            if (tid == 0) set_status(a.status, bad_ptr ? MEDUSA_DEV_BAD_CACHE : MEDUSA_DEV_BAD_PREFIX);
            return;
        }
        krow = kc + (size_t)(P + i0) * a.Hkv * DH;
        vrow = vc + (size_t)(P + i0) * a.Hkv * DH;
    } else {
        krow = static_cast<T *>(a.k_out) + ((long long)b * a.R + i0) * a.Hkv * DH;
    }
    const int nq = a.H, nqk = a.H + a.Hkv, nv = nqk + (a.kc ? a.Hkv : 0);
    const int v0 = blockIdx.y * (VPP * NP) + tid / LPV;
    // the row's vectors, as if each kind went on from the one before
    const long long row = (long long)b * a.R + i0;
    const T *qin = static_cast<const T *>(a.q) + row * a.q_stride;
    const T *kin = static_cast<const T *>(a.k) + row * a.k_stride - (long long)nq * DH;
    const T *vin = static_cast<const T *>(a.v) + row * a.v_stride - (long long)nqk * DH;
    T *qout = static_cast<T *>(a.q_out) + row * nq * DH;
    T *kout = krow - (long long)nq * DH;
    T *vout = vrow - (long long)nqk * DH;
    Piece<T> raw[NP][2];
    auto load = [&] {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int v = v0 + n * VPP;
            const T *src = (v < nq ? qin : v < nqk ? kin : vin) + v * DH;
            raw[n][0] = v < nv ? ld_piece(src + e_lo) : Piece<T>{};
            raw[n][1] = v < nv ? ld_piece(src + e_hi) : Piece<T>{};
        }
    };
    load();
    if (angle) {
        // fraction of a turn, in [-1/2, 1/2)
        const int64_t frac = (int64_t)((uint64_t)(int64_t)pos * turns_per_position(freq));
        float s, c;
        sincospif((float)frac * 0x1p-63f, &s, &c);
        if (!(fabsf(freq) < INFINITY)) s = c = NAN;
        cosine[jr][j] = c;
        sine[jr][j] = s;
    }
    __syncthreads();
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
        float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (turned) {
            c4 = *reinterpret_cast<const float4 *>(&cosine[r][4 * sub]);
            s4 = *reinterpret_cast<const float4 *>(&sine[r][4 * sub]);
        }
        const float2 c2[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
        const float2 s2[2] = {make_float2(s4.x, s4.y), make_float2(s4.z, s4.w)};
        const float2 m2[2] = {make_float2(-s4.x, -s4.y), make_float2(-s4.z, -s4.w)};
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int v = v0 + n * VPP;
            T *dst = (v < nq ? qout : v < nqk ? kout : vout) + v * DH;
            if (v >= nqk && v < nv) {  // values: copied
                *reinterpret_cast<Piece<T> *>(dst + e_lo) = raw[n][0];
                *reinterpret_cast<Piece<T> *>(dst + e_hi) = raw[n][1];
            }
            if (__all_sync(0xffffffffu, v >= nqk)) continue;
            // u, w: the first and second elements of the four pairs
            float x[8];
            widen(raw[n][0], raw[n][1], x);
            float2 u[2], w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                u[e] = IL ? make_float2(x[4 * e], x[4 * e + 2]) : make_float2(x[2 * e], x[2 * e + 1]);
                w[e] = IL ? make_float2(x[4 * e + 1], x[4 * e + 3]) : make_float2(x[2 * e + 4], x[2 * e + 5]);
            }
            if (a.norm) {  // uniform: the shuffles run in every lane
                float2 q2 = __fmul2_rn(u[0], u[0]);
                q2 = __ffma2_rn(u[1], u[1], q2);
                q2 = __ffma2_rn(w[0], w[0], q2);
                q2 = __ffma2_rn(w[1], w[1], q2);
                float ss = q2.x + q2.y;
#pragma unroll
                for (int o = LPV / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = rsqrtf(fmaf(ss, 1.f / DH, a.eps));  // within 2 units in the last place
                const float2 i2 = make_float2(inv, inv);
                const bool is_q = v < nq;
                if (is_q ? a.qw : a.kw) {
                    float f[8];
                    widen(is_q ? wraw[0][0] : wraw[1][0], is_q ? wraw[0][1] : wraw[1][1], f);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 fu = IL ? make_float2(f[4 * e], f[4 * e + 2]) : make_float2(f[2 * e], f[2 * e + 1]);
                        const float2 fw = IL ? make_float2(f[4 * e + 1], f[4 * e + 3]) : make_float2(f[2 * e + 4], f[2 * e + 5]);
                        u[e] = __fmul2_rn(u[e], __fmul2_rn(i2, fu));
                        w[e] = __fmul2_rn(w[e], __fmul2_rn(i2, fw));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        u[e] = __fmul2_rn(u[e], i2);
                        w[e] = __fmul2_rn(w[e], i2);
                    }
                }
            }
            if (turned) {  // (the other elements stay what they are: inf * 0 is not 0)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 t = __ffma2_rn(w[e], m2[e], __fmul2_rn(u[e], c2[e]));
                    w[e] = __ffma2_rn(u[e], s2[e], __fmul2_rn(w[e], c2[e]));
                    u[e] = t;
                }
            }
            if (v < nqk) {
                if (IL) {
                    store4(dst + e_lo, u[0].x, w[0].x, u[0].y, w[0].y);
                    store4(dst + e_hi, u[1].x, w[1].x, u[1].y, w[1].y);
                } else {
                    store4(dst + e_lo, u[0].x, u[0].y, u[1].x, u[1].y);
                    store4(dst + e_hi, w[0].x, w[0].y, w[1].x, w[1].y);
                }
            }
        }
        if (NR == 1 || r + 1 == rows) break;
        qin += a.q_stride;
        kin += a.k_stride;
        vin += a.v_stride;
        qout += nq * DH;
        kout += a.Hkv * DH;
        vout += a.Hkv * DH;
        load();
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
    // With few rows one row and pass per CTA puts more CTAs to work (65 rows of 96
    // vectors: 2.9 us); with enough of them three passes over four rows share what
    // comes before the first vector (the prompt above: 31.4 us; with two passes
    // 39.1, with two rows 31.8).
    const int passes = (nv + vpp - 1) / vpp;
    const bool many = rows * passes >= 16LL * device_sm_count();
    auto of = [&](auto t, auto il) {
        using T = decltype(t);
        constexpr bool IL = decltype(il)::value;
        return dh == 128 ? (many ? qk_norm_rope_kernel<T, 128, kManyPasses, kManyRows, IL>
                                 : qk_norm_rope_kernel<T, 128, 1, 1, IL>)
                         : (many ? qk_norm_rope_kernel<T, 64, kManyPasses, kManyRows, IL>
                                 : qk_norm_rope_kernel<T, 64, 1, 1, IL>);
    };
    auto kern = dtype == MEDUSA_F32 ? (interleaved ? of(float{}, std::true_type{}) : of(float{}, std::false_type{}))
                                    : (interleaved ? of(bf16{}, std::true_type{}) : of(bf16{}, std::false_type{}));
    const int per_cta = many ? kManyPasses : 1;
    cudaError_t e = launch_pdl(kern, dim3(many ? (R + kManyRows - 1) / kManyRows : R,
                                    (passes + per_cta - 1) / per_cta, B),
                               dim3(kRopeThreads), 0, stream, a);
    note_launch();
    return e;
}

}  // namespace medusa
