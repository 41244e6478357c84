// cache_attention.cu -- tree attention with a sliding window and sinks, with
// grouped KV heads, over a bf16/fp32 cache or a cache held in 4 bits.
//
// Positions: prefix slot j of sequence b is position j, tree slot P + t is
// position P + depth[t].  Row i (position P + depth[i]) sees
//     prefix slot j   iff  j < sinks  or  P + depth[i] - j < window
//     tree slot P+t   iff  bit t of anc_mask[b,i] is set and
//                          (P + depth[t] < sinks or depth[i] - depth[t] < window)
// and with window = 0 the whole prefix and every set bit.  Query head h reads
// KV head h / (H / Hkv).  A row that sees nothing gets zeros.
//
// With a window a sequence's keys are two runs of slots: the sinks that lie
// before the window of the first row (position P), and everything from
// P - window + 1 on.  They are numbered 0 .. len-1 without a gap (KeyRun), so
// the work does not grow with the prefix.  The numbered keys are split into
// ranges of `chunk` keys; one CTA computes an unnormalised partial (O, m, l)
// of a tile of rows over one range, and cache_attn_combine_kernel joins the
// ranges.  With one range the CTA writes the output itself.
//
// The rows of a tile are the R * G (G = H / Hkv) rows that share a KV head,
// row r * G + g being tree row r and query head hk * G + g.
#include <algorithm>

#include "kv4.cuh"
#include "launch.h"

namespace medusa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct CacheAttnArgs {
    const void *q;
    const void *const *kc;
    const void *const *vc;
    const int32_t *prefix_len;
    const uint64_t *anc_mask;
    const int32_t *depth;  // null without a window
    int B, R, H, Hkv, P_max;
    int window, sinks;
    int chunk, ns, row_tiles;
    float scale_log2;
    float *part_o;         // [B, H, ns, R, dh]
    float2 *part_ml;       // [B, H, ns, R] (m in log2 units, l)
    void *out;
    int *status;
};

// A sequence's visible slots, numbered without a gap.
struct KeyRun {
    int n_sink, lo, len;
    __device__ __forceinline__ KeyRun(int P, int R, int window, int sinks) {
        lo = window ? max(0, P - window + 1) : 0;
        n_sink = min(sinks, lo);
        len = n_sink + (P + R - lo);
    }
    __device__ __forceinline__ int slot(int x) const { return x < n_sink ? x : x - n_sink + lo; }
};

// depth of tree row t, clamped into 0..R-1 (out of range: BAD_DEPTH)
__device__ __forceinline__ int row_depth(const CacheAttnArgs &a, int b, int t) {
    if (!a.depth) return 0;
    const int d = a.depth[(size_t)b * a.R + t];
    if (d < 0 || d >= a.R) {
        set_status(a.status, MEDUSA_DEV_BAD_DEPTH);
        return d < 0 ? 0 : a.R - 1;
    }
    return d;
}

// Sequence b's prefix and caches, checked; false (and the status set) when
// the sequence cannot run.
__device__ __forceinline__ bool sequence_ok(const CacheAttnArgs &a, int b, int &P, const void *&kc,
                                            const void *&vc) {
    P = a.prefix_len[b];
    kc = a.kc[b];
    vc = a.vc[b];
    if (!kc || !vc || ((reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) & 15u)) {
        set_status(a.status, MEDUSA_DEV_BAD_CACHE);
        return false;
    }
    if (P < 0 || P > a.P_max) {
        set_status(a.status, MEDUSA_DEV_BAD_PREFIX);
        return false;
    }
    return true;
}

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(bf16 *p, float v) { *p = __float2bfloat16_rn(v); }

// ------------------------------------------------------------- CUDA cores ---
//
// 128 threads, 16 rows, 32 keys at a time: K and V of the tile are widened to
// fp32 in shared memory, thread (row tid/8, u = tid%8) scores keys u, u+8,
// u+16, u+24 and owns output columns 4u + 32c .. +3.  The running maximum and sum of a row live
// in its eight threads.
constexpr int kRows = 16, kKeys = 32, kSimtThreads = 128;

// eight elements of head g of cache row `slot` from element e0 on
template <typename T, bool KV4, int DH>
__device__ __forceinline__ void cache_load8(const void *cache, int slot, int Hkv, int g, int e0,
                                            float (&x)[8]) {
    if constexpr (KV4) {
        const uint8_t *row = static_cast<const uint8_t *>(cache) + (size_t)slot * kv4_row_bytes(Hkv, DH);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(row + (g * DH + e0) / 2);
        const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(
            row[kv4_code_bytes(Hkv, DH) + (g * DH + e0) / 16], __NV_E4M3)));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2 f = __half22float2(e2m1x2_half2(w >> (8 * u)));
            x[2 * u] = f.x * s;
            x[2 * u + 1] = f.y * s;
        }
    } else {
        const T *p = static_cast<const T *>(cache) + ((size_t)slot * Hkv + g) * DH + e0;
        constexpr int N = Vec16<T>::N;
#pragma unroll
        for (int u = 0; u < 8 / N; ++u) {
            float f[N];
            Vec16<T>::widen(*reinterpret_cast<const uint4 *>(p + u * N), f);
#pragma unroll
            for (int e = 0; e < N; ++e) x[u * N + e] = f[e];
        }
    }
}

template <typename T, bool KV4, int DH>
__global__ void __launch_bounds__(kSimtThreads) cache_attn_simt_kernel(CacheAttnArgs a) {
    pdl_enter();
    constexpr int LD = DH + 4;
    __shared__ float qs[kRows][LD], ks[kKeys][LD], vs[kKeys][LD];
    __shared__ float ps[kRows][kKeys];
    const int g = blockIdx.x / a.row_tiles, rt = blockIdx.x - g * a.row_tiles;  // KV head, tile
    const int split = blockIdx.y, b = blockIdx.z;
    const int R = a.R, G = a.H / a.Hkv, M = R * G;
    const int tid = threadIdx.x, lr = tid >> 3, u = tid & 7;
    const int m = rt * kRows + lr;  // row of the KV head
    const bool live = m < M;
    const int r = live ? m / G : 0, h = g * G + (live ? m - r * G : 0);
    const size_t prow = (((size_t)b * a.H + h) * a.ns + split) * R + r;
    T *dst = static_cast<T *>(a.out) + (((size_t)b * R + r) * a.H + h) * DH;
    int P;
    const void *kc, *vc;
    const bool ok = sequence_ok(a, b, P, kc, vc);
    const KeyRun run(ok ? P : 0, R, a.window, a.sinks);
    const int kbeg = split * a.chunk, kend = ok ? min(kbeg + a.chunk, run.len) : 0;
    if (kbeg >= kend) {  // uniform over the CTA
        if (!live) return;
        if (a.ns == 1)
            for (int c = u; c < DH; c += 8) store_out(dst + c, 0.f);
        else if (u == 0)
            a.part_ml[prow] = make_float2(-INFINITY, 0.f);
        return;
    }
    const uint64_t *mask = a.anc_mask + ((size_t)b * R + r) * ((R + 63) / 64);
    const int my_depth = row_depth(a, b, r);
    for (int e = tid; e < kRows * DH; e += kSimtThreads) {
        const int row = e / DH, c = e - row * DH, mm = rt * kRows + row;
        float x = 0.f;
        if (mm < M) {
            const int rr = mm / G, hh = g * G + mm - rr * G;
            x = Vec16<T>::load1(static_cast<const T *>(a.q) + (((size_t)b * R + rr) * a.H + hh) * DH + c);
        }
        qs[row][c] = x;
    }
    float acc[DH / 8];
#pragma unroll
    for (int c = 0; c < DH / 8; ++c) acc[c] = 0.f;
    float m_run = -INFINITY, l_run = 0.f;
    for (int k0 = kbeg; k0 < kend; k0 += kKeys) {
        __syncthreads();
        for (int e = tid; e < kKeys * DH / 8; e += kSimtThreads) {
            const int kk = e / (DH / 8), e0 = (e - kk * (DH / 8)) * 8;
            float x[8] = {}, y[8] = {};
            if (k0 + kk < kend) {
                const int slot = run.slot(k0 + kk);
                cache_load8<T, KV4, DH>(kc, slot, a.Hkv, g, e0, x);
                cache_load8<T, KV4, DH>(vc, slot, a.Hkv, g, e0, y);
            }
#pragma unroll
            for (int c = 0; c < 8; c += 4) {
                *reinterpret_cast<float4 *>(&ks[kk][e0 + c]) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
                *reinterpret_cast<float4 *>(&vs[kk][e0 + c]) = make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]);
            }
        }
        __syncthreads();
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int c = 0; c < DH; c += 4) {
            const float4 qv = *reinterpret_cast<const float4 *>(&qs[lr][c]);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float4 kv = *reinterpret_cast<const float4 *>(&ks[u + 8 * n][c]);
                s[n] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[n]))));
            }
        }
        float cm = -INFINITY;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int x = k0 + u + 8 * n;
            bool vis = live && x < kend;
            if (vis) {
                const int slot = run.slot(x);
                if (slot < P) {
                    vis = !a.window || slot < a.sinks || P + my_depth - slot < a.window;
                } else {
                    const int t = slot - P;
                    vis = (mask[t >> 6] >> (t & 63)) & 1u;
                    if (vis && a.window) {
                        const int td = row_depth(a, b, t);
                        vis = P + td < a.sinks || my_depth - td < a.window;
                    }
                }
            }
            s[n] = vis ? s[n] * a.scale_log2 : -INFINITY;
            cm = fmaxf(cm, s[n]);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, o));
        const float m_new = fmaxf(m_run, cm);
        const float mu = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = m_run == m_new ? 1.f : exp2f(m_run - mu);
        m_run = m_new;
        l_run *= alpha;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float p = exp2f(s[n] - mu);
            l_run += p;
            ps[lr][u + 8 * n] = p;
        }
        __syncwarp();  // a row's eight threads are in one warp
#pragma unroll
        for (int c = 0; c < DH / 8; ++c) acc[c] *= alpha;
#pragma unroll 4
        for (int kk = 0; kk < kKeys; ++kk) {
            const float p = ps[lr][kk];
            if (p != 0.f) {  // a key the row does not see adds nothing, whatever V holds
#pragma unroll
                for (int c = 0; c < DH / 32; ++c) {
                    const float4 v = *reinterpret_cast<const float4 *>(&vs[kk][c * 32 + u * 4]);
                    acc[4 * c] = fmaf(p, v.x, acc[4 * c]);
                    acc[4 * c + 1] = fmaf(p, v.y, acc[4 * c + 1]);
                    acc[4 * c + 2] = fmaf(p, v.z, acc[4 * c + 2]);
                    acc[4 * c + 3] = fmaf(p, v.w, acc[4 * c + 3]);
                }
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) l_run += __shfl_xor_sync(0xffffffffu, l_run, o);
    if (!live) return;
    if (a.ns == 1) {
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
#pragma unroll
        for (int c = 0; c < DH / 8; ++c) store_out(dst + (c / 4) * 32 + u * 4 + c % 4, acc[c] * inv);
    } else {
        float *po = a.part_o + prow * DH;
#pragma unroll
        for (int c = 0; c < DH / 32; ++c)
            *reinterpret_cast<float4 *>(po + c * 32 + u * 4) =
                make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
        if (u == 0) a.part_ml[prow] = make_float2(m_run, l_run);
    }
}

// ---------------------------------------------------------------- combine ---

// One warp per (sequence, head, row): out = sum_s 2^(m_s - M) O_s / sum_s
// 2^(m_s - M) l_s over the key ranges.  An empty range (l = 0) has no O row.
template <typename T, int DH>
__global__ void __launch_bounds__(256)
cache_attn_combine_kernel(const float *__restrict__ part_o, const float2 *__restrict__ part_ml,
                          int B, int R, int H, int NS, T *__restrict__ out) {
    pdl_enter();
    constexpr int PER = DH / 32;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= (long long)B * H * R) return;
    const int r = (int)(item % R);
    const long long bh = item / R;
    const float2 *ml = part_ml + bh * NS * R + r;
    float M = -INFINITY;
    for (int s = lane; s < NS; s += 32) {
        const float2 x = ml[(size_t)s * R];
        if (x.y != 0.f) M = fmaxf(M, x.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) acc[p] = 0.f;
#pragma unroll 4
    for (int s = 0; s < NS; ++s) {
        const float2 x = ml[(size_t)s * R];
        if (x.y == 0.f) continue;
        const float w = exp2f(x.x - mu);
        L = fmaf(w, x.y, L);
        const float *o = part_o + ((bh * NS + s) * R + r) * DH + lane * PER;
#pragma unroll
        for (int p = 0; p < PER; ++p) acc[p] = fmaf(w, o[p], acc[p]);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    T *dst = out + (((bh / H) * R + r) * H + bh % H) * DH + lane * PER;
#pragma unroll
    for (int p = 0; p < PER; ++p) store_out(dst + p, acc[p] * inv);
}

// ------------------------------------------------------------------- host ---

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct CachePlan {
    int row_tiles, ns, chunk, window, sinks;
};

CachePlan cache_plan(int B, int R, int H, int Hkv, int P_max, int window, int sinks) {
    CachePlan p;
    // a window no row's oldest key falls out of is none
    p.window = window >= P_max + R ? 0 : window;
    p.sinks = p.window ? std::min(sinks, P_max + R) : 0;
    const int keys =
        p.window ? std::min(P_max, p.sinks + p.window - 1) + R : P_max + R;  // longest KeyRun
    const int M = R * (H / Hkv);
    p.row_tiles = (M + kRows - 1) / kRows;
    const int subs = (keys + kKeys - 1) / kKeys;
    const long long ctas = (long long)B * Hkv * p.row_tiles;
    const int want = (int)std::max<long long>(1, 4LL * device_sm_count() / ctas);
    const int per = std::max(2, (subs + want - 1) / want);
    p.ns = (subs + per - 1) / per;
    p.chunk = per * kKeys;
    return p;
}

}  // namespace

size_t cache_attention_workspace_bytes(medusa_dtype, bool, int B, int R, int H, int Hkv, int dh,
                                       int P_max, int window, int sinks) {
    const CachePlan p = cache_plan(B, R, H, Hkv, P_max, window, sinks);
    if (p.ns == 1) return MEDUSA_WS_HEADER;
    const size_t rows = (size_t)B * H * p.ns * R;
    return MEDUSA_WS_HEADER + align256(rows * dh * sizeof(float)) + align256(rows * sizeof(float2));
}

cudaError_t launch_cache_attention(medusa_dtype dtype, bool kv4, const void *q,
                                   const void *const *k_cache, const void *const *v_cache,
                                   const int32_t *prefix_len, int P_max, const uint64_t *anc_mask,
                                   const int32_t *depth, int window, int sinks, int B, int R, int H,
                                   int Hkv, int dh, float scale, void *out, void *ws,
                                   cudaStream_t stream) {
    const CachePlan p = cache_plan(B, R, H, Hkv, P_max, window, sinks);
    CacheAttnArgs a;
    a.q = q;
    a.kc = k_cache;
    a.vc = v_cache;
    a.prefix_len = prefix_len;
    a.anc_mask = anc_mask;
    a.depth = p.window ? depth : nullptr;
    a.B = B;
    a.R = R;
    a.H = H;
    a.Hkv = Hkv;
    a.P_max = P_max;
    a.window = p.window;
    a.sinks = p.sinks;
    a.chunk = p.chunk;
    a.ns = p.ns;
    a.row_tiles = p.row_tiles;
    a.scale_log2 = scale * kLog2e;
    const size_t rows = (size_t)B * H * p.ns * R;
    char *w = static_cast<char *>(ws) + MEDUSA_WS_HEADER;
    a.part_o = reinterpret_cast<float *>(w);
    a.part_ml = reinterpret_cast<float2 *>(w + align256(rows * dh * sizeof(float)));
    a.out = out;
    a.status = static_cast<int *>(ws);
    const bool f32 = dtype == MEDUSA_F32;
    auto kern =
        f32 ? (kv4 ? (dh == 128 ? cache_attn_simt_kernel<float, true, 128> : cache_attn_simt_kernel<float, true, 64>)
                   : (dh == 128 ? cache_attn_simt_kernel<float, false, 128> : cache_attn_simt_kernel<float, false, 64>))
            : (kv4 ? (dh == 128 ? cache_attn_simt_kernel<bf16, true, 128> : cache_attn_simt_kernel<bf16, true, 64>)
                   : (dh == 128 ? cache_attn_simt_kernel<bf16, false, 128> : cache_attn_simt_kernel<bf16, false, 64>));
    cudaError_t e = launch_pdl(kern, dim3(Hkv * p.row_tiles, p.ns, B), dim3(kSimtThreads), 0, stream, a);
    note_launch();
    if (e || p.ns == 1) return e;
    const unsigned blocks = (unsigned)(((long long)B * H * R + 7) / 8);
    const float *po = a.part_o;
    const float2 *pm = a.part_ml;
    if (f32)
        e = launch_pdl(dh == 128 ? cache_attn_combine_kernel<float, 128> : cache_attn_combine_kernel<float, 64>,
                       dim3(blocks), dim3(256), 0, stream, po, pm, B, R, H, p.ns, static_cast<float *>(out));
    else
        e = launch_pdl(dh == 128 ? cache_attn_combine_kernel<bf16, 128> : cache_attn_combine_kernel<bf16, 64>,
                       dim3(blocks), dim3(256), 0, stream, po, pm, B, R, H, p.ns, static_cast<bf16 *>(out));
    note_launch();
    return e;
}

}  // namespace medusa
