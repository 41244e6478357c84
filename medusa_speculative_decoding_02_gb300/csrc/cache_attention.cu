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
#include "tcgen05.cuh"

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
    uint32_t wait_polls;   // poll limit of the tensor-core path's waits
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

// ----------------------------------------------------------- tensor cores ---
//
// bf16 queries.  One CTA (nine warps, two CTAs an SM) per (128-row tile, KV
// head, key range, sequence), its keys in stages of 64:
//   warps 4-7  load: K and V of a stage into shared memory as 128-byte swizzled
//              tiles, a ring of three stages.  A bf16 cache comes by cp.async;
//              a 4-bit row is read into registers three stages ahead, widened
//              to fp16 (exact) and stored.
//   warp 8     one thread issues the products: S = Q K^T, then, when the
//              weights are there, O += P V.
//   warps 0-3  softmax: thread t owns row t of the tile, reads its 64 scores
//              from tensor memory, keeps the row's reference m and sum l in
//              registers (no exchange between threads), and writes the
//              weights P over the scores.
// Tensor memory (256 columns): [0,64) S in fp32, then P in 16 bits; [64,128)
// Q; [128,256) O.  S of stage j+1 overwrites P of stage j, so it is issued
// after O of stage j has arrived; the other CTA of the SM fills that gap.
// The reference m moves only when a stage's maximum exceeds it by 2^8, and O
// is then rescaled in tensor memory; P may thus reach 2^8.
//
// 4-bit caches run in fp16: a value c * s is exact there.  A query row is
// scaled by a power of two to a largest magnitude in [1, 2), which the score
// scale takes back (bf16 elements keep their eight bits down to 2^-14 of the
// largest, and an absolute 2^-25 of it below).  The weights are biased by 2^7:
// they reach 2^15, and what fp16 drops is below 2^-32 of the reference, so
// even 2^20 keys there lose less than 2^-12 of the sum.
//
// Masks are built as 64 bits a row and stage.  Products run over masked keys
// too, with weight 0, so a non-finite V element there would reach every row
// as 0 * inf: in stages that are not wholly visible the softmax warps look for
// such elements, add them to the rows that see them and clear them before the
// product.  Every wait is bounded; on a timeout the CTA sets the status, waits
// (bounded) for its products, frees its tensor memory and publishes nothing.
constexpr int kSub = 64, kStages = 3, kTcThreads = 288;
constexpr float kRescaleLog2 = 8.f;
constexpr float kF16Bias = 7.f;
constexpr uint32_t kDrainPolls = 1u << 16;

template <int DH>
struct CacheSmem {
    static constexpr int NB = DH / 64;
    static constexpr int TILE = NB * kSub * 128;
    static constexpr int STAGE = 2 * TILE;
    static constexpr int BAR = kStages * STAGE;
    // full[3], empty[3], s, p, o, drain; then words
    static constexpr int WORDS = BAR + 10 * 8;
    static constexpr int TOTAL = WORDS + 12 * 4;
    static_assert(2 * (TOTAL + 1024) <= 196 * 1024, "two CTAs per SM in the heads' carveout");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0));
}

// barrier of the 128 softmax threads that also ORs a predicate
__device__ __forceinline__ bool softmax_any(bool p) {
    int r;
    asm volatile(
        "{\n.reg .pred p, q;\n"
        "setp.ne.b32 p, %1, 0;\n"
        "barrier.cta.red.or.pred q, 1, 128, p;\n"
        "selp.b32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((int)p)
        : "memory");
    return r != 0;
}

// Wait for a phase, giving up after `limit` polls or once the CTA has failed.
__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t parity, uint32_t limit,
                                             volatile int *failed) {
    for (uint32_t i = 0; i < limit; ++i) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if (*failed) return false;
    }
    *failed = 1;
    return false;
}

// the lowest n bits (n may be negative or past 64)
__device__ __forceinline__ uint64_t bits_below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// 16-bit pairs with at least one infinity or NaN (all exponent bits set)
template <bool KV4>
__device__ __forceinline__ bool pair_bad(uint32_t w) {
    constexpr uint32_t E = KV4 ? 0x7c00u : 0x7f80u;
    return (w & E) == E || ((w >> 16) & E) == E;
}
template <bool KV4>
__device__ __forceinline__ float half_of_pair(uint32_t w, int hi) {
    const uint16_t v = (uint16_t)(hi ? w >> 16 : w);
    if constexpr (KV4) {
        __half_raw r;
        r.x = v;
        return __half2float(__half(r));
    } else {
        return bf16_to_f(v);
    }
}

template <bool KV4>
__device__ __forceinline__ uint32_t pack_weights(float a, float b) {
    if constexpr (KV4) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// ---- loader, bf16 cache: 128 threads; thread t copies 16-byte column t % CPR
// of key rows t / CPR + RPP u (rows RPP apart share the swizzle phase)
template <int DH>
__device__ __forceinline__ void load_stage_bf16(unsigned char *st, const bf16 *kc, const bf16 *vc,
                                                const KeyRun &run, int k0, int kend, int Hkv, int g,
                                                int t) {
    constexpr int CPR = DH / 8, RPP = 128 / CPR;
    static_assert(RPP % 8 == 0, "passes keep the swizzle phase");
    const int c16 = t % CPR, r0 = t / CPR;
    const uint32_t so0 =
        tc::smem_addr(st) + (c16 >> 3) * kSub * 128 + tc::sw128(r0, c16 & 7);
    const size_t row = (size_t)Hkv * DH;
    const size_t col = (size_t)g * DH + c16 * 8;
#pragma unroll
    for (int u = 0; u < kSub / RPP; ++u) {
        const int x = k0 + r0 + u * RPP;
        const bool ok = x < kend;
        const size_t off = ok ? (size_t)run.slot(x) * row + col : 0;
        cp_async16(so0 + u * RPP * 128, kc + off, ok);
        cp_async16(so0 + u * RPP * 128 + CacheSmem<DH>::TILE, vc + off, ok);
    }
    asm volatile("cp.async.commit_group;\n");
}

// ---- loader, 4-bit cache: a stage of one of K and V is 64 keys x DH/32 groups
// of 32 elements (16 code bytes, two scales); thread t takes groups t + 128 u
template <int DH>
struct Kv4Regs {
    static constexpr int N = DH / 64;
    uint4 code[2][N];
    uint32_t scale[2][N];
};

template <int DH>
__device__ __forceinline__ void load_regs_kv4(Kv4Regs<DH> &r, const uint8_t *kc, const uint8_t *vc,
                                              const KeyRun &run, int k0, int kend, int Hkv, int g,
                                              int t) {
    constexpr int GPK = DH / 32;  // groups per key
    const int rb = kv4_row_bytes(Hkv, DH), cb = kv4_code_bytes(Hkv, DH);
#pragma unroll
    for (int u = 0; u < Kv4Regs<DH>::N; ++u) {
        const int c = t + 128 * u, x = k0 + c / GPK, q = c % GPK;
        if (x < kend) {
            const size_t off = (size_t)run.slot(x) * rb;
            const int co = g * (DH / 2) + q * 16, so = cb + g * (DH / 16) + q * 2;
            r.code[0][u] = ld_stream16(kc + off + co);
            r.code[1][u] = ld_stream16(vc + off + co);
            r.scale[0][u] = __ldg(reinterpret_cast<const unsigned short *>(kc + off + so));
            r.scale[1][u] = __ldg(reinterpret_cast<const unsigned short *>(vc + off + so));
        } else {
            r.code[0][u] = r.code[1][u] = make_uint4(0, 0, 0, 0);
            r.scale[0][u] = r.scale[1][u] = 0;
        }
    }
}

__device__ __forceinline__ uint32_t widen_pair(uint32_t byte, __half2 s) {
    const __half2 v = __hmul2(e2m1x2_half2(byte), s);  // exact
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int DH>
__device__ __forceinline__ void store_regs_kv4(const Kv4Regs<DH> &r, unsigned char *st, int t) {
    constexpr int GPK = DH / 32;
#pragma unroll
    for (int u = 0; u < Kv4Regs<DH>::N; ++u) {
        const int c = t + 128 * u, key = c / GPK, q = c % GPK;
        // groups of the second column block store their 16-byte chunks in the
        // order 2,3,0,1: the eight lanes of a store phase (two keys, four
        // groups) then hit eight different bank groups
        const bool flip = (q >> 1) & 1;
        const uint32_t base = (q >> 1) * kSub * 128;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint4 w = r.code[kv][u];
            const __half2_raw sr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)r.scale[kv][u], __NV_E4M3);
            const __half2 s2 = __half2(sr);
            const __half2 sa = flip ? __high2half2(s2) : __low2half2(s2);
            const __half2 sb = flip ? __low2half2(s2) : __high2half2(s2);
            const uint32_t word[4] = {flip ? w.z : w.x, flip ? w.w : w.y, flip ? w.x : w.z, flip ? w.y : w.w};
            unsigned char *tile = st + kv * CacheSmem<DH>::TILE + base;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 s = i < 2 ? sa : sb;
                const int ch = (q & 1) * 4 + (i ^ (flip ? 2 : 0));
                *reinterpret_cast<uint4 *>(tile + tc::sw128(key, ch)) =
                    make_uint4(widen_pair(word[i], s), widen_pair(word[i] >> 8, s),
                               widen_pair(word[i] >> 16, s), widen_pair(word[i] >> 24, s));
            }
        }
    }
}

template <int DH, bool KV4>
__global__ void __launch_bounds__(kTcThreads, 2) cache_attn_tc_kernel(CacheAttnArgs a) {
    pdl_enter();
    using L = CacheSmem<DH>;
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BAR), *empty = full + kStages;
    uint64_t *bar_s = full + 6, *bar_p = full + 7, *bar_o = full + 8, *bar_drain = full + 9;
    volatile int *failed = reinterpret_cast<volatile int *>(sm + L::WORDS);
    volatile int *o_started = failed + 1;                        // O holds something before stage 0
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(sm + L::WORDS + 8);
    int *warp_depth = reinterpret_cast<int *>(sm + L::WORDS + 16);       // [4]
    uint32_t *bad_keys = reinterpret_cast<uint32_t *>(sm + L::WORDS + 32);  // [2]

    const int g = blockIdx.x / a.row_tiles, rt = blockIdx.x - g * a.row_tiles;
    const int split = blockIdx.y, b = blockIdx.z;
    const int R = a.R, G = a.H / a.Hkv, M = R * G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int P;
    const void *kc, *vc;
    const bool ok = sequence_ok(a, b, P, kc, vc);
    const KeyRun run(ok ? P : 0, R, a.window, a.sinks);
    const int kbeg = split * a.chunk, kend = ok ? min(kbeg + a.chunk, run.len) : 0;

    // row of a softmax thread
    const int m = rt * 128 + tid;
    const bool live = tid < 128 && m < M;
    const int r = live ? m / G : 0, h = g * G + (live ? m - r * G : 0);
    const size_t prow = (((size_t)b * a.H + h) * a.ns + split) * R + r;
    bf16 *dst = static_cast<bf16 *>(a.out) + (((size_t)b * R + r) * a.H + h) * DH;
    auto publish_nothing = [&] {
        if (!live) return;
        if (a.ns == 1) {
#pragma unroll
            for (int c = 0; c < DH; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
        } else {
            a.part_ml[prow] = make_float2(-INFINITY, 0.f);
        }
    };
    if (kbeg >= kend) {  // uniform over the CTA
        publish_nothing();
        return;
    }
    const int nsub = (kend - kbeg + kSub - 1) / kSub;

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(full + i, 128);
            tc::mbar_init(empty + i, 1);
        }
        tc::mbar_init(bar_s, 1);
        tc::mbar_init(bar_p, 128);
        tc::mbar_init(bar_o, 1);
        tc::mbar_init(bar_drain, 1);
        *failed = 0;
        *o_started = 0;
        bad_keys[0] = bad_keys[1] = 0;
        tc::fence_mbarrier_init();
    }
    if (warp == 8) tc::tmem_alloc(tmem_holder, 256);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_holder;
    const uint32_t t_s = tmem, t_q = tmem + 64, t_o = tmem + 128;

    if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ loaders
        const int t = tid - 128;
        auto wait_empty = [&](int j) {  // stage of j free: the product of j - 3 is done
            return j < kStages ||
                   wait_or_fail(empty + j % kStages, (j / kStages - 1) & 1, a.wait_polls, failed);
        };
        if constexpr (KV4) {
            const uint8_t *k8 = static_cast<const uint8_t *>(kc), *v8 = static_cast<const uint8_t *>(vc);
            Kv4Regs<DH> buf[kStages];
#pragma unroll
            for (int u = 0; u < kStages; ++u)
                load_regs_kv4<DH>(buf[u], k8, v8, run, kbeg + u * kSub, kend, a.Hkv, g, t);
            bool go = true;
            for (int j0 = 0; j0 < nsub && go; j0 += kStages) {
#pragma unroll
                for (int u = 0; u < kStages; ++u) {
                    const int j = j0 + u;
                    if (j < nsub && go) {
                        go = wait_empty(j);
                        if (go) {
                            store_regs_kv4<DH>(buf[u], sm + u * L::STAGE, t);
                            tc::fence_proxy_async_smem();
                            tc::mbar_arrive(full + u);
                            load_regs_kv4<DH>(buf[u], k8, v8, run, kbeg + (j + kStages) * kSub, kend,
                                              a.Hkv, g, t);
                        }
                    }
                }
            }
        } else {
            const bf16 *k16 = static_cast<const bf16 *>(kc), *v16 = static_cast<const bf16 *>(vc);
            int j = 0;
            for (; j < nsub; ++j) {
                if (!wait_empty(j)) break;
                load_stage_bf16<DH>(sm + (j % kStages) * L::STAGE, k16, v16, run, kbeg + j * kSub, kend,
                                    a.Hkv, g, t);
                if (j >= 2) {  // two younger groups stay in flight
                    asm volatile("cp.async.wait_group 2;\n");
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(full + (j - 2) % kStages);
                }
            }
            if (j == nsub) {
                if (nsub >= 2) {
                    asm volatile("cp.async.wait_group 1;\n");
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(full + (nsub - 2) % kStages);
                }
                asm volatile("cp.async.wait_group 0;\n");
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(full + (nsub - 1) % kStages);
            }
            asm volatile("cp.async.wait_group 0;\n");
        }
    } else if (warp == 8) {
        // ----------------------------------------------------------- products
        // (Q is in tensor memory before the softmax warps' first arrival on bar_p)
        if (lane == 0) {
            constexpr uint32_t id_s = KV4 ? tc::idesc_f16(128, kSub, 0) : tc::idesc_bf16(128, kSub, 0);
            constexpr uint32_t id_o = KV4 ? tc::idesc_f16(128, DH, 1) : tc::idesc_bf16(128, DH, 1);
            bool go = wait_or_fail(bar_p, 0, a.wait_polls, failed);  // Q written
            for (int j = 0; j < nsub && go; ++j) {
                const unsigned char *st = sm + (j % kStages) * L::STAGE;
                go = wait_or_fail(full + j % kStages, (j / kStages) & 1, a.wait_polls, failed);
                // S overwrites P of j - 1, which the product of j - 1 reads
                if (go && j > 0) go = wait_or_fail(bar_o, (j - 1) & 1, a.wait_polls, failed);
                if (!go) break;
                tc::fence_after_sync();
                const uint64_t kd = tc::sdesc_sw128(tc::smem_addr(st), 16, 1024);
#pragma unroll
                for (int ks = 0; ks < DH / 16; ++ks)
                    tc::mma_bf16_ts(t_s, t_q + ks * 8, kd + (((ks >> 2) * kSub * 128 + (ks & 3) * 32) >> 4),
                                    id_s, ks > 0);
                tc::mma_commit(bar_s);
                go = wait_or_fail(bar_p, (j + 1) & 1, a.wait_polls, failed);
                if (!go) break;
                tc::fence_after_sync();
                const uint64_t vd = tc::sdesc_sw128(tc::smem_addr(st + L::TILE), kSub * 128, 1024);
                const uint32_t acc0 = j > 0 || *o_started;
#pragma unroll
                for (int ks = 0; ks < kSub / 16; ++ks)
                    tc::mma_bf16_ts(t_o, t_s + ks * 8, vd + ((ks * 16 * 128) >> 4), id_o,
                                    ks > 0 ? 1u : acc0);
                tc::mma_commit(empty + j % kStages);
                tc::mma_commit(bar_o);
            }
            // every product issued above is done before the tensor memory is freed
            tc::mma_commit(bar_drain);
            if (!tc::mbar_wait_bounded(bar_drain, 0, kDrainPolls)) {
                *failed = 1;
                if (a.status) atomicExch(a.status, MEDUSA_DEV_DRAIN_TIMEOUT);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const bool rows_live = rt * 128 + warp * 32 < M;  // warp-uniform
        float row_scale = a.scale_log2;
        {
            // Q row into tensor memory, half a row (64 elements) at a time
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const bf16 *>(a.q) + (((size_t)b * R + r) * a.H + h) * DH);
            float factor = 1.f;
            if (KV4) {
                float amax = 0.f;
                if (live) {
#pragma unroll
                    for (int i = 0; i < DH / 8; ++i) {
                        float f[8];
                        Vec16<bf16>::widen(src[i], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
                    }
                }
                if (amax > 0.f && amax < INFINITY) {
                    // 2^floor(log2 amax), from the exponent bits (subnormals: 2^-126)
                    const uint32_t eb = max(1u, __float_as_uint(amax) >> 23);
                    factor = eb < 254u ? __uint_as_float((254u - eb) << 23) : 0x1p-127f;
                    row_scale *= __uint_as_float(eb << 23);
                }
            }
#pragma unroll
            for (int half = 0; half < DH / 64; ++half) {
                uint32_t qr[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (live) v = src[half * 8 + i];
                    if (KV4) {
                        float f[8];
                        Vec16<bf16>::widen(v, f);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            qr[4 * i + e] = pack_weights<true>(f[2 * e] * factor, f[2 * e + 1] * factor);
                    } else {
                        qr[4 * i] = v.x;
                        qr[4 * i + 1] = v.y;
                        qr[4 * i + 2] = v.z;
                        qr[4 * i + 3] = v.w;
                    }
                }
                tc::tmem_st32u(t_q + lane_base + half * 32, qr);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bar_p);
        }
        // ---- what this row sees, in numbered keys
        const int my_depth = a.window ? row_depth(a, b, r) : 0;
        int dmax = 0;
        uint64_t am[4] = {0, 0, 0, 0};
        const int x_tree = run.n_sink + P - run.lo;  // number of tree slot 0
        if (live && kend > x_tree) {
            const int W = (R + 63) / 64;
            const uint64_t *mr = a.anc_mask + ((size_t)b * R + r) * W;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                if (w < W) am[w] = mr[w];
        }
        if (a.window) {
            dmax = __reduce_max_sync(0xffffffffu, live ? my_depth : 0);
            if (lane == 0) warp_depth[warp] = dmax;
            softmax_any(false);
            dmax = max(max(warp_depth[0], warp_depth[1]), max(warp_depth[2], warp_depth[3]));
            if (dmax >= a.window && live && kend > x_tree) {
                // ancestors out of the window (and not among the sinks)
                for (int t = 0; t < R; ++t) {
                    const int td = row_depth(a, b, t);
                    if (!(P + td < a.sinks || my_depth - td < a.window)) {
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            if (w == (t >> 6)) am[w] &= ~(1ull << (t & 63));
                    }
                }
            }
        }
        // numbers [x_win, x_tree) are the row's window, [n_sink, x_sink) slots
        // under `sinks` that the first row's window holds as well
        const int x_win = a.window ? run.n_sink + max(0, P + my_depth - a.window + 1 - run.lo) : 0;
        const int x_sink = min(run.n_sink + max(0, a.sinks - run.lo), x_tree);
        // keys that every row of the tile sees: numbers below n_sink, and
        // [x_all, x_tree)
        const int x_all = a.window ? run.n_sink + max(0, P + dmax - a.window + 1 - run.lo) : 0;

        float m_run = -INFINITY, l_run = 0.f;
        bool dead = false;  // warp-uniform; a dead warp keeps up with the barriers
        for (int j = 0; j < nsub; ++j) {
            const int k0 = kbeg + j * kSub;
            const bool masked = !(k0 + kSub <= min(kend, x_tree) && (k0 >= x_all || k0 + kSub <= run.n_sink));
            if (!dead)
                dead = !__all_sync(0xffffffffu, wait_or_fail(bar_s, j & 1, a.wait_polls, failed));
            tc::fence_after_sync();
            bool grew = false;
            float alpha = 1.f;
            if (!dead && rows_live) {
                float x[kSub];
                {
                    float (&lo)[32] = *reinterpret_cast<float (*)[32]>(x);
                    float (&hi)[32] = *reinterpret_cast<float (*)[32]>(x + 32);
                    tc::tmem_ld32(t_s + lane_base, lo);
                    tc::tmem_ld32(t_s + lane_base + 32, hi);
                }
                if (masked) {
                    uint64_t vis = (bits_below(x_tree - k0) & ~bits_below(x_win - k0)) |
                                   (bits_below(x_sink - k0) & ~bits_below(run.n_sink - k0)) |
                                   bits_below(run.n_sink - k0);
                    const int t0 = k0 - x_tree;  // tree slot of the stage's first key
                    if (t0 > -kSub) {
                        if (t0 < 0) {
                            vis |= am[0] << -t0;
                        } else {
                            const int w = t0 >> 6, s = t0 & 63;
                            const uint64_t lo = w == 0 ? am[0] : w == 1 ? am[1] : w == 2 ? am[2] : w == 3 ? am[3] : 0ull;
                            const uint64_t hi = w == 0 ? am[1] : w == 1 ? am[2] : w == 2 ? am[3] : 0ull;
                            vis |= (lo >> s) | (s ? hi << (64 - s) : 0ull);
                        }
                    }
                    vis &= bits_below(kend - k0);
                    if (!live) vis = 0;
                    const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        x[e] = (v0 >> e) & 1u ? x[e] : -INFINITY;
                        x[e + 32] = (v1 >> e) & 1u ? x[e + 32] : -INFINITY;
                    }
                }
                float ma = max3f(x[0], x[1], x[2]), mb = max3f(x[3], x[4], x[5]);
#pragma unroll
                for (int e = 6; e + 3 < kSub; e += 4) {
                    ma = max3f(ma, x[e], x[e + 1]);
                    mb = max3f(mb, x[e + 2], x[e + 3]);
                }
                ma = max3f(ma, x[kSub - 2], x[kSub - 1]);
                const float cm = fmaxf(ma, mb) * row_scale;
                if (cm > m_run + kRescaleLog2) {  // m_run = -inf: the first visible key
                    alpha = exp2f(m_run - cm);
                    m_run = cm;
                    l_run *= alpha;
                    grew = true;
                }
                const float mu = (m_run == -INFINITY ? 0.f : m_run) - (KV4 ? kF16Bias : 0.f);
                // the fused x * scale - m keeps bits that m = round(max * scale)
                // lost: harmless below 2^16 (2^-8 in the exponent), but past 2^24
                // the largest weight would leave 1, so there the scores are
                // rounded first
                float sc = row_scale;
                if (__any_sync(0xffffffffu, fabsf(mu) > 65536.f)) {
#pragma unroll
                    for (int e = 0; e < kSub; ++e) x[e] *= row_scale;
                    sc = 1.f;
                }
                const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-mu, -mu);
                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 t = __ffma2_rn(make_float2(x[q * 32 + e], x[q * 32 + e + 1]), sc2, nm2);
                        const float p0 = ex2_approx(t.x), p1 = ex2_approx(t.y);
                        // rounded for the product only; the sum adds the fp32 weights
                        pk[e / 2] = pack_weights<KV4>(p0, p1);
                        ls[(e / 2) & 1] = __fadd2_rn(ls[(e / 2) & 1], make_float2(p0, p1));
                    }
                    tc::tmem_st16(t_s + lane_base + q * 16, pk);
                }
                l_run += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                if (__any_sync(0xffffffffu, grew && (j > 0 || *o_started))) {
                    // O of the stages before is complete: S of j came after it
#pragma unroll 1
                    for (int c = 0; c < DH; c += 32) {
                        float ov[32];
                        tc::tmem_ld32(t_o + lane_base + c, ov);
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] *= alpha;
                        tc::tmem_st32(t_o + lane_base + c, ov);
                    }
                }
                tc::tmem_wait_st();
            }
            if (masked) {
                // ---- infinities and NaNs in V of a stage that some row does not see
                unsigned char *vt = sm + (j % kStages) * L::STAGE + L::TILE;
                if (!dead)
                    dead = !__all_sync(0xffffffffu, wait_or_fail(full + j % kStages, (j / kStages) & 1,
                                                                 a.wait_polls, failed));
                // thread t scans half a key row: 128-byte rows t, t + 128, ... of the tile
                bool bad = false;
                if (!dead)
                    for (int row = tid; row < L::NB * kSub; row += 128)
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(
                                vt + row * 128 + (c ^ (row & 7)) * 16);
                            if (pair_bad<KV4>(w.x) || pair_bad<KV4>(w.y) || pair_bad<KV4>(w.z) ||
                                pair_bad<KV4>(w.w)) {
                                bad = true;
                                atomicOr(bad_keys + ((row & 63) >> 5), 1u << (row & 31));
                            }
                        }
                if (softmax_any(bad)) {
                    if (!dead && j == 0) {  // O has no product yet: it starts from zeros
                        float z[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) z[e] = 0.f;
#pragma unroll 1
                        for (int c = 0; c < DH; c += 32) tc::tmem_st32(t_o + lane_base + c, z);
                        *o_started = 1;
                    }
                    if (!dead && rows_live) {
#pragma unroll 1
                        for (int key = 0; key < kSub; ++key) {
                            if (!((bad_keys[key >> 5] >> (key & 31)) & 1u)) continue;
                            const uint32_t pw = __float_as_uint(tc::tmem_ld1(t_s + lane_base + key / 2));
                            const float p = half_of_pair<KV4>(pw, key & 1);
#pragma unroll 1
                            for (int c = 0; c < DH; ++c) {
                                const uint32_t w = *reinterpret_cast<const uint16_t *>(
                                    vt + (c >> 6) * kSub * 128 + tc::sw128(key, (c & 63) >> 3) + (c & 7) * 2);
                                if (!pair_bad<KV4>(w)) continue;  // uniform: one address
                                float o = tc::tmem_ld1(t_o + lane_base + c);
                                if (p != 0.f) o += p * half_of_pair<KV4>(w, 0);
                                tc::tmem_st1(t_o + lane_base + c, o);
                                tc::tmem_wait_st();
                            }
                        }
                    }
                    softmax_any(false);  // every row has read V
                    if (!dead)
                        for (int row = tid; row < L::NB * kSub; row += 128)
#pragma unroll 1
                            for (int c = 0; c < 64; ++c) {
                                uint16_t *e = reinterpret_cast<uint16_t *>(vt + row * 128) + c;
                                if (pair_bad<KV4>(*e)) *e = 0;
                            }
                    if (tid == 0) bad_keys[0] = bad_keys[1] = 0;
                    tc::fence_proxy_async_smem();
                }
            }
            if (!dead) {
                tc::fence_before_sync();
                tc::mbar_arrive(bar_p);
            }
        }
        // ---- the last product, then the row
        if (!dead)
            dead = !__all_sync(0xffffffffu, wait_or_fail(bar_o, (nsub - 1) & 1, a.wait_polls, failed));
        tc::fence_after_sync();
        if (dead) {
            publish_nothing();
        } else if (rows_live) {
            const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
#pragma unroll 1
            for (int c = 0; c < DH; c += 32) {
                float ov[32];
                tc::tmem_ld32(t_o + lane_base + c, ov);
                if (!live) continue;
                if (a.ns == 1) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = pack_weights<false>(ov[e + 2 * i] * inv, ov[e + 2 * i + 1] * inv);
                        *reinterpret_cast<uint4 *>(dst + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    float *po = a.part_o + prow * DH + c;
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4 *>(po + e) = make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                }
            }
            if (live && a.ns > 1)
                a.part_ml[prow] = make_float2(m_run - (KV4 ? kF16Bias : 0.f), l_run);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && *failed) set_status(a.status, MEDUSA_DEV_TIMEOUT);
    if (warp == 8) tc::tmem_dealloc(tmem, 256);
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

// Key ranges: the count that makes (waves of CTAs) x (stages per CTA + the
// fixed cost of a CTA, in stages) smallest, joining included.
CachePlan cache_plan(medusa_dtype dtype, int B, int R, int H, int Hkv, int P_max, int window,
                     int sinks) {
    CachePlan p;
    // a window no row's oldest key falls out of is none
    p.window = window >= P_max + R ? 0 : window;
    p.sinks = p.window ? std::min(sinks, P_max + R) : 0;
    const int keys =
        p.window ? std::min(P_max, p.sinks + p.window - 1) + R : P_max + R;  // longest KeyRun
    const int M = R * (H / Hkv);
    const bool simt = dtype == MEDUSA_F32;
    const int rows = simt ? kRows : 128, sub = simt ? kKeys : kSub;
    const int slots = (simt ? 4 : 2) * device_sm_count();
    p.row_tiles = (M + rows - 1) / rows;
    const int subs = (keys + sub - 1) / sub;
    const long long ctas = (long long)B * Hkv * p.row_tiles;
    double best = 0;
    p.ns = 1;
    int per_best = subs;
    for (int ns = 1; ns <= std::min(subs, 512); ++ns) {
        const int per = (subs + ns - 1) / ns;
        if ((subs + per - 1) / per != ns) continue;  // the same split as a smaller ns
        const double waves = (double)((ctas * ns + slots - 1) / slots);
        const double cost = waves * (per + 3) + (ns > 1 ? 3.0 + 0.05 * ns : 0.0);
        if (ns == 1 || cost < best) {
            best = cost;
            p.ns = ns;
            per_best = per;
        }
    }
    p.chunk = per_best * sub;
    return p;
}

}  // namespace

size_t cache_attention_workspace_bytes(medusa_dtype dtype, bool, int B, int R, int H, int Hkv, int dh,
                                       int P_max, int window, int sinks) {
    const CachePlan p = cache_plan(dtype, B, R, H, Hkv, P_max, window, sinks);
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
    const CachePlan p = cache_plan(dtype, B, R, H, Hkv, P_max, window, sinks);
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
    a.wait_polls = wait_budget();
    const bool f32 = dtype == MEDUSA_F32;
    const dim3 grid(Hkv * p.row_tiles, p.ns, B);
    cudaError_t e;
    if (f32) {
        auto kern = kv4 ? (dh == 128 ? cache_attn_simt_kernel<float, true, 128>
                                     : cache_attn_simt_kernel<float, true, 64>)
                        : (dh == 128 ? cache_attn_simt_kernel<float, false, 128>
                                     : cache_attn_simt_kernel<float, false, 64>);
        e = launch_pdl(kern, grid, dim3(kSimtThreads), 0, stream, a);
    } else {
        auto kern = kv4 ? (dh == 128 ? cache_attn_tc_kernel<128, true> : cache_attn_tc_kernel<64, true>)
                        : (dh == 128 ? cache_attn_tc_kernel<128, false> : cache_attn_tc_kernel<64, false>);
        const int smem = dh == 128 ? CacheSmem<128>::TOTAL : CacheSmem<64>::TOTAL;
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)))
            return e;
        e = launch_pdl(kern, grid, dim3(kTcThreads), (size_t)smem, stream, a);
    }
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
