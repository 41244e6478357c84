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
// ranges (find_item); one CTA computes an unnormalised partial (O, m, l) of a
// tile of rows over one range, and cache_attn_combine_kernel joins the ranges.
// With one range the CTA writes the output itself.
//
// Three kernels: fp32 on the CUDA cores and bf16 on the tensor cores here, and
// bf16 with at most 16 rows a KV head in cache_attention_few.cu.
//
// The rows of a tile are the R * G (G = H / Hkv) rows that share a KV head,
// row r * G + g being tree row r and query head hk * G + g.
#include <algorithm>

#include "cache_attention.cuh"
#include "tcgen05.cuh"

namespace medusa {

namespace {

// ------------------------------------------------------------- CUDA cores ---
//
// fp32.  128 threads, 16 rows, 32 keys at a time: K and V of the tile are widened to
// fp32 in shared memory, thread (row tid/8, u = tid%8) scores keys u, u+8,
// u+16, u+24 and owns output columns 4u + 32c .. +3.  The running maximum and sum of a row live
// in its eight threads.
constexpr int kRows = 16, kKeys = 32, kSimtThreads = 128;

// eight elements of head g of cache row `slot` from element e0 on
template <bool KV4, int DH>
__device__ __forceinline__ void cache_load8(const void *cache, int slot, int Hkv, int g, int e0,
                                            float (&x)[8]) {
    if constexpr (KV4) {
        const uint8_t *row = static_cast<const uint8_t *>(cache) + (size_t)slot * kv4_row_bytes(Hkv, DH);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(row + (g * DH + e0) / 2);
        kv4_widen(w, e4m3_half(row[kv4_code_bytes(Hkv, DH) + (g * DH + e0) / 16]), x);
    } else {
        const float *p = static_cast<const float *>(cache) + ((size_t)slot * Hkv + g) * DH + e0;
        constexpr int N = Vec16<float>::N;
#pragma unroll
        for (int u = 0; u < 8 / N; ++u) {
            float f[N];
            Vec16<float>::widen(*reinterpret_cast<const uint4 *>(p + u * N), f);
#pragma unroll
            for (int e = 0; e < N; ++e) x[u * N + e] = f[e];
        }
    }
}

template <bool KV4, int DH>
__global__ void __launch_bounds__(kSimtThreads) cache_attn_simt_kernel(CacheAttnArgs a) {
    pdl_enter();
    constexpr int LD = DH + 4;
    __shared__ float qs[kRows][LD], ks[kKeys][LD], vs[kKeys][LD];
    __shared__ float ps[kRows][kKeys];
    const int g = blockIdx.x / a.row_tiles, rt = blockIdx.x - g * a.row_tiles;  // KV head, tile
    const int R = a.R, G = a.H / a.Hkv, M = R * G;
    const int tid = threadIdx.x, lr = tid >> 3, u = tid & 7;
    const int m = rt * kRows + lr;  // row of the KV head
    const bool live = m < M;
    const int r = live ? m / G : 0, h = g * G + (live ? m - r * G : 0);
    CacheItem it;
    find_item<false, kKeys>(a, [&](int P) { return KeyRun(P, R, a.window, a.sinks).len; }, it);
    const int b = it.b, P = it.P, kbeg = it.kbeg, kend = it.kend;
    const void *kc = it.kc, *vc = it.vc;
    const KeyRun run(P, R, a.window, a.sinks);
    const size_t prow = ((size_t)it.range * a.H + h) * R + r;
    float *dst = static_cast<float *>(a.out) + (((size_t)b * R + r) * a.H + h) * DH;
    if (kbeg >= kend) {  // uniform over the CTA
        if (!live) return;
        if (a.ns == 1)
            for (int c = u; c < DH; c += 8) dst[c] = 0.f;
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
            x = Vec16<float>::load1(static_cast<const float *>(a.q) + (((size_t)b * R + rr) * a.H + hh) * DH + c);
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
                cache_load8<KV4, DH>(kc, slot, a.Hkv, g, e0, x);
                cache_load8<KV4, DH>(vc, slot, a.Hkv, g, e0, y);
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
        for (int c = 0; c < DH / 8; ++c) dst[(c / 4) * 32 + u * 4 + c % 4] = acc[c] * inv;
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
//   warps 4-7  load: K and V tiles of a stage into shared memory as 128-byte
//              swizzled blocks, a ring of tiles in the order of their use
//              (K0 K1 V0 K2 V1 ..).  A bf16 cache comes by cp.async; a 4-bit
//              tile is read into registers four tiles ahead, widened to fp16
//              (exact) and stored.
//   warp 8     one thread issues the products: S_j+1 = Q K^T as soon as the
//              scores of stage j are in registers, then O += P_j V.
//   warps 0-3  softmax: thread t owns row t of the tile, reads its 64 scores
//              from tensor memory, keeps the row's reference m and sum l in
//              registers (no exchange between threads), and writes the
//              weights P to shared memory, the product's A operand.
// Tensor memory (256 columns): [0,64) S in fp32, [64,128) Q, [128,256) O.
// P in shared memory costs 32 KB of its traffic a stage; over the S columns
// it made each stage wait for the product before (S, softmax, O in a chain).
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
// What bounds it is neither the products (a stage's take 0.33 us of an SM at the
// measured bf16 rate) nor the bytes, but passing a stage between the warps:
// about 1 us a stage with two CTAs on the SM, whatever the cache's type; a CTA
// costs 6 us more at its ends.  Without the loads and conversions after the first
// ring 0.80-0.85 of a call's time remains, without the exponentials 0.91-0.94,
// without both 0.72-0.79 (the last three cases here).  Measured: 65 rows x 32
// heads over a 1024 window 16.1 us; eight sequences of 65 rows, 32 heads over 8 KV
// heads, 4096 window 85.3 us (35 GFLOP: 0.41 PFLOP/s); 4 bits, 65 rows x 32 heads
// over 8192 slots 29.8 us, eight ragged sequences up to 4096 slots 65.2 us.
// Measured and not kept: the whole ring in flight before a tile is announced (92
// against 82 us: each tile then waits for the slot of the one NT before it),
// weights in tensor memory, 16 warps, one CTA walking several ranges, and the rows
// behind the last whole tile (260 rows are two tiles and four) on the few-row
// kernel, launched to overlap this one (5 us less to 7 us more).
//
// Masks are built as 64 bits a row and stage.  Products run over masked keys
// too, with weight 0, so a non-finite V element there would reach every row
// as 0 * inf: in stages that are not wholly visible the softmax warps look for
// such elements, add them to the rows that see them and clear them before the
// product.  Every wait is bounded; on a timeout the CTA sets the status, waits
// (bounded) for its products, frees its tensor memory and publishes nothing.
constexpr int kSub = 64, kTcThreads = 288;
constexpr uint32_t kDrainPolls = 1u << 16;
constexpr int kAhead = 4;  // 4-bit tiles held in a loader's registers

template <int DH>
struct CacheSmem {
    static constexpr int NB = DH / 64;
    static constexpr int TILE = NB * kSub * 128;
    // ring tiles: what fits beside P
    static constexpr int NT = 4 * (128 / DH);
    static constexpr int PW = NT * TILE;          // two P buffers: 128 rows of 64 weights
    static constexpr int P_BYTES = 128 * 128;
    static constexpr int BAR = PW + 2 * P_BYTES;
    // full[NT], empty[NT], q, s, sfree, drain, p[2], o[2]; then words
    static constexpr int WORDS = BAR + (2 * NT + 8) * 8;
    static constexpr int TOTAL = WORDS + 12 * 4;
    static_assert(2 * (TOTAL + 1024) <= 196 * 1024, "two CTAs per SM in the heads' carveout");
};

// Tile `i` of a range of n stages, in the order K0 K1 V0 K2 V1 .. V(n-1).
__device__ __forceinline__ bool tile_is_v(int i, int n) {
    return (i > 0 && (i & 1) == 0) || i == 2 * n - 1;
}
__device__ __forceinline__ int tile_stage(int i, int n) {
    return i == 0 ? 0 : i == 2 * n - 1 ? n - 1 : (i & 1) ? (i + 1) / 2 : i / 2 - 1;
}
__device__ __forceinline__ int k_tile(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int v_tile(int j, int n) { return min(2 * j + 2, 2 * n - 1); }

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

// Wait of a converged warp for a phase, giving up after `limit` polls or once
// the CTA has failed.  The votes keep the loop free of divergence.
__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t parity, uint32_t limit,
                                             volatile int *failed) {
    for (uint32_t i = 0; i < limit; ++i) {
        if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *failed)) return false;
    }
    *failed = 1;
    return false;
}

// the lowest n bits (n may be negative or past 64)
__device__ __forceinline__ uint64_t bits_below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// ---- loader, bf16 cache: 128 threads; thread t copies 16-byte column t % CPR
// of key rows t / CPR + RPP u (rows RPP apart share the swizzle phase)
template <int DH>
__device__ __forceinline__ void load_tile_bf16(unsigned char *tile, const bf16 *cache,
                                               const KeyRun &run, int k0, int kend, int Hkv, int g,
                                               int t) {
    constexpr int CPR = DH / 8, RPP = 128 / CPR;
    static_assert(RPP % 8 == 0, "passes keep the swizzle phase");
    const int c16 = t % CPR, r0 = t / CPR;
    const uint32_t so0 = tc::smem_addr(tile) + (c16 >> 3) * kSub * 128 + tc::sw128(r0, c16 & 7);
    const size_t row = (size_t)Hkv * DH;
    const size_t col = (size_t)g * DH + c16 * 8;
#pragma unroll
    for (int u = 0; u < kSub / RPP; ++u) {
        const int x = k0 + r0 + u * RPP;
        const bool ok = x < kend;
        const size_t off = ok ? (size_t)run.slot(x) * row + col : 0;
        cp_async16(so0 + u * RPP * 128, cache + off, ok);
    }
    asm volatile("cp.async.commit_group;\n");
}

// ---- loader, 4-bit cache: a tile is 64 keys x DH/32 groups of 32 elements (16
// code bytes, two scales); thread t takes groups t + 128 u
template <int DH>
struct Kv4Regs {
    static constexpr int N = DH / 64;
    uint4 code[N];
    uint32_t scale[N];
};

// Loads that stay where they are written, ahead of their use by kAhead tiles.
// The condition is inside: a load in a branch would be waited for where its
// register is merged with the other side's.
__device__ __forceinline__ void ld_ahead16(uint4 &r, const void *p, bool on) {
    asm volatile(
        "{\n.reg .pred q;\n"
        "setp.ne.b32 q, %5, 0;\n"
        "@q ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n}\n"
        : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
        : "l"(p), "r"((int)on));
}
__device__ __forceinline__ void ld_ahead2(uint32_t &r, const void *p, bool on) {
    asm volatile(
        "{\n.reg .pred q;\n"
        "setp.ne.b32 q, %2, 0;\n"
        "@q ld.global.nc.u16 %0, [%1];\n}\n"
        : "+r"(r)
        : "l"(p), "r"((int)on));
}

// (keys past the range read its last row; their scale is cleared on the way to
// shared memory)
template <int DH>
__device__ __forceinline__ void load_regs_kv4(Kv4Regs<DH> &r, const uint8_t *cache,
                                              const KeyRun &run, int k0, int kend, int Hkv, int g,
                                              int t, bool on) {
    constexpr int GPK = DH / 32;  // groups per key
    const int rb = kv4_row_bytes(Hkv, DH), cb = kv4_code_bytes(Hkv, DH);
#pragma unroll
    for (int u = 0; u < Kv4Regs<DH>::N; ++u) {
        const int c = t + 128 * u, x = min(k0 + c / GPK, kend - 1), q = c % GPK;
        const uint8_t *row = cache + (size_t)run.slot(x) * rb;
        ld_ahead16(r.code[u], row + g * (DH / 2) + q * 16, on);
        ld_ahead2(r.scale[u], row + cb + g * (DH / 16) + q * 2, on);
    }
}

template <int DH>
__device__ __forceinline__ void store_regs_kv4(const Kv4Regs<DH> &r, unsigned char *tile, int k0,
                                               int kend, int t) {
    constexpr int GPK = DH / 32;
#pragma unroll
    for (int u = 0; u < Kv4Regs<DH>::N; ++u) {
        const int c = t + 128 * u, key = c / GPK, q = c % GPK;
        // groups of the second column block store their 16-byte chunks in the
        // order 2,3,0,1: the eight lanes of a store phase (two keys, four
        // groups) then hit eight different bank groups
        const bool flip = (q >> 1) & 1;
        unsigned char *blk = tile + (q >> 1) * kSub * 128;
        const uint4 w = r.code[u];
        const __half2 s2 =
            __half2(__nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(k0 + key < kend ? r.scale[u] : 0u), __NV_E4M3));
        const __half2 sa = flip ? __high2half2(s2) : __low2half2(s2);
        const __half2 sb = flip ? __low2half2(s2) : __high2half2(s2);
        const uint32_t word[4] = {flip ? w.z : w.x, flip ? w.w : w.y, flip ? w.x : w.z, flip ? w.y : w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = (q & 1) * 4 + (i ^ (flip ? 2 : 0));
            *reinterpret_cast<uint4 *>(blk + tc::sw128(key, ch)) = kv4_widen(word[i], i < 2 ? sa : sb);
        }
    }
}

template <int DH, bool KV4, bool DEAL>
__global__ void __launch_bounds__(kTcThreads, 2) cache_attn_tc_kernel(CacheAttnArgs a) {
    pdl_enter();
    using L = CacheSmem<DH>;
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BAR), *empty = full + L::NT;
    // p and o have a barrier for each P buffer: a warp may be a stage ahead of
    // another, and its arrival for the next stage must not count for this one
    // (at stage j + 2 the scores it has waited for came after the product of j)
    uint64_t *bar_q = empty + L::NT, *bar_s = bar_q + 1, *bar_sfree = bar_q + 2,
             *bar_drain = bar_q + 3, *bar_p = bar_q + 4, *bar_o = bar_q + 6;
    volatile int *failed = reinterpret_cast<volatile int *>(sm + L::WORDS);
    volatile int *o_started = failed + 1;                        // O holds something before stage 0
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(sm + L::WORDS + 8);
    int *warp_depth = reinterpret_cast<int *>(sm + L::WORDS + 16);       // [4]
    // Keys of a stage whose V is not finite, a pair of words for each parity of the
    // stage: a warp may mark the next stage's keys while thread 0 still clears
    // this one's.  The pair's next use, two stages on, follows thread 0's arrival
    // on bar_sfree after the clearing.
    uint32_t *bad_keys = reinterpret_cast<uint32_t *>(sm + L::WORDS + 32);  // [2][2]

    const int g = blockIdx.x / a.row_tiles, rt = blockIdx.x - g * a.row_tiles;
    const int R = a.R, G = a.H / a.Hkv, M = R * G;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    CacheItem it;
    if (!find_item<DEAL>(a, [&](int P) { return KeyRun(P, R, a.window, a.sinks).len; }, it)) return;
    const int b = it.b, P = it.P, kbeg = it.kbeg, kend = it.kend;
    const void *kc = it.kc, *vc = it.vc;
    const KeyRun run(P, R, a.window, a.sinks);

    // row of a softmax thread
    const int m = rt * 128 + tid;
    const bool live = tid < 128 && m < M;
    const int r = live ? m / G : 0, h = g * G + (live ? m - r * G : 0);
    const size_t prow = ((size_t)it.range * a.H + h) * R + r;
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
        for (int i = 0; i < L::NT; ++i) {
            tc::mbar_init(full + i, 128);
            tc::mbar_init(empty + i, 1);
        }
        tc::mbar_init(bar_q, 128);
        tc::mbar_init(bar_s, 1);
        tc::mbar_init(bar_sfree, 128);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar_p + i, 128);
            tc::mbar_init(bar_o + i, 1);
        }
        tc::mbar_init(bar_drain, 1);
        *failed = 0;
        *o_started = 0;
        bad_keys[0] = bad_keys[1] = bad_keys[2] = bad_keys[3] = 0;
        tc::fence_mbarrier_init();
    }
    if (warp == 8) tc::tmem_alloc(tmem_holder, 256);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_holder;
    const uint32_t t_s = tmem, t_q = tmem + 64, t_o = tmem + 128;

    auto slot_of = [&](int i) { return sm + (i % L::NT) * L::TILE; };
    auto wait_full = [&](int i) {
        return wait_or_fail(full + i % L::NT, (i / L::NT) & 1, a.wait_polls, failed);
    };
    auto wait_product = [&](int j) {  // O += P_j V done
        return wait_or_fail(bar_o + (j & 1), (j >> 1) & 1, a.wait_polls, failed);
    };
    if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ loaders
        const int t = tid - 128, n_tiles = 2 * nsub;
        auto wait_empty = [&](int i) {  // slot of tile i free: tile i - NT was used
            return i < L::NT ||
                   wait_or_fail(empty + i % L::NT, (i / L::NT - 1) & 1, a.wait_polls, failed);
        };
        if constexpr (KV4) {
            const uint8_t *k8 = static_cast<const uint8_t *>(kc), *v8 = static_cast<const uint8_t *>(vc);
            Kv4Regs<DH> buf[kAhead] = {};
            auto fetch = [&](Kv4Regs<DH> &r, int i) {
                load_regs_kv4<DH>(r, tile_is_v(i, nsub) ? v8 : k8, run,
                                  kbeg + tile_stage(i, nsub) * kSub, kend, a.Hkv, g, t, i < n_tiles);
            };
#pragma unroll
            for (int u = 0; u < kAhead; ++u) fetch(buf[u], u);
            bool go = true;
            for (int i0 = 0; i0 < n_tiles && go; i0 += kAhead) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = i0 + u;
                    if (i < n_tiles && go) {
                        go = wait_empty(i);
                        if (go) {
                            store_regs_kv4<DH>(buf[u], slot_of(i), kbeg + tile_stage(i, nsub) * kSub,
                                               kend, t);
                            tc::fence_proxy_async_smem();
                            tc::mbar_arrive(full + i % L::NT);
                        }
                    }
                    fetch(buf[u], i + kAhead);
                }
            }
        } else {
            // half the ring of younger copies stays in flight when a tile is announced
            constexpr int LAG = L::NT / 2;
            const bf16 *k16 = static_cast<const bf16 *>(kc), *v16 = static_cast<const bf16 *>(vc);
            bool go = true;
            for (int i = 0; i < n_tiles + LAG && go; ++i) {
                if (i < n_tiles) {
                    go = wait_empty(i);
                    if (!go) break;
                    load_tile_bf16<DH>(slot_of(i), tile_is_v(i, nsub) ? v16 : k16, run,
                                       kbeg + tile_stage(i, nsub) * kSub, kend, a.Hkv, g, t);
                } else {
                    asm volatile("cp.async.commit_group;\n");  // keeps the count of groups
                }
                if (i >= LAG) {
                    asm volatile("cp.async.wait_group %0;\n" ::"n"(LAG));
                    tc::fence_proxy_async_smem();
                    tc::mbar_arrive(full + (i - LAG) % L::NT);
                }
            }
            asm volatile("cp.async.wait_group 0;\n");
        }
    } else if (warp == 8) {
        // ----------------------------------------------------------- products
        // (the warp stays converged; one elected lane issues)
        constexpr uint32_t id_s = KV4 ? tc::idesc_f16(128, kSub, 0) : tc::idesc_bf16(128, kSub, 0);
        constexpr uint32_t id_o = KV4 ? tc::idesc_f16(128, DH, 1) : tc::idesc_bf16(128, DH, 1);
        const uint64_t kd0 = tc::sdesc_sw128(tc::smem_addr(sm), 16, 1024);
        const uint64_t vd0 = tc::sdesc_sw128(tc::smem_addr(sm), kSub * 128, 1024);
        const uint64_t pd0 = tc::sdesc_sw128(tc::smem_addr(sm + L::PW), 16, 1024);
        auto scores = [&](int j) {
            const int i = k_tile(j);
            // the scores before are in registers
            if (!wait_full(i)) return false;
            if (j > 0 && !wait_or_fail(bar_sfree, (j - 1) & 1, a.wait_polls, failed)) return false;
            tc::fence_after_sync();
            const int slot = i % L::NT;
            if (tc::elect_one()) {
                const uint64_t kd = kd0 + (uint64_t)(slot * (L::TILE >> 4));
#pragma unroll
                for (int ks = 0; ks < DH / 16; ++ks)
                    tc::mma_bf16_ts(t_s, t_q + ks * 8, kd + (((ks >> 2) * kSub * 128 + (ks & 3) * 32) >> 4),
                                    id_s, ks > 0);
                tc::mma_commit(bar_s);
                tc::mma_commit(empty + slot);
            }
            __syncwarp();
            return true;
        };
        bool go = wait_or_fail(bar_q, 0, a.wait_polls, failed) && scores(0);
        for (int j = 0; j < nsub && go; ++j) {
            if (j + 1 < nsub && !scores(j + 1)) break;
            const int i = v_tile(j, nsub);
            if (!wait_or_fail(bar_p + (j & 1), (j >> 1) & 1, a.wait_polls, failed) || !wait_full(i)) break;
            tc::fence_after_sync();
            const uint32_t acc0 = j > 0 || *o_started;
            const int slot = i % L::NT;
            if (tc::elect_one()) {
                const uint64_t vd = vd0 + (uint64_t)(slot * (L::TILE >> 4));
                const uint64_t pd = pd0 + (uint64_t)((j & 1) * (L::P_BYTES >> 4));
#pragma unroll
                for (int ks = 0; ks < kSub / 16; ++ks)
                    tc::mma_bf16_ss(t_o, pd + ((ks * 32) >> 4), vd + ((ks * 16 * 128) >> 4), id_o,
                                    ks > 0 ? 1u : acc0);
                tc::mma_commit(bar_o + (j & 1));
                tc::mma_commit(empty + slot);
            }
            __syncwarp();
        }
        // every product issued above is done before the tensor memory is freed
        if (tc::elect_one()) tc::mma_commit(bar_drain);
        __syncwarp();
        if (!__all_sync(0xffffffffu, tc::mbar_wait_bounded(bar_drain, 0, kDrainPolls))) {
            *failed = 1;
            if (lane == 0 && a.status) atomicExch(a.status, MEDUSA_DEV_DRAIN_TIMEOUT);
        }
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
            // a masked score, -inf, times the scale has to stay -inf
            row_scale = fmaxf(row_scale, 0x1p-126f);
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
            tc::mbar_arrive(bar_q);
        }
        // ---- what this row sees, in numbered keys
        const int my_depth = row_depth(a, b, r);
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
            unsigned char *p_row = sm + L::PW + (j & 1) * L::P_BYTES;
            // the scores are there; their commit also covers the product of j - 2,
            // issued before them, which read this P buffer
            if (!dead) dead = !wait_or_fail(bar_s, j & 1, a.wait_polls, failed);
            tc::fence_after_sync();
            if (!dead && !rows_live) tc::mbar_arrive(bar_sfree);
            if (!dead && rows_live) {
                float x[kSub];
                tc::tmem_ld64(t_s + lane_base, x);
                tc::fence_before_sync();
                tc::mbar_arrive(bar_sfree);
                bool grew = false;
                float alpha = 1.f;
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
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mx[q] = max3f(x[q], x[q + 4], x[q + 8]);
#pragma unroll
                    for (int e = 12; e + 4 < kSub; e += 8) mx[q] = max3f(mx[q], x[q + e], x[q + e + 4]);
                    mx[q] = fmaxf(mx[q], x[q + kSub - 4]);
                }
                const float cm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * row_scale;
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
                for (int c = 0; c < kSub / 8; ++c) {
                    uint32_t pk[4];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float2 t = __ffma2_rn(make_float2(x[c * 8 + e], x[c * 8 + e + 1]), sc2, nm2);
                        const float p0 = ex2_approx(t.x), p1 = ex2_approx(t.y);
                        // Rounded for the product only, whose operands have 16 bits:
                        // to bf16 beside a bf16 V (fp16 has not its range, and both
                        // operands are of one type), at most 2^-8 of a weight; the
                        // sum adds the fp32 weights.
                        pk[e / 2] = pack_weights<KV4>(p0, p1);
                        ls[(e / 2) & 1] = __fadd2_rn(ls[(e / 2) & 1], make_float2(p0, p1));
                    }
                    *reinterpret_cast<uint4 *>(p_row + tc::sw128(tid, c)) =
                        make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
                l_run += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                tc::fence_proxy_async_smem();
                if (__any_sync(0xffffffffu, grew && j > 0)) {
                    dead = !wait_product(j - 1);
                    tc::fence_after_sync();
                    if (!dead) {
#pragma unroll 1
                        for (int c = 0; c < DH; c += 32) {
                            float ov[32];
                            tc::tmem_ld32(t_o + lane_base + c, ov);
#pragma unroll
                            for (int e = 0; e < 32; ++e) ov[e] *= alpha;
                            tc::tmem_st32(t_o + lane_base + c, ov);
                        }
                    }
                }
            }
            if (masked) {
                // ---- infinities and NaNs in V of a stage that some row does not see
                unsigned char *vt = slot_of(v_tile(j, nsub));
                uint32_t *bad_now = bad_keys + 2 * (j & 1);
                if (!dead) dead = !wait_full(v_tile(j, nsub));
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
                                atomicOr(bad_now + ((row & 63) >> 5), 1u << (row & 31));
                            }
                        }
                if (softmax_any(bad)) {
                    if (!dead && j > 0) {
                        dead = !wait_product(j - 1);
                        tc::fence_after_sync();
                    }
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
                            if (!((bad_now[key >> 5] >> (key & 31)) & 1u)) continue;
                            const float p = half_of_pair<KV4>(*reinterpret_cast<const uint16_t *>(
                                p_row + tc::sw128(tid, key >> 3) + (key & 7) * 2), 0);
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
                    if (tid == 0) bad_now[0] = bad_now[1] = 0;
                    tc::fence_proxy_async_smem();
                }
            }
            if (!dead) {
                tc::fence_before_sync();
                tc::mbar_arrive(bar_p + (j & 1));
            }
        }
        // ---- the last product, then the row
        if (!dead)
            dead = !wait_product(nsub - 1);
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
// Lane s reads range s's (m, l); the O rows do not depend on them and are
// loaded eight at a time, the first eight in the same round.
template <typename T, int DH>
__global__ void __launch_bounds__(256)
cache_attn_combine_kernel(const float *__restrict__ part_o, const float2 *__restrict__ part_ml,
                          const int *__restrict__ starts, int B, int R, int H, int ns,
                          T *__restrict__ out) {
    pdl_enter();
    constexpr int PER = DH / 32, AHEAD = 8;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= (long long)B * H * R) return;
    const int r = (int)(item % R);
    const long long bh = item / R;
    const int b = (int)(bh / H), first_range = starts ? starts[b] : b * ns;
    const int NS = starts ? starts[b + 1] - first_range : ns;
    const size_t ml_step = (size_t)H * R, step = ml_step * DH;
    const float2 *ml = part_ml + first_range * ml_step + (bh % H) * R + r;
    const float *po = part_o + (first_range * ml_step + (bh % H) * R + r) * DH + lane * PER;
    float2 row[AHEAD][PER / 2];
    auto load = [&](int s0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (s0 + i < NS) {
                const float *p = po + (s0 + i) * step;
                if constexpr (PER == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(p);
                    row[i][0] = make_float2(v.x, v.y);
                    row[i][1] = make_float2(v.z, v.w);
                } else {
                    row[i][0] = *reinterpret_cast<const float2 *>(p);
                }
            }
    };
    const float2 empty = make_float2(-INFINITY, 0.f);
    const float2 first = lane < NS ? ml[lane * ml_step] : empty;
    load(0);
    float M = first.y != 0.f ? first.x : -INFINITY;
    for (int s = lane + 32; s < NS; s += 32) {
        const float2 x = ml[s * ml_step];
        if (x.y != 0.f) M = fmaxf(M, x.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) acc[p] = 0.f;
    float w_l = 0.f;
    for (int s0 = 0; s0 < NS; s0 += AHEAD) {
        if (s0 > 0) load(s0);
        if ((s0 & 31) == 0) {
            const float2 x = s0 == 0 ? first : s0 + lane < NS ? ml[(s0 + lane) * ml_step] : empty;
            w_l = x.y != 0.f ? exp2f(x.x - mu) : 0.f;
            if (x.y != 0.f) L = fmaf(w_l, x.y, L);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const float w = __shfl_sync(0xffffffffu, w_l, (s0 + i) & 31);
            if (s0 + i < NS && w != 0.f) {
#pragma unroll
                for (int p = 0; p < PER / 2; ++p) {
                    acc[2 * p] = fmaf(w, row[i][p].x, acc[2 * p]);
                    acc[2 * p + 1] = fmaf(w, row[i][p].y, acc[2 * p + 1]);
                }
            }
        }
    }
    L = warp_sum(L);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    T *dst = out + (((bh / H) * R + r) * H + bh % H) * DH + lane * PER;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int p = 0; p < PER; ++p) dst[p] = acc[p] * inv;
    } else {
#pragma unroll
        for (int p = 0; p < PER; p += 2)
            *reinterpret_cast<__nv_bfloat162 *>(dst + p) =
                __floats2bfloat162_rn(acc[p] * inv, acc[p + 1] * inv);
    }
}

// ------------------------------------------------------------------- host ---

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct CachePlan {
    int row_tiles, ns, window, sinks;
    bool few;   // at most kFewRows rows a KV head
    bool deal;  // ranges dealt out by the sequences' lengths
};

// Key ranges: the count that makes (waves of CTAs) x (stages per CTA + 3)
// smallest, joining included.  The 3 stands for the fixed cost of a CTA in all three
// kernels: over 42 shapes of them every choice from 3 to 8 gave the same times
// within 1 %, 1 and 2 the few-row kernel up to 20 % more (eight single tokens over
// 4000 slots 18.9 against 15.7 us).
CachePlan cache_plan(medusa_dtype dtype, bool kv4, int B, int R, int H, int Hkv, int P_max, int window,
                     int sinks) {
    CachePlan p;
    // a window no row's oldest key falls out of is none
    p.window = window >= P_max + R ? 0 : window;
    p.sinks = p.window ? std::min(sinks, P_max + R) : 0;
    const int keys =
        p.window ? std::min(P_max, p.sinks + p.window - 1) + R : P_max + R;  // longest KeyRun
    const int M = R * (H / Hkv);
    const bool simt = dtype == MEDUSA_F32;
    p.few = !simt && M <= kFewRows;
    const int rows = simt ? kRows : 128;
    const int sub = simt ? kKeys : kRangeUnit;
    const int slots = (simt ? 4 : p.few ? cache_few_ctas_per_sm(kv4, M) : 2) * device_sm_count();
    p.row_tiles = (M + rows - 1) / rows;
    const int subs = (keys + (p.few && p.sinks ? 15 : 0) + sub - 1) / sub;  // (few: a gap after the sinks)
    const long long ctas = (long long)B * Hkv * p.row_tiles;
    double best = 0;
    p.ns = 1;
    // (more than four waves only add to the fixed cost)
    const int most = std::min<long long>(subs, std::max<long long>(1, 4LL * slots / ctas));
    for (int ns = 1; ns <= most; ++ns) {
        const int per = (subs + ns - 1) / ns;
        if ((subs + per - 1) / per != ns) continue;  // the same split as a smaller ns
        const double waves = (double)((ctas * ns + slots - 1) / slots);
        const double cost = waves * (per + 3) + (ns > 1 ? 3.0 + 0.05 * ns : 0.0);
        if (ns == 1 || cost < best) {
            best = cost;
            p.ns = ns;
        }
    }
    // Sequences of different lengths (behind a window they are about alike): ranges
    // dealt out by length.  Single tokens, eight sequences of 7.5k to 32k 4-bit slots:
    // 75 -> 56 us.  It costs 1-2 us at the start and in the join (a 65-row step over
    // a 1024 window 15.8 -> 17.2 us).
    p.deal = !simt && p.ns > 1 && B > 1 && B <= 32 && !p.window;
    return p;
}

}  // namespace

size_t cache_attention_workspace_bytes(medusa_dtype dtype, bool kv4, int B, int R, int H, int Hkv, int dh,
                                       int P_max, int window, int sinks) {
    const CachePlan p = cache_plan(dtype, kv4, B, R, H, Hkv, P_max, window, sinks);
    if (p.ns == 1) return MEDUSA_WS_HEADER;
    const size_t rows = (size_t)B * H * p.ns * R;
    return MEDUSA_WS_HEADER + align256(rows * dh * sizeof(float)) + align256(rows * sizeof(float2)) +
           (p.deal ? align256((B + 1) * sizeof(int)) : 0);
}

cudaError_t launch_cache_attention(medusa_dtype dtype, bool kv4, const void *q,
                                   const void *const *k_cache, const void *const *v_cache,
                                   const int32_t *prefix_len, int P_max, const uint64_t *anc_mask,
                                   const int32_t *depth, int window, int sinks, int B, int R, int H,
                                   int Hkv, int dh, float scale, void *out, void *ws,
                                   cudaStream_t stream) {
    const CachePlan p = cache_plan(dtype, kv4, B, R, H, Hkv, P_max, window, sinks);
    CacheAttnArgs a;
    a.q = q;
    a.kc = k_cache;
    a.vc = v_cache;
    a.prefix_len = prefix_len;
    a.anc_mask = anc_mask;
    a.depth = window ? depth : nullptr;  // checked also where no slot falls out of the window
    a.B = B;
    a.R = R;
    a.H = H;
    a.Hkv = Hkv;
    a.P_max = P_max;
    a.window = p.window;
    a.sinks = p.sinks;
    a.ns = p.ns;
    a.row_tiles = p.row_tiles;
    a.scale_log2 = scale * kLog2e;
    const size_t rows = (size_t)B * H * p.ns * R;
    char *w = static_cast<char *>(ws) + MEDUSA_WS_HEADER;
    a.part_o = reinterpret_cast<float *>(w);
    a.part_ml = reinterpret_cast<float2 *>(w + align256(rows * dh * sizeof(float)));
    a.starts = p.deal ? reinterpret_cast<int *>(reinterpret_cast<char *>(a.part_ml) +
                                                     align256(rows * sizeof(float2)))
                           : nullptr;
    a.out = out;
    a.status = static_cast<int *>(ws);
    a.wait_polls = wait_budget();
    const bool f32 = dtype == MEDUSA_F32;
    const dim3 grid(Hkv * p.row_tiles, p.ns, B);
    cudaError_t e;
    if (f32) {
        auto kern = kv4 ? (dh == 128 ? cache_attn_simt_kernel<true, 128> : cache_attn_simt_kernel<true, 64>)
                        : (dh == 128 ? cache_attn_simt_kernel<false, 128> : cache_attn_simt_kernel<false, 64>);
        e = launch_pdl(kern, grid, dim3(kSimtThreads), 0, stream, a);
    } else if (p.few) {
        e = launch_cache_attention_few(a, kv4, dh, stream);
    } else {
        auto pick = [&](auto own, auto deal) { return p.deal ? deal : own; };
        auto kern =
            kv4 ? (dh == 128 ? pick(cache_attn_tc_kernel<128, true, false>, cache_attn_tc_kernel<128, true, true>)
                             : pick(cache_attn_tc_kernel<64, true, false>, cache_attn_tc_kernel<64, true, true>))
                : (dh == 128 ? pick(cache_attn_tc_kernel<128, false, false>, cache_attn_tc_kernel<128, false, true>)
                             : pick(cache_attn_tc_kernel<64, false, false>, cache_attn_tc_kernel<64, false, true>));
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
                       dim3(blocks), dim3(256), 0, stream, po, pm, (const int *)a.starts, B, R, H, p.ns,
                       static_cast<float *>(out));
    else
        e = launch_pdl(dh == 128 ? cache_attn_combine_kernel<bf16, 128> : cache_attn_combine_kernel<bf16, 64>,
                       dim3(blocks), dim3(256), 0, stream, po, pm, (const int *)a.starts, B, R, H, p.ns,
                       static_cast<bf16 *>(out));
    note_launch();
    return e;
}

}  // namespace medusa
