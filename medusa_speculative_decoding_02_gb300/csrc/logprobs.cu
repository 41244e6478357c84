// logprobs.cu -- log probabilities of given tokens, with their ranks, the entropy
// of each row and its top alternatives, in one pass over the logits.
//
// Row x of V logits, temperature T, token t, y = x log2(e) / T, m the row's largest y:
//     S = sum 2^(y - m),  A = sum 2^(y - m) (y - m)
//     logp = ln2 (y_t - m - log2 S)       entropy = ln2 (log2 S - A / S)
//     rank = number of tokens before t in the order (larger logit, then smaller id)
//     alternatives: the first `top` tokens of that order
//
// A CTA (four warps that compute, one that copies) takes a row at a time, in chunks of
// 512 16-byte vectors that come by bulk copies into a ring; with few rows a cluster of
// CTAs shares each row.  A thread keeps its own reference, S and A, and moves the
// reference when a chunk's maximum (packed, NaNs kept) exceeds it by 2^8; references in
// base 2 are rounded by products that are not fused, so that all sums are relative
// to the same number.
// Ranks are packed comparisons with the token's logit, or up to its place with the
// number below it.  Alternatives: the k-th largest of 32 groups of threads' maxima so
// far is at most the row's k-th largest logit (T0, looked at again after 1, 2, 4, ..
// chunks); vectors whose maximum reaches it are kept, at the row's end their elements that
// do are the candidates (some tens), and a candidate's place in the order is the number
// of better ones among them.
//
// What this form does not take (a NaN, +inf or nothing above -1e29 in the row, the token
// at -inf, too many candidates because of ties, fewer possible tokens
// than alternatives, temperatures below 1e-7) is done by slow_row, by plain passes over
// the row: the results are the same by definition.
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace medusa {

namespace {

constexpr int kConsumers = 128, kLpThreads = kConsumers + 32, kWarps = kConsumers / 32;
constexpr int kChunk = 512, kPer = kChunk / kConsumers;  // vectors of a chunk, of a thread
constexpr int kRing = 3, kLpCtas = 6;
constexpr int kVectors = 256, kCandidates = 512;  // kept of a row
constexpr int kMaxCluster = 8;
constexpr uint32_t kLpPolls = 1u << 20;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -1e30f, kNothing = -1e29f, kHighest = 1e30f, kLag = 8.f;
static_assert(32 >= MEDUSA_MAX_TOP_S && kMaxCluster * MEDUSA_MAX_TOP_S <= kConsumers, "groups, and parts' lists");

struct LogprobArgs {
    const void *logits;
    long long stride;
    const int32_t *tokens;
    int N, V, top;
    float inv_T, y_scale;  // 1 / T, log2(e) / T
    float *logp, *entropy;
    int32_t *rank;
    int32_t *top_ids;
    float *top_logp;
    int *status;
};

// What a CTA of a cluster knows of its part of a row.
struct RowPart {
    float m;       // largest logit (NaN if there is one)
    float S, A;    // relative to m
    int before, n; // tokens before the row's token; candidates (-1: too many)
    uint64_t key[MEDUSA_MAX_TOP_S];  // the part's first tokens (0: none)
};

struct LpSmem {
    static constexpr int RING = 0;
    static constexpr int VEC = kRing * kChunk * 16;  // vectors kept
    static constexpr int CAND = VEC + kVectors * 16;  // candidates: see key_of
    static constexpr int AT = CAND + kCandidates * 8; // the vectors' places
    static constexpr int PART = AT + kVectors * 4;
    static constexpr int RED = PART + (int)(sizeof(RowPart) + 15) / 16 * 16;  // [4][kWarps]
    static constexpr int GROUP = RED + 4 * kWarps * 4;                        // [2][kWarps][32]
    static constexpr int BAR = GROUP + 2 * kWarps * 32 * 4;
    static constexpr int WORDS = BAR + 2 * kRing * 8;  // vectors, candidates of even and odd rows; failed
    static constexpr int TOTAL = WORDS + 32;
    static_assert(kLpCtas * (TOTAL + 1024) <= 228 * 1024, "CTAs of an SM");
};

__device__ __forceinline__ void consumers_sync() { asm volatile("barrier.cta.sync 1, %0;\n" ::"n"(kConsumers) : "memory"); }

// floats in order as unsigned numbers (a NaN: 0, below all)
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);  // (-0 is 0)
    return isnan(f) ? 0u : u ^ ((int)u < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k ^ ((int)k < 0 ? 0x80000000u : 0xffffffffu));
}
// a token in the order: the larger key comes first
__device__ __forceinline__ uint64_t key_of(float f, int id) { return (uint64_t)ordered(f) << 32 | (uint32_t)~id; }
__device__ __forceinline__ float key_logit(uint64_t k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_id(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Sixteen bytes of logits: the packed steps of a vector.
template <typename T> struct Lp;
template <> struct Lp<bf16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ float value(bf16 x) { return __bfloat162float(x); }
    using Pair = __nv_bfloat162;
    __device__ static __forceinline__ uint4 nothing() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    __device__ static __forceinline__ Pair pair(uint32_t w) { return *reinterpret_cast<const Pair *>(&w); }
    // the largest of a vector, in two halves, of two such, and as a number
    using Top = Pair;
    __device__ static __forceinline__ Top top(const uint4 &v) {
        return __hmax2_nan(__hmax2_nan(pair(v.x), pair(v.y)), __hmax2_nan(pair(v.z), pair(v.w)));
    }
    __device__ static __forceinline__ Top top(Top a, Top b) { return __hmax2_nan(a, b); }
    __device__ static __forceinline__ float number(Top p) { return max_nan(__low2float(p), __high2float(p)); }
    // how many elements of a chunk's vectors lie above a bound
    using Bound = Pair;
    __device__ static __forceinline__ Bound bound(float x) { return __float2bfloat162_rn(x); }
    struct Count {
        float2 all = make_float2(0.f, 0.f);
        Pair n;
        __device__ __forceinline__ void start() { n = __float2bfloat162_rn(0.f); }
        __device__ __forceinline__ void add(const uint4 &v, Bound b) {
            n = __hadd2(n, __hadd2(__hadd2(__hgt2(pair(v.x), b), __hgt2(pair(v.y), b)),
                                   __hadd2(__hgt2(pair(v.z), b), __hgt2(pair(v.w), b))));
        }
        __device__ __forceinline__ void end() {  // (up to 16 in a half, and 2^24 in all, are exact)
            const uint32_t u = *reinterpret_cast<const uint32_t *>(&n);
            all = __fadd2_rn(all, make_float2(bf_lo(u), bf_hi(u)));
        }
        __device__ __forceinline__ int total() const { return (int)(all.x + all.y); }
    };
    // the largest number of the type below x
    __device__ static __forceinline__ float below(float x) {
        const uint32_t u = __float_as_uint(x);
        return __uint_as_float(x == 0.f ? 0x80010000u : (int)u < 0 ? u + 0x10000u : u - 0x10000u);
    }
    __device__ static __forceinline__ void add(const uint4 &v, float ys, float m2, float2 (&S)[2], float2 (&A)[2]) {
        const Pair low = __float2bfloat162_rn(kLowest);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // (-inf is lifted: 0 * -inf would make A a NaN)
            const Pair c = __hmax2(pair(w[i]), low);
            const uint32_t u = *reinterpret_cast<const uint32_t *>(&c);
            const float2 t = __ffma2_rn(make_float2(bf_lo(u), bf_hi(u)), make_float2(ys, ys), make_float2(-m2, -m2));
            const float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
            S[i & 1] = __fadd2_rn(S[i & 1], p);
            A[i & 1] = __ffma2_rn(p, t, A[i & 1]);
        }
    }
};
template <> struct Lp<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ float value(float x) { return x; }
    __device__ static __forceinline__ uint4 nothing() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    using Top = float;
    __device__ static __forceinline__ Top top(const uint4 &v) {
        return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                       max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    __device__ static __forceinline__ Top top(Top a, Top b) { return max_nan(a, b); }
    __device__ static __forceinline__ float number(Top p) { return p; }
    using Bound = float;
    __device__ static __forceinline__ Bound bound(float x) { return x; }
    struct Count {
        int n = 0;
        __device__ __forceinline__ void start() {}
        __device__ __forceinline__ void add(const uint4 &v, Bound b) {
            n += (__uint_as_float(v.x) > b) + (__uint_as_float(v.y) > b) + (__uint_as_float(v.z) > b) +
                 (__uint_as_float(v.w) > b);
        }
        __device__ __forceinline__ void end() {}
        __device__ __forceinline__ int total() const { return n; }
    };
    __device__ static __forceinline__ float below(float x) {
        const uint32_t u = __float_as_uint(x);
        return __uint_as_float(x == 0.f ? 0x80000001u : (int)u < 0 ? u + 1u : u - 1u);
    }
    __device__ static __forceinline__ void add(const uint4 &v, float ys, float m2, float2 (&S)[2], float2 (&A)[2]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 f = make_float2(fmaxf(__uint_as_float(w[2 * i]), kLowest), fmaxf(__uint_as_float(w[2 * i + 1]), kLowest));
            const float2 t = __ffma2_rn(f, make_float2(ys, ys), make_float2(-m2, -m2));
            const float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
            S[i] = __fadd2_rn(S[i], p);
            A[i] = __ffma2_rn(p, t, A[i]);
        }
    }
};

// Where a row's vectors lie: elements N i - off .. of whole 16-byte blocks i in [first,
// last), the others at the row's ends one by one.
template <typename T>
struct RowShape {
    const char *block;  // block 0: the 16 bytes that hold element 0
    int off, first, last;
    int left, edges;    // elements before block `first`; and all outside the whole blocks
    __device__ __forceinline__ RowShape(const LogprobArgs &a, int row) {
        constexpr int N = Lp<T>::N;
        const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T *>(a.logits) + (long long)row * a.stride);
        block = reinterpret_cast<const char *>(at & ~(uintptr_t)15);
        off = (int)(at & 15) / (int)sizeof(T);
        first = off ? 1 : 0;
        last = (off + a.V) / N;
        left = off ? min(N - off, a.V) : 0;
        if (last < first) last = first;
        edges = a.V - (last - first) * N;
    }
    // id of the i-th of the edge elements
    __device__ __forceinline__ int edge(int i) const { return i < left ? i : i + (last - first) * Lp<T>::N; }
};

template <typename F>
__device__ __forceinline__ float fold_consumers(float v, float *s, F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    consumers_sync();
    if (lane == 0) s[warp] = v;
    consumers_sync();
    v = s[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v = f(v, s[w]);
    return v;
}

// A row by the definition: a pass for the maximum, one for the sums, one for each
// alternative.
template <typename T>
__device__ __noinline__ void slow_row(const LogprobArgs &a, int row, int tok, float *s_f, int *s_i) {
    const int tid = threadIdx.x;
    const T *x = static_cast<const T *>(a.logits) + (long long)row * a.stride;
    auto add = [](float p, float q) { return p + q; };
    auto larger = [](float p, float q) { return fmaxf(p, q); };
    const float xt = tok >= 0 ? Vec16<T>::load1(x + tok) : NAN;
    float m = -INFINITY, odd = 0.f;
    for (int i = tid; i < a.V; i += kConsumers) {
        const float f = Vec16<T>::load1(x + i);
        m = fmaxf(m, f);
        if (!(f < INFINITY)) odd = 1.f;
    }
    m = fold_consumers(m, s_f, larger);
    const bool bad = fold_consumers(odd, s_f, larger) != 0.f;  // +inf or NaN in the row
    float S = 0.f, A = 0.f, before = 0.f;
    for (int i = tid; i < a.V; i += kConsumers) {
        const float f = Vec16<T>::load1(x + i);
        const float t = fmaxf((f - m) * a.y_scale, -127.f), p = ex2_approx(t);
        S += p;
        A = fmaf(p, t, A);
        if (f > xt || (f == xt && i < tok)) before += 1.f;
    }
    S = fold_consumers(S, s_f, add);
    A = fold_consumers(A, s_f, add);
    before = fold_consumers(before, s_f, add);
    const bool none = m == -INFINITY;  // nothing is possible
    const float ls = log2f(S);
    auto logp_of = [&](float f) { return bad ? NAN : none ? -INFINITY : (f - m) * a.inv_T - ls * kLn2; };
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
            for (int i = tid; i < a.V; i += kConsumers) {
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
        consumers_sync();
        if ((tid & 31) == 0) s_f[tid >> 5] = bv, s_i[tid >> 5] = bi;
        consumers_sync();
        for (int w = 0; w < kWarps; ++w)
            if (better(s_f[w], s_i[w], bv, bi)) bv = s_f[w], bi = s_i[w];
        any = bi != INT_MAX;
        if (tid == 0) {
            a.top_ids[(size_t)row * a.top + k] = any ? bi : -1;
            a.top_logp[(size_t)row * a.top + k] = any ? logp_of(bv) : NAN;
        }
        lv = bv;
        li = bi;
    }
    consumers_sync();
}

__device__ __forceinline__ void bulk_copy(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                     tc::smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}
// generic address of `p` in the shared memory of CTA `rank` of the cluster
template <typename P>
__device__ __forceinline__ const P *cluster_ptr(const P *p, uint32_t rank) {
    uint64_t r;
    asm("mapa.u64 %0, %1, %2;\n" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<const P *>(r);
}

// What the one pass holds for; otherwise slow_row.
__device__ __forceinline__ bool fast_form(const LogprobArgs &a, float top, bool many, int n, int tok, float xt) {
    return top >= kNothing && top <= kHighest && !many && n >= a.top && (tok < 0 || xt > -INFINITY) &&
           a.y_scale <= 1e7f;
}

// ln p of logits of a row whose largest is `top`, with the sum relative to it
struct LogP {
    float y_scale, inv_T, t2, ls;
    __device__ __forceinline__ LogP(const LogprobArgs &a, float top, float sum) {
        y_scale = a.y_scale;
        inv_T = a.inv_T;
        t2 = __fmul_rn(top, a.y_scale);
        ls = log2f(sum);
    }
    __device__ __forceinline__ float operator()(float f) const {
        const float l = (fmaf(f, y_scale, -t2) - ls) * kLn2;
        return l == -INFINITY && f > -INFINITY ? f * inv_T : l;
    }
};

// grid: C CTAs (a cluster) a row; with C = 1 a CTA takes rows blockIdx.x, + gridDim.x, ..
template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kLpThreads, kLpCtas) token_logprobs_kernel(LogprobArgs a, int C) {
    pdl_enter();
    constexpr int N = Lp<T>::N;
    extern __shared__ __align__(128) unsigned char sm[];
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + LpSmem::BAR), *empty = full + kRing;
    uint4 *kept = reinterpret_cast<uint4 *>(sm + LpSmem::VEC);
    uint64_t *cand = reinterpret_cast<uint64_t *>(sm + LpSmem::CAND);
    int *kept_at = reinterpret_cast<int *>(sm + LpSmem::AT);
    RowPart *part = reinterpret_cast<RowPart *>(sm + LpSmem::PART);
    float *red = reinterpret_cast<float *>(sm + LpSmem::RED), *group_max = reinterpret_cast<float *>(sm + LpSmem::GROUP);
    int *counts = reinterpret_cast<int *>(sm + LpSmem::WORDS);
    volatile int *failed = reinterpret_cast<volatile int *>(counts + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank_in = CLUSTER ? (int)cluster_rank() : 0;
    const int row0 = CLUSTER ? (int)blockIdx.x / C : blockIdx.x, row_step = CLUSTER ? a.N : gridDim.x;
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(full + i, 1);
            tc::mbar_init(empty + i, kWarps);
        }
        counts[0] = counts[1] = counts[2] = counts[3] = 0;
        *failed = 0;
        tc::fence_mbarrier_init();
    }
    __syncthreads();
    auto slice = [&](const RowShape<T> &s, int &lo, int &hi) {
        const long long n = s.last - s.first;
        lo = s.first + (int)(n * rank_in / C);
        hi = s.first + (int)(n * (rank_in + 1) / C);
    };
    // a row's token (-1: none) and its logit
    auto token_of = [&](int row) { return row < a.N ? a.tokens[row] : -1; };
    auto logit_of = [&](int row, int tok) {
        return tok >= 0 && tok < a.V
                   ? Vec16<T>::load1(static_cast<const T *>(a.logits) + (long long)row * a.stride + tok)
                   : INFINITY;
    };

    if (warp == kWarps) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            int it = 0;
            bool go = true;
            for (int row = row0; row < a.N && go; row += row_step) {
                const RowShape<T> s(a, row);
                int lo, hi;
                slice(s, lo, hi);
                for (int v = lo; v < hi; v += kChunk, ++it) {
                    const int at = it % kRing;
                    if (it >= kRing) {
                        uint32_t i = 0;
                        while (go && !tc::mbar_try_wait(empty + at, (it / kRing - 1) & 1))
                            go = !*failed && ++i < kLpPolls;
                        if (!go) {
                            *failed = 1;
                            break;
                        }
                    }
                    const uint32_t bytes = (uint32_t)min(kChunk, hi - v) * 16;
                    tc::mbar_arrive_expect_tx(full + at, bytes);
                    bulk_copy(sm + LpSmem::RING + at * kChunk * 16, s.block + (size_t)v * 16, bytes, full + at);
                }
            }
            // every copy has landed before the shared memory goes
            for (int i = max(0, it - kRing); i < it; ++i)
                if (!tc::mbar_wait_bounded(full + i % kRing, (i / kRing) & 1, kLpPolls)) *failed = 1;
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ rows
        int it = 0, tok = token_of(row0), odd = 0, look = 0;
        float xt = logit_of(row0, tok);
        for (int row = row0; row < a.N; row += row_step, odd ^= 1) {
            // (the next row's token and logit are on their way while this row is done)
            const int next_tok = CLUSTER ? -1 : token_of(row + row_step);
            const RowShape<T> s(a, row);
            int lo, hi;
            slice(s, lo, hi);
            if (tok >= a.V || tok < -1) {
                if (tid == 0 && rank_in == 0) set_status(a.status, MEDUSA_DEV_BAD_TOKEN);
                tok = -1;
            }
            // Tokens before the row's own: logits above xt, in the blocks up to the token's
            // own xt too (above the number below it), less the equal ones in that block
            // from the token on, which are counted back here.
            const int tv = tok >= 0 ? (s.off + tok) / N : -1;
            const typename Lp<T>::Bound after_it = Lp<T>::bound(xt), up_to_it = Lp<T>::bound(Lp<T>::below(xt));
            typename Lp<T>::Count above;
            bool not_before = false;
            if (tid < N && tv >= lo && tv < hi && tv * N - s.off + tid >= tok)
                not_before = logit_of(row, tv * N - s.off + tid) == xt;
            // m: the thread's largest logit; m2: what its sums are relative to, in base 2
            // (-inf: nothing summed yet), at most kLag below the largest
            float m = -INFINITY, m2 = -INFINITY;
            int before = not_before ? -1 : 0;
            float2 S[2] = {}, A[2] = {};
            float T0 = kLowest;  // candidates reach it
            auto grow = [&](float top) {
                m = max_nan(m, top);
                const float n2 = __fmul_rn(top, a.y_scale);
                if (n2 > m2 + kLag && top >= kNothing) {  // m2 = -inf: the first possible token
                    const float d = m2 - n2, f = exp2f(d);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        A[i] = f == 0.f ? make_float2(0.f, 0.f)
                                        : make_float2(f * fmaf(S[i].x, d, A[i].x), f * fmaf(S[i].y, d, A[i].y));
                        S[i] = make_float2(f * S[i].x, f * S[i].y);
                    }
                    m2 = n2;
                }
            };
            // Counters of this row.  The row before has done with its own, and with what is
            // kept, behind the first barrier of this row: of T0, or here.
            int *n_kept = counts + 2 * odd, *n_cand = n_kept + 1;
            auto other_counters = [&] {
                if (tid == 0) counts[2 * (odd ^ 1)] = counts[2 * (odd ^ 1) + 1] = 0;
            };
            if (lo >= hi) {
                consumers_sync();
                other_counters();
            }
            auto candidate = [&](float f, int id) {
                if (f >= T0) {
                    const int at = atomicAdd(n_cand, 1);
                    if (at < kCandidates) cand[at] = key_of(f, id);
                }
            };
            for (int v0 = lo; v0 < hi; v0 += kChunk, ++it) {
                const int at = it % kRing;
                uint32_t polls = 0;
                while (!tc::mbar_try_wait(full + at, (it / kRing) & 1))
                    if (*failed || ++polls == kLpPolls) {
                        *failed = 1;
                        break;
                    }
                const uint4 *src = reinterpret_cast<const uint4 *>(sm + LpSmem::RING + at * kChunk * 16);
                uint4 w[kPer];
#pragma unroll
                for (int u = 0; u < kPer; ++u)
                    w[u] = v0 + u * kConsumers + tid < hi ? src[u * kConsumers + tid] : Lp<T>::nothing();
                typename Lp<T>::Top vm[kPer], all;
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    vm[u] = Lp<T>::top(w[u]);
                    all = u ? Lp<T>::top(all, vm[u]) : vm[u];
                }
                const float top = Lp<T>::number(all);
                grow(top);
                const int chunk = (v0 - lo) / kChunk;
                if (a.top && (chunk & (chunk + 1)) == 0 && (chunk == 0 || v0 + kChunk < hi)) {
                    // (two places by turns: a warp may be a look ahead of another)
                    float *gm = group_max + look * kWarps * 32;
                    look ^= 1;
                    gm[warp * 32 + lane] = m;
                    consumers_sync();
                    if (chunk == 0) other_counters();
                    uint32_t mine = 0, best = 0;
#pragma unroll
                    for (int x = 0; x < kWarps; ++x) mine = max(mine, ordered(gm[x * 32 + lane]));
                    // (equal ones go at once: the bound may only be lower)
                    for (int k = 0; k < a.top; ++k) {
                        best = __reduce_max_sync(0xffffffffu, mine);
                        if (mine == best) mine = 0;
                    }
                    if (best) T0 = fmaxf(T0, unordered(best));
                }
                if (m2 > -INFINITY) {
#pragma unroll
                    for (int u = 0; u < kPer; ++u) Lp<T>::add(w[u], a.y_scale, m2, S, A);
                }
                above.start();
#pragma unroll
                for (int u = 0; u < kPer; ++u) above.add(w[u], v0 + u * kConsumers + tid <= tv ? up_to_it : after_it);
                above.end();
                if (top >= T0 && a.top) {
#pragma unroll
                    for (int u = 0; u < kPer; ++u)
                        if (Lp<T>::number(vm[u]) >= T0) {
                            const int at = atomicAdd(n_kept, 1);
                            if (at < kVectors) {
                                kept[at] = w[u];
                                kept_at[at] = (v0 + u * kConsumers + tid) * N - s.off;
                            }
                        }
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(empty + at);
            }
            if (rank_in == 0 && tid < s.edges) {  // the row's ends
                const int id = s.edge(tid);
                const float f = Vec16<T>::load1(static_cast<const T *>(a.logits) + (long long)row * a.stride + id);
                grow(f);
                if (m2 > -INFINITY) {
                    const float t = fmaf(fmaxf(f, kLowest), a.y_scale, -m2), p = ex2_approx(t);
                    S[0].x += p;
                    A[0].x = fmaf(p, t, A[0].x);
                }
                before += f > xt || (f == xt && id < tok);
                if (a.top) candidate(f, id);
            }
            const float next_xt = CLUSTER ? 0.f : logit_of(row + row_step, next_tok);
            // ---- the CTA's part: the reference first, then plain sums
            float top;
            asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;\n" : "=f"(top) : "f"(m));
            if (lane == 0) red[warp] = top;
            consumers_sync();
            top = red[0];
#pragma unroll
            for (int x = 1; x < kWarps; ++x) top = max_nan(top, red[x]);
            // the kept vectors' elements that reach T0
            bool many = false;
            if (a.top) {
                const int n = *n_kept;
                many = n > kVectors;
                for (int i = tid; i < min(n, kVectors) * N; i += kConsumers)
                    candidate(Lp<T>::value(reinterpret_cast<const T *>(kept)[i]), kept_at[i / N] + i % N);
            }
            float sum = 0.f, asum = 0.f;
            if (m2 > -INFINITY) {
                const float d = m2 - __fmul_rn(top, a.y_scale), f = exp2f(d);
                sum = (S[0].x + S[0].y) + (S[1].x + S[1].y);
                asum = f * fmaf(sum, d, (A[0].x + A[0].y) + (A[1].x + A[1].y));
                sum *= f;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                asum += __shfl_xor_sync(0xffffffffu, asum, o);
            }
            before = __reduce_add_sync(0xffffffffu, before + above.total());
            if (lane == 0) {
                red[kWarps + warp] = sum;
                red[2 * kWarps + warp] = asum;
                red[3 * kWarps + warp] = __int_as_float(before);
            }
            consumers_sync();
            sum = red[kWarps];
            asum = red[2 * kWarps];
            before = __float_as_int(red[3 * kWarps]);
#pragma unroll
            for (int x = 1; x < kWarps; ++x) {
                sum += red[kWarps + x];
                asum += red[2 * kWarps + x];
                before += __float_as_int(red[3 * kWarps + x]);
            }
            int n = *n_cand;
            many = many || n > kCandidates;
            if (many) n = 0;
            // places of the candidates in the order
            auto place_of = [&](uint64_t c) {
                int p = 0;
#pragma unroll 4
                for (int i = 0; i < n; ++i) p += cand[i] > c;
                return p;
            };
            if constexpr (CLUSTER) {
                if (tid < a.top) part->key[tid] = 0;
                consumers_sync();
                for (int i = tid; i < n; i += kConsumers) {
                    const uint64_t c = cand[i];
                    const int p = place_of(c);
                    if (p < a.top) part->key[p] = c;
                }
                if (tid == 0) {
                    part->m = top;
                    part->S = sum;
                    part->A = asum;
                    part->before = before;
                    part->n = many ? -1 : min(n, a.top);
                }
                break;  // (to the cluster's barriers, which are for all its warps)
            } else {
                if (fast_form(a, top, many, n, tok, xt)) {
                    const LogP logp_of(a, top, sum);
                    if (tid == 0) {
                        a.logp[row] = tok < 0 ? 0.f : logp_of(xt);
                        a.rank[row] = tok < 0 ? -1 : before;
                        a.entropy[row] = fmaxf(kLn2 * (logp_of.ls - asum / sum), 0.f);
                    }
                    if (a.top)
                        for (int i = tid; i < n; i += kConsumers) {
                            const uint64_t c = cand[i];
                            const int p = place_of(c);
                            if (p < a.top) {
                                a.top_ids[(size_t)row * a.top + p] = key_id(c);
                                a.top_logp[(size_t)row * a.top + p] = logp_of(key_logit(c));
                            }
                        }
                } else {
                    slow_row<T>(a, row, tok, red, reinterpret_cast<int *>(group_max));
                }
                tok = next_tok;
                xt = next_xt;
            }
        }
    }
    if constexpr (CLUSTER) {
        __syncthreads();
        cluster_sync();  // every part is written
        if (rank_in == 0 && warp < kWarps) {
            const int row = row0;
            int tok = a.tokens[row];
            if (tok >= a.V || tok < -1) tok = -1;
            const float xt = logit_of(row, tok);
            const RowPart *p = cluster_ptr(part, lane < C ? lane : 0);
            const bool mine = lane < C;
            const float m = mine ? p->m : -INFINITY;
            float top = m, sum = 0.f, asum = 0.f;
            int before = mine ? p->before : 0, n = mine ? p->n : 0;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = __shfl_sync(0xffffffffu, top, 0);
            if (mine && m >= kNothing) {
                const float d = __fmul_rn(m, a.y_scale) - __fmul_rn(top, a.y_scale), f = exp2f(d);
                sum = f * p->S;
                asum = f * fmaf(p->S, d, p->A);
            }
            const bool many = __any_sync(0xffffffffu, n < 0);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                asum += __shfl_xor_sync(0xffffffffu, asum, o);
                before += __shfl_xor_sync(0xffffffffu, before, o);
                n += __shfl_xor_sync(0xffffffffu, n, o);
            }
            sum = __shfl_sync(0xffffffffu, sum, 0);
            asum = __shfl_sync(0xffffffffu, asum, 0);
            before = __shfl_sync(0xffffffffu, before, 0);
            n = __shfl_sync(0xffffffffu, n, 0);
            if (fast_form(a, top, many, n, tok, xt)) {
                const LogP logp_of(a, top, sum);
                if (tid == 0) {
                    a.logp[row] = tok < 0 ? 0.f : logp_of(xt);
                    a.rank[row] = tok < 0 ? -1 : before;
                    a.entropy[row] = fmaxf(kLn2 * (logp_of.ls - asum / sum), 0.f);
                }
                // the parts' first tokens, gathered, then placed as the candidates are
                if (tid < C * a.top) cand[tid] = cluster_ptr(part, tid / a.top)->key[tid % a.top];
                consumers_sync();
                if (tid < C * a.top) {
                    const uint64_t c = cand[tid];
                    int at = 0;
                    for (int i = 0; i < C * a.top; ++i) at += cand[i] > c;
                    if (at < a.top && c) {
                        a.top_ids[(size_t)row * a.top + at] = key_id(c);
                        a.top_logp[(size_t)row * a.top + at] = logp_of(key_logit(c));
                    }
                }
            } else {
                slow_row<T>(a, row, tok, red, reinterpret_cast<int *>(group_max));
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while its part may be read
    }
    if (tid == 0 && *failed) set_status(a.status, MEDUSA_DEV_TIMEOUT);
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
    a.N = N;
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
    // CTAs a row: as many as fit at once, none with less than a chunk
    const int slots = kLpCtas * device_sm_count();
    const int chunks = (int)(((long long)V * (dtype == MEDUSA_F32 ? 4 : 2) + kChunk * 16 - 1) / (kChunk * 16));
    int C = 1;
    while (C < kMaxCluster && (long long)N * C * 2 <= slots && 2 * C <= chunks) C *= 2;
    auto kern = dtype == MEDUSA_F32
                    ? (C > 1 ? token_logprobs_kernel<float, true> : token_logprobs_kernel<float, false>)
                    : (C > 1 ? token_logprobs_kernel<bf16, true> : token_logprobs_kernel<bf16, false>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LpSmem::TOTAL);
    if (e) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C > 1 ? N * C : std::min(N, slots));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = LpSmem::TOTAL;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, a, C);
    note_launch();
    return e;
}

}  // namespace medusa
