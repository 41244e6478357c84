// logprobs.cu -- log probabilities of given tokens, with their ranks, the entropy
// of each row and its top alternatives, in one pass over the logits.
//
// Row x of V logits, temperature T, token t, y = x log2(e) / T, m the row's largest y:
//     S = sum 2^(y - m),  A = sum 2^(y - m) (y - m)
//     logp = ln2 (y_t - m - log2 S)       entropy = ln2 (log2 S - A / S)
//     rank = number of tokens before t in the order (larger logit, then smaller id)
//     alternatives: the first `top` tokens of that order
//
// A CTA takes a row at a time, in chunks of 1024 16-byte vectors; with few rows a
// cluster of CTAs shares each row.
//   warps 0-3  a thread keeps the largest logit of its vectors, and S and A relative to
//              a reference of its own, which moves when a chunk's maximum (packed, NaNs
//              kept) exceeds it by 2^8.  References in base 2 are rounded by products
//              that are not fused, so that all sums are relative to the same number.
//              Ranks are packed comparisons with the token's logit, or up to its place
//              with the number below it.
//   warp 4     bulk copies into a ring of three chunks.  A wait whose polls run out sets the
//              status, and the rows from there on get NaN
//   warp 5     ends a row while the others are at the next: it joins the threads' sums,
//              and finds the alternatives.  The k-th largest of 32 groups of threads'
//              maxima (T0) is at most the row's k-th largest logit.  The few threads
//              whose maximum reaches it have their vectors of that chunk read again
//              (from L2; of the whole row where the largest of their other chunks
//              reaches it as well), the elements that reach it are the candidates, and
//              a candidate's place in the order is the number of better ones among them.
//
// What this form does not take (a NaN or +inf in the row, a largest y outside -2^29 .. 2^30,
// the token at -inf, too many candidates because of ties, fewer possible tokens than
// alternatives, temperatures below 1.44e-7 or above 1.44e18) is done by slow_row, by plain
// passes of one warp over the row: the results are the same by definition, at 50 us a pass of
// 32000 logits (10 alternatives: 65 such rows 620 us for 24, 4093 of them 4.9 ms for 74).
//
// Bound by issue (50 % of the slots over a launch, 67 % while all four CTAs of an SM are
// in their rows): conversions, two packed products, an exponential and two packed sums an
// element.  4093 x 32000 bf16 (262 MB): 51.4 us without alternatives, 5.1 TB/s, 61.8 with 10;
// 2048 x 50257 fp32 (412 MB) with 10: 74.9, 5.5 TB/s; 301 of them 16.0; 65 x 32000: 5.0, with 5
// 7.7, a chain of copies, sums, the cluster's join and the second read.
// Against it, with 10 alternatives: a pass for each result 1164; one pass with 256 summing
// threads 121, four warps and kept vectors 100; counts of elements one by one 82, references
// that follow every chunk's maximum 77; rows ended by the warps that sum 70; all of a row read
// again for the candidates 69.
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace medusa {

namespace {

constexpr int kConsumers = 128, kWarps = kConsumers / 32, kLpThreads = kConsumers + 64;
// (chunks of 512 with six CTAs an SM: 68 us for 4093 x 32000 with 10 alternatives, these
// 60.5; two rounds of rows of which the last is even, at six CTAs, 75)
constexpr int kChunk = 1024, kPer = kChunk / kConsumers;  // vectors of a chunk, of a thread
constexpr int kRing = 3, kLpCtas = 4;
constexpr int kCandidates = 256;
constexpr int kMaxCluster = 4;  // 65 x 32000: 7.0 us, with 8 8.5
constexpr uint32_t kLpDrain = 1u << 16;  // polls for a CTA's own copies before its shared memory goes
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -1e30f, kLag = 8.f;
// References in base 2.  One of 2^30 is off by up to 32, and weights relative to it reach 2^32
// (2^40 with kLag); further out they would leave fp32 (2^439 at a logit of -1e10).  Below -kFar
// a thread sums nothing, which is nothing beside a row's largest of -kFar / 2 at least.
constexpr float kFar = 0x1p30f;
constexpr float kMostScale = 1e7f, kLeastScale = 1e-18f;  // log2(e) / T
static_assert(kMaxCluster * MEDUSA_MAX_TOP_S <= kCandidates, "the parts' lists");

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
    uint32_t wait_polls;  // after which a wait gives up
};

// What a CTA of a cluster knows of its part of a row.
struct RowPart {
    float m;       // largest logit (NaN if there is one)
    float S, A;    // relative to m
    int before, n; // tokens before the row's token; candidates (-1: too many, kLost)
    uint64_t key[MEDUSA_MAX_TOP_S];  // the part's first tokens (0: none)
};

constexpr int kLost = -2;  // a wait for the row's logits ran out

// A thread's share of a row: the largest logit of its vectors, the chunk that holds it (or
// kLost), the largest of the other chunks; its sums and their reference in base 2.
struct Sums {
    float m, other;
    int chunk;
    float m2, S, A;
    int before;
};

struct LpSmem {
    static constexpr int RING = 0;
    static constexpr int CAND = kRing * kChunk * 16;  // candidates: see key_of
    static constexpr int VECTORS = CAND + kCandidates * 8;  // that hold them
    static constexpr int PART = VECTORS + kCandidates * 4;
    static constexpr int SUMS = PART + (int)(sizeof(RowPart) + 15) / 16 * 16;  // of the threads
    static constexpr int COLUMNS = SUMS + kConsumers * (int)sizeof(Sums);      // [kConsumers]
    static constexpr int BAR = (COLUMNS + kConsumers * 4 + 7) / 8 * 8;
    static constexpr int WORDS = BAR + 2 * kRing * 8;  // vectors; failed; beat
    static constexpr int TOTAL = WORDS + 32;
    static_assert(kLpCtas * (TOTAL + 1024) <= 228 * 1024, "CTAs of an SM");
};

// Barriers between the warps that sum and the one that ends rows: the sums of a row
// are there, and they have been read.
template <int ID>
__device__ __forceinline__ void row_arrive() {
    asm volatile("barrier.cta.arrive %0, %1;\n" ::"n"(ID), "n"(kConsumers + 32) : "memory");
}
template <int ID>
__device__ __forceinline__ void row_sync() {
    asm volatile("barrier.cta.sync %0, %1;\n" ::"n"(ID), "n"(kConsumers + 32) : "memory");
}
constexpr int kSummed = 1, kRead = 2;

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
        static_assert(4 * kPer <= 256, "a chunk's count in a half is exact in bf16");
        __device__ __forceinline__ void end() {  // (2^24 in all are exact as well)
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

// f(i) for the lane's share of the row's logits.  `beat` goes on with every kBeat of them, some
// 50 us where all SMs are at this.
constexpr int kBeat = 4096;
template <typename F>
__device__ __forceinline__ void each_logit(int V, volatile int *beat, F f) {
    const int lane = threadIdx.x & 31;
    for (int at = 0; at < V; at += kBeat) {
        const int end = min(at + kBeat, V);
#pragma unroll 8
        for (int i = at + lane; i < end; i += 32) f(i);
        if (lane == 0) *beat = *beat + 1;
    }
}

// A sum that carries what its last addition lost: off by two roundings, however many terms.
struct LongSum {
    float s = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float y = x - lost, t = s + y;
        lost = (t - s) - y;
        s = t;
    }
};

// A row by the definition, by one warp: a pass for the maximum, one for the sums, one
// for each alternative.
template <typename T>
__device__ __noinline__ void slow_row(const LogprobArgs &a, int row, int tok, volatile int *beat) {
    const int lane = threadIdx.x & 31;
    const T *x = static_cast<const T *>(a.logits) + (long long)row * a.stride;
    const float xt = tok >= 0 ? Vec16<T>::load1(x + tok) : NAN;
    float m = -INFINITY;
    bool bad = false;  // +inf or NaN in the row
    each_logit(a.V, beat, [&](int i) {
        const float f = Vec16<T>::load1(x + i);
        m = fmaxf(m, f);
        bad = bad || !(f < INFINITY);
    });
    bad = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    LongSum S_lane, A_lane;  // (a lane adds V / 32 terms)
    int before = 0;
    each_logit(a.V, beat, [&](int i) {
        const float f = Vec16<T>::load1(x + i);
        const float t = fmaxf((f - m) * a.y_scale, -127.f), p = ex2_approx(t);
        S_lane.add(p);
        A_lane.add(p * t);
        before += f > xt || (f == xt && i < tok);
    });
    const float S = warp_sum(S_lane.s), A = warp_sum(A_lane.s);
    before = __reduce_add_sync(0xffffffffu, before);
    const bool none = m == -INFINITY;  // nothing is possible
    const float ls = log2f(S);
    // (halves: logits may lie further apart than fp32 reaches)
    auto logp_of = [&](float f) {
        return bad ? NAN : none ? -INFINITY : (0.5f * f - 0.5f * m) * (2.f * a.inv_T) - ls * kLn2;
    };
    if (lane == 0) {
        a.logp[row] = tok < 0 ? 0.f : logp_of(xt);
        a.rank[row] = tok < 0 || isnan(xt) ? -1 : before;
        a.entropy[row] = bad ? NAN : none ? 0.f : fmaxf(kLn2 * (ls - A / S), 0.f);
    }
    uint64_t last = ~0ull;  // the alternative before
    for (int k = 0; k < a.top; ++k) {
        uint64_t best = 0;
        if (last)
            each_logit(a.V, beat, [&](int i) {
                const float f = Vec16<T>::load1(x + i);
                const uint64_t c = isnan(f) ? 0 : key_of(f, i);
                if (c < last && c > best) best = c;
            });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t c = __shfl_xor_sync(0xffffffffu, (unsigned long long)best, o);
            if (c > best) best = c;
        }
        if (lane == 0) {
            a.top_ids[(size_t)row * a.top + k] = best ? key_id(best) : -1;
            a.top_logp[(size_t)row * a.top + k] = best ? logp_of(key_logit(best)) : NAN;
        }
        last = best;
    }
}

__device__ __forceinline__ void bulk_copy(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                     tc::smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_addr(bar))
                 : "memory");
}

// A row whose logits did not come: nothing is said of it.
__device__ __forceinline__ void lost_row(const LogprobArgs &a, int row) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        a.logp[row] = a.entropy[row] = NAN;
        a.rank[row] = -1;
    }
    if (lane < a.top) {
        a.top_ids[(size_t)row * a.top + lane] = -1;
        a.top_logp[(size_t)row * a.top + lane] = NAN;
    }
}

// Wait of a converged warp for a chunk; false: the polls or another warp's ran out.
__device__ __forceinline__ bool wait_chunk(uint64_t *bar, uint32_t parity, uint32_t limit, volatile int *failed) {
    for (uint32_t i = 0; i < limit; ++i) {
        if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *failed)) return false;
    }
    *failed = 1;
    return false;
}

// What the one pass holds for; otherwise slow_row.  Below kLeastScale (temperatures above
// 1.4e18) kLowest, to which smaller logits and -inf are lifted, would no longer lie far below a
// largest y of -kFar / 2 or above: there it does, by 1e30 kLeastScale - kFar / 2 > 9e11.
__device__ __forceinline__ bool fast_form(const LogprobArgs &a, float top, bool many, int n, int tok, float xt) {
    const float t2 = __fmul_rn(top, a.y_scale);
    return t2 >= -kFar / 2 && t2 <= kFar && !many && n >= a.top && (tok < 0 || xt > -INFINITY) &&
           a.y_scale <= kMostScale && a.y_scale >= kLeastScale;
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
    uint64_t *cand = reinterpret_cast<uint64_t *>(sm + LpSmem::CAND);
    RowPart *part = reinterpret_cast<RowPart *>(sm + LpSmem::PART);
    Sums *sums = reinterpret_cast<Sums *>(sm + LpSmem::SUMS);
    int *columns = reinterpret_cast<int *>(sm + LpSmem::COLUMNS);
    int *vectors = reinterpret_cast<int *>(sm + LpSmem::VECTORS), *n_vec = reinterpret_cast<int *>(sm + LpSmem::WORDS);
    volatile int *failed = reinterpret_cast<volatile int *>(n_vec + 1), *beat = failed + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank_in = CLUSTER ? (int)cluster_rank() : 0;
    const int row0 = CLUSTER ? (int)blockIdx.x / C : blockIdx.x, row_step = CLUSTER ? a.N : gridDim.x;
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(full + i, 1);
            tc::mbar_init(empty + i, kWarps);
        }
        *failed = *beat = 0;
        tc::fence_mbarrier_init();
    }
    __syncthreads();
    auto slice = [&](const RowShape<T> &s, int &lo, int &hi) {
        lo = s.first;
        hi = s.last;
        if constexpr (CLUSTER) {
            const int per = (hi - lo + C - 1) / C;
            lo = min(lo + rank_in * per, hi);
            hi = min(lo + per, hi);
        }
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
                        // (a row by plain passes may hold this place up for longer than the
                        // polls last, 0.1 to 1.4 us each: they count from its last beat)
                        int seen = *beat;
                        go = false;
                        for (uint32_t i = 0; i < a.wait_polls && !go && !*failed; ++i) {
                            go = tc::mbar_try_wait(empty + at, (it / kRing - 1) & 1);
                            if (const int now = *beat; now != seen) {
                                seen = now;
                                i = 0;
                            }
                        }
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
                if (!tc::mbar_wait_bounded(full + i % kRing, (i / kRing) & 1, kLpDrain)) *failed = 1;
        }
        __syncwarp();
    } else if (warp < kWarps) {
        // -------------------------------------------------------------- sums
        // (it: the chunk's number, or kLost for good once a wait of the warp has run out)
        int it = 0, tok = token_of(row0), next_tok = CLUSTER ? -1 : token_of(row0 + row_step);
        float xt = logit_of(row0, tok);
        for (int row = row0; row < a.N; row += row_step) {
            // (the next row's logit, and the token after it, are on their way while this row is
            // done)
            const float next_xt = CLUSTER ? 0.f : logit_of(row + row_step, next_tok);
            const int tok_after = CLUSTER ? -1 : token_of(row + 2 * row_step);
            const RowShape<T> s(a, row);
            int lo, hi;
            slice(s, lo, hi);
            if (tok >= a.V || tok < 0) {
                tok = -1;
                xt = INFINITY;
            }
            // Tokens before the row's own: logits above xt, in the blocks up to the token's
            // own xt too (above the number below it); the equal ones of that block from the
            // token on are counted back at the row's end.
            const int tv = tok >= 0 ? (s.off + tok) / N : -1;
            const typename Lp<T>::Bound after_it = Lp<T>::bound(xt), up_to_it = Lp<T>::bound(Lp<T>::below(xt));
            typename Lp<T>::Count above;
            // m2: what the sums are relative to, in base 2 (-inf: nothing summed yet), at
            // most kLag below the largest, and -kFar or above
            float m = -INFINITY, other = -INFINITY, m2 = -INFINITY;
            int before = 0, chunk = 0;
            float2 S[2] = {}, A[2] = {};
            auto grow = [&](float top) {
                const float n2 = __fmul_rn(top, a.y_scale);
                if (n2 > m2 + kLag && n2 >= -kFar) {  // m2 = -inf: the first token that counts
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
            for (int v0 = lo; v0 < hi; v0 += kChunk, ++it) {
                const int at = it % kRing;
                if (it < 0 || !wait_chunk(full + at, (it / kRing) & 1, a.wait_polls, failed)) {
                    it = chunk = kLost;
                    break;
                }
                const uint4 *src = reinterpret_cast<const uint4 *>(sm + LpSmem::RING + at * kChunk * 16);
                uint4 w[kPer];
#pragma unroll
                for (int u = 0; u < kPer; ++u)
                    w[u] = v0 + u * kConsumers + tid < hi ? src[u * kConsumers + tid] : Lp<T>::nothing();
                typename Lp<T>::Top all = Lp<T>::top(w[0]);
#pragma unroll
                for (int u = 1; u < kPer; ++u) all = Lp<T>::top(all, Lp<T>::top(w[u]));
                const float top = Lp<T>::number(all);
                other = fmaxf(other, fminf(m, top));
                if (top > m) chunk = (v0 - lo) / kChunk;
                m = max_nan(m, top);
                grow(top);
                if (m2 > -INFINITY) {
#pragma unroll
                    for (int u = 0; u < kPer; ++u) Lp<T>::add(w[u], a.y_scale, m2, S, A);
                }
                above.start();
#pragma unroll
                for (int u = 0; u < kPer; ++u) above.add(w[u], v0 + u * kConsumers + tid <= tv ? up_to_it : after_it);
                above.end();
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
            }
            if (row != row0) row_sync<kRead>();  // the sums of the row before
            sums[tid] = Sums{m, other, chunk, m2, (S[0].x + S[0].y) + (S[1].x + S[1].y), (A[0].x + A[0].y) + (A[1].x + A[1].y),
                             before + above.total()};
            row_arrive<kSummed>();
            tok = next_tok;
            next_tok = tok_after;
            xt = next_xt;
        }
    } else {
        // ----------------------------------------------------------- rows' ends
        for (int row = row0; row < a.N; row += row_step) {
            const RowShape<T> s(a, row);
            int lo, hi;
            slice(s, lo, hi);
            int tok = token_of(row);
            if (tok >= a.V || tok < -1) {
                if (lane == 0 && rank_in == 0) set_status(a.status, MEDUSA_DEV_BAD_TOKEN);
                tok = -1;
            }
            const float xt = logit_of(row, tok);
            // equal logits of the token's block from the token on
            const int tv = tok >= 0 ? (s.off + tok) / N : -1, beside = tv * N - s.off + lane;
            const bool back = lane < N && tv >= lo && tv < hi && beside >= tok && logit_of(row, beside) == xt;
            const bool at_edge = rank_in == 0 && lane < s.edges;
            const float f_edge = at_edge ? logit_of(row, s.edge(lane)) : 0.f;
            row_sync<kSummed>();
            Sums x[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) x[w] = sums[w * 32 + lane];
            if (row + row_step < a.N) row_arrive<kRead>();
            const bool lost = __any_sync(0xffffffffu, (x[0].chunk | x[1].chunk | x[2].chunk | x[3].chunk) < 0);
            if (!CLUSTER && lost) {
                lost_row(a, row);
                continue;
            }
            float top = max_nan(max_nan(x[0].m, x[1].m), max_nan(x[2].m, x[3].m));
            static_assert(kWarps == 4, "four shares a lane");
            if (at_edge) top = max_nan(top, f_edge);
            asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;\n" : "=f"(top) : "f"(top));
            const float t2 = __fmul_rn(top, a.y_scale);
            float sum = 0.f, asum = 0.f;
            int before = back ? -1 : 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                before += x[w].before;
                if (x[w].m2 > -INFINITY) {
                    const float d = x[w].m2 - t2, f = exp2f(d);
                    sum = fmaf(f, x[w].S, sum);
                    asum = fmaf(f, fmaf(x[w].S, d, x[w].A), asum);
                }
            }
            sum = warp_sum(sum);
            asum = warp_sum(asum);
            before = __reduce_add_sync(0xffffffffu, before);
            int n = 0;
            if (a.top && !(CLUSTER && lost)) {
                float mine = -INFINITY;  // (NaNs are left out: such a row is not done here)
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mine = fmaxf(mine, x[w].m);
                int place = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float o = __shfl_sync(0xffffffffu, mine, i);
                    place += o > mine || (o == mine && i < lane);
                }
                const uint32_t kth = __ballot_sync(0xffffffffu, place == a.top - 1);
                const float T0 = fmaxf(kth ? __shfl_sync(0xffffffffu, mine, __ffs(kth) - 1) : kLowest, kLowest);
                int n_col = 0;  // the threads that reach it
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const bool is = x[w].m >= T0;
                    const uint32_t who = __ballot_sync(0xffffffffu, is);
                    if (is) columns[n_col + __popc(who & ((1u << lane) - 1))] = w * 32 + lane + x[w].chunk * kChunk;
                    n_col += __popc(who);
                }
                if (lane == 0) *n_vec = 0;
                __syncwarp();
                const uint4 *blocks = reinterpret_cast<const uint4 *>(s.block);
                auto keep = [&](int v) {
                    const int at = atomicAdd(n_vec, 1);
                    if (at < kCandidates) vectors[at] = v;
                };
                constexpr int kAhead = 4;
                for (int i0 = lane; i0 - lane < n_col * kPer; i0 += 32 * kAhead) {
                    uint4 y[kAhead];
                    int v[kAhead];
#pragma unroll
                    for (int q = 0; q < kAhead; ++q) {
                        const int i = i0 + 32 * q;
                        v[q] = i < n_col * kPer ? lo + columns[i / kPer] + i % kPer * kConsumers : hi;
                        y[q] = v[q] < hi ? __ldg(blocks + v[q]) : Lp<T>::nothing();
                    }
#pragma unroll
                    for (int q = 0; q < kAhead; ++q)
                        if (Lp<T>::number(Lp<T>::top(y[q])) >= T0) keep(v[q]);
                }
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    for (uint32_t who = __ballot_sync(0xffffffffu, x[w].other >= T0); who; who &= who - 1) {
                        const int t = __ffs(who) - 1, done = __shfl_sync(0xffffffffu, x[w].chunk, t);
                        for (int v = lo + w * 32 + t + lane * kConsumers; v < hi; v += 32 * kConsumers)
                            if ((v - lo) / kChunk != done && Lp<T>::number(Lp<T>::top(__ldg(blocks + v))) >= T0) keep(v);
                    }
                __syncwarp();
                // the candidates, numbered by the warp
                auto candidates = [&](bool is, float f, int id) {
                    const uint32_t who = __ballot_sync(0xffffffffu, is && f >= T0);
                    const int at = n + __popc(who & ((1u << lane) - 1));
                    if (is && f >= T0 && at < kCandidates) cand[at] = key_of(f, id);
                    n += __popc(who);
                };
                const int nv = *n_vec;
                if (nv > kCandidates) n = kCandidates + 1;
                for (int i = lane; i - lane < nv * N && nv <= kCandidates; i += 32) {
                    const bool is = i < nv * N;
                    const int id = is ? vectors[i / N] * N - s.off + i % N : 0;
                    candidates(is, is ? logit_of(row, id) : 0.f, id);
                }
                if (s.edges) candidates(at_edge, f_edge, s.edge(lane));
                __syncwarp();
            }
            const bool many = n > kCandidates;
            if (many) n = 0;
            // places of the candidates in the order
            auto place_of = [&](uint64_t c, int n) {
                int p = 0;
#pragma unroll 4
                for (int i = 0; i < n; ++i) p += cand[i] > c;
                return p;
            };
            auto finish = [&](bool many, int n) {
                if (!fast_form(a, top, many, n, tok, xt)) {
                    slow_row<T>(a, row, tok, beat);
                    return;
                }
                const LogP logp_of(a, top, sum);
                if (lane == 0) {
                    a.logp[row] = tok < 0 ? 0.f : logp_of(xt);
                    a.rank[row] = tok < 0 ? -1 : before;
                    a.entropy[row] = fmaxf(kLn2 * (logp_of.ls - asum / sum), 0.f);
                }
                for (int i = lane; i < n; i += 32) {
                    const uint64_t c = cand[i];
                    const int p = place_of(c, n);
                    if (p < a.top && c) {
                        a.top_ids[(size_t)row * a.top + p] = key_id(c);
                        a.top_logp[(size_t)row * a.top + p] = logp_of(key_logit(c));
                    }
                }
                __syncwarp();
            };
            if constexpr (CLUSTER) {
                if (lane < a.top) part->key[lane] = 0;
                __syncwarp();
                for (int i = lane; i < n; i += 32) {
                    const uint64_t c = cand[i];
                    const int p = place_of(c, n);
                    if (p < a.top) part->key[p] = c;
                }
                if (lane == 0) {
                    part->m = top;
                    part->S = sum;
                    part->A = asum;
                    part->before = before;
                    part->n = lost ? kLost : many ? -1 : min(n, a.top);
                }
                cluster_arrive();  // the part is written
                cluster_wait();
                if (rank_in == 0) {
                    const RowPart *p = cluster_ptr(part, lane < C ? lane : 0);
                    const bool mine = lane < C;
                    const float m = mine ? p->m : -INFINITY;
                    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;\n" : "=f"(top) : "f"(m));
                    sum = asum = 0.f;
                    if (mine && __fmul_rn(m, a.y_scale) >= -kFar) {  // (something was summed)
                        const float d = __fmul_rn(m, a.y_scale) - __fmul_rn(top, a.y_scale), f = exp2f(d);
                        sum = f * p->S;
                        asum = f * fmaf(p->S, d, p->A);
                    }
                    sum = warp_sum(sum);
                    asum = warp_sum(asum);
                    before = __reduce_add_sync(0xffffffffu, mine ? p->before : 0);
                    n = mine ? p->n : 0;
                    const bool over = __any_sync(0xffffffffu, n < 0), gone = __any_sync(0xffffffffu, n == kLost);
                    n = __reduce_add_sync(0xffffffffu, n);
                    if (!gone && fast_form(a, top, over, n, tok, xt)) {
                        // the parts' first tokens, gathered, then placed as the candidates are
                        for (int i = lane; i < C * a.top; i += 32)
                            cand[i] = cluster_ptr(part, i / a.top)->key[i % a.top];
                        n = C * a.top;
                        __syncwarp();
                    }
                    if (gone)
                        lost_row(a, row);
                    else
                        finish(over, n);
                }
                __syncwarp();
            } else {
                finish(many, n);
            }
        }
    }
    if constexpr (CLUSTER) {
        if (warp != kWarps + 1) {
            cluster_arrive();
            cluster_wait();
        }
        cluster_arrive();  // no CTA leaves while its part may be read
        cluster_wait();
    }
    __syncthreads();
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
    a.wait_polls = wait_budget();
    // CTAs a row: as many as run at once, none with less than a chunk, or than three chunks
    // where half the SMs have a row of their own.  Rows of 4 chunks (32000 in bf16): 65 of
    // them 7.8 us with one CTA a row and 7.1 with four, 100 8.0 and 8.0, 200 9.6 and (two CTAs)
    // 10.5; of 16 chunks: 65 22.8 and 14.0, 300 28.3 and (two) 23.8.  Clusters of four get no more than
    // about 5/6 of the places: 125 of them 8.3 us, 150 14.2.
    const int slots = kLpCtas * device_sm_count(), least = 2 * N > device_sm_count() ? 3 : 1;
    const int chunks = (int)(((long long)V * (dtype == MEDUSA_F32 ? 4 : 2) + kChunk * 16 - 1) / (kChunk * 16));
    int C = 1;
    while (C < kMaxCluster && (long long)N * C * 2 <= (C == 1 ? slots : slots * 5 / 6) && 2 * C * least <= chunks) C *= 2;
    auto kern = dtype == MEDUSA_F32
                    ? (C > 1 ? token_logprobs_kernel<float, true> : token_logprobs_kernel<float, false>)
                    : (C > 1 ? token_logprobs_kernel<bf16, true> : token_logprobs_kernel<bf16, false>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LpSmem::TOTAL);
    if (e) return e;
    // (as many rows for each CTA, rather than a last round of a few)
    const int rounds = (N + slots - 1) / slots;
    const dim3 grid(C > 1 ? N * C : (N + rounds - 1) / rounds), block(kLpThreads);
    e = C > 1 ? launch_pdl_cluster(kern, grid, block, dim3(C), LpSmem::TOTAL, stream, a, C)
              : launch_pdl(kern, grid, block, LpSmem::TOTAL, stream, a, C);
    note_launch();
    return e;
}

}  // namespace medusa
