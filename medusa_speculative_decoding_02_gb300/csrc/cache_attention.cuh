// cache_attention.cuh -- what the attention kernels over the caches share: the
// arguments of a launch, the numbering of the visible keys, the checks.
#pragma once

#include "kv4.cuh"
#include "launch.h"

namespace medusa {

constexpr float kLog2e = 1.4426950408889634f;

struct CacheAttnArgs {
    const void *q;
    const void *const *kc;
    const void *const *vc;
    const int32_t *prefix_len;
    const uint64_t *anc_mask;
    const int32_t *depth;  // null in calls without a window
    int B, R, H, Hkv, P_max;
    int window, sinks;     // 0, 0 where no slot falls out of the window
    int ns, row_tiles;
    float scale_log2;
    uint32_t wait_polls;   // poll limit of the tensor-core path's waits
    float *part_o;         // [B * ns, H, R, dh]
    float2 *part_ml;       // [B * ns, H, R] (m in log2 units, l)
    int *starts;           // [B + 1] first range of each sequence, where they are dealt out
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

// What a CTA works on: keys [kbeg, kend) of sequence b, whose partial result is
// number `range` of the B * ns; kend = 0: a range without keys.
struct CacheItem {
    int b, range, kbeg, kend, P;
    const void *kc, *vc;
};

// Keys of a range on the tensor-core paths are a multiple of this.
constexpr int kRangeUnit = 64;

// The CTA's item.  The host chooses ns, from P_max.  Without DEAL each sequence
// is cut into ns ranges of its own length.  With DEAL (B <= 32) the B * ns
// ranges are dealt out by the sequences' lengths: the shortest range size with
// which all of them together need no more.  The first CTA leaves the first
// numbers of the sequences' ranges for the join.  `len(P)`: numbered keys of a
// prefix of P slots.  Called by whole warps; false: no item for this CTA.
template <bool DEAL, int UNIT = kRangeUnit, typename Len>
__device__ __forceinline__ bool find_item(const CacheAttnArgs &a, Len len, CacheItem &it) {
    const int idx = blockIdx.z * a.ns + blockIdx.y, lane = threadIdx.x & 31;
    it.range = idx;
    if constexpr (!DEAL) {
        it.b = blockIdx.z;
        const bool ok = sequence_ok(a, it.b, it.P, it.kc, it.vc);
        if (!ok) it.P = 0;
        const int n = ok ? len(it.P) : 0;
        const int size = ((n + UNIT - 1) / UNIT + a.ns - 1) / a.ns * UNIT;
        it.kbeg = blockIdx.y * size;
        it.kend = min(it.kbeg + size, n);
        return true;
    }
    int P = 0, units = 0;
    const void *kc = nullptr, *vc = nullptr;
    if (lane < a.B) {
        if (sequence_ok(a, lane, P, kc, vc))
            units = (len(P) + UNIT - 1) / UNIT;
        else
            P = 0;
    }
    const int all = a.B * a.ns;
    // (a range size that max / ns allows is enough for every sequence)
    int lo = max(1, (__reduce_add_sync(0xffffffffu, units) + all - 1) / all);
    int size = max(1, (__reduce_max_sync(0xffffffffu, units) + a.ns - 1) / a.ns);
    while (lo < size) {
        const int mid = (lo + size) >> 1;
        if (__reduce_add_sync(0xffffffffu, (units + mid - 1) / mid) <= all)
            size = mid;
        else
            lo = mid + 1;
    }
    const int n = (units + size - 1) / size;
    int end = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, end, d);
        if (lane >= d) end += y;
    }
    if (idx == 0 && blockIdx.x == 0 && threadIdx.x < a.B) {
        if (threadIdx.x == 0) a.starts[0] = 0;
        a.starts[threadIdx.x + 1] = end;
    }
    const int b = __popc(__ballot_sync(0xffffffffu, idx >= end));
    if (b >= a.B) return false;
    it.b = b;
    it.P = __shfl_sync(0xffffffffu, P, b);
    it.kc = reinterpret_cast<const void *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(kc), b));
    it.vc = reinterpret_cast<const void *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vc), b));
    it.kbeg = (idx - __shfl_sync(0xffffffffu, end - n, b)) * size * UNIT;
    it.kend = min(it.kbeg + size * UNIT, len(it.P));
    return true;
}

// The softmax reference of a row moves only when a maximum exceeds it by 2^8,
// so weights reach 2^8; fp16 weights (4-bit caches) are biased by 2^7.
constexpr float kRescaleLog2 = 8.f;
constexpr float kF16Bias = 7.f;

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

// Kernel for few rows (cache_attention_few.cu): rows a KV head may have, and the
// launch.  At 16 rows, eight sequences of 8192 slots and eight KV heads it takes
// 47.2 us against 50.1 of the 128-row tiles (4 bits 32.5 against 42.5), at 1 row
// 44.6 against 48.5 (23.1 against 42.2), over 1000 slots 10.2 against 14.6.
constexpr int kFewRows = 16;
int cache_few_ctas_per_sm(bool kv4, int rows);
cudaError_t launch_cache_attention_few(const CacheAttnArgs &a, bool kv4, int dh, cudaStream_t stream);

}  // namespace medusa
