// kv4.cu -- rows into and out of the 4-bit cache (layout: kv4.cuh).
//
// kv4_append_kernel: one thread per block of 16 elements of K or V: it reads
// them, picks the scale and the codes and stores eight bytes of codes and one
// scale byte.  Consecutive threads take consecutive blocks of a row, so both
// stores of a warp are contiguous.  kv4_unpack_kernel is the inverse.  Both
// are bound by the bytes they move (per element 2 or 4 bytes on the wide side
// and 9/16 on the narrow one).
#include <algorithm>

#include "kv4.cuh"
#include "launch.h"

namespace medusa {

namespace {

constexpr int kKv4Threads = 256;

struct Kv4Args {
    const void *k, *v;        // wide rows (append: in; unpack: out)
    long long k_stride, v_stride;  // elements between wide rows
    uint8_t *const *kc;
    uint8_t *const *vc;
    const int32_t *prefix_len;
    const int32_t *n_rows;    // or null: all R
    int R, Hkv, dh, P_max;
    int *status;
};

// Row checks shared by both directions: the cache row of wide row i of
// sequence b, or null when there is nothing to do.
__device__ __forceinline__ uint8_t *kv4_row(const Kv4Args &a, int b, int i, bool is_v) {
    if (a.n_rows && i >= a.n_rows[b]) return nullptr;
    uint8_t *kc = a.kc[b], *vc = a.vc[b];
    if (!kc || !vc || ((reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) & 15u)) {
        set_status(a.status, MEDUSA_DEV_BAD_CACHE);
        return nullptr;
    }
    const int P = a.prefix_len[b];
    if (P < 0 || P > a.P_max) {
        set_status(a.status, MEDUSA_DEV_BAD_PREFIX);
        return nullptr;
    }
    return (is_v ? vc : kc) + (size_t)(P + i) * kv4_row_bytes(a.Hkv, a.dh);
}

template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]) {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int u = 0; u < 16 / N; ++u) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p + u * N);
        float f[N];
        Vec16<T>::widen(w, f);
#pragma unroll
        for (int e = 0; e < N; ++e) x[u * N + e] = f[e];
    }
}

// grid (blocks of a row pair over 256 threads, R, B)
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(Kv4Args a) {
    pdl_enter();
    const int per = a.Hkv * a.dh / 16;  // blocks of a K row, and of a V row
    const int blk = blockIdx.x * kKv4Threads + threadIdx.x;
    if (blk >= 2 * per) return;
    const bool is_v = blk >= per;
    const int e = is_v ? blk - per : blk;
    const int i = blockIdx.y, b = blockIdx.z;
    uint8_t *row = kv4_row(a, b, i, is_v);
    if (!row) return;
    const long long r = (long long)b * a.R + i;
    const T *src = is_v ? static_cast<const T *>(a.v) + r * a.v_stride
                        : static_cast<const T *>(a.k) + r * a.k_stride;
    float x[16];
    load16(src + e * 16, x);
    float amax = 0.f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        amax = fmaxf(amax, fabsf(x[j]));
        finite = finite && fabsf(x[j]) < INFINITY;  // false for NaN too
    }
    uint32_t sb = kE4m3Nan, lo = 0, hi = 0;
    if (finite) {
        sb = kv4_scale_byte(amax);
        if (sb) {
            const float s = e4m3_value(sb);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                lo |= kv4_code(x[j], s) << (4 * j);
                hi |= kv4_code(x[j + 8], s) << (4 * j);
            }
        }
    }
    *reinterpret_cast<uint2 *>(row + e * 8) = make_uint2(lo, hi);
    row[kv4_code_bytes(a.Hkv, a.dh) + e] = (uint8_t)sb;
}

template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_unpack_kernel(Kv4Args a) {
    pdl_enter();
    const int per = a.Hkv * a.dh / 16;
    const int blk = blockIdx.x * kKv4Threads + threadIdx.x;
    if (blk >= 2 * per) return;
    const bool is_v = blk >= per;
    const int e = is_v ? blk - per : blk;
    const int i = blockIdx.y, b = blockIdx.z;
    const uint8_t *row = kv4_row(a, b, i, is_v);
    if (!row) return;
    const long long r = (long long)b * a.R + i;
    T *dst = is_v ? static_cast<T *>(const_cast<void *>(a.v)) + r * a.v_stride
                  : static_cast<T *>(const_cast<void *>(a.k)) + r * a.k_stride;
    dst += e * 16;
    const uint2 c = *reinterpret_cast<const uint2 *>(row + e * 8);
    const __half s =
        __half(__nv_cvt_fp8_to_halfraw(row[kv4_code_bytes(a.Hkv, a.dh) + e], __NV_E4M3));
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t byte = (j < 4 ? c.x : c.y) >> (8 * (j & 3));
        const float2 f = __half22float2(__hmul2(e2m1x2_half2(byte), __half2half2(s)));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            *reinterpret_cast<float4 *>(dst + 4 * u) =
                make_float4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * u], x[2 * u + 1]);
            w[u] = *reinterpret_cast<const uint32_t *>(&p);
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

}  // namespace

cudaError_t launch_kv4_rows(medusa_dtype dtype, bool append, const void *k, const void *v,
                            long long k_stride, long long v_stride, void *const *k_cache,
                            void *const *v_cache, const int32_t *prefix_len, int P_max,
                            const int32_t *n_rows, int B, int R, int Hkv, int dh, void *ws,
                            cudaStream_t stream) {
    Kv4Args a;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.kc = reinterpret_cast<uint8_t *const *>(k_cache);
    a.vc = reinterpret_cast<uint8_t *const *>(v_cache);
    a.prefix_len = prefix_len;
    a.n_rows = n_rows;
    a.R = R;
    a.Hkv = Hkv;
    a.dh = dh;
    a.P_max = P_max;
    a.status = static_cast<int *>(ws);
    const int gx = (2 * Hkv * dh / 16 + kKv4Threads - 1) / kKv4Threads;
    auto kern = append ? (dtype == MEDUSA_F32 ? kv4_append_kernel<float> : kv4_append_kernel<bf16>)
                       : (dtype == MEDUSA_F32 ? kv4_unpack_kernel<float> : kv4_unpack_kernel<bf16>);
    cudaError_t e = launch_pdl(kern, dim3(gx, R, B), dim3(kKv4Threads), 0, stream, a);
    note_launch();
    return e;
}

}  // namespace medusa
