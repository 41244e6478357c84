// kv4.cu -- rows into and out of the 4-bit cache (layout: kv4.cuh).
//
// kv4_append_kernel: one thread per block of 16 elements of K or V: it picks the
// scale and the codes and stores eight bytes of codes and one scale byte.
// Consecutive threads take consecutive blocks of a sequence's rows, K's then
// V's, so both stores of a warp are contiguous.  kv4_unpack_kernel is the
// inverse.  They move 2 or 4 bytes an element on the wide side and 9/16 on the
// narrow one, and are bound by issue (append) and by the latency of two dependent
// rounds of loads (unpack).  Four ragged bf16 prompts of up to 4001 rows of 8 x 128
// elements (58 MB each way): append 13.6 us, 4.2 TB/s, unpack 11.2 us, 5.2 TB/s
// (fp32, 103 MB: 27.0 and 24.8 us); 65 rows of 32 x 128: 2.2 and 2.1 us.  Two
// blocks a thread gained nothing on the prompts and took 5.5 us for both calls at
// the 65 rows; with divisions by 6 and by the blocks of a slot, and the largest
// magnitude taken element by element, both calls took 27.5 us on the prompts.
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
    unsigned per_magic, per_shift;  // division by the blocks of a slot (K and V)
    int *status;
};

// One block of a call: the wide elements and the cache row they belong to, or
// row = null when there is nothing to do (past the end, or the sequence's
// checks failed).
template <typename T>
struct Kv4Block {
    T *wide;
    uint8_t *row;
    int e;  // block within the row
    __device__ __forceinline__ Kv4Block(const Kv4Args &a, int b, unsigned idx, int live) {
        const unsigned per = (unsigned)(a.Hkv * a.dh / 16);  // blocks of a K row, and of a V row
        const unsigned i = __umulhi(idx, a.per_magic) >> a.per_shift;
        unsigned blk = idx - i * (2 * per);
        const bool is_v = blk >= per;
        if (is_v) blk -= per;
        e = (int)blk;
        row = nullptr;
        if ((int)i >= live) return;
        row = (is_v ? a.vc : a.kc)[b] + (size_t)(a.prefix_len[b] + (int)i) * kv4_row_bytes(a.Hkv, a.dh);
        const long long r = (long long)b * a.R + i;
        wide = static_cast<T *>(const_cast<void *>(is_v ? a.v : a.k)) +
               r * (is_v ? a.v_stride : a.k_stride) + blk * 16;
    }
};

// Rows of sequence b to handle: 0 when its checks fail.
__device__ __forceinline__ int kv4_live_rows(const Kv4Args &a, int b) {
    const uint8_t *kc = a.kc[b], *vc = a.vc[b];
    if (!kc || !vc || ((reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) & 15u)) {
        set_status(a.status, MEDUSA_DEV_BAD_CACHE);
        return 0;
    }
    const int P = a.prefix_len[b];
    if (P < 0 || P > a.P_max) {
        set_status(a.status, MEDUSA_DEV_BAD_PREFIX);
        return 0;
    }
    return a.n_rows ? min(a.R, a.n_rows[b]) : a.R;
}

// grid (blocks of a sequence over 256, B)
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(Kv4Args a) {
    pdl_enter();
    constexpr int N = Vec16<T>::N, V = 16 / N;
    const int b = blockIdx.y;
    const Kv4Block<T> k(a, b, blockIdx.x * kKv4Threads + threadIdx.x, kv4_live_rows(a, b));
    if (!k.row) return;
    uint4 raw[V];
#pragma unroll
    for (int c = 0; c < V; ++c) raw[c] = ld_stream16(k.wide + c * N);
    float x[16];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        float f[N];
        Vec16<T>::widen(raw[c], f);
#pragma unroll
        for (int j = 0; j < N; ++j) x[c * N + j] = f[j];
    }
    // the largest magnitude, by its bits: infinities and NaNs come out on top
    uint32_t top = 0;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = __vmaxu2(top, w[j] & 0x7fff7fffu);
        }
        top = max(top & 0xffff0000u, top << 16);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
    }
    uint32_t sb = kE4m3Nan, lo = 0, hi = 0;
    if (top < 0x7f800000u) {
        sb = kv4_scale_byte(__uint_as_float(top));
        if (sb) {
            const float s = e4m3_value(sb);
            lo = kv4_codes(x, s, T());
            hi = kv4_codes(x + 8, s, T());
        }
    }
    *reinterpret_cast<uint2 *>(k.row + k.e * 8) = make_uint2(lo, hi);
    k.row[kv4_code_bytes(a.Hkv, a.dh) + k.e] = (uint8_t)sb;
}

template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_unpack_kernel(Kv4Args a) {
    pdl_enter();
    const int b = blockIdx.y;
    const Kv4Block<T> k(a, b, blockIdx.x * kKv4Threads + threadIdx.x, kv4_live_rows(a, b));
    if (!k.row) return;
    const uint2 codes = *reinterpret_cast<const uint2 *>(k.row + k.e * 8);
    const __half s = e4m3_half(k.row[kv4_code_bytes(a.Hkv, a.dh) + k.e]);
    float x[2][8];
    kv4_widen(codes.x, s, x[0]);
    kv4_widen(codes.y, s, x[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        T *dst = k.wide + 8 * h;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(dst) = make_float4(x[h][0], x[h][1], x[h][2], x[h][3]);
            *reinterpret_cast<float4 *>(dst + 4) = make_float4(x[h][4], x[h][5], x[h][6], x[h][7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(x[h][2 * c], x[h][2 * c + 1]);
                w[c] = *reinterpret_cast<const uint32_t *>(&p);
            }
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
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
    // i / d = (i m) >> (32 + s) for all i < 2^30, with 2^s the power of two below d
    // and m = 2^(32 + s) / d + 1: m is too large by less than one, so i m / 2^(32 + s)
    // by less than i / 2^(32 + s) < 1 / d (i < 2^30 < 2^(32 + s) / d, as d <= 2^(s + 1))
    const unsigned d = 2u * (unsigned)(Hkv * dh / 16);
    unsigned s = 0;
    while ((2u << s) < d) ++s;
    a.per_shift = s;
    a.per_magic = (unsigned)((1ull << (32 + s)) / d + 1);
    static_assert(2ll * kKv4MaxRows * 1024 * 128 / 16 < 1 << 30, "blocks of a sequence (1024 heads of 128)");
    const unsigned blocks = (unsigned)R * (unsigned)(2 * Hkv * dh / 16);
    const unsigned gx = (blocks + kKv4Threads - 1) / kKv4Threads;
    auto kern = append ? (dtype == MEDUSA_F32 ? kv4_append_kernel<float> : kv4_append_kernel<bf16>)
                       : (dtype == MEDUSA_F32 ? kv4_unpack_kernel<float> : kv4_unpack_kernel<bf16>);
    cudaError_t e = launch_pdl(kern, dim3(gx, B), dim3(kKv4Threads), 0, stream, a);
    note_launch();
    return e;
}

}  // namespace medusa
