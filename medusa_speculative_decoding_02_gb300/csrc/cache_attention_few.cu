// cache_attention_few.cu -- attention over the caches for few rows: plain
// decoding, where a KV head has at most 16 rows (R * H / Hkv).
//
// Such a call reads the cache once and computes little, and the 128-row tiles
// of the other kernel spend their time on passing stages between warps.  Here
// every warp is on its own: it copies 16 keys at a time into a ring of its own and
// reads them from there in the lane layout of a matrix instruction whose operands
// are registers, so that no barrier lies between the cache and the product until
// the warps of a CTA join at the end.
//
// Keys are the 16 rows of the instruction, query rows its 8 columns:
//     S^T = K Q^T   (16 keys x 8 rows, over dh in steps of 16)
//     O^T = V^T P^T (16 elements x 8 rows, over the 16 keys)
// Lane 4g + t holds keys g and g + 8 of K, and elements of keys 2t, 2t+1, 2t+8,
// 2t+9 of V.  Which elements of a head stand at which place of a product is
// free as long as both operands (or the result) agree, so a lane takes 16-byte
// pieces of the rows as they lie: element order below is by lane, not by index.
// The weights change lanes between the two products by an 8x8 transposition.
// A 4-bit row is widened to fp16 in registers; for V the codes of two keys are
// joined in a byte first, so that the conversion gives the pair of keys that the
// product wants.  Its numerics are those of the other kernel: fp16 products of
// query rows scaled by a power of two, weights biased by 2^7, a reference that
// moves by jumps of at least 2^8.
//
// The rows come by asynchronous copies into a ring of three tiles that is the
// warp's own (4-bit: 2.3 KB a tile, three CTAs of four warps an SM; bf16: 8 KB, two
// CTAs).  Loaded straight into registers the next tile had 2.1 us to come at 12
// warps an SM and still was waited for (64 us where the ring takes 47); rings of 2
// KB tiles deeper than three, more warps with fewer registers (51 us) and two tiles
// a step (50 us) were slower.
//
// Bound by the bytes for a bf16 cache: eight sequences x 32 KV heads x 8192 slots
// (1.07 GB) in 148 us, 7.2 TB/s; eight single tokens behind a 2047 window (69 MB)
// in 16.4 us with a cold L2, 11.3 us with the rows in it, of which the second launch,
// the join, is 2-3 us.  A 4-bit cache takes some 330 instructions a tile of 16 keys, of
// which 64 conversions, 64 products with scales and 16 matrix instructions, and is
// bound by issue and the latency of that chain (57 % of the issue slots at 12 warps
// an SM): 186 MB in 46.9 us, 4.0 TB/s.
#include "cache_attention.cuh"

namespace medusa {

namespace {

constexpr int kFewThreads = 128, kFewWarps = kFewThreads / 32;

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

// c += A (16 x 16) B (16 x 8)
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transposition: lane 4i + j gives elements (i, 2j), (i, 2j+1) of a matrix
// and gets (2j, i), (2j+1, i)
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_halves(uint32_t bytes) {  // two e4m3 -> fp16 pair
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)bytes, __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }

// Sixteen keys of a KV head in shared memory: rows of K, rows of V, and for a
// 4-bit cache the scales of K, the scales of V.  The 16-byte pieces of a
// 128-byte line are permuted so that the reads below, eight (or sixteen) lanes at
// a time, meet every bank once.
template <int DH, bool KV4>
struct FewTile {
    static constexpr int NI = DH / 32, NJ = DH / 64;
    static constexpr int ROW = KV4 ? DH / 2 : DH * 2, SCALES = KV4 ? DH / 16 : 0;
    static constexpr int BYTES = 32 * (ROW + SCALES);
    const char *at;  // this tile
    // the lane's pieces: of key g of K, of keys 2t and 2t+1 of V, and their scales
    // (eight rows further on a piece has the same place in its line)
    struct Lane {
        int k, v[2], ks, vs;
        __device__ __forceinline__ Lane(int g, int t) {
            if constexpr (KV4 && DH == 64)
                k = g * ROW + t * 8;
            else
                k = piece(g, t);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[i] = 16 * ROW + (!KV4        ? piece(2 * t + i, g)
                                   : DH == 128 ? piece(2 * t + i, g >> 1) + (g & 1) * 8
                                               : (2 * t + i) * ROW + g * 4);
            ks = 32 * ROW + g * SCALES + t * (DH / 64);
            vs = 32 * ROW + (16 + 2 * t) * SCALES + g * SCALES / 8;
        }
    };
    const Lane &p;

    // byte of a row's piece c (16 bytes)
    static __device__ __forceinline__ int piece(int row, int c) {
        if constexpr (ROW >= 128)
            return row * ROW + ((c ^ ((row & 6) | (row & 1) << 2)) << 4);
        else if constexpr (ROW == 64)
            return (row >> 1) * 128 + ((((row & 1) << 2 | c) ^ (row & 6)) << 4);
        else
            return row * ROW + (c << 4);
    }
    // Copies of slots s0 .. s0 + 15 (past the last slot: the last): a lane's pieces
    // of the rows and its scales, and where they go.
    struct Copy {
        static constexpr int C = ROW / 16, RPP = 32 / C;  // pieces a row, rows a pass
        const char *k, *v, *s;
        int row, to, s_to;
        __device__ __forceinline__ Copy(const CacheItem &it, int head, int scales_at, int lane) {
            const int c = lane % C;
            row = lane / C;
            to = piece(row, c);
            k = static_cast<const char *>(it.kc) + head * ROW + c * 16;
            v = static_cast<const char *>(it.vc) + head * ROW + c * 16;
            s = static_cast<const char *>(lane < 16 ? it.kc : it.vc) + scales_at + head * SCALES;
            s_to = 32 * ROW + lane * SCALES;
        }
        __device__ __forceinline__ void operator()(uint32_t dst, uint32_t row_bytes, int s0, int last,
                                                   int lane) const {
#pragma unroll
            for (int p = 0; p < 16 / RPP; ++p) {
                // (a pass of fewer than eight rows changes the place in the line)
                const int place = RPP % 8 == 0 ? to + p * RPP * ROW : piece(row + p * RPP, lane % C);
                const size_t off = (size_t)(uint32_t)min(s0 + row + p * RPP, last) * row_bytes;
                copy_async<16>(dst + place, k + off);
                copy_async<16>(dst + place + 16 * ROW, v + off);
            }
            if constexpr (KV4)
                copy_async<SCALES>(dst + s_to, s + (size_t)(uint32_t)min(s0 + (lane & 15), last) * row_bytes);
        }
    };
    // the lane's elements 8i .. 8i+7 of key g + 8h, as four pairs
    struct KWords {
        uint4 w[NI];
    };
    __device__ __forceinline__ KWords k_words(int h) const {
        KWords r;
        const char *k = at + p.k + 8 * h * ROW, *ks = at + p.ks + 8 * h * SCALES;
        if constexpr (KV4) {
            uint32_t w[NI], s;
            if constexpr (DH == 128) {
                const uint4 x = *reinterpret_cast<const uint4 *>(k);
                w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
                s = *reinterpret_cast<const uint16_t *>(ks);
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(k);
                w[0] = x.x, w[1] = x.y;
                s = *reinterpret_cast<const uint8_t *>(ks);
            }
            const uint32_t s2 = e4m3_halves(s);  // DH = 128: of words 0, 1 and of words 2, 3
#pragma unroll
            for (int i = 0; i < NI; ++i)
                r.w[i] = kv4_widen(w[i], as_half2(__byte_perm(s2, 0, i >= 2 ? 0x3232 : 0x1010)));
        } else {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                r.w[i] = *reinterpret_cast<const uint4 *>(at + ((p.k ^ (i & 1) << 6) + (i >> 1) * 128 + 8 * h * ROW));
        }
        return r;
    }
    // the lane's elements of keys 2t, 2t+1, 2t+8, 2t+9 as they are stored
    struct VRaw {
        uint32_t w[4][KV4 ? NJ : 4 * NJ], s[2];
    };
    __device__ __forceinline__ VRaw v_raw() const {
        VRaw r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const char *v = at + p.v[i & 1] + 8 * (i >> 1) * ROW;
            if constexpr (KV4) {
                if constexpr (DH == 128) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(v);
                    r.w[i][0] = x.x, r.w[i][NJ - 1] = x.y;
                } else {
                    r.w[i][0] = *reinterpret_cast<const uint32_t *>(v);
                }
            } else {
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(v + j * 128);
                    r.w[i][4 * j] = x.x, r.w[i][4 * j + 1] = x.y, r.w[i][4 * j + 2] = x.z, r.w[i][4 * j + 3] = x.w;
                }
            }
        }
        if constexpr (KV4) {
            const uint8_t *s = reinterpret_cast<const uint8_t *>(at + p.vs);
#pragma unroll
            for (int h = 0; h < 2; ++h) r.s[h] = s[8 * h * SCALES] | (uint32_t)s[(8 * h + 1) * SCALES] << 8;
        }
        return r;
    }
    // A operands of the products for the lane's elements 8j .. 8j+7 of V: element
    // 2n and 2n+1 (rows g and g+8 of product n) of its four keys
    static __device__ __forceinline__ void v_words(const VRaw &r, int j, uint32_t (&a)[4][4]) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {  // keys 2t, 2t+1 and 2t+8, 2t+9
            uint32_t ev[4], od[4];
            if constexpr (KV4) {
                const uint32_t wa = r.w[2 * p][j], wb = r.w[2 * p + 1][j];
                constexpr uint32_t L = 0x0f0f0f0fu;
                const __half2 s = as_half2(e4m3_halves(r.s[p]));
                const uint4 e = kv4_widen((wa & L) | ((wb << 4) & ~L), s);
                const uint4 o = kv4_widen(((wa >> 4) & L) | (wb & ~L), s);
                ev[0] = e.x, ev[1] = e.y, ev[2] = e.z, ev[3] = e.w;
                od[0] = o.x, od[1] = o.y, od[2] = o.z, od[3] = o.w;
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint32_t x = r.w[2 * p][4 * j + n], y = r.w[2 * p + 1][4 * j + n];
                    ev[n] = __byte_perm(x, y, 0x5410);
                    od[n] = __byte_perm(x, y, 0x7632);
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                a[n][2 * p] = ev[n];
                a[n][2 * p + 1] = od[n];
            }
        }
    }
    // index within the head of the lane's element 8j + 2n
    __device__ static __forceinline__ int v_element(int g, int j, int n) {
        return KV4 ? g * (DH / 8) + 8 * j + 2 * n : j * 64 + g * 8 + 2 * n;
    }
    // an infinity or a NaN among the lane's elements of V
    static __device__ __forceinline__ bool v_bad(const VRaw &r) {
        bool bad = false;
        if constexpr (KV4) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
                bad = bad || (r.s[p] & 0x7fu) == kE4m3Nan || ((r.s[p] >> 8) & 0x7fu) == kE4m3Nan;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4 * NJ; ++j) bad = bad || pair_bad<false>(r.w[i][j]);
        }
        return bad;
    }
};

// Tiles of a warp's ring (all but one of them in flight) and CTAs an SM.
constexpr int kFewRing = 3;
template <bool KV4, int NQ> constexpr int kFewCtas = KV4 && NQ == 1 ? 3 : 2;

template <int DH, bool KV4, int NQ>
struct FewSmem {
    static constexpr int WARP = kFewRing * FewTile<DH, KV4>::BYTES;
    static constexpr int LD = DH + 4, Q = 8 * NQ;
    // after the loop, in place of the rings: O of each warp [Q][LD], then (m, l)
    static constexpr int JOIN = kFewWarps * Q * (LD * 4 + 8);
    static constexpr int TOTAL = kFewWarps * WARP > JOIN ? kFewWarps * WARP : JOIN;
    static_assert(kFewCtas<KV4, NQ> * (TOTAL + 512 + 1024) <= 196 * 1024, "in the heads' carveout");
};

template <int DH, bool KV4, int NQ, bool DEAL>
__global__ void __launch_bounds__(kFewThreads, kFewCtas<KV4, NQ>) cache_attn_few_kernel(CacheAttnArgs a) {
    pdl_enter();
    using Tile = FewTile<DH, KV4>;
    using S = FewSmem<DH, KV4, NQ>;
    constexpr int NI = Tile::NI, NJ = Tile::NJ, Q = 8 * NQ, LD = S::LD, D = kFewRing;
    constexpr float kBias = KV4 ? kF16Bias : 0.f;
    extern __shared__ __align__(128) char sm[];
    __shared__ uint64_t row_mask[Q];  // tree slots a row sees
    __shared__ int row_win[Q], row_far[Q];

    const int head = blockIdx.x;
    const int R = a.R, G = a.H / a.Hkv, M = R * G;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    // The numbers here leave a gap after the sinks, up to a multiple of 16, so
    // that a tile's slots are consecutive.
    auto pad16 = [](int n) { return (n + 15) & ~15; };
    CacheItem it;
    if (!find_item<DEAL>(a, [&](int P) {
            const KeyRun r(P, R, a.window, a.sinks);
            return r.len - r.n_sink + pad16(r.n_sink);
        }, it))
        return;
    const int b = it.b, P = it.P, kbeg = it.kbeg, kend = it.kend;
    const KeyRun run(P, R, a.window, a.sinks);
    const int n_pad = pad16(run.n_sink), last = P + R - 1;
    auto slot = [&](int x) { return x < n_pad ? x : x - n_pad + run.lo; };
    bf16 *out = static_cast<bf16 *>(a.out);
    auto out_row = [&](int m) { return out + (((size_t)b * R + m / G) * a.H + head * G + m % G) * DH; };
    auto part_row = [&](int m) { return ((size_t)it.range * a.H + head * G + m % G) * R + m / G; };
    if (kbeg >= kend) {  // uniform over the CTA
        if (a.ns == 1) {
            for (int i = tid; i < M * (DH / 8); i += kFewThreads)
                reinterpret_cast<uint4 *>(out_row(i / (DH / 8)))[i % (DH / 8)] = make_uint4(0, 0, 0, 0);
        } else if (tid < M) {
            a.part_ml[part_row(tid)] = make_float2(-INFINITY, 0.f);
        }
        return;
    }

    constexpr int kStep = 16 * kFewWarps;
    static_assert(kRangeUnit % 16 == 0, "ranges begin at a tile");
    const int x_warp = kbeg + warp * 16;
    const int row_bytes = KV4 ? kv4_row_bytes(a.Hkv, DH) : a.Hkv * DH * 2;
    char *ring = sm + warp * S::WARP;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    const typename Tile::Copy copy_tile(it, head, KV4 ? kv4_code_bytes(a.Hkv, DH) : 0, lane);
    auto copy = [&](int x, int place) {
        if (x < kend) copy_tile(ring_at + place * Tile::BYTES, row_bytes, slot(x), last, lane);
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) copy(x_warp + i * kStep, i);

    // ---- what each row sees, in numbered keys
    const int x_tree = n_pad + P - run.lo;  // number of tree slot 0
    if (tid < Q) {
        uint64_t am = 0;
        int win = 0, far = 0;
        if (tid < M) {
            const int r = tid / G, d = row_depth(a, b, r);
            am = a.anc_mask[(size_t)b * R + r];  // R <= 16: one word
            if (a.window) {
                far = max(0, P + d - a.window + 1 - run.lo);
                win = n_pad + far;
                if (d >= a.window)  // ancestors out of the window (and not among the sinks)
                    for (int s = 0; s < R; ++s) {
                        const int sd = row_depth(a, b, s);
                        if (!(P + sd < a.sinks || d - sd < a.window)) am &= ~(1ull << s);
                    }
            }
        }
        row_mask[tid] = am;
        row_win[tid] = win;
        row_far[tid] = far;
    }

    // ---- Q: lane (g, t) holds its elements of row 8n + g
    uint32_t qf[NQ][4 * NI];
    float scale[NQ][2];  // of rows 8n + 2t and 8n + 2t + 1
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int m = 8 * n + g;
        const bool live = m < M;
        const bf16 *src = static_cast<const bf16 *>(a.q) +
                          (((size_t)b * R + (live ? m / G : 0)) * a.H + head * G + (live ? m % G : 0)) * DH;
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) w = *reinterpret_cast<const uint4 *>(src + (KV4 ? t * (DH / 4) + i * 8 : i * 32 + t * 8));
            qf[n][4 * i] = w.x, qf[n][4 * i + 1] = w.y, qf[n][4 * i + 2] = w.z, qf[n][4 * i + 3] = w.w;
            if (KV4) {
                float f[8];
                Vec16<bf16>::widen(w, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
            }
        }
        float row_scale = a.scale_log2;
        if (KV4) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            float factor = 1.f;
            if (amax > 0.f && amax < INFINITY) {
                // 2^floor(log2 amax), from the exponent bits (subnormals: 2^-126)
                const uint32_t eb = max(1u, __float_as_uint(amax) >> 23);
                factor = eb < 254u ? __uint_as_float((254u - eb) << 23) : 0x1p-127f;
                row_scale *= __uint_as_float(eb << 23);
            }
#pragma unroll
            for (int i = 0; i < 4 * NI; ++i)
                qf[n][i] = pack_weights<true>(bf_lo(qf[n][i]) * factor, bf_hi(qf[n][i]) * factor);
        }
        // a masked score, -inf, times the scale has to stay -inf
        row_scale = fmaxf(row_scale, 0x1p-126f);
        scale[n][0] = __shfl_sync(0xffffffffu, row_scale, 8 * t);
        scale[n][1] = __shfl_sync(0xffffffffu, row_scale, 8 * t + 4);
    }
    __syncthreads();
    // keys that every row sees: numbers below n_sink, and [x_all, x_tree)
    int far = 0;
    for (int m = 0; m < M && a.window; ++m) far = max(far, row_far[m]);
    const int x_all = a.window ? n_pad + far : 0;
    // [n_pad, x_sink): slots under `sinks` that the first row's window holds as well
    const int x_sink = min(n_pad + max(0, a.sinks - run.lo), x_tree);
    auto sees = [&](int m, int x) {
        if (x >= kend) return false;
        if (x >= x_tree) return ((row_mask[m] >> (x - x_tree)) & 1u) != 0;
        return x >= row_win[m] || x < run.n_sink || (x >= n_pad && x < x_sink);
    };

    float o[NQ][4 * NJ][4], m_run[NQ][2], mu[NQ][2], l_run[NQ][2];
    bool huge = false;  // uniform over the warp
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int i = 0; i < 4 * NJ; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        m_run[n][0] = m_run[n][1] = -INFINITY;
        mu[n][0] = mu[n][1] = -kBias;
        l_run[n][0] = l_run[n][1] = 0.f;
    }

    const typename Tile::Lane place(g, t);
    int at = 0;  // ring place of the tile at x0
#pragma unroll 1
    for (int x0 = x_warp; x0 < kend; x0 += kStep) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(D - 2) : "memory");
        __syncwarp();  // every lane's copies are there, and the tile before is read
        copy(x0 + (D - 1) * kStep, at == 0 ? D - 1 : at - 1);
        const Tile tl{ring + at * Tile::BYTES, place};
        at = at == D - 1 ? 0 : at + 1;
        // s[..][0], [1]: key g, rows 8n + 2t and + 1; s[..][2], [3]: key g + 8
        float s[NQ][4];
        {
            const typename Tile::KWords k0 = tl.k_words(0), k1 = tl.k_words(1);
            float s2[NQ][4];  // two chains of products, added up: half the latency
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const uint4 lo = k0.w[i], hi = k1.w[i];
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    mma16816<KV4>(s[n], lo.x, hi.x, lo.y, hi.y, qf[n][4 * i], qf[n][4 * i + 1]);
                    mma16816<KV4>(s2[n], lo.z, hi.z, lo.w, hi.w, qf[n][4 * i + 2], qf[n][4 * i + 3]);
                }
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] += s2[n][e];
        }
        const bool masked =
            !(x0 + 16 <= min(kend, x_tree) && (x0 >= x_all || x0 + 16 <= run.n_sink));
        if (masked) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!sees(8 * n + 2 * t + (e & 1), x0 + g + 8 * (e >> 1))) s[n][e] = -INFINITY;
        }
        bool grew = false;
        float cm[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                cm[n][c] = fmaxf(s[n][c], s[n][c + 2]) * scale[n][c];
                grew = grew || cm[n][c] > m_run[n][c] + kRescaleLog2;  // m_run = -inf: the first visible key
            }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = cm[n][c];
#pragma unroll
                    for (int d = 4; d <= 16; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    if (x > m_run[n][c] + kRescaleLog2) {
                        const float alpha = exp2f(m_run[n][c] - x);
                        m_run[n][c] = x;
                        mu[n][c] = x - kBias;
                        l_run[n][c] *= alpha;
#pragma unroll
                        for (int i = 0; i < 4 * NJ; ++i) {
                            o[n][i][c] *= alpha;
                            o[n][i][c + 2] *= alpha;
                        }
                    }
                    // past 2^16 the scores are rounded before the difference, as the
                    // maximum was: the fused form keeps bits of the product that the
                    // maximum lost, and the largest weight would leave 1
                    huge = huge || __any_sync(0xffffffffu, fabsf(mu[n][c]) > 65536.f);
                }
        }
        uint32_t pb[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float p[4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (huge) {
                    p[c] = ex2_approx(__fmul_rn(s[n][c], scale[n][c]) - mu[n][c]);
                    p[c + 2] = ex2_approx(__fmul_rn(s[n][c + 2], scale[n][c]) - mu[n][c]);
                } else {
                    p[c] = ex2_approx(fmaf(s[n][c], scale[n][c], -mu[n][c]));
                    p[c + 2] = ex2_approx(fmaf(s[n][c + 2], scale[n][c], -mu[n][c]));
                }
                l_run[n][c] += p[c] + p[c + 2];  // the sum adds the fp32 weights
            }
            pb[n][0] = transpose8(pack_weights<KV4>(p[0], p[1]));
            pb[n][1] = transpose8(pack_weights<KV4>(p[2], p[3]));
        }
        const typename Tile::VRaw vr = tl.v_raw();
        if (masked && __any_sync(0xffffffffu, Tile::v_bad(vr))) {
            // Infinities or NaNs in V where some row may not see them: one row at a
            // time, with the keys of weight 0 cleared from V for it.
#pragma unroll 1
            for (int row = 0; row < 8; ++row) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    uint32_t keep[2];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const uint32_t w = __shfl_sync(0xffffffffu, pb[n][p], row * 4 + t);
                        keep[p] = ((w & 0x7fffu) ? 0xffffu : 0u) | ((w & 0x7fff0000u) ? 0xffff0000u : 0u);
                    }
                    const uint32_t b0 = g == row ? pb[n][0] : 0u, b1 = g == row ? pb[n][1] : 0u;
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        uint32_t v[4][4];
                        Tile::v_words(vr, j, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float d[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) d[e] = o[n][4 * j + i][e];
                            mma16816<KV4>(d, v[i][0] & keep[0], v[i][1] & keep[0], v[i][2] & keep[1],
                                          v[i][3] & keep[1], b0, b1);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (2 * t + (e & 1) == row) o[n][4 * j + i][e] = d[e];
                        }
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                uint32_t v[4][4];
                Tile::v_words(vr, j, v);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma16816<KV4>(o[n][4 * j + i], v[i][0], v[i][1], v[i][2], v[i][3], pb[n][0],
                                      pb[n][1]);
            }
        }
    }

    // ---- the warps' parts joined (every copy has landed, or none was begun)
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncthreads();
    float *so = reinterpret_cast<float *>(sm);
    float2 *sml = reinterpret_cast<float2 *>(so + kFewWarps * Q * LD);
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int m = 8 * n + 2 * t + c;
            float l = l_run[n][c];
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            if (g == 0) sml[warp * Q + m] = make_float2(m_run[n][c], l);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float2 *>(so + (warp * Q + m) * LD + Tile::v_element(g, j, i)) =
                        make_float2(o[n][4 * j + i][c], o[n][4 * j + i][c + 2]);
        }
    __syncthreads();
    for (int i = tid; i < M * (DH / 4); i += kFewThreads) {
        const int m = i / (DH / 4), c = (i % (DH / 4)) * 4;
        float top = -INFINITY, l = 0.f;
        float2 ml[kFewWarps];
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            ml[w] = sml[w * Q + m];
            top = fmaxf(top, ml[w].x);
        }
        const float mu = top == -INFINITY ? 0.f : top;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float f = exp2f(ml[w].x - mu);
            l = fmaf(f, ml[w].y, l);  // (also with f = 0: a row of NaN scores has m = -inf, l = NaN)
            if (f == 0.f) continue;
            const float4 v = *reinterpret_cast<const float4 *>(so + (w * Q + m) * LD + c);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
        }
        if (a.ns == 1) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            *reinterpret_cast<uint2 *>(out_row(m) + c) =
                make_uint2(pack_weights<false>(acc.x * inv, acc.y * inv), pack_weights<false>(acc.z * inv, acc.w * inv));
        } else {
            const size_t pr = part_row(m);
            *reinterpret_cast<float4 *>(a.part_o + pr * DH + c) = acc;
            if (c == 0) a.part_ml[pr] = make_float2(top - kBias, l);
        }
    }
}

template <int DH, bool KV4, int NQ>
cudaError_t launch_few(const CacheAttnArgs &a, cudaStream_t stream) {
    auto kern = a.starts ? cache_attn_few_kernel<DH, KV4, NQ, true> : cache_attn_few_kernel<DH, KV4, NQ, false>;
    constexpr int smem = FewSmem<DH, KV4, NQ>::TOTAL;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e) return e;
    return launch_pdl(kern, dim3(a.Hkv, a.ns, a.B), dim3(kFewThreads), (size_t)smem, stream, a);
}

}  // namespace

int cache_few_ctas_per_sm(bool kv4, int rows) {
    return rows <= 8 ? (kv4 ? kFewCtas<true, 1> : kFewCtas<false, 1>) : (kv4 ? kFewCtas<true, 2> : kFewCtas<false, 2>);
}

cudaError_t launch_cache_attention_few(const CacheAttnArgs &a, bool kv4, int dh, cudaStream_t stream) {
    const bool two = a.R * (a.H / a.Hkv) > 8;
    if (kv4 && dh == 128) return two ? launch_few<128, true, 2>(a, stream) : launch_few<128, true, 1>(a, stream);
    if (kv4) return two ? launch_few<64, true, 2>(a, stream) : launch_few<64, true, 1>(a, stream);
    if (dh == 128) return two ? launch_few<128, false, 2>(a, stream) : launch_few<128, false, 1>(a, stream);
    return two ? launch_few<64, false, 2>(a, stream) : launch_few<64, false, 1>(a, stream);
}

}  // namespace medusa
