// paged_attention.cu -- attention over a cache in pages: a chunk of new tokens
// (row i of sequence b sees slots 0 .. P + i) or a candidate tree (row i sees the
// prefix and the slots of its ancestors).
//
// Query head h reads KV head h / G (G = H / Hkv).  The rows of a tile are rows that
// share a KV head, row r * G + g being new row r and query head hk * G + g.  A
// tile's keys are split into ranges where there are few tiles (find_item), which a
// cluster of CTAs or a second kernel joins.  A slot whose page number is outside the pool is
// not seen (and the status is set).  A row that sees nothing gets zeros; rows behind
// a sequence's n_rows are neither read nor written.
//
// Three kernels: fp32 on the CUDA cores here, bf16 with at most 16 rows a KV head in
// cache_attention_few.cu, bf16 with more in paged_attention_tc.cu.
#include <algorithm>

#include "cache_attention.cuh"

namespace medusa {

namespace {

// ------------------------------------------------------------- CUDA cores ---
//
// fp32.  ROWS rows and 32 keys at a time, four threads a row: thread (ty, tx) of ROWS / 4 x
// 16 scores rows 4 ty .. +3 against keys tx and tx + 16, and owns columns 4 tx + 64 c .. +3
// of those rows' outputs.  The running maximum and sum of a row live in its 16 threads.
// K and V of the next keys are copied while these are at work.
//
// Bound by the reads of shared memory and their latency: the scores read 96 bytes a thread
// for every 32 products.  8 sequences x 8 heads behind 2048 slots, dh 128: 64 rows 171 us
// (26 TFLOP/s), 32 rows 114; a single 32 x 64 tile with copies between the stages took
// 295 and 167.  Tiles of 64 rows lose where they are too few for the SMs (two trees of 65
// rows behind 300 slots: 17.5 us for 14.4).
constexpr int kKeys = 32;

template <int DH, int ROWS>
struct SimtSmem {
    static constexpr int LD = DH + 4, LP = kKeys + 4, TILE = 2 * kKeys * LD;  // K and V of a stage
    static constexpr int WORDS = (ROWS * LD + 2 * TILE + ROWS * LP) * 4;
    static constexpr int TOTAL = WORDS + (2 * kKeys + 2) * 4;
    static_assert(2 * (TOTAL + 1024) <= 228 * 1024, "two CTAs an SM");
};

template <int DH, int ROWS>
__global__ void __launch_bounds__(4 * ROWS, 2) paged_attn_simt_kernel(CacheAttnArgs a) {
    pdl_enter();
    using L = SimtSmem<DH, ROWS>;
    constexpr int LD = L::LD, LP = L::LP, C = DH / 64, THREADS = 4 * ROWS;
    extern __shared__ __align__(16) float sf[];
    auto smem_at = [](const float *p) { return (uint32_t)__cvta_generic_to_shared(p); };
    float *qs = sf, *tiles = qs + ROWS * LD, *ps = tiles + 2 * L::TILE;
    int *key_ok = reinterpret_cast<int *>(sf + L::WORDS / 4);  // [2][kKeys]: the key's page is in the pool
    int *bad_at = key_ok + 2 * kKeys;  // [2]: the stage, if it has keys whose page is not
    const int g = blockIdx.x / a.row_tiles, rt = a.row_tiles - 1 - (blockIdx.x - g * a.row_tiles);
    const int R = a.R, G = a.H / a.Hkv;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    CacheItem it;
    find_item<false, kRangeUnit, true>(a, [&](int P, int b) {
        const int n = live_rows(a, b);
        return n == 0 ? 0 : P + (a.anc_mask ? n : min(n, (rt * ROWS + ROWS - 1) / G + 1));
    }, it);
    const int b = it.b, P = it.P, kbeg = it.kbeg, kend = it.kend;
    const int M = live_rows(a, b) * G;
    if (rt * ROWS >= M) return;  // uniform over the CTA
    int row[4], head[4];
    bool live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = rt * ROWS + ty * 4 + i;
        live[i] = m < M;
        row[i] = live[i] ? m / G : 0;
        head[i] = g * G + (live[i] ? m - row[i] * G : 0);
    }
    auto out_row = [&](int i) {
        return static_cast<float *>(a.out) + (((size_t)b * R + row[i]) * a.H + head[i]) * DH;
    };
    auto part_row = [&](int i) { return ((size_t)it.range * a.H + head[i]) * R + row[i]; };
    auto store4 = [&](float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; };
    if (kbeg >= kend) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!live[i]) continue;
            if (a.ns == 1) {
#pragma unroll
                for (int c = 0; c < C; ++c) store4(out_row(i) + tx * 4 + 64 * c, make_float4(0.f, 0.f, 0.f, 0.f));
            } else if (tx == 0) {
                a.part_ml[part_row(i)] = make_float2(-INFINITY, 0.f);
            }
        }
        return;
    }
    auto put = [&](float *dst, const float *src) {
        *reinterpret_cast<float4 *>(dst) = *reinterpret_cast<const float4 *>(src);
    };
    constexpr int VR = DH / 4;  // 16-byte vectors a row
    for (int e = tid; e < ROWS * VR; e += THREADS) {
        const int lr = e / VR, c = (e - lr * VR) * 4, m = rt * ROWS + lr;
        const int r = m < M ? m / G : 0, h = g * G + (m < M ? m - r * G : 0);
        put(qs + lr * LD + c, static_cast<const float *>(a.q) + (((size_t)b * R + r) * a.H + h) * DH + c);
    }
    float acc[4][C][4], m_run[4], l_run[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m_run[i] = -INFINITY;
        l_run[i] = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][c][e] = 0.f;
    }
    const int W = (R + 63) / 64;
    const float *kp = static_cast<const float *>(a.kp), *vp = static_cast<const float *>(a.vp);
    // slots below this are seen by every row of the tile
    const int all = a.anc_mask ? P : P + rt * ROWS / G + 1;
    auto load = [&](int k0, int buf) {
        float *ks = tiles + buf * L::TILE, *vs = ks + kKeys * LD;
#pragma unroll
        for (int u = 0; u < kKeys * VR / THREADS; ++u) {
            const int e = tid + u * THREADS, kk = e / VR, c = (e - kk * VR) * 4, slot = k0 + kk;
            bool ok = slot < kend;
            size_t at = 0;
            if (ok) {
                const int page = a.map.page_of(b, slot);
                ok = a.map.good(page);
                if (ok) {
                    at = (a.map.row(page, slot) * a.Hkv + g) * DH + c;
                } else if (c == 0) {
                    bad_at[buf] = k0;
                    set_status(a.status, MEDUSA_DEV_BAD_PAGE);
                }
            }
            cp_async16(smem_at(ks + kk * LD + c), kp + at, ok);
            cp_async16(smem_at(vs + kk * LD + c), vp + at, ok);
            if (c == 0) key_ok[buf * kKeys + kk] = ok;
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    if (tid < 2) bad_at[tid] = -1;
    __syncthreads();
    load(kbeg, 0);
    int buf = 0;
    for (int k0 = kbeg; k0 < kend; k0 += kKeys, buf ^= 1) {
        asm volatile("cp.async.wait_group 0;\n" ::: "memory");
        __syncthreads();  // the stage is there, and the other place is free
        if (k0 + kKeys < kend) load(k0 + kKeys, buf ^ 1);
        const float *ks = tiles + buf * L::TILE, *vs = ks + kKeys * LD;
        const bool masked = bad_at[buf] == k0 || k0 + kKeys > min(all, kend);
        float s[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int c = 0; c < DH; c += 4) {
            float4 q[4], k[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4 *>(qs + (ty * 4 + i) * LD + c);
#pragma unroll
            for (int j = 0; j < 2; ++j) k[j] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * j) * LD + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    s[i][j] = fmaf(q[i].x, k[j].x, fmaf(q[i].y, k[j].y, fmaf(q[i].z, k[j].z, fmaf(q[i].w, k[j].w, s[i][j]))));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float cm = -INFINITY;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                bool see = true;
                if (masked) {
                    const int kk = tx + 16 * j, slot = k0 + kk, t = slot - P;
                    see = live[i] && key_ok[buf * kKeys + kk];
                    if (see && t >= 0)
                        see = a.anc_mask ? (a.anc_mask[((size_t)b * R + row[i]) * W + (t >> 6)] >> (t & 63)) & 1u
                                         : t <= row[i];
                }
                s[i][j] = see ? s[i][j] * a.scale_log2 : -INFINITY;
                cm = fmaxf(cm, s[i][j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, o));
            const float m_new = fmaxf(m_run[i], cm);
            const float mu = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = m_run[i] == m_new ? 1.f : exp2f(m_run[i] - mu);
            m_run[i] = m_new;
            l_run[i] *= alpha;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p = exp2f(s[i][j] - mu);
                l_run[i] += p;
                ps[(ty * 4 + i) * LP + tx + 16 * j] = p;
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][c][e] *= alpha;
        }
        __syncwarp();  // a row's 16 threads are in one warp
#pragma unroll 2
        for (int kk = 0; kk < kKeys; kk += 4) {
            float4 p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(ps + (ty * 4 + i) * LP + kk);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float4 v = *reinterpret_cast<const float4 *>(vs + (kk + u) * LD + tx * 4 + 64 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
                        // a key the row does not see adds nothing, whatever V holds
                        if (!masked || w != 0.f) {
                            acc[i][c][0] = fmaf(w, v.x, acc[i][c][0]);
                            acc[i][c][1] = fmaf(w, v.y, acc[i][c][1]);
                            acc[i][c][2] = fmaf(w, v.z, acc[i][c][2]);
                            acc[i][c][3] = fmaf(w, v.w, acc[i][c][3]);
                        }
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], o);
        if (!live[i]) continue;
        const float inv = a.ns > 1 ? 1.f : l_run[i] == 0.f ? 0.f : 1.f / l_run[i];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float4 v = make_float4(acc[i][c][0] * inv, acc[i][c][1] * inv, acc[i][c][2] * inv, acc[i][c][3] * inv);
            if (a.ns == 1)
                store4(out_row(i) + tx * 4 + 64 * c, v);
            else
                *reinterpret_cast<float4 *>(a.part_o + part_row(i) * DH + tx * 4 + 64 * c) = v;
        }
        if (a.ns > 1 && tx == 0) a.part_ml[part_row(i)] = make_float2(m_run[i], l_run[i]);
    }
}

// ---- few rows
//
// fp32, at most kVecRows rows a KV head.  128 threads, ROWS rows: a warp scores four keys
// at a time, eight lanes a key, a lane holding DH / 8 of its elements and of the rows'
// outputs; the next keys are on their way meanwhile.  Every eight lanes keep a running
// maximum and sum of their own, which are joined at the end.
//
// Bound by the bytes for a row or two: 8 single tokens x 8 heads behind 2048 slots, dh 128
// (134 MB): 26.6 us, 5.1 TB/s, then by the fp32 products and the exchanges that sum a score
// over its lanes: 4 rows 38, 8 rows 60, 16 rows 100, where tiles of 32 rows take 114 whatever
// they hold.
constexpr int kVecRows = 16, kVecTile = 4, kVecThreads = 128;
constexpr int vec_ctas_per_sm(int rows) { return rows == 1 ? 4 : rows == 2 ? 3 : 2; }  // registers

template <int DH, int ROWS>
__global__ void __launch_bounds__(kVecThreads, vec_ctas_per_sm(ROWS)) paged_attn_vec_kernel(CacheAttnArgs a) {
    pdl_enter();
    constexpr int V = DH / 32, WARPS = kVecThreads / 32, STEP = 4 * WARPS;
    __shared__ float s_o[WARPS][ROWS][DH];
    __shared__ float2 s_ml[WARPS][ROWS];
    const int g = blockIdx.x / a.row_tiles, m0 = (blockIdx.x - g * a.row_tiles) * ROWS;
    const int R = a.R, G = a.H / a.Hkv, W = (R + 63) / 64;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, part = lane & 7, mine = lane >> 3;
    CacheItem it;
    find_item<false, kRangeUnit, true>(a, [&](int P, int b) {
        const int n = live_rows(a, b);
        return n == 0 ? 0 : P + (a.anc_mask ? n : min(n, (m0 + ROWS - 1) / G + 1));
    }, it);
    const int b = it.b, P = it.P, kend = it.kend, M = live_rows(a, b) * G;
    if (m0 >= M) return;  // uniform over the CTA
    int row[ROWS], head[ROWS];
    float4 q[ROWS][V], acc[ROWS][V];
    float m_run[ROWS], l_run[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const int m = min(m0 + u, M - 1);
        row[u] = m / G;
        head[u] = g * G + m - row[u] * G;
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) +
                                                             (((size_t)b * R + row[u]) * a.H + head[u]) * DH);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            q[u][v] = src[8 * v + part];
            acc[u][v] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        m_run[u] = -INFINITY;
        l_run[u] = 0.f;
    }
    float4 k[V], v[V];
    bool ok = false;
    int page = 0;
    auto look_up = [&](int k0) { page = k0 < kend ? a.map.page_of(b, k0) : 0; };
    // the lane's piece of key k0 + mine, whose page has been looked up (the four are in one);
    // looks up the next ones'
    auto load = [&](int k0) {
        const int slot = k0 + mine;
        ok = slot < kend;
        if (k0 < kend && !a.map.good(page)) {
            set_status(a.status, MEDUSA_DEV_BAD_PAGE);
            ok = false;
        }
        if (ok) {
            const size_t at = (a.map.row(page, slot) * a.Hkv + g) * DH;
            const float4 *ks = reinterpret_cast<const float4 *>(static_cast<const float *>(a.kp) + at) + part;
            const float4 *vs = reinterpret_cast<const float4 *>(static_cast<const float *>(a.vp) + at) + part;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                k[e] = ks[8 * e];
                v[e] = vs[8 * e];
            }
        }
        look_up(k0 + STEP);
    };
    auto dot4 = [](const float4 &x, const float4 &y, float s) {
        return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
    };
    const int first = it.kbeg + 4 * warp;
    look_up(first);
    load(first);
    for (int k0 = first; k0 < kend; k0 += STEP) {
        float s[ROWS];
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            s[u] = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) s[u] = dot4(q[u][e], k[e], s[u]);
        }
        float4 x[V];
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = v[e];
        const bool here = ok;
        const int t = k0 + mine - P;
        load(k0 + STEP);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < ROWS; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            bool see = here;
            if (see && t >= 0)
                see = a.anc_mask ? (a.anc_mask[((size_t)b * R + row[u]) * W + (t >> 6)] >> (t & 63)) & 1u : t <= row[u];
            if (!see) continue;  // (whatever V holds)
            const float y = s[u] * a.scale_log2;
            if (y > m_run[u]) {
                const float alpha = exp2f(m_run[u] - y);
                m_run[u] = y;
                l_run[u] *= alpha;
#pragma unroll
                for (int e = 0; e < V; ++e)
                    acc[u][e] = make_float4(acc[u][e].x * alpha, acc[u][e].y * alpha, acc[u][e].z * alpha, acc[u][e].w * alpha);
            }
            const float p = exp2f(y - (m_run[u] == -INFINITY ? 0.f : m_run[u]));
            l_run[u] += p;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                acc[u][e].x = fmaf(p, x[e].x, acc[u][e].x);
                acc[u][e].y = fmaf(p, x[e].y, acc[u][e].y);
                acc[u][e].z = fmaf(p, x[e].z, acc[u][e].z);
                acc[u][e].w = fmaf(p, x[e].w, acc[u][e].w);
            }
        }
        __syncwarp();
    }
    // ---- the warp's four sums, then the CTA's
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        float top = m_run[u];
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float f = exp2f(m_run[u] - (top == -INFINITY ? 0.f : top));
        float l = f * l_run[u];
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (lane == 0) s_ml[warp][u] = make_float2(top, l);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            // (a sum with a weight of zero adds nothing)
            float y[4] = {acc[u][e].x, acc[u][e].y, acc[u][e].z, acc[u][e].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = f == 0.f ? 0.f : y[i] * f;
                y[i] += __shfl_xor_sync(0xffffffffu, y[i], 8);
                y[i] += __shfl_xor_sync(0xffffffffu, y[i], 16);
            }
            if (mine == 0)
                *reinterpret_cast<float4 *>(&s_o[warp][u][(8 * e + part) * 4]) = make_float4(y[0], y[1], y[2], y[3]);
        }
    }
    __syncthreads();
    for (int i = tid; i < ROWS * DH; i += kVecThreads) {
        const int u = i / DH, c = i - u * DH;
        if (m0 + u >= M) break;
        float top = -INFINITY, l = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_ml[w][u].x);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = exp2f(s_ml[w][u].x - (top == -INFINITY ? 0.f : top));
            l = fmaf(f, s_ml[w][u].y, l);
            if (f != 0.f) y = fmaf(f, s_o[w][u][c], y);
        }
        const int m = m0 + u, r = m / G, h = g * G + m - r * G;
        if (a.ns == 1) {
            static_cast<float *>(a.out)[(((size_t)b * R + r) * a.H + h) * DH + c] = l == 0.f ? 0.f : y / l;
        } else {
            const size_t at = ((size_t)it.range * a.H + h) * R + r;
            a.part_o[at * DH + c] = y;
            if (c == 0) a.part_ml[at] = make_float2(top, l);
        }
    }
}

// ------------------------------------------------------------------- join ---

// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over a row's key ranges.  An empty range
// (l = 0) has no O row.  The O rows do not depend on the weights: the first of them are
// on their way while those are computed.

// Many rows: eight lanes a row, so that many rows are on their way.
template <typename T, int DH>
__global__ void __launch_bounds__(128, 4) paged_join_rows_kernel(CacheAttnArgs a) {
    pdl_enter();
    constexpr int C = DH / 8, V = C / 4, AHEAD = 4;  // a lane's columns, vectors of them
    const int lane = threadIdx.x & 31, c = lane & 7, R = a.R, H = a.H;
    const int groups = (R + 3) / 4;
    const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (item >= (long long)a.B * H * groups) return;
    const int r = (int)(item % groups) * 4 + (lane >> 3);
    const int bh = (int)(item / groups), b = bh / H, h = bh - b * H;
    const bool live = r < live_rows(a, b);
    const int first = a.starts ? a.starts[b] : b * a.ns, NS = a.starts ? a.starts[b + 1] - first : a.ns;
    if (a.ranges && NS == 1) return;  // written already
    const size_t step = (size_t)H * R, at = first * step + (size_t)h * R + (live ? r : 0);
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + at * DH) + c * V;
    float4 row[AHEAD][V];
    auto load = [&](int s, float4 (&x)[V]) {
        if (s < NS)
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = po[s * step * (DH / 4) + v];
    };
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) load(s, row[s]);
    const float2 empty = make_float2(-INFINITY, 0.f);
    auto ml = [&](int s) { return s < NS ? a.part_ml[at + s * step] : empty; };
    const float2 mine = ml(c);  // of range c; ranges from 8 on are read again below
    float M = mine.y != 0.f ? mine.x : -INFINITY;
    for (int s = c + 8; s < NS; s += 8) {
        const float2 x = ml(s);
        if (x.y != 0.f) M = fmaxf(M, x.x);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f, w = 0.f, acc[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v][0] = acc[v][1] = acc[v][2] = acc[v][3] = 0.f;
    for (int s0 = 0; s0 < NS; s0 += AHEAD) {
        if ((s0 & 7) == 0) {
            const float2 x = s0 == 0 ? mine : ml(s0 + c);
            w = x.y != 0.f ? exp2f(x.x - mu) : 0.f;
            if (x.y != 0.f) L = fmaf(w, x.y, L);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const float f = __shfl_sync(0xffffffffu, w, (lane & 24) | ((s0 + i) & 7));
            if (s0 + i < NS && f != 0.f) {
#pragma unroll
                for (int v = 0; v < V; ++v) add4(acc[v], f, row[i][v]);
            }
            load(s0 + AHEAD + i, row[i]);
        }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (!live) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    T *dst = static_cast<T *>(a.out) + (((size_t)b * R + r) * H + h) * DH + c * C;
#pragma unroll
    for (int v = 0; v < V; ++v) store_row4(dst + 4 * v, acc[v], inv);
}

// Few rows: a CTA a row, its ranges dealt to groups of DH / 4 threads (32 rows of some 60
// ranges: 14 us for the whole call, 29 with eight lanes a row).  grid B * H * R
template <typename T, int DH>
__global__ void __launch_bounds__(256) paged_join_ranges_kernel(CacheAttnArgs a) {
    pdl_enter();
    constexpr int COLS = DH / 4, GROUPS = 256 / COLS, AHEAD = 4;
    __shared__ float s_o[GROUPS][COLS][4];
    const int tid = threadIdx.x, lane = tid & 31, c = tid % COLS, group = tid / COLS, R = a.R, H = a.H;
    const int r = blockIdx.x % R, bh = blockIdx.x / R, b = bh / H, h = bh - b * H;
    if (r >= live_rows(a, b)) return;  // uniform over the CTA
    const int first = a.starts ? a.starts[b] : b * a.ns, NS = a.starts ? a.starts[b + 1] - first : a.ns;
    if (a.ranges && NS == 1) return;  // written already
    const size_t step = (size_t)H * R, at = first * step + (size_t)h * R + r;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + at * DH) + c;
    const float2 *ml = a.part_ml + at;
    float4 row[AHEAD];
    auto load = [&](int s, float4 &x) {
        if (s < NS) x = po[s * step * (DH / 4)];
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(group + i * GROUPS, row[i]);
    float M = -INFINITY;
    for (int s = lane; s < NS; s += 32) {
        const float2 x = ml[s * step];
        if (x.y != 0.f) M = fmaxf(M, x.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = lane; s < NS; s += 32) {  // (every warp for itself; from the cache)
        const float2 x = ml[s * step];
        if (x.y != 0.f) L = fmaf(exp2f(x.x - mu), x.y, L);
    }
    L = warp_sum(L);
    for (int s0 = group; s0 < NS; s0 += AHEAD * GROUPS)
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int s = s0 + i * GROUPS;
            if (s < NS) {
                const float2 x = ml[s * step];
                const float f = x.y != 0.f ? exp2f(x.x - mu) : 0.f;
                if (f != 0.f) add4(acc, f, row[i]);
            }
            load(s + AHEAD * GROUPS, row[i]);
        }
#pragma unroll
    for (int e = 0; e < 4; ++e) s_o[group][c][e] = acc[e];
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int x = 1; x < GROUPS; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += s_o[x][c][e];
    store_row4(static_cast<T *>(a.out) + (((size_t)b * R + r) * H + h) * DH + c * 4, acc, L == 0.f ? 0.f : 1.f / L);
}

// Up to kJoinFewRows rows the time is the latency of a row's ranges, beyond it is how
// many rows are on their way: a CTA a row takes 8.9 us for 2080 rows of 2 ranges, eight
// lanes a row 4.3; 42.7 and 7.5 for 16384.
constexpr int kJoinFewRows = 1024;

template <typename T, int DH>
cudaError_t launch_join(const CacheAttnArgs &a, cudaStream_t stream) {
    const long long rows = (long long)a.B * a.H * a.R;
    if (rows <= kJoinFewRows)
        return launch_pdl(paged_join_ranges_kernel<T, DH>, dim3((unsigned)rows), dim3(256), 0, stream, a);
    const long long warps = (long long)a.B * a.H * ((a.R + 3) / 4);
    return launch_pdl(paged_join_rows_kernel<T, DH>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, stream, a);
}

// ------------------------------------------------------------------- host ---

constexpr int kLongStages = 64, kClusterStages = 16;
constexpr int kPairStages = 24;
constexpr double kPairStage = 1.7;  // a stage of two heads, in stages of one

// Key ranges: the count that makes (waves of CTAs) x (stages per CTA + 3) smallest, with 3
// stages (4 of one tile) for the join, 2 where a cluster of up to 8 CTAs joins its own ranges.
//
// Clusters are for at most 128 rows a KV head: 65 rows, 32 heads, prefix 1024 (3 ranges)
// 14.3 -> 12.5 us, prefix 4096 (4) 18.5 -> 14.9, 17 rows 14.7 -> 10.9; 32 rows, 32 heads over
// 8 (5) 14.1 -> 10.8.  Two tiles of rows are more than a few CTAs join as fast: 256 rows,
// prefix 1024, in 2 ranges 15.6 -> 21.4, in 5 12.9 -> 13.8.  Clusters that do not all run
// at once wait for one another: 24 of 6 CTAs (23 fit) 19.0 -> 24.3.  A batch's ranges are not
// dealt out in clusters, so those are for up to kClusterStages stages a CTA: 3 x 65 rows, 8
// heads, up to 3000 slots 19.1 -> 13.0; 4 x 65 up to 8000 (16 stages) 24.9 -> 22.1, equally
// long 35.0 -> 30.2, but with one long sequence among short ones up to 11 stages more.
//
// More tiles of at most 128 rows than SMs: two KV heads a CTA, whose ends are then those of
// one and whose products hide one another's softmax.  Trees of 65 rows, 32 heads, prefix 1024:
// 8 39.0 -> 31.1 us, 16 76.4 -> 60.4, 5 29.5 -> 21.3; 128 of 16 rows, 32 heads over 8, 133 -> 117.
// In one wave that is nearly full the longest sequence sets the time, so that long
// ones (kPairStages) stay apart there: 8 ragged ones up to 4096 slots would take 69 us for 63
// (equally long 86 for 95).  In ranges they lose to single heads (12 up to 2048: 105 for 87).
PagedPlan plan_ranges(medusa_dtype dtype, int B, int R, int H, int Hkv, int dh, int P_max) {
    PagedPlan p;
    const int M = R * (H / Hkv);
    const bool simt = dtype == MEDUSA_F32;
    p.few = !simt && M <= kFewRows;
    p.vec = simt && M <= kVecRows;
    // (tiles of 64 rows where there are enough of them to go round)
    const long long wide = (long long)B * Hkv * ((M + 63) / 64) * ((P_max + R + kRangeUnit - 1) / kRangeUnit);
    p.simt_rows = M > 32 && 2 * wide >= 3 * device_sm_count() ? 64 : 32;
    const int rows = p.vec ? kVecTile : simt ? p.simt_rows : kPagedTileRows, sub = simt || p.few ? kRangeUnit : kPagedStage;
    const int slots = (p.few ? cache_few_ctas_per_sm(false, M) : p.vec ? vec_ctas_per_sm(M) : simt ? 2 : 1) * device_sm_count();
    p.row_tiles = p.few ? 1 : (M + rows - 1) / rows;
    const int subs = (P_max + R + sub - 1) / sub;
    double best = 0;
    p.ns = 1;
    p.cluster = p.pair = false;
    const bool split = !simt && !p.few && M <= kPagedTileRows / 2;
    long long ctas = 0;
    for (int pair = 0; pair <= (split && Hkv > 1 && B * (long long)Hkv > slots); ++pair) {
        const long long of_ns = (long long)B * (pair ? (Hkv + 1) / 2 : Hkv) * p.row_tiles;
        const double stage = pair ? kPairStage : 1.0;
        if (pair && of_ns <= slots && 4 * of_ns > 3 * slots && subs > kPairStages) continue;
        const int most = pair ? 1 : std::min<long long>(subs, std::max<long long>(1, 4LL * slots / of_ns));
        for (int ns = 1; ns <= most; ++ns) {
            const int per = (subs + ns - 1) / ns;
            if ((subs + per - 1) / per != ns) continue;
            const bool cluster = split && ns > 1 && ns <= kClusterRanges &&
                                 (B == 1 || per <= kClusterStages) && of_ns <= paged_cluster_slots(dh, ns);
            const double waves = cluster ? 1.0 : (double)((of_ns * ns + slots - 1) / slots);
            const double cost =
                waves * (stage * per + 3) + (cluster ? 2.0 : ns > 1 ? (split ? 4.0 : 3.0) + 0.05 * ns : 0.0);
            if (best == 0 || cost < best) {
                best = cost;
                ctas = of_ns;
                p.ns = ns;
                p.cluster = cluster;
                p.pair = pair;
            }
        }
    }
    p.deal = !simt && p.ns > 1 && !p.cluster && B > 1 && B <= 32;
    p.ranges = B * p.ns;
    // One range a sequence, two tiles of rows a CTA and a wave of CTAs or less: the longest
    // sequence would set the time, so where it is long half as many ranges again are dealt
    // out, which the longer ones take.  Trees of 64 or 65 rows, 32 heads over 8, dh 128, half the
    // sequences short: 8 of up to 8192 slots 91 -> 65 us and 16 of them 94 -> 74 (all
    // equally long 94 -> 98, 101 -> 106), but 16 of up to 4096 53 -> 53 and 8 of up to
    // 2048 30 -> 35.  By the stages of the longest, 8 of 65 rows: 33 51 -> 45 (equally long 52
    // -> 55), 40 60 -> 52 (61 -> 64), 48 70 -> 53 (71 -> 74), 56 80 -> 58 (81 -> 84); 16 of 64:
    // 40 63 -> 59 (67 -> 71), 48 73 -> 64 (78 -> 83), 56 84 -> 69 (89 -> 93).  From
    // kLongStages on it saves four to seven times what it costs where all are equally long.
    // With one tile of rows a CTA (4 of 65 rows, 32 heads over 32), where
    // the copies set the time, 71 -> 78.
    if (!simt && !p.few && p.ns == 1 && B > 1 && B <= 32 && M > kPagedTileRows / 2 &&
        subs >= kLongStages && ctas <= slots) {
        p.deal = true;
        p.ranges = B + (B + 1) / 2;
    }
    return p;
}

template <int DH, int ROWS>
cudaError_t launch_simt(const CacheAttnArgs &a, const PagedPlan &p, cudaStream_t stream) {
    auto kern = paged_attn_simt_kernel<DH, ROWS>;
    constexpr int smem = SimtSmem<DH, ROWS>::TOTAL;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e) return e;
    return launch_pdl(kern, dim3(a.Hkv * p.row_tiles, p.ns, a.B), dim3(4 * ROWS), (size_t)smem, stream, a);
}

}  // namespace

PagedPlan paged_plan(medusa_dtype dtype, int B, int R, int H, int Hkv, int dh, int P_max) {
    PagedPlan p = plan_ranges(dtype, B, R, H, Hkv, dh, P_max);
    const size_t rows = (size_t)p.ranges * H * R;
    p.workspace = MEDUSA_WS_HEADER;
    if (!p.cluster && (p.ns > 1 || p.deal))
        p.workspace += align256(rows * dh * sizeof(float)) + align256(rows * sizeof(float2)) +
                       (p.deal ? align256((B + 1) * sizeof(int)) : 0);
    return p;
}

cudaError_t launch_paged_attention(const PagedPlan &p, medusa_dtype dtype, const void *q, const void *k_pages,
                                   const void *v_pages, const PagedCache &cache,
                                   const int32_t *prefix_len, int P_max, const uint64_t *anc_mask,
                                   const int32_t *n_rows, int B, int R, int H, int Hkv, int dh,
                                   float scale, void *out, void *ws, cudaStream_t stream) {
    CacheAttnArgs a = {};
    a.q = q;
    a.kp = k_pages;
    a.vp = v_pages;
    a.map = PageMap{cache.table, cache.stride, cache.n_pages, cache.shift};
    a.prefix_len = prefix_len;
    a.anc_mask = anc_mask;
    a.n_rows = n_rows;
    a.B = B;
    a.R = R;
    a.H = H;
    a.Hkv = Hkv;
    a.P_max = P_max;
    a.ns = p.ns;
    a.row_tiles = p.row_tiles;
    a.scale_log2 = scale * kLog2e;
    const size_t rows = (size_t)p.ranges * H * R;
    char *w = static_cast<char *>(ws) + MEDUSA_WS_HEADER;
    a.part_o = reinterpret_cast<float *>(w);
    a.part_ml = reinterpret_cast<float2 *>(w + align256(rows * dh * sizeof(float)));
    a.starts = p.deal ? reinterpret_cast<int *>(reinterpret_cast<char *>(a.part_ml) +
                                                align256(rows * sizeof(float2)))
                      : nullptr;
    a.out = out;
    a.status = static_cast<int *>(ws);
    a.wait_polls = wait_budget();
    a.ranges = p.deal && !p.few ? p.ranges : 0;
    a.cluster = p.cluster;
    a.pair = p.pair;
    const int M = R * (H / Hkv);
    cudaError_t e;
    if (p.vec) {
        auto kern = dh == 128 ? (M == 1   ? paged_attn_vec_kernel<128, 1>
                                 : M == 2 ? paged_attn_vec_kernel<128, 2>
                                          : paged_attn_vec_kernel<128, kVecTile>)
                              : (M == 1   ? paged_attn_vec_kernel<64, 1>
                                 : M == 2 ? paged_attn_vec_kernel<64, 2>
                                          : paged_attn_vec_kernel<64, kVecTile>);
        e = launch_pdl(kern, dim3(Hkv * p.row_tiles, p.ns, B), dim3(kVecThreads), 0, stream, a);
    } else if (dtype == MEDUSA_F32) {
        e = p.simt_rows == 32 ? (dh == 128 ? launch_simt<128, 32>(a, p, stream) : launch_simt<64, 32>(a, p, stream))
                              : (dh == 128 ? launch_simt<128, 64>(a, p, stream) : launch_simt<64, 64>(a, p, stream));
    } else {
        e = p.few ? launch_cache_attention_few(a, false, dh, stream) : launch_paged_attention_tc(a, dh, stream);
    }
    note_launch();
    if (e || p.cluster || (p.ns == 1 && !p.deal)) return e;
    e = dtype == MEDUSA_F32 ? (dh == 128 ? launch_join<float, 128>(a, stream) : launch_join<float, 64>(a, stream))
                            : (dh == 128 ? launch_join<bf16, 128>(a, stream) : launch_join<bf16, 64>(a, stream));
    note_launch();
    return e;
}

}  // namespace medusa
