// paged.cu -- rows into the pages of a cache, and the commit of the accepted
// path on them (layout: paged.cuh).
#include <algorithm>

#include "launch.h"
#include "paged.cuh"

namespace medusa {

namespace {

constexpr int kAppendThreads = 256, kCommitThreads = 128;

struct AppendArgs {
    const uint4 *k, *v;
    long long k_step, v_step;  // 16-byte vectors between rows
    uint4 *kp, *vp;
    PageMap map;
    const int32_t *prefix_len;
    const int32_t *n_rows;  // or null: all R
    int R, P_max, row_vecs;
    int *status;
};

// One warp a row of K or of V: its lanes copy 16-byte vectors, kAhead loads ahead of their
// stores, the first of them before the row's place is known (places first: 5.4 us for 8 x
// 65 rows of 32 heads, 12.6 for four ragged prompts of up to 4001 rows of 8 heads, 66 MB;
// as it is 5.1 and 12.0).  Bound by the bytes: 16 x 512 rows of 32 heads, bf16, 268 MB in
// 41.6 us, 6.45 TB/s; small calls by the launch.
// grid (2 R rows over 8 warps, B)
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(AppendArgs a) {
    pdl_enter();
    constexpr int kAhead = 4;
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const int w = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int i = w >> 1;
    const bool is_v = w & 1;
    if (i >= a.R || (a.n_rows && i >= a.n_rows[b])) return;  // (rows behind the last are not read)
    const long long r = (long long)b * a.R + i;
    const uint4 *src = is_v ? a.v + r * a.v_step : a.k + r * a.k_step;
    uint4 x[kAhead];
    auto load = [&](int c) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (c + 32 * u < a.row_vecs) x[u] = ld_stream16(src + c + 32 * u);
    };
    load(lane);
    const int P = a.prefix_len[b];
    if (P < 0 || P > a.P_max) {
        set_status(a.status, MEDUSA_DEV_BAD_PREFIX);
        return;
    }
    const int page = a.map.page_of(b, P + i);
    if (!a.map.good(page)) {
        set_status(a.status, MEDUSA_DEV_BAD_PAGE);
        return;
    }
    uint4 *dst = (is_v ? a.vp : a.kp) + a.map.row(page, P + i) * a.row_vecs;
    for (int c = lane; c < a.row_vecs;) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (c + 32 * u < a.row_vecs) dst[c + 32 * u] = x[u];
        c += 32 * kAhead;
        load(c);
    }
}

struct PagedCommitArgs {
    uint4 *kp, *vp;
    PageMap map;
    const int32_t *prefix_len, *path, *accept_len;
    int32_t *new_prefix_len;
    int K, R, P_max, row_vecs;
    int *status;
};

// The commit of commit.cuh with a page looked up for every slot.  A thread owns
// whole 16-byte columns and reads all rows of a column before it writes one, so
// no barrier separates sources from targets.  Bound by the launch and two dependent
// lookups: one sequence 2.2 us, 32 sequences of 32 heads 2.5.  grid (column blocks, B)
__global__ void __launch_bounds__(kCommitThreads) paged_commit_kernel(PagedCommitArgs a) {
    pdl_enter();
    __shared__ size_t s_src[MEDUSA_MAX_HEADS + 1], s_dst[MEDUSA_MAX_HEADS + 1];
    __shared__ int s_code;
    const int b = blockIdx.y, tid = threadIdx.x;
    const int L = a.accept_len[b], P = a.prefix_len[b];
    if (tid == 0) s_code = P < 0 || P > a.P_max                       ? MEDUSA_DEV_BAD_PREFIX
                           : L < 0 || L > min(a.K, a.R - 1) ? MEDUSA_DEV_BAD_PATH
                                                            : MEDUSA_DEV_OK;
    __syncthreads();
    if (s_code == MEDUSA_DEV_OK && tid <= L) {
        const int node = a.path[(size_t)b * (a.K + 1) + tid];
        if (node < 0 || node >= a.R) {
            atomicMax(&s_code, MEDUSA_DEV_BAD_PATH);
        } else {
            const int from = a.map.page_of(b, P + node), to = a.map.page_of(b, P + tid);
            if (!a.map.good(from) || !a.map.good(to)) atomicMax(&s_code, MEDUSA_DEV_BAD_PAGE);
            s_src[tid] = a.map.row(from, P + node) * a.row_vecs;
            s_dst[tid] = a.map.row(to, P + tid) * a.row_vecs;
        }
    }
    __syncthreads();
    const int code = s_code;
    if (tid == 0) {
        if (code != MEDUSA_DEV_OK) set_status(a.status, code);
        if (blockIdx.x == 0) a.new_prefix_len[b] = code == MEDUSA_DEV_OK ? P + L + 1 : P;
    }
    if (code != MEDUSA_DEV_OK) return;
    for (int c = blockIdx.x * kCommitThreads + tid; c < a.row_vecs; c += gridDim.x * kCommitThreads) {
        uint4 kb[MEDUSA_MAX_HEADS + 1], vb[MEDUSA_MAX_HEADS + 1];
#pragma unroll
        for (int q = 0; q <= MEDUSA_MAX_HEADS; ++q)
            if (q <= L && s_src[q] != s_dst[q]) {
                kb[q] = a.kp[s_src[q] + c];
                vb[q] = a.vp[s_src[q] + c];
            }
#pragma unroll
        for (int q = 0; q <= MEDUSA_MAX_HEADS; ++q)
            if (q <= L && s_src[q] != s_dst[q]) {
                a.kp[s_dst[q] + c] = kb[q];
                a.vp[s_dst[q] + c] = vb[q];
            }
    }
}

}  // namespace

cudaError_t launch_paged_append(size_t elt, const void *k, const void *v, long long k_stride,
                                long long v_stride, void *k_pages, void *v_pages,
                                const PagedCache &cache, const int32_t *prefix_len, int P_max,
                                const int32_t *n_rows, int B, int R, int Hkv, int dh, void *ws,
                                cudaStream_t stream) {
    AppendArgs a;
    a.k = static_cast<const uint4 *>(k);
    a.v = static_cast<const uint4 *>(v);
    a.k_step = k_stride * (long long)elt / 16;
    a.v_step = v_stride * (long long)elt / 16;
    a.kp = static_cast<uint4 *>(k_pages);
    a.vp = static_cast<uint4 *>(v_pages);
    a.map = PageMap{cache.table, cache.stride, cache.n_pages, cache.shift};
    a.prefix_len = prefix_len;
    a.n_rows = n_rows;
    a.R = R;
    a.P_max = P_max;
    a.row_vecs = (int)((size_t)Hkv * dh * elt / 16);
    a.status = static_cast<int *>(ws);
    const unsigned gx = (unsigned)((2LL * R + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
    cudaError_t e = launch_pdl(paged_append_kernel, dim3(gx, B), dim3(kAppendThreads), 0, stream, a);
    note_launch();
    return e;
}

cudaError_t launch_commit_paged(size_t elt, void *k_pages, void *v_pages, const PagedCache &cache,
                                const int32_t *prefix_len, int P_max, const int32_t *path,
                                const int32_t *accept_len, int B, int K, int R, int Hkv, int dh,
                                int32_t *new_prefix_len, void *ws, cudaStream_t stream) {
    PagedCommitArgs a;
    a.kp = static_cast<uint4 *>(k_pages);
    a.vp = static_cast<uint4 *>(v_pages);
    a.map = PageMap{cache.table, cache.stride, cache.n_pages, cache.shift};
    a.prefix_len = prefix_len;
    a.path = path;
    a.accept_len = accept_len;
    a.new_prefix_len = new_prefix_len;
    a.K = K;
    a.R = R;
    a.P_max = P_max;
    a.row_vecs = (int)((size_t)Hkv * dh * elt / 16);
    a.status = static_cast<int *>(ws);
    const int cx = std::max(1, std::min(64, (a.row_vecs + kCommitThreads - 1) / kCommitThreads));
    cudaError_t e = launch_pdl(paged_commit_kernel, dim3(cx, B), dim3(kCommitThreads), 0, stream, a);
    note_launch();
    return e;
}

}  // namespace medusa
