// api.cu -- the extern "C" boundary of libmedusa_gb300.so.
//
// Every entry point validates its arguments on the host, launches nothing on
// a bad argument, and maps CUDA failures to MEDUSA_ERR_CUDA.  The message of
// the last failure on the calling thread is kept for medusa_last_error().
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "launch.h"

namespace medusa {

namespace {

thread_local char g_err[512] = "";
std::atomic<uint64_t> g_launches{0};

medusa_status fail(medusa_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}

medusa_status cuda_fail(cudaError_t e, const char *where) {
    return fail(MEDUSA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

medusa_status check_ws(const void *ws, size_t have, size_t need, const char *who) {
    if (!ws) return fail(MEDUSA_ERR_WORKSPACE, "%s: workspace is NULL", who);
    if (!aligned256(ws)) return fail(MEDUSA_ERR_WORKSPACE, "%s: workspace not 256-byte aligned", who);
    if (have < need)
        return fail(MEDUSA_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", who, have, need);
    return MEDUSA_OK;
}

}  // namespace

namespace {

// Poll limit of the bounded device waits; MEDUSA_FAULT_WAIT_BUDGET sets the
// first value (fault injection), medusa_set_wait_budget any later one.
constexpr uint32_t kDefaultWaitPolls = 1u << 16;
std::atomic<uint32_t> g_wait_polls{kDefaultWaitPolls};
std::once_flag g_wait_env_once;

void read_wait_env() {
    const char *v = std::getenv("MEDUSA_FAULT_WAIT_BUDGET");
    if (!v || !*v) return;
    char *end = nullptr;
    const unsigned long n = std::strtoul(v, &end, 10);
    if (end && *end == '\0' && n <= 0xffffffffUL) g_wait_polls.store((uint32_t)n);
}

}  // namespace

uint32_t wait_budget() {
    std::call_once(g_wait_env_once, read_wait_env);
    return g_wait_polls.load(std::memory_order_relaxed);
}

NvtxRange::NvtxRange(const char *name) { nvtxRangePushA(name); }
NvtxRange::~NvtxRange() { nvtxRangePop(); }

int device_sm_count() {
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    std::lock_guard<std::mutex> lk(mu);
    if (!cache[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 152;
        cache[dev] = n;
    }
    return cache[dev];
}

void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

void set_last_error(const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
}

}  // namespace medusa

using namespace medusa;

extern "C" {

const char *medusa_status_string(medusa_status s) {
    switch (s) {
    case MEDUSA_OK: return "MEDUSA_OK";
    case MEDUSA_ERR_INVALID_ARG: return "MEDUSA_ERR_INVALID_ARG";
    case MEDUSA_ERR_UNSUPPORTED: return "MEDUSA_ERR_UNSUPPORTED";
    case MEDUSA_ERR_WORKSPACE: return "MEDUSA_ERR_WORKSPACE";
    case MEDUSA_ERR_CUDA: return "MEDUSA_ERR_CUDA";
    case MEDUSA_ERR_TIMEOUT: return "MEDUSA_ERR_TIMEOUT";
    case MEDUSA_ERR_DEVICE_CHECK: return "MEDUSA_ERR_DEVICE_CHECK";
    }
    return "MEDUSA_ERR_UNKNOWN";
}

const char *medusa_last_error(void) { return g_err; }

uint64_t medusa_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

uint32_t medusa_wait_budget(void) { return wait_budget(); }

void medusa_set_wait_budget(uint32_t polls) {
    std::call_once(g_wait_env_once, read_wait_env);
    g_wait_polls.store(polls, std::memory_order_relaxed);
}

medusa_status medusa_read_device_status(const void *ws, int32_t *status_host, medusa_stream stream) {
    if (!ws || !status_host) return fail(MEDUSA_ERR_INVALID_ARG, "read_device_status: NULL pointer");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(status_host, ws, sizeof(int32_t), cudaMemcpyDeviceToHost, st);
    if (e) return cuda_fail(e, "read_device_status");
    e = cudaStreamSynchronize(st);
    if (e) return cuda_fail(e, "read_device_status");
    return MEDUSA_OK;
}

medusa_status medusa_clear_device_status(void *ws, medusa_stream stream) {
    if (!ws) return fail(MEDUSA_ERR_INVALID_ARG, "clear_device_status: NULL workspace");
    cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, "clear_device_status");
    return MEDUSA_OK;
}

// ----------------------------------------------------------------- heads ---

size_t medusa_heads_workspace_size(int B, int K, int d, int V, int top_s) {
    if (B < 1 || K < 1 || d < 1 || V < 1 || top_s < 1) return 0;
    return heads_workspace_bytes(B, K, d, V, top_s);
}

size_t medusa_heads_lm_workspace_size(int B, int K, int d, int V, int top_s) {
    if (B < 1 || K < 1 || d < 1 || V < 1 || top_s < 1) return 0;
    return heads_workspace_bytes(B, K, d, V, top_s, true);
}

}  // extern "C"

namespace {

medusa_status check_heads(const char *who, medusa_dtype dtype, const void *h, const void *W1,
                          const void *b1, const void *W2, int B, int d, int V, int K, int top_s,
                          const int32_t *topk_ids, const float *topk_logp, bool need_logp = true) {
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dtype);
    if (!h || !W1 || !W2 || !topk_ids || (need_logp && !topk_logp))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
    if (B < 1 || B > MEDUSA_MAX_BATCH)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: B=%d outside 1..%d", who, B, MEDUSA_MAX_BATCH);
    if (K < 1 || K > MEDUSA_MAX_HEADS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: K=%d outside 1..%d", who, K, MEDUSA_MAX_HEADS);
    if (d < 8 || d % 8)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: d=%d must be a positive multiple of 8", who, d);
    if (top_s < 1 || top_s > MEDUSA_MAX_TOP_S || top_s > V)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: top_s=%d outside 1..min(16, V)", who, top_s);
    const int nb = B <= 1 ? 1 : B <= 2 ? 2 : B <= 4 ? 4 : 8;  // batch bucket held in smem
    if ((size_t)nb * d * sizeof(float) > 160 * 1024)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: %d x d x 4 = %zu bytes exceeds 160 KiB", who, nb,
                    (size_t)nb * d * sizeof(float));
    if (!aligned16(h) || !aligned16(W1) || !aligned16(W2) || (b1 && !aligned16(b1)))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: tensor pointers must be 16-byte aligned", who);
    return MEDUSA_OK;
}

}  // namespace

extern "C" {

medusa_status medusa_heads(medusa_dtype dtype, const void *h, const void *W1, const void *b1,
                           const void *W2, int B, int d, int V, int K, int top_s,
                           int32_t *topk_ids, float *topk_logp, void *ws, size_t ws_bytes,
                           medusa_stream stream) {
    const NvtxRange range("medusa_heads");
    const char *who = "medusa_heads";
    if (medusa_status s = check_heads(who, dtype, h, W1, b1, W2, B, d, V, K, top_s, topk_ids,
                                      topk_logp))
        return s;
    if (medusa_status s = check_ws(ws, ws_bytes, heads_workspace_bytes(B, K, d, V, top_s), who))
        return s;
    cudaError_t e = launch_heads(dtype, h, nullptr, W1, b1, W2, B, d, V, K, top_s, topk_ids,
                                 topk_logp, nullptr, nullptr, nullptr, ws,
                                 static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

medusa_status medusa_heads_lm(medusa_dtype dtype, const void *h, const void *W_lm, const void *W1,
                              const void *b1, const void *W2, int B, int d, int V, int K,
                              int top_s, int32_t *root, float *root_logp, int32_t *topk_ids,
                              float *topk_logp, void *ws, size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_heads_lm");
    const char *who = "medusa_heads_lm";
    if (medusa_status s = check_heads(who, dtype, h, W1, b1, W2, B, d, V, K, top_s, topk_ids,
                                      topk_logp))
        return s;
    if (!W_lm || !root || !root_logp)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned16(W_lm))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: W_lm must be 16-byte aligned", who);
    if (medusa_status s =
            check_ws(ws, ws_bytes, heads_workspace_bytes(B, K, d, V, top_s, true), who))
        return s;
    cudaError_t e = launch_heads(dtype, h, W_lm, W1, b1, W2, B, d, V, K, top_s, topk_ids,
                                 topk_logp, root, root_logp, nullptr, ws,
                                 static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

medusa_status medusa_heads_sample(medusa_dtype dtype, const void *h, const void *W1,
                                  const void *b1, const void *W2, int B, int d, int V, int K,
                                  float temperature, uint64_t seed, uint64_t step,
                                  int32_t *drafts, float *draft_logits, void *ws,
                                  size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_heads_sample");
    const char *who = "medusa_heads_sample";
    // drafts is the top-1 list of the perturbed keys; no log-probabilities
    if (medusa_status s =
            check_heads(who, dtype, h, W1, b1, W2, B, d, V, K, 1, drafts, nullptr, false))
        return s;
    if (!draft_logits) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL draft_logits", who);
    if (!(temperature > 0.f) || !(temperature < 1e30f))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: temperature must be positive and finite", who);
    if (medusa_status s = check_ws(ws, ws_bytes, heads_workspace_bytes(B, K, d, V, 1), who))
        return s;
    SampleArgs smp;
    smp.on = 1;
    smp.inv_T = 1.f / temperature;
    smp.seed = seed;
    smp.step = step;
    smp.logits_out = draft_logits;
    cudaError_t e = launch_heads(dtype, h, nullptr, W1, b1, W2, B, d, V, K, 1, drafts, nullptr,
                                 nullptr, nullptr, &smp, ws, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

// ------------------------------------------------------------------ tree ---

size_t medusa_build_tree_workspace_size(int B, int K, int top_s, int n) {
    return tree_workspace_bytes(B, K, top_s, n);
}

}  // extern "C"

namespace {

medusa_status check_tree(const char *who, const int32_t *root, const int32_t *topk_ids,
                         const float *weights, int B, int K, const int32_t *s_host, int top_s,
                         int n, const int32_t *tokens, const int32_t *parent,
                         const int32_t *depth, const int32_t *pos_id, const uint64_t *anc_mask,
                         const int32_t *paths, const int32_t *n_leaf, const void *ws,
                         size_t ws_bytes) {
    if (!root || !topk_ids || !weights || !s_host || !tokens || !parent || !depth || !pos_id ||
        !anc_mask || !paths || !n_leaf)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (B < 1) return fail(MEDUSA_ERR_INVALID_ARG, "%s: B=%d", who, B);
    if (K < 1 || K > MEDUSA_MAX_HEADS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: K=%d outside 1..%d", who, K, MEDUSA_MAX_HEADS);
    if (top_s < 1 || top_s > MEDUSA_MAX_TOP_S)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: top_s=%d outside 1..16", who, top_s);
    long long total = 0, level = 1;
    for (int k = 0; k < K; ++k) {
        if (s_host[k] < 1 || s_host[k] > top_s)
            return fail(MEDUSA_ERR_INVALID_ARG, "%s: s[%d]=%d outside 1..top_s", who, k, s_host[k]);
        level *= s_host[k];
        total += level;
        if (total > (1 << 20)) break;
    }
    if (n < 1 || n + 1 > MEDUSA_MAX_TREE_ROWS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: n=%d outside 1..%d", who, n,
                    MEDUSA_MAX_TREE_ROWS - 1);
    if (n > total)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: n=%d exceeds the %lld nodes of the full tree",
                    who, n, total);
    return check_ws(ws, ws_bytes, tree_workspace_bytes(B, K, top_s, n), who);
}

}  // namespace

extern "C" {

medusa_status medusa_build_tree(const int32_t *root, const int32_t *topk_ids,
                                const float *topk_logp, int B, int K, const int32_t *s_host,
                                int top_s, int n, const int32_t *prefix_len, int32_t *tokens,
                                int32_t *parent, int32_t *depth, int32_t *pos_id,
                                uint64_t *anc_mask, int32_t *paths, int32_t *n_leaf, void *ws,
                                size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_build_tree");
    const char *who = "medusa_build_tree";
    if (medusa_status s = check_tree(who, root, topk_ids, topk_logp, B, K, s_host, top_s, n,
                                     tokens, parent, depth, pos_id, anc_mask, paths, n_leaf, ws,
                                     ws_bytes))
        return s;
    cudaError_t e = launch_build_tree(root, topk_ids, topk_logp, false, B, K, s_host, top_s, n,
                                      prefix_len, tokens, parent, depth, pos_id, anc_mask, paths,
                                      n_leaf, ws, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

medusa_status medusa_build_tree_static(const int32_t *root, const int32_t *topk_ids,
                                       const float *log_a, int B, int K, const int32_t *s_host,
                                       int top_s, int n, const int32_t *prefix_len,
                                       int32_t *tokens, int32_t *parent, int32_t *depth,
                                       int32_t *pos_id, uint64_t *anc_mask, int32_t *paths,
                                       int32_t *n_leaf, void *ws, size_t ws_bytes,
                                       medusa_stream stream) {
    const NvtxRange range("medusa_build_tree_static");
    const char *who = "medusa_build_tree_static";
    if (medusa_status s = check_tree(who, root, topk_ids, log_a, B, K, s_host, top_s, n, tokens,
                                     parent, depth, pos_id, anc_mask, paths, n_leaf, ws,
                                     ws_bytes))
        return s;
    cudaError_t e = launch_build_tree(root, topk_ids, log_a, true, B, K, s_host, top_s, n,
                                      prefix_len, tokens, parent, depth, pos_id, anc_mask, paths,
                                      n_leaf, ws, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

// ------------------------------------------------------------- attention ---

size_t medusa_tree_attention_workspace_size(medusa_dtype dtype, int B, int R, int H, int dh,
                                            int P_max) {
    if (B < 1 || R < 1 || H < 1 || dh < 1 || P_max < 0) return 0;
    return attention_workspace_bytes(dtype, B, R, H, dh, P_max);
}

medusa_status medusa_tree_attention(medusa_dtype dtype, const void *q, const void *const *k_cache,
                                    const void *const *v_cache, const int32_t *prefix_len,
                                    int P_max, const uint64_t *anc_mask, int B, int R, int H,
                                    int dh, float scale, void *out, void *ws, size_t ws_bytes,
                                    medusa_stream stream) {
    const NvtxRange range("medusa_tree_attention");
    const char *who = "medusa_tree_attention";
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dtype);
    if (!q || !k_cache || !v_cache || !prefix_len || !anc_mask || !out)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (B < 1 || H < 1) return fail(MEDUSA_ERR_INVALID_ARG, "%s: B=%d H=%d", who, B, H);
    if (R < 1 || R > MEDUSA_MAX_TREE_ROWS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: R=%d outside 1..%d", who, R, MEDUSA_MAX_TREE_ROWS);
    if (dh != 64 && dh != 128)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: dh=%d (supported: 64, 128)", who, dh);
    if (P_max < 0) return fail(MEDUSA_ERR_INVALID_ARG, "%s: P_max=%d", who, P_max);
    if (dtype == MEDUSA_F32 && (long long)P_max + R > 16384)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: f32 path needs P_max + R <= 16384", who);
    if (!(scale > 0.f)) return fail(MEDUSA_ERR_INVALID_ARG, "%s: scale must be > 0", who);
    if (!aligned16(q) || !aligned16(out) || !aligned16(anc_mask) || !aligned16(k_cache) ||
        !aligned16(v_cache))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
    if (medusa_status s = check_ws(ws, ws_bytes, attention_workspace_bytes(dtype, B, R, H, dh, P_max), who))
        return s;
    cudaError_t e = launch_tree_attention(dtype, q, k_cache, v_cache, prefix_len, P_max, anc_mask,
                                          B, R, H, dh, scale, out, ws,
                                          static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

// ------------------------------------------------------------- posterior ---

size_t medusa_posterior_workspace_size(int B, int R) {
    if (B < 1 || R < 1) return 0;
    return posterior_workspace_bytes(B, R);
}

}  // extern "C"

namespace {

// The posterior's results may go to device memory or straight to page-locked
// host memory that the device addresses at the same pointer (cudaHostAlloc,
// or cudaHostRegister with mapping, under unified addressing): the select
// kernel writes them there, and the host reads them after the stream syncs.
// Pageable host memory is refused.  If the runtime cannot answer (no device)
// the check is left to the launch.
medusa_status check_result_pointer(const void *p, const char *who) {
    if (!p) return MEDUSA_OK;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return MEDUSA_OK;
    }
    if (at.type == cudaMemoryTypeUnregistered)
        return fail(MEDUSA_ERR_INVALID_ARG,
                    "%s: a result pointer is pageable host memory (device or pinned host memory)",
                    who);
    if (at.type == cudaMemoryTypeHost && at.devicePointer != p)
        return fail(MEDUSA_ERR_INVALID_ARG,
                    "%s: a pinned host result buffer is not mapped at the same device address",
                    who);
    return MEDUSA_OK;
}

medusa_status check_posterior(const char *who, medusa_dtype dtype, const void *logits,
                              const int32_t *tokens, const int32_t *parent, const int32_t *depth,
                              int B, int R, int V, int K, medusa_accept_mode mode, float eps,
                              float delta, float temperature, const int32_t *accept_len,
                              const int32_t *path, const int32_t *path_tokens,
                              const int32_t *next_token, const void *ws, size_t ws_bytes) {
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dtype);
    if (mode != MEDUSA_GREEDY && mode != MEDUSA_TYPICAL)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: unknown mode %d", who, (int)mode);
    if (!logits || !tokens || !parent || !depth || !accept_len || !path || !path_tokens ||
        !next_token)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (B < 1) return fail(MEDUSA_ERR_INVALID_ARG, "%s: B=%d", who, B);
    if (R < 1 || R > MEDUSA_MAX_TREE_ROWS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: R=%d outside 1..%d", who, R, MEDUSA_MAX_TREE_ROWS);
    if (K < 0 || K > MEDUSA_MAX_HEADS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: K=%d outside 0..%d", who, K, MEDUSA_MAX_HEADS);
    const int vn = dtype == MEDUSA_BF16 ? 8 : 4;
    if (V < 1 || V % vn)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: V=%d must be a positive multiple of %d", who, V, vn);
    if (!(temperature > 0.f) || !(eps > 0.f) || !(delta > 0.f))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: eps, delta and temperature must be > 0", who);
    if (!aligned16(logits))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: logits must be 16-byte aligned", who);
    if (medusa_status s = check_ws(ws, ws_bytes, posterior_workspace_bytes(B, R), who)) return s;
    const void *outs[4] = {accept_len, path, path_tokens, next_token};
    for (const void *o : outs)
        if (medusa_status s = check_result_pointer(o, who)) return s;
    return MEDUSA_OK;
}

// Host checks of the commit arguments shared by both commit entry points.
medusa_status check_commit(const char *who, medusa_dtype dtype, const void *const *k_cache,
                           const void *const *v_cache, const int32_t *prefix_len,
                           const int32_t *new_prefix_len, int H, int dh) {
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dtype);
    if (!k_cache || !v_cache || !prefix_len || !new_prefix_len)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (static_cast<const void *>(new_prefix_len) == static_cast<const void *>(prefix_len))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: new_prefix_len must not alias prefix_len", who);
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: cache pointer arrays must be 16-byte aligned", who);
    const size_t elt = dtype == MEDUSA_BF16 ? 2 : 4;
    if (H < 1 || dh < 1 || (long long)H * dh > (1LL << 26))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: H=%d dh=%d", who, H, dh);
    if (((size_t)H * dh * elt) % 16)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: a cache row (H*dh elements) must be a multiple of 16 bytes",
                    who);
    return MEDUSA_OK;
}

}  // namespace

// The posterior with or without the commit (k_cache non-null) and with an
// optional completion word per sequence (the step executor's).
medusa_status medusa::evaluate_posterior_signalled(
    medusa_dtype dtype, const void *logits, const int32_t *tokens, const int32_t *parent,
    const int32_t *depth, int B, int R, int V, int K, medusa_accept_mode mode, float eps,
    float delta, float temperature, int32_t *accept_len, int32_t *path, int32_t *path_tokens,
    int32_t *next_token, int32_t *accept, void *const *k_cache, void *const *v_cache,
    const int32_t *prefix_len, int H, int dh, int32_t *new_prefix_len, void *ws,
    size_t ws_bytes, cudaStream_t stream, uint32_t *done) {
    const char *who = k_cache ? "medusa_evaluate_posterior_commit" : "medusa_evaluate_posterior";
    if (medusa_status s = check_posterior(who, dtype, logits, tokens, parent, depth, B, R, V, K,
                                          mode, eps, delta, temperature, accept_len, path,
                                          path_tokens, next_token, ws, ws_bytes))
        return s;
    if (medusa_status s = check_result_pointer(accept, who)) return s;
    if (k_cache) {
        if (medusa_status s = check_commit(who, dtype, k_cache, v_cache, prefix_len,
                                           new_prefix_len, H, dh))
            return s;
    }
    cudaError_t e = launch_posterior(dtype, logits, tokens, parent, depth, B, R, V, K, mode, eps,
                                     delta, temperature, accept_len, path, path_tokens, next_token,
                                     accept, k_cache, v_cache, prefix_len, H, dh, new_prefix_len,
                                     ws, stream, done);
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

extern "C" {

medusa_status medusa_evaluate_posterior(medusa_dtype dtype, const void *logits,
                                        const int32_t *tokens, const int32_t *parent,
                                        const int32_t *depth, int B, int R, int V, int K,
                                        medusa_accept_mode mode, float eps, float delta,
                                        float temperature, int32_t *accept_len, int32_t *path,
                                        int32_t *path_tokens, int32_t *next_token,
                                        int32_t *accept, void *ws, size_t ws_bytes,
                                        medusa_stream stream) {
    const NvtxRange range("medusa_evaluate_posterior");
    return evaluate_posterior_signalled(dtype, logits, tokens, parent, depth, B, R, V, K, mode,
                                        eps, delta, temperature, accept_len, path, path_tokens,
                                        next_token, accept, nullptr, nullptr, nullptr, 0, 0,
                                        nullptr, ws, ws_bytes, static_cast<cudaStream_t>(stream),
                                        nullptr);
}

medusa_status medusa_evaluate_posterior_commit(
    medusa_dtype dtype, const void *logits, const int32_t *tokens, const int32_t *parent,
    const int32_t *depth, int B, int R, int V, int K, medusa_accept_mode mode, float eps,
    float delta, float temperature, int32_t *accept_len, int32_t *path, int32_t *path_tokens,
    int32_t *next_token, int32_t *accept, void *const *k_cache, void *const *v_cache,
    const int32_t *prefix_len, int H, int dh, int32_t *new_prefix_len, void *ws,
    size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_evaluate_posterior_commit");
    if (!k_cache)
        return fail(MEDUSA_ERR_INVALID_ARG, "medusa_evaluate_posterior_commit: NULL pointer");
    return evaluate_posterior_signalled(dtype, logits, tokens, parent, depth, B, R, V, K, mode,
                                        eps, delta, temperature, accept_len, path, path_tokens,
                                        next_token, accept, k_cache, v_cache, prefix_len, H, dh,
                                        new_prefix_len, ws, ws_bytes,
                                        static_cast<cudaStream_t>(stream), nullptr);
}

// ----------------------------------------------------------- speculative ---

size_t medusa_speculative_workspace_size(int B, int K) {
    if (B < 1 || K < 1) return 0;
    return speculative_workspace_bytes(B, K);
}

medusa_status medusa_speculative_posterior(medusa_dtype dtype, const void *logits,
                                           const int32_t *tokens, const float *draft_logits,
                                           int B, int V, int K, float temperature, uint64_t seed,
                                           uint64_t step, int32_t *accept_len,
                                           int32_t *path_tokens, int32_t *next_token,
                                           int32_t *accept, void *ws, size_t ws_bytes,
                                           medusa_stream stream) {
    const NvtxRange range("medusa_speculative_posterior");
    const char *who = "medusa_speculative_posterior";
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dtype);
    if (!logits || !tokens || !draft_logits || !accept_len || !path_tokens || !next_token)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (B < 1) return fail(MEDUSA_ERR_INVALID_ARG, "%s: B=%d", who, B);
    if (K < 1 || K > MEDUSA_MAX_HEADS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: K=%d outside 1..%d", who, K, MEDUSA_MAX_HEADS);
    if (V < 1 || V % 8)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: V=%d must be a positive multiple of 8", who, V);
    if (!(temperature > 0.f) || !(temperature < 1e30f))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: temperature must be positive and finite", who);
    if (medusa_status s = check_ws(ws, ws_bytes, speculative_workspace_bytes(B, K), who)) return s;
    cudaError_t e = launch_speculative(dtype, logits, tokens, draft_logits, B, V, K, temperature,
                                       seed, step, accept_len, path_tokens, next_token, accept, ws,
                                       static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

// ---------------------------------------------------------------- commit ---

medusa_status medusa_commit_kv(medusa_dtype dtype, void *const *k_cache, void *const *v_cache,
                               const int32_t *prefix_len, const int32_t *path,
                               const int32_t *accept_len, int B, int K, int R, int H, int dh,
                               int32_t *new_prefix_len, void *ws, size_t ws_bytes,
                               medusa_stream stream) {
    const NvtxRange range("medusa_commit_kv");
    const char *who = "medusa_commit_kv";
    if (medusa_status s = check_commit(who, dtype, k_cache, v_cache, prefix_len, new_prefix_len,
                                       H, dh))
        return s;
    if (!path || !accept_len) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (B < 1) return fail(MEDUSA_ERR_INVALID_ARG, "%s: B=%d", who, B);
    if (K < 0 || K > MEDUSA_MAX_HEADS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: K=%d outside 0..%d", who, K, MEDUSA_MAX_HEADS);
    if (R < 1 || R > MEDUSA_MAX_TREE_ROWS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: R=%d outside 1..%d", who, R, MEDUSA_MAX_TREE_ROWS);
    if (medusa_status s = check_ws(ws, ws_bytes, MEDUSA_WS_HEADER, who)) return s;
    cudaError_t e = launch_commit_kv(dtype == MEDUSA_BF16 ? 2 : 4, k_cache, v_cache, prefix_len,
                                     path, accept_len, B, K, R, H, dh, new_prefix_len, ws,
                                     static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

}  // extern "C"

// ------------------------------------------ rotation, 4-bit cache, windows ---

namespace {

constexpr int kMaxPrefix = 1 << 29;  // sums of prefix, sinks and window stay in an int

bool is_dtype(medusa_dtype d) { return d == MEDUSA_F32 || d == MEDUSA_BF16; }

// Shape checks shared by every call on cache rows: B sequences, R rows (at
// most max_rows), H query heads over Hkv KV heads of dh elements.
medusa_status check_heads_shape(const char *who, medusa_dtype dtype, int B, int R, int max_rows,
                                int H, int Hkv, int dh) {
    if (!is_dtype(dtype)) return fail(MEDUSA_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dtype);
    if (B < 1 || B > 65535) return fail(MEDUSA_ERR_INVALID_ARG, "%s: B=%d outside 1..65535", who, B);
    if (R < 1 || R > max_rows)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: R=%d outside 1..%d", who, R, max_rows);
    if (Hkv < 1 || H < Hkv || H > 1024 || H % Hkv)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: H=%d query heads over Hkv=%d KV heads (H <= 1024, "
                    "a multiple of Hkv)", who, H, Hkv);
    if (dh != 64 && dh != 128)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: dh=%d (64 or 128)", who, dh);
    return MEDUSA_OK;
}

medusa_status check_caches(const char *who, const void *k_cache, const void *v_cache,
                           const void *prefix_len, int P_max) {
    if (!k_cache || !v_cache || !prefix_len)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: cache pointer arrays must be 16-byte aligned", who);
    if (P_max < 0 || P_max > kMaxPrefix)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: P_max=%d outside 0..%d", who, P_max, kMaxPrefix);
    return MEDUSA_OK;
}

// Distance between consecutive rows of `heads` vectors (in elements): at
// least a row, and rows keep 16-byte alignment.
medusa_status check_row_stride(const char *who, const char *name, medusa_dtype dtype, int64_t stride,
                               int heads, int dh) {
    const int64_t align = dtype == MEDUSA_BF16 ? 8 : 4;
    if (stride < (int64_t)heads * dh || stride % align || stride > (int64_t)1 << 40)
        return fail(MEDUSA_ERR_INVALID_ARG,
                    "%s: %s=%lld must be at least a row (%d) and a multiple of 16 bytes", who, name,
                    (long long)stride, heads * dh);
    return MEDUSA_OK;
}

medusa_status check_rope(const char *who, medusa_dtype dtype, const void *q, const void *k,
                         int64_t q_stride, int64_t k_stride, const void *q_weight,
                         const void *k_weight, float eps, int norm, const int32_t *pos,
                         const float *inv_freq, int rot, int B, int R, int H, int Hkv, int dh,
                         const void *q_out) {
    if (medusa_status s = check_heads_shape(who, dtype, B, R, 1 << 24, H, Hkv, dh)) return s;
    if ((long long)B * R > 0x7fffffffLL)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: B * R exceeds 2^31 - 1 rows", who);
    if (!q || !k || !q_out || !pos) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (rot < 0 || rot > dh || rot % 16)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: rot=%d must be a multiple of 16 in 0..dh", who, rot);
    if (rot && !inv_freq) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL inv_freq", who);
    if (!norm && (q_weight || k_weight))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: weights given, but norm is 0", who);
    if (norm && (!(eps >= 0.f) || !(eps < 1e30f)))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: eps must be finite and not negative", who);
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || (q_weight && !aligned16(q_weight)) ||
        (k_weight && !aligned16(k_weight)))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: tensor pointers must be 16-byte aligned", who);
    if (medusa_status s = check_row_stride(who, "q_stride", dtype, q_stride, H, dh)) return s;
    return check_row_stride(who, "k_stride", dtype, k_stride, Hkv, dh);
}

medusa_status check_kv4_rows(const char *who, medusa_dtype dtype, const void *k, const void *v,
                             int64_t k_stride, int64_t v_stride, const void *k_cache,
                             const void *v_cache, const int32_t *prefix_len, int P_max, int B,
                             int R, int Hkv, int dh, const void *ws, size_t ws_bytes) {
    if (medusa_status s = check_heads_shape(who, dtype, B, R, kKv4MaxRows, Hkv, Hkv, dh)) return s;
    if (!k || !v) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned16(k) || !aligned16(v))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: tensor pointers must be 16-byte aligned", who);
    if (medusa_status s = check_row_stride(who, "k_stride", dtype, k_stride, Hkv, dh)) return s;
    if (medusa_status s = check_row_stride(who, "v_stride", dtype, v_stride, Hkv, dh)) return s;
    if (medusa_status s = check_caches(who, k_cache, v_cache, prefix_len, P_max)) return s;
    return check_ws(ws, ws_bytes, MEDUSA_WS_HEADER, who);
}

bool attention_shape_ok(medusa_dtype dtype, int B, int R, int H, int Hkv, int dh, int P_max,
                        int window, int sinks) {
    return is_dtype(dtype) && B >= 1 && B <= 65535 && R >= 1 && R <= MEDUSA_MAX_TREE_ROWS &&
           Hkv >= 1 && H >= Hkv && H <= 1024 && H % Hkv == 0 && (dh == 64 || dh == 128) &&
           P_max >= 0 && P_max <= kMaxPrefix && window >= 0 && sinks >= 0;
}

medusa_status cache_attention(const char *who, bool kv4, medusa_dtype dtype, const void *q,
                              const void *const *k_cache, const void *const *v_cache,
                              const int32_t *prefix_len, int P_max, const uint64_t *anc_mask,
                              const int32_t *depth, int window, int sinks, int B, int R, int H,
                              int Hkv, int dh, float scale, void *out, void *ws, size_t ws_bytes,
                              medusa_stream stream) {
    if (medusa_status s = check_heads_shape(who, dtype, B, R, MEDUSA_MAX_TREE_ROWS, H, Hkv, dh))
        return s;
    if (!q || !anc_mask || !out) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (medusa_status s = check_caches(who, k_cache, v_cache, prefix_len, P_max)) return s;
    if (window < 0 || sinks < 0)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: window=%d, sinks=%d", who, window, sinks);
    if (window == 0 && sinks != 0)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: sinks=%d without a window", who, sinks);
    if (window && !depth)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: a window needs the rows' depth", who);
    if (!(scale > 0.f) || !(scale < 1e30f))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
    if (!aligned16(q) || !aligned16(out))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: tensor pointers must be 16-byte aligned", who);
    if (medusa_status s = check_ws(ws, ws_bytes,
                                   cache_attention_workspace_bytes(dtype, kv4, B, R, H, Hkv, dh,
                                                                   P_max, window, sinks),
                                   who))
        return s;
    cudaError_t e = launch_cache_attention(dtype, kv4, q, k_cache, v_cache, prefix_len, P_max,
                                           anc_mask, depth, window, sinks, B, R, H, Hkv, dh, scale,
                                           out, ws, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

}  // namespace

extern "C" {

medusa_status medusa_qk_norm_rope(medusa_dtype dtype, const void *q, const void *k,
                                  int64_t q_stride, int64_t k_stride, const void *q_weight,
                                  const void *k_weight, float eps, int norm, const int32_t *pos,
                                  const float *inv_freq, int rot, int interleaved,
                                  const int32_t *n_rows, int B, int R, int H, int Hkv, int dh,
                                  void *q_out, void *k_out, medusa_stream stream) {
    const NvtxRange range("medusa_qk_norm_rope");
    const char *who = "medusa_qk_norm_rope";
    if (medusa_status s = check_rope(who, dtype, q, k, q_stride, k_stride, q_weight, k_weight, eps,
                                     norm, pos, inv_freq, rot, B, R, H, Hkv, dh, q_out))
        return s;
    if (!k_out) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned16(k_out))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: tensor pointers must be 16-byte aligned", who);
    cudaError_t e = launch_qk_norm_rope(dtype, q, k, nullptr, q_stride, k_stride, 0, q_weight,
                                        k_weight, eps, norm, pos, inv_freq, rot, interleaved,
                                        n_rows, nullptr, nullptr, nullptr, 0, B, R, H, Hkv, dh,
                                        q_out, k_out, nullptr, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

medusa_status medusa_qk_norm_rope_append(
    medusa_dtype dtype, const void *q, const void *k, const void *v, int64_t q_stride,
    int64_t k_stride, int64_t v_stride, const void *q_weight, const void *k_weight, float eps,
    int norm, const int32_t *pos, const float *inv_freq, int rot, int interleaved,
    const int32_t *n_rows, void *const *k_cache, void *const *v_cache, const int32_t *prefix_len,
    int P_max, int B, int R, int H, int Hkv, int dh, void *q_out, void *ws, size_t ws_bytes,
    medusa_stream stream) {
    const NvtxRange range("medusa_qk_norm_rope_append");
    const char *who = "medusa_qk_norm_rope_append";
    if (medusa_status s = check_rope(who, dtype, q, k, q_stride, k_stride, q_weight, k_weight, eps,
                                     norm, pos, inv_freq, rot, B, R, H, Hkv, dh, q_out))
        return s;
    if (!v) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned16(v))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: tensor pointers must be 16-byte aligned", who);
    if (medusa_status s = check_row_stride(who, "v_stride", dtype, v_stride, Hkv, dh)) return s;
    if (medusa_status s = check_caches(who, k_cache, v_cache, prefix_len, P_max)) return s;
    if (medusa_status s = check_ws(ws, ws_bytes, MEDUSA_WS_HEADER, who)) return s;
    cudaError_t e = launch_qk_norm_rope(dtype, q, k, v, q_stride, k_stride, v_stride, q_weight,
                                        k_weight, eps, norm, pos, inv_freq, rot, interleaved,
                                        n_rows, k_cache, v_cache, prefix_len, P_max, B, R, H, Hkv,
                                        dh, q_out, nullptr, ws, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

size_t medusa_kv4_row_bytes(int Hkv, int dh) {
    if (Hkv < 1 || Hkv > 1024 || (dh != 64 && dh != 128)) return 0;
    return ((size_t)Hkv * dh / 2 + (size_t)Hkv * dh / 16 + 15) / 16 * 16;
}

medusa_status medusa_kv4_append(medusa_dtype dtype, const void *k, const void *v, int64_t k_stride,
                                int64_t v_stride, void *const *k_cache, void *const *v_cache,
                                const int32_t *prefix_len, int P_max, const int32_t *n_rows, int B,
                                int R, int Hkv, int dh, void *ws, size_t ws_bytes,
                                medusa_stream stream) {
    const NvtxRange range("medusa_kv4_append");
    const char *who = "medusa_kv4_append";
    if (medusa_status s = check_kv4_rows(who, dtype, k, v, k_stride, v_stride, k_cache, v_cache,
                                         prefix_len, P_max, B, R, Hkv, dh, ws, ws_bytes))
        return s;
    cudaError_t e = launch_kv4_rows(dtype, true, k, v, k_stride, v_stride, k_cache, v_cache,
                                    prefix_len, P_max, n_rows, B, R, Hkv, dh, ws,
                                    static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

medusa_status medusa_kv4_unpack(medusa_dtype dtype, const void *const *k_cache,
                                const void *const *v_cache, const int32_t *prefix_len, int P_max,
                                const int32_t *n_rows, int B, int R, int Hkv, int dh, void *k_out,
                                void *v_out, void *ws, size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_kv4_unpack");
    const char *who = "medusa_kv4_unpack";
    const int64_t row = (int64_t)Hkv * dh;
    if (medusa_status s = check_kv4_rows(who, dtype, k_out, v_out, row, row, k_cache, v_cache,
                                         prefix_len, P_max, B, R, Hkv, dh, ws, ws_bytes))
        return s;
    cudaError_t e = launch_kv4_rows(dtype, false, k_out, v_out, row, row,
                                    const_cast<void *const *>(k_cache),
                                    const_cast<void *const *>(v_cache), prefix_len, P_max, n_rows,
                                    B, R, Hkv, dh, ws, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

medusa_status medusa_commit_kv4(void *const *k_cache, void *const *v_cache,
                                const int32_t *prefix_len, const int32_t *path,
                                const int32_t *accept_len, int B, int K, int R, int Hkv, int dh,
                                int32_t *new_prefix_len, void *ws, size_t ws_bytes,
                                medusa_stream stream) {
    const NvtxRange range("medusa_commit_kv4");
    const char *who = "medusa_commit_kv4";
    if (medusa_status s = check_heads_shape(who, MEDUSA_BF16, B, R, MEDUSA_MAX_TREE_ROWS, Hkv, Hkv, dh))
        return s;
    // the row is moved as raw bytes: 2-byte elements, one head of row_bytes / 2
    const int row = (int)medusa_kv4_row_bytes(Hkv, dh);
    if (medusa_status s = check_commit(who, MEDUSA_BF16, k_cache, v_cache, prefix_len,
                                       new_prefix_len, 1, row / 2))
        return s;
    if (!path || !accept_len) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (K < 0 || K > MEDUSA_MAX_HEADS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: K=%d outside 0..%d", who, K, MEDUSA_MAX_HEADS);
    if (medusa_status s = check_ws(ws, ws_bytes, MEDUSA_WS_HEADER, who)) return s;
    cudaError_t e = launch_commit_kv(1, k_cache, v_cache, prefix_len, path, accept_len, B, K, R, 1,
                                     row, new_prefix_len, ws, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

size_t medusa_tree_attention_window_workspace_size(medusa_dtype dtype, int B, int R, int H, int Hkv,
                                                   int dh, int P_max, int window, int sinks) {
    if (!attention_shape_ok(dtype, B, R, H, Hkv, dh, P_max, window, sinks)) return 0;
    return cache_attention_workspace_bytes(dtype, false, B, R, H, Hkv, dh, P_max, window, sinks);
}

size_t medusa_tree_attention_kv4_workspace_size(medusa_dtype dtype, int B, int R, int H, int Hkv,
                                                int dh, int P_max, int window, int sinks) {
    if (!attention_shape_ok(dtype, B, R, H, Hkv, dh, P_max, window, sinks)) return 0;
    return cache_attention_workspace_bytes(dtype, true, B, R, H, Hkv, dh, P_max, window, sinks);
}

medusa_status medusa_tree_attention_window(
    medusa_dtype dtype, const void *q, const void *const *k_cache, const void *const *v_cache,
    const int32_t *prefix_len, int P_max, const uint64_t *anc_mask, const int32_t *depth,
    int window, int sinks, int B, int R, int H, int Hkv, int dh, float scale, void *out, void *ws,
    size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_tree_attention_window");
    return cache_attention("medusa_tree_attention_window", false, dtype, q, k_cache, v_cache,
                           prefix_len, P_max, anc_mask, depth, window, sinks, B, R, H, Hkv, dh,
                           scale, out, ws, ws_bytes, stream);
}

medusa_status medusa_tree_attention_kv4(
    medusa_dtype dtype, const void *q, const void *const *k_cache, const void *const *v_cache,
    const int32_t *prefix_len, int P_max, const uint64_t *anc_mask, const int32_t *depth,
    int window, int sinks, int B, int R, int H, int Hkv, int dh, float scale, void *out, void *ws,
    size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_tree_attention_kv4");
    return cache_attention("medusa_tree_attention_kv4", true, dtype, q, k_cache, v_cache,
                           prefix_len, P_max, anc_mask, depth, window, sinks, B, R, H, Hkv, dh,
                           scale, out, ws, ws_bytes, stream);
}

}  // extern "C"

// ------------------------------------------------- paged cache, log probs ---

namespace {

constexpr int kMaxChunkRows = 1 << 20;  // rows times query heads of a KV head stay below 2^30

medusa_status check_pages(const char *who, const void *k_pages, const void *v_pages, int n_pages,
                          int page, const int32_t *page_table, int table_stride,
                          const int32_t *prefix_len, int P_max, int R, PagedCache &cache) {
    if (!k_pages || !v_pages || !page_table || !prefix_len)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned16(k_pages) || !aligned16(v_pages))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: the pools must be 16-byte aligned", who);
    if (page < MEDUSA_MIN_PAGE || page > MEDUSA_MAX_PAGE || (page & (page - 1)))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: page=%d must be a power of two in %d..%d", who, page,
                    MEDUSA_MIN_PAGE, MEDUSA_MAX_PAGE);
    if (n_pages < 1 || (long long)n_pages * page > 0x7fffffffLL)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: n_pages=%d pages of %d slots (1 to 2^31 - 1 slots)",
                    who, n_pages, page);
    if (P_max < 0 || P_max > kMaxPrefix)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: P_max=%d outside 0..%d", who, P_max, kMaxPrefix);
    if (table_stride < 1 || (long long)table_stride * page < (long long)P_max + R)
        return fail(MEDUSA_ERR_INVALID_ARG,
                    "%s: table_stride=%d pages of %d slots do not hold P_max + R = %lld slots", who,
                    table_stride, page, (long long)P_max + R);
    cache.table = page_table;
    cache.stride = table_stride;
    cache.n_pages = n_pages;
    cache.shift = 0;
    while ((1 << cache.shift) < page) ++cache.shift;
    return MEDUSA_OK;
}

medusa_status paged_attention(const char *who, medusa_dtype dtype, const void *q,
                              const void *k_pages, const void *v_pages, int n_pages, int page,
                              const int32_t *page_table, int table_stride, const int32_t *prefix_len,
                              int P_max, const uint64_t *anc_mask, const int32_t *n_rows, int max_rows,
                              int B, int R, int H, int Hkv, int dh, float scale, void *out, void *ws,
                              size_t ws_bytes, medusa_stream stream) {
    if (medusa_status s = check_heads_shape(who, dtype, B, R, max_rows, H, Hkv, dh)) return s;
    if (!q || !out) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    PagedCache cache;
    if (medusa_status s = check_pages(who, k_pages, v_pages, n_pages, page, page_table, table_stride,
                                      prefix_len, P_max, R, cache))
        return s;
    if (!(scale > 0.f) || !(scale < 1e30f))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
    if (!aligned16(q) || !aligned16(out))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: tensor pointers must be 16-byte aligned", who);
    const PagedPlan plan = paged_plan(dtype, B, R, H, Hkv, dh, P_max);
    if (medusa_status s = check_ws(ws, ws_bytes, plan.workspace, who)) return s;
    cudaError_t e = launch_paged_attention(plan, dtype, q, k_pages, v_pages, cache, prefix_len, P_max,
                                           anc_mask, n_rows, B, R, H, Hkv, dh, scale, out, ws,
                                           static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

}  // namespace

extern "C" {

medusa_status medusa_paged_append(medusa_dtype dtype, const void *k, const void *v, int64_t k_stride,
                                  int64_t v_stride, void *k_pages, void *v_pages, int n_pages,
                                  int page, const int32_t *page_table, int table_stride,
                                  const int32_t *prefix_len, int P_max, const int32_t *n_rows, int B,
                                  int R, int Hkv, int dh, void *ws, size_t ws_bytes,
                                  medusa_stream stream) {
    const NvtxRange range("medusa_paged_append");
    const char *who = "medusa_paged_append";
    if (medusa_status s = check_heads_shape(who, dtype, B, R, kMaxChunkRows, Hkv, Hkv, dh)) return s;
    if (!k || !v) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned16(k) || !aligned16(v))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: tensor pointers must be 16-byte aligned", who);
    if (medusa_status s = check_row_stride(who, "k_stride", dtype, k_stride, Hkv, dh)) return s;
    if (medusa_status s = check_row_stride(who, "v_stride", dtype, v_stride, Hkv, dh)) return s;
    PagedCache cache;
    if (medusa_status s = check_pages(who, k_pages, v_pages, n_pages, page, page_table, table_stride,
                                      prefix_len, P_max, R, cache))
        return s;
    if (medusa_status s = check_ws(ws, ws_bytes, MEDUSA_WS_HEADER, who)) return s;
    cudaError_t e = launch_paged_append(dtype == MEDUSA_BF16 ? 2 : 4, k, v, k_stride, v_stride,
                                        k_pages, v_pages, cache, prefix_len, P_max, n_rows, B, R,
                                        Hkv, dh, ws, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

medusa_status medusa_commit_paged(medusa_dtype dtype, void *k_pages, void *v_pages, int n_pages,
                                  int page, const int32_t *page_table, int table_stride,
                                  const int32_t *prefix_len, int P_max, const int32_t *path,
                                  const int32_t *accept_len, int B, int K, int R, int Hkv, int dh,
                                  int32_t *new_prefix_len, void *ws, size_t ws_bytes,
                                  medusa_stream stream) {
    const NvtxRange range("medusa_commit_paged");
    const char *who = "medusa_commit_paged";
    if (medusa_status s = check_heads_shape(who, dtype, B, R, MEDUSA_MAX_TREE_ROWS, Hkv, Hkv, dh))
        return s;
    PagedCache cache;
    if (medusa_status s = check_pages(who, k_pages, v_pages, n_pages, page, page_table, table_stride,
                                      prefix_len, P_max, R, cache))
        return s;
    if (!path || !accept_len || !new_prefix_len)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (new_prefix_len == prefix_len)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: new_prefix_len must not alias prefix_len", who);
    if (K < 0 || K > MEDUSA_MAX_HEADS)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: K=%d outside 0..%d", who, K, MEDUSA_MAX_HEADS);
    if (medusa_status s = check_ws(ws, ws_bytes, MEDUSA_WS_HEADER, who)) return s;
    cudaError_t e = launch_commit_paged(dtype == MEDUSA_BF16 ? 2 : 4, k_pages, v_pages, cache,
                                        prefix_len, P_max, path, accept_len, B, K, R, Hkv, dh,
                                        new_prefix_len, ws, static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

size_t medusa_paged_attention_workspace_size(medusa_dtype dtype, int B, int R, int H, int Hkv, int dh,
                                             int P_max) {
    if (!is_dtype(dtype) || B < 1 || B > 65535 || R < 1 || R > kMaxChunkRows || Hkv < 1 || H < Hkv ||
        H > 1024 || H % Hkv || (dh != 64 && dh != 128) || P_max < 0 || P_max > kMaxPrefix)
        return 0;
    return paged_plan(dtype, B, R, H, Hkv, dh, P_max).workspace;
}

medusa_status medusa_chunk_attention_paged(
    medusa_dtype dtype, const void *q, const void *k_pages, const void *v_pages, int n_pages, int page,
    const int32_t *page_table, int table_stride, const int32_t *prefix_len, int P_max,
    const int32_t *n_rows, int B, int R, int H, int Hkv, int dh, float scale, void *out, void *ws,
    size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_chunk_attention_paged");
    return paged_attention("medusa_chunk_attention_paged", dtype, q, k_pages, v_pages, n_pages, page,
                           page_table, table_stride, prefix_len, P_max, nullptr, n_rows,
                           kMaxChunkRows, B, R, H, Hkv, dh, scale, out, ws, ws_bytes, stream);
}

medusa_status medusa_tree_attention_paged(
    medusa_dtype dtype, const void *q, const void *k_pages, const void *v_pages, int n_pages, int page,
    const int32_t *page_table, int table_stride, const int32_t *prefix_len, int P_max,
    const uint64_t *anc_mask, int B, int R, int H, int Hkv, int dh, float scale, void *out, void *ws,
    size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_tree_attention_paged");
    const char *who = "medusa_tree_attention_paged";
    if (!anc_mask) return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    return paged_attention(who, dtype, q, k_pages, v_pages, n_pages, page, page_table, table_stride,
                           prefix_len, P_max, anc_mask, nullptr, MEDUSA_MAX_TREE_ROWS, B, R, H, Hkv,
                           dh, scale, out, ws, ws_bytes, stream);
}

medusa_status medusa_token_logprobs(medusa_dtype dtype, const void *logits, int64_t stride,
                                    const int32_t *tokens, int N, int V, int top, float temperature,
                                    float *logp, float *entropy, int32_t *rank, int32_t *top_ids,
                                    float *top_logp, void *ws, size_t ws_bytes, medusa_stream stream) {
    const NvtxRange range("medusa_token_logprobs");
    const char *who = "medusa_token_logprobs";
    if (!is_dtype(dtype)) return fail(MEDUSA_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dtype);
    if (!logits || !tokens || !logp || !entropy || !rank || (top > 0 && (!top_ids || !top_logp)))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (reinterpret_cast<uintptr_t>(logits) % (dtype == MEDUSA_F32 ? 4 : 2))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: logits must be aligned to their elements", who);
    if (N < 1 || N > 1 << 30) return fail(MEDUSA_ERR_INVALID_ARG, "%s: N=%d outside 1..2^30", who, N);
    if (V < 1 || V > MEDUSA_MAX_VOCAB)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: V=%d outside 1..%d", who, V, MEDUSA_MAX_VOCAB);
    if (stride < V || stride > (int64_t)1 << 40)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: stride=%lld below V=%d", who, (long long)stride, V);
    if (top < 0 || top > MEDUSA_MAX_TOP_S || top > V)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: top=%d outside 0..min(V, %d)", who, top,
                    MEDUSA_MAX_TOP_S);
    if (!(temperature > 1e-30f) || !(temperature < 1e30f))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: temperature must be in 1e-30..1e30", who);
    if (medusa_status s = check_ws(ws, ws_bytes, MEDUSA_WS_HEADER, who)) return s;
    cudaError_t e = launch_token_logprobs(dtype, logits, stride, tokens, N, V, top, temperature, logp,
                                          entropy, rank, top_ids, top_logp, ws,
                                          static_cast<cudaStream_t>(stream));
    if (e) return cuda_fail(e, who);
    return MEDUSA_OK;
}

}  // extern "C"
