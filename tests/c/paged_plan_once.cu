// Calls medusa_tree_attention_paged with a fake of the query for clusters that run at once, whose
// answer changes from one plan to the next, and a fake launch that takes down what it is given.
// Exits with 1 if a launch gets ranges to join and no workspace for them.  Touches no GPU.
#include <cstdio>

#include "cache_attention.cuh"

namespace medusa {

int g_turn = 0, g_last = 1 << 30, g_launches = 0, g_bad = 0;
size_t g_ws_bytes = 0;

int paged_cluster_slots(int, int size) {  // (a plan asks for sizes in ascending order)
    if (size <= g_last) ++g_turn;
    g_last = size;
    return g_turn & 1 ? 100 : 0;
}

cudaError_t launch_paged_attention_tc(const CacheAttnArgs &a, int dh, cudaStream_t) {
    ++g_launches;
    const size_t rows = (size_t)a.B * a.ns * a.H * a.R;
    const size_t need = a.ns > 1 && !a.cluster ? MEDUSA_WS_HEADER + rows * dh * 4 : (size_t)MEDUSA_WS_HEADER;
    if (need > g_ws_bytes) {
        std::printf("%d ranges to join, cluster %d: %zu bytes of %zu\n", a.ns, a.cluster, need, g_ws_bytes);
        g_bad = 1;
    }
    return cudaErrorUnknown;  // nothing is launched behind it
}

}  // namespace medusa

int main() {
    using namespace medusa;
    void *p = reinterpret_cast<void *>(4096);  // never dereferenced
    const int B = 1, R = 65, H = 32, Hkv = 32, dh = 128, P = 1024;
    for (int first = 0; first < 2; ++first)
        for (size_t bytes : {(size_t)MEDUSA_WS_HEADER, (size_t)1 << 30}) {
            g_turn = first;
            g_ws_bytes = bytes;
            medusa_tree_attention_paged(MEDUSA_BF16, p, p, p, 100, 64, static_cast<int32_t *>(p), 40,
                                        static_cast<int32_t *>(p), P, static_cast<uint64_t *>(p), B, R, H, Hkv,
                                        dh, 0.1f, p, reinterpret_cast<void *>(1 << 20), bytes, nullptr);
        }
    std::printf("%d launches\n", g_launches);
    return g_bad || g_launches < 2;
}
