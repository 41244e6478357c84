// paged_attention_tc.cu -- attention over a cache in pages on the tensor cores:
// prompt chunks and trees with more than 16 rows a KV head, bf16.
//
// One CTA an SM (twelve warps) works on up to 256 rows that share a KV head, in two
// tiles A and B of 128 rows, over stages of 128 keys:
//   warps 0-3, 4-7  softmax of tile A and of tile B: thread t owns row t, reads its 128
//              scores from tensor memory, keeps the row's reference m and sum l in
//              registers, and writes the weights P over the scores, as the bf16 A
//              operand of the second product.
//   warp 8     products: S = Q K^T (both operands in shared memory), O += P V (P in
//              tensor memory).  The tiles take turns: while the softmax of one
//              works, the products of the other run.
//   warps 9, 10  copies: K and V of a stage, one TMA box a page (and 64 columns),
//              into a ring each.
//   warp 11    sets the barriers up, then nothing (register budgets are by four warps).
// With at most 128 rows the two tiles hold the same rows, A the even stages and B the
// odd ones, so that the work still takes turns; their results are joined at the end, and
// those of the CTAs of a cluster after that, where each has a range of the keys.  Where
// there are more such tiles than SMs, A and B are the same rows of two KV heads, and the
// ring holds the stages of one and of the other by turns.
//
// Tensor memory (512 columns): S / P of A, S / P of B, O of A, O of B.  The reference
// m moves only when a stage's maximum exceeds it by 2^8, and O is then rescaled in
// tensor memory.
//
// Masks are built as 128 bits a row and stage, in stages that a warp's rows do not
// see wholly.  A weight of zero times an infinity in V would be a NaN in every row, so
// the softmax warps (of B, or of the stage's half) look for such elements before those
// stages and clear them; a row that does see one adds it at the end, from the cache
// itself.  Every wait is bounded; on a timeout the CTA sets the status, waits
// (bounded) for its products and copies, frees its tensor memory and publishes
// nothing.
//
// What bounds it: the products and what feeds them.  A stage of two tiles takes
// 2490-2550 cycles, of which 2048 are its four products at the rate of the tensor cores;
// the two of them that read both operands from shared memory leave its ports no room.  A
// stage of one tile, by halves, takes 1470-1830.  A CTA's ends cost some 12000 cycles: 1900
// to learn where its keys are, 3000 for the first copies and 900 for the first scores; 900
// behind the last weights for the last product, 3900 for a tile's rows and 1600 for the
// other's.  Nothing of the next CTA overlaps them, as one takes the SM's shared memory.
// Measured: a prompt of 8192 rows, 32 heads over 8, dh 128: 342 us, 1610 TFLOP/s (370 us where
// it runs without a break, at the power limit; dh 64 275 us); six chunks of 1 to 509 rows
// behind up to 5001 slots, 28 heads over 4: 79 us, 1170 TFLOP/s, where the busiest SM has
// two CTAs and 48 stages against 40 on average; eight trees of 65 rows behind up to 8192
// slots, 32 heads over 8: 64 us, 2.8 TB/s; one of 32 heads behind 1024: 12.5 us (14.7 with
// a cold L2), nearly all of it the ends.
// Pages: a page is a TMA box of up to 128 rows, whose row a lane has looked up while the
// stage before was under way, so that 16-row pages cost what 128-row pages do (338 and 350
// us); copies issued by one lane took 571 us at 16 rows.
// Measured and not kept: K and V copied by one warp (367, and 468 us at 16 rows), Q and O
// moved by their rows' threads (375), weights computed against the reference before the
// stage's maximum is known (394; registers spill), one arrival for a stage's weights instead
// of two (383 against 376), 64 of a row's columns at a time on its way out (no change, partial
// rows 2-4 % slower), the rows behind the last whole tile (260 rows are 256 and 4)
// on register-operand products by warp 11 from the same stages (112-119 us against 91:
// 58 cycles an instruction beside the others').
#include "cache_attention.cuh"
#include "tensor_map.h"

#include <atomic>

namespace medusa {

namespace {

constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // 256 * 216 + 128 * 72 = 384 * 168
constexpr int kMaskedStages = 4;  // stages that hold new rows: at most 3 (255 keys apart)

template <int DH>
struct PagedSmem {
    static constexpr int NB = DH / 64;
    static constexpr int BLOCK = 128 * 128;          // 128 rows of 64 elements
    static constexpr int TILE = NB * BLOCK;          // Q tile, K or V of a stage
    static constexpr int NK = 2 * (128 / DH), NT = 2 * NK;  // stages in the rings of K and of V
    static constexpr int RING = 2 * TILE;
    static constexpr int BAR = RING + NT * TILE;
    // full[NT], empty[NT], q[2], s[2], o[2], p[2][2], drain, armed and clean[kMaskedStages]
    static constexpr int WORDS = BAR + (2 * NT + 11 + 2 * kMaskedStages) * 8;
    // failed, tmem, bad (a V element is not finite), pad; bad keys [kMaskedStages][4]
    // CLUSTER: (m, l) of the rows of a range
    static constexpr int PART_ML = (WORDS + 16 + kMaskedStages * 16 + 15) / 16 * 16;
    static constexpr int TOTAL = PART_ML + 128 * 8;
    // B's rows and their (m, l) for the join of the halves, in place of the Q tiles and
    // the ring
    static constexpr int LD = DH + 4;
    static_assert(128 * (LD * 4 + 8) <= BAR, "the join fits before the barriers");
    // CLUSTER: the range's rows, beside those
    static constexpr int PART = 3 * TILE;
    static_assert(128 * (LD * 4 + 8) <= PART && PART + 128 * LD * 4 <= BAR, "rows for the cluster");
    static_assert(TOTAL + 1024 <= 227 * 1024, "shared memory of an SM");
};

// Division of numbers below 2^31 by d, as a product and a shift.  With 2^s the power of
// two below d and m = 2^(32 + s) / d + 1, m is too large by less than one, so that
// i m / 2^(32 + s) is by less than i / 2^(32 + s) < 1 / d (d <= 2^(s + 1)).
struct Divisor {
    unsigned magic, shift;  // magic 0: d = 1
    __host__ explicit Divisor(unsigned d = 1) : magic(0), shift(0) {
        while ((2u << shift) < d) ++shift;
        if (d > 1) magic = (unsigned)((1ull << (32 + shift)) / d + 1);
    }
    __device__ __forceinline__ int operator()(int x) const {
        return magic ? (int)(__umulhi((unsigned)x, magic) >> shift) : x;
    }
};

struct PagedMaps {
    CUtensorMap k, v;
    Divisor by_g, by_units;  // division by G and by the CTAs of a row tile
};

__device__ __forceinline__ bool pair_not_finite(uint4 w) {
    return pair_bad<false>(w.x) || pair_bad<false>(w.y) || pair_bad<false>(w.z) || pair_bad<false>(w.w);
}

// 32 lanes x 128 consecutive 32-bit columns: four loads in flight, one wait
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
    uint32_t r[128];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        uint32_t *q = r + 32 * h;
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
            "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
            : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]),
              "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]),
              "=r"(q[14]), "=r"(q[15]), "=r"(q[16]), "=r"(q[17]), "=r"(q[18]), "=r"(q[19]),
              "=r"(q[20]), "=r"(q[21]), "=r"(q[22]), "=r"(q[23]), "=r"(q[24]), "=r"(q[25]),
              "=r"(q[26]), "=r"(q[27]), "=r"(q[28]), "=r"(q[29]), "=r"(q[30]), "=r"(q[31])
            : "r"(taddr + 32 * h));
    }
    // the wait names the registers, so no use can move above it
    tc::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 128; ++i) {
        asm volatile("" : "+r"(r[i]));
        v[i] = __uint_as_float(r[i]);
    }
}

// What a CTA's tiles are: 256 rows or the halves of 128; halves whose CTAs are a cluster; 128
// rows of two KV heads.
enum Rows { kTiles, kCluster, kPair };

template <int DH, bool DEAL, Rows MODE>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_tc_kernel(const __grid_constant__ PagedMaps maps, const CacheAttnArgs a) {
    using L = PagedSmem<DH>;
    constexpr bool CLUSTER = MODE == kCluster, PAIR = MODE == kPair;
    constexpr int NK = L::NK, NT = 2 * NK;
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::BAR), *empty = full + NT, *bar_q = empty + NT,
             *bar_s = bar_q + 2, *bar_o = bar_q + 4, *bar_p = bar_q + 6, *bar_drain = bar_q + 10,
             *armed = bar_q + 11, *clean = armed + kMaskedStages;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    volatile int *failed = reinterpret_cast<volatile int *>(sm + L::WORDS);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(sm + L::WORDS + 4);
    int *bad_v = reinterpret_cast<int *>(sm + L::WORDS + 8);
    uint32_t *bad_keys = reinterpret_cast<uint32_t *>(sm + L::WORDS + 16);

    // (done while the grid before ends, and by a warp that is free)
    if (tid == kThreads - 1) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            tc::mbar_init(full + i, 1);
            tc::mbar_init(empty + i, 1);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar_q + i, 128);
            tc::mbar_init(bar_s + i, 1);
            tc::mbar_init(bar_p + 2 * i, 128);
            tc::mbar_init(bar_p + 2 * i + 1, 128);
            tc::mbar_init(bar_o + i, 1);
        }
        tc::mbar_init(bar_drain, 1);
#pragma unroll
        for (int i = 0; i < kMaskedStages; ++i) {
            tc::mbar_init(armed + i, 1);
            tc::mbar_init(clean + i, 128);
#pragma unroll
            for (int w = 0; w < 4; ++w) bad_keys[4 * i + w] = 0;
        }
        *failed = 0;
        *bad_v = 0;
        tc::fence_mbarrier_init();
    }
    if (warp == 9) tc::prefetch_tmap(&maps.k);
    if (warp == 10) tc::prefetch_tmap(&maps.v);
    // (the copying warps do not wait for the others to be set up)
    if (warp >= 9) asm volatile("barrier.cta.sync 3, 96;\n" ::: "memory");
    pdl_enter();

    // the longest first: a chunk's last rows see the most keys, a tree's last tile has the fewest rows
    const int units = PAIR ? (a.Hkv + 1) / 2 : a.Hkv;
    const int rt_up = maps.by_units(blockIdx.x), g = (blockIdx.x - rt_up * units) * (PAIR ? 2 : 1);
    const int rt = a.anc_mask ? rt_up : a.row_tiles - 1 - rt_up;
    const int R = a.R, G = a.H / a.Hkv;
    const bool tree = a.anc_mask != nullptr;
    const int m0 = rt * kPagedTileRows;
    const int box = min(1 << a.map.shift, 128);
    // lane of a copying warp: one box of the tile (a box of 128 rows brings all columns)
    const int per = box == 128 ? 1 : L::NB, copy_boxes = box == 128 ? 1 : 128 / box * L::NB;
    const int my = lane / per, half = lane % per;
    // What the first copies need is read at once with the prefix, not after it: the rows of the
    // sequence, and the pages where its keys begin (of its first keys, if all are this CTA's)
    int n_first = 0, page_first = 0;
    if (!DEAL) {
        n_first = live_rows(a, blockIdx.z);
        const int at = my * box >> a.map.shift;
        if (a.ns == 1 && warp >= 9 && at < a.map.stride) page_first = a.map.table[(size_t)blockIdx.z * a.map.stride + at];
    }
    CacheItem it;
    // slots that the last of the first `rows` rows sees (a tree's rows: all)
    auto by_g = [&](int x) { return maps.by_g(x); };  // x / G
    auto keys_of = [&](int P, int n, int rows) { return P + (tree ? n : min(n, by_g(rows - 1) + 1)); };
    if (!find_item<DEAL, kPagedStage, true>(a, [&](int P, int b) {
            const int n = DEAL ? live_rows(a, b) : n_first;
            return n == 0 ? 0 : DEAL ? P + n : keys_of(P, n, m0 + kPagedTileRows);
        }, it))
        return;
    const bool direct = DEAL ? it.alone : a.ns == 1;  // no join
    const int b = it.b, P = it.P;
    const int n = DEAL ? live_rows(a, b) : n_first, M = n * G;
    if (m0 >= M) return;  // uniform over the CTA
    const int rows = min(kPagedTileRows, M - m0);
    // PAIR: A and B are the same rows of two KV heads, but for the last head of an odd number
    const bool pair = PAIR && g + 1 < a.Hkv;
    const bool turns = CLUSTER || PAIR || rows <= 128;  // A and B take turns at the stages
    const bool split = turns && !pair;                  // ... and are the same rows
    const int kbeg = it.kbeg, kend = min(it.kend, keys_of(P, n, m0 + rows));

    // row of a softmax thread
    const int side = (warp >> 2) & 1, t = tid & 127, gs = pair ? g + side : g;
    const int m = m0 + (turns ? 0 : side * 128) + t;
    const bool live = tid < 256 && m < M;
    const int r = live ? by_g(m) : 0;
    const int mw = m0 + (turns ? 0 : side * 128) + (warp & 3) * 32;  // the warp's first row
    // row of q and out, and of the partial results, in rows of DH elements
    auto row_at = [&](int r, int gq) { return ((size_t)b * R + r) * a.H + gs * G + gq; };
    auto part_at = [&](int r, int gq) { return ((size_t)it.range * a.H + gs * G + gq) * R + r; };
    float *const part_o = reinterpret_cast<float *>(sm + L::PART);  // CLUSTER: [128][LD]
    float2 *const part_ml = reinterpret_cast<float2 *>(sm + L::PART_ML);
    auto publish_nothing = [&] {
        if (!live || (split && side)) return;
        if (CLUSTER) {
            part_ml[t] = make_float2(-INFINITY, 0.f);
        } else if (direct) {
            bf16 *dst = static_cast<bf16 *>(a.out) + row_at(r, m - r * G) * DH;
#pragma unroll
            for (int c = 0; c < DH; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
        } else {
            a.part_ml[part_at(r, m - r * G)] = make_float2(-INFINITY, 0.f);
        }
    };
    // The warp's 32 rows in pieces of 16 bytes, kCols pieces a row: f(row of the 32, piece,
    // the row's number) for the lane's of each kPass rows, so that a warp's accesses to global
    // memory are whole rows.  Row numbers are at(new row, query head of the group): `head` apart
    // from head to head, `next` from the last head of a row to the first of the one after it.
    constexpr int kCols = DH / 8, kPass = 32 / kCols;
    auto for_rows = [&](auto at, long long head, long long next, auto f) {
        const int first = mw + lane / kCols;
        const int rr = by_g(first), dr = by_g(kPass), dg = kPass - dr * G;
        int gg = first - rr * G;
        const long long wrap = next - head, step = kPass * head + dr * wrap;  // (a row of G heads is passed dr times)
        long long row = at(rr, gg);
#pragma unroll 8
        for (int i = 0; i < 32; i += kPass) {
            f(i + lane / kCols, lane % kCols, row);
            row += step;
            gg += dg;
            if (gg >= G) {
                gg -= G;
                row += wrap;
            }
        }
    };
    // CLUSTER: the CTAs of the cluster hold a range of the same rows each, and take turns at
    // joining them, DH / 4 threads a row.  (Several rows at once, for few ranges, spills at the
    // 72 registers that the copying warps keep: 14.6 us for 10.8.)
    auto join_cluster = [&] {
        cluster_arrive();
        cluster_wait();
        constexpr int COLS = DH / 4;
        if (tid < 256)
            for (int i = blockIdx.y + a.ns * (tid / COLS); i < M; i += a.ns * (256 / COLS)) {
                float2 ml[kClusterRanges];
                float4 o[kClusterRanges];
                float top = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kClusterRanges; ++s)
                    if (s < a.ns) {
                        ml[s] = *cluster_ptr(part_ml + i, s);
                        o[s] = *reinterpret_cast<const float4 *>(cluster_ptr(part_o + i * L::LD + tid % COLS * 4, s));
                    }
#pragma unroll
                for (int s = 0; s < kClusterRanges; ++s)
                    if (s < a.ns && ml[s].y != 0.f) top = fmaxf(top, ml[s].x);
                const float mu = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int s = 0; s < kClusterRanges; ++s)
                    if (s < a.ns && ml[s].y != 0.f) {  // (an empty range has no row)
                        const float f = exp2f(ml[s].x - mu);
                        l = fmaf(f, ml[s].y, l);
                        if (f != 0.f) add4(acc, f, o[s]);
                    }
                const int rr = by_g(i);
                store_row4(static_cast<bf16 *>(a.out) + row_at(rr, i - rr * G) * DH + tid % COLS * 4, acc,
                           l == 0.f ? 0.f : 1.f / l);
            }
        cluster_arrive();  // no CTA leaves while its rows may be read
        cluster_wait();
    };
    if (kbeg >= kend) {  // uniform over the CTA
        publish_nothing();
        if constexpr (CLUSTER) join_cluster();
        return;
    }
    // stages; of a pair by turns, A's first
    const int nsub = ((kend - kbeg + kPagedStage - 1) / kPagedStage) << pair;
    // stages of tile A that hold keys one of its rows sees (of B: all nsub)
    const int nsub_a = turns ? nsub
                             : max(0, min(nsub, (keys_of(P, n, m0 + 128) - kbeg + kPagedStage - 1) / kPagedStage));
    // the first stage that some row of the CTA does not see wholly
    const int all = tree ? P : min(P + by_g(m0) + 1, kend);
    const int j_masked = max(0, (all - kbeg) / kPagedStage) << pair;
    auto first_key = [&](int j) { return kbeg + (j >> pair) * kPagedStage; };

    // place of stage j's K or V among the slots, a ring for each
    auto slot_of = [&](int j, bool vs) { return (vs ? NK : 0) + j % NK; };
    auto wait_full = [&](int j, bool vs) {
        return wait_or_fail(full + slot_of(j, vs), (j / NK) & 1, a.wait_polls, failed);
    };

    const uint32_t to = half * L::BLOCK + my * box * 128;
    const int rows_end = a.map.n_pages << a.map.shift;  // past the pool: zeros
    const int end = P + n;
    const bool vs = warp == 10;
    auto row_of = [&](int j) {  // the lane's pool row of stage j
        const int slot = first_key(j) + my * box;
        if (lane >= copy_boxes || slot >= end) return rows_end;
        const int page = !DEAL && a.ns == 1 && first_key(j) == 0 ? page_first : a.map.page_of(b, slot);
        return a.map.good(page) ? (int)a.map.row(page, slot) : rows_end;
    };
    // The copies of stage j, whose row the lane has looked up; looks up the next stage's.
    // -1: failed.
    auto copy_stage = [&](int j, int row) {
        const int i = slot_of(j, vs), next = j + 1 < nsub ? row_of(j + 1) : 0;
        if (j >= NK && !wait_or_fail(empty + i, (j / NK - 1) & 1, a.wait_polls, failed)) return -1;
        if (lane == 0) tc::mbar_arrive_expect_tx(full + i, L::TILE);
        __syncwarp();
        if (lane < copy_boxes)
            tc::tma_load_3d(sm + L::RING + i * L::TILE + to, vs ? &maps.v : &maps.k, 0, row,
                            (pair ? g + (j & 1) : g) * L::NB + half, full + i);
        // (a phase of `full` can be told from the one two before it only by who knows
        // which stage is in the slot: the checking warps wait from here on)
        if (vs && j >= j_masked && lane == 0) tc::mbar_arrive(armed + (j - j_masked));
        return next;
    };
    int issued = 0, next = 0;
    if (warp == 9 || warp == 10) {
        next = copy_stage(0, row_of(0));
        issued = 1;
    }
    if (warp == 8) tc::tmem_alloc(tmem_holder, 512);
    if (warp < 8 && !(split && side)) {  // Q: rows that are not there are zeros
        const uint32_t qt = tc::smem_addr(sm + side * L::TILE);
        const bf16 *q = static_cast<const bf16 *>(a.q);
        for_rows(row_at, 1, a.H - G + 1, [&](int i, int c, long long row) {
            const bool ok = mw + i < M;
            cp_async16(qt + (c >> 3) * L::BLOCK + tc::sw128((warp & 3) * 32 + i, c & 7),
                       ok ? q + row * DH + c * 8 : q, ok);
        });
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_holder;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
        if (warp == 9 || warp == 10) {
            // -------------------------------------------------------- copies
            for (; issued < nsub; ++issued) {
                next = copy_stage(issued, next);
                if (next < 0) break;
            }
            // every copy has landed before the shared memory goes
            for (int j = max(0, issued - NK); j < issued; ++j)
                if (!__all_sync(0xffffffffu,
                                tc::mbar_wait_bounded(full + slot_of(j, vs), (j / NK) & 1, kDrainPolls)))
                    *failed = 1;
        } else if (warp == 8) {
            // ------------------------------------------------------ products
            // (the warp stays converged; one elected lane issues)
            constexpr uint32_t id_s = tc::idesc_bf16(128, kPagedStage, 0), id_o = tc::idesc_bf16(128, DH, 1);
            const uint64_t qd0 = tc::sdesc_sw128(tc::smem_addr(sm), 16, 1024);
            const uint64_t kd0 = tc::sdesc_sw128(tc::smem_addr(sm + L::RING), 16, 1024);
            const uint64_t vd0 = tc::sdesc_sw128(tc::smem_addr(sm + L::RING), L::BLOCK, 1024);
            auto scores = [&](int x, int j, bool last) {  // S of tile x; `last`: K is free then
                const int slot = slot_of(j, false);
                if (!wait_full(j, false)) return false;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint64_t kd = kd0 + (uint64_t)(slot * (L::TILE >> 4));
                    const uint64_t qd = qd0 + (uint64_t)((split ? 0 : x) * (L::TILE >> 4));
#pragma unroll
                    for (int ks = 0; ks < DH / 16; ++ks) {
                        const int o = ((ks >> 2) * L::BLOCK + (ks & 3) * 32) >> 4;
                        tc::mma_bf16_ss(tmem + x * 128, qd + o, kd + o, id_s, ks > 0);
                    }
                    tc::mma_commit(bar_s + x);
                    if (last) tc::mma_commit(empty + slot);
                }
                __syncwarp();
                return true;
            };
            auto values = [&](int x, int j, int use, bool last) {  // O += P V, the tile's product `use`
                const int slot = slot_of(j, true);
                if (!wait_full(j, true)) return false;
                if (j >= j_masked && !wait_or_fail(clean + (j - j_masked), 0, a.wait_polls, failed)) return false;
                const uint64_t vd = vd0 + (uint64_t)(slot * (L::TILE >> 4));
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // weights of 64 keys each
                    if (!wait_or_fail(bar_p + 2 * x + half, use & 1, a.wait_polls, failed)) return false;
                    tc::fence_after_sync();
                    if (tc::elect_one()) {
#pragma unroll
                        for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                            tc::mma_bf16_ts(tmem + 256 + x * DH, tmem + x * 128 + ks * 8,
                                            vd + ((ks * 16 * 128) >> 4), id_o, use > 0 || ks > 0);
                        if (half) tc::mma_commit(bar_o + x);
                        if (half && last) tc::mma_commit(empty + slot);
                    }
                    __syncwarp();
                }
                return true;
            };
            bool go = wait_or_fail(bar_q, 0, a.wait_polls, failed);
            if (turns) {
                go = go && scores(0, 0, true) && (!pair || wait_or_fail(bar_q + 1, 0, a.wait_polls, failed)) &&
                     (nsub == 1 || scores(1, 1, true));
                for (int j = 0; j < nsub && go; ++j)
                    go = values(j & 1, j, j >> 1, true) && (j + 2 >= nsub || scores(j & 1, j + 2, true));
            } else {
                if (go && nsub_a > 0) go = scores(0, 0, false);
                go = go && wait_or_fail(bar_q + 1, 0, a.wait_polls, failed) && scores(1, 0, true);
                for (int j = 0; j < nsub && go; ++j) {
                    if (j < nsub_a) go = values(0, j, j, false) && (j + 1 >= nsub_a || scores(0, j + 1, false));
                    go = go && values(1, j, j, true) && (j + 1 >= nsub || scores(1, j + 1, true));
                }
            }
            // every product issued above is done before the tensor memory is freed
            if (tc::elect_one()) tc::mma_commit(bar_drain);
            __syncwarp();
            if (!__all_sync(0xffffffffu, tc::mbar_wait_bounded(bar_drain, 0, kDrainPolls))) {
                *failed = 1;
                if (lane == 0 && a.status) atomicExch(a.status, MEDUSA_DEV_DRAIN_TIMEOUT);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
        // ------------------------------------------------------------ softmax
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + side * 128 + lane_base, t_o = tmem + 256 + side * DH + lane_base;
        const bool rows_live = mw < M;  // warp-uniform
        const float row_scale = a.scale_log2;
        if (!(split && side)) {
            asm volatile("cp.async.wait_group 0;\n" ::: "memory");
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(bar_q + side);
        }
        // ---- what this row sees: slots below `mine` and the tree's bits from P on
        const int mine = tree ? P : P + r + 1;
        const int warp_all = tree ? P : P + by_g(mw) + 1;  // slots that every row of the warp sees
        // 64 keys from slot k0 on that this row sees
        auto sees64 = [&](int k0) {
            uint64_t vis = bits_below(mine - k0);
            if (tree && k0 + 64 > P && live) {
                const int t0 = k0 - P, W = (R + 63) / 64;  // tree slot of the first key
                const uint64_t *mr = a.anc_mask + ((size_t)b * R + r) * W;
                if (t0 < 0) {
                    vis |= mr[0] << -t0;
                } else {
                    const int w = t0 >> 6, s = t0 & 63;
                    vis |= w < W ? mr[w] >> s : 0ull;
                    if (s && w + 1 < W) vis |= mr[w + 1] << (64 - s);
                }
            }
            vis &= bits_below(kend - k0);
            return live ? vis : 0ull;
        };
        const int box_log2 = min(a.map.shift, 7), boxes = 128 >> box_log2;
        const int step = turns ? 2 : 1, mine_n = side == 0 ? nsub_a : nsub;

        float m_run = -INFINITY, l_run = 0.f;
        bool dead = false;  // warp-uniform
        int use = 0;
        for (int j = turns ? side : 0; j < mine_n && !dead; j += step, ++use) {
            const int k0 = first_key(j);
            // pages of the stage, one a lane
            bool bad_page = false;
            if (lane < boxes && k0 + (lane << box_log2) < kend)
                bad_page = !a.map.good(a.map.page_of(b, k0 + (lane << box_log2)));
            if (j >= j_masked && (turns || side)) {
                // ---- infinities and NaNs in V of a stage that some row does not see wholly
                dead = !wait_or_fail(armed + (j - j_masked), 0, a.wait_polls, failed) || !wait_full(j, true);
                if (dead) break;
                unsigned char *vt = sm + L::RING + slot_of(j, true) * L::TILE;
#pragma unroll
                for (int u = 0; u < L::NB; ++u) {  // key t's 64 elements of a column block
                    uint4 w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] = *reinterpret_cast<const uint4 *>(vt + u * L::BLOCK + t * 128 + (e ^ (t & 7)) * 16);
                    bool bad = false;
#pragma unroll
                    for (int e = 0; e < 8; ++e) bad = bad || pair_not_finite(w[e]);
                    if (bad) {
                        *bad_v = 1;
                        atomicOr(bad_keys + 4 * (j - j_masked) + (t >> 5), 1u << (t & 31));
#pragma unroll 1
                        for (int e = 0; e < 64; ++e) {
                            uint16_t *x = reinterpret_cast<uint16_t *>(vt + u * L::BLOCK + t * 128) + e;
                            if (pair_bad<false>(*x)) *x = 0;
                        }
                    }
                }
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(clean + (j - j_masked));
            }
            dead = !wait_or_fail(bar_s + side, use & 1, a.wait_polls, failed);
            if (dead) break;
            tc::fence_after_sync();
            if (rows_live) {
                float x[kPagedStage];
                tmem_ld128(t_s, x);
                const uint32_t bad_pages = __ballot_sync(0xffffffffu, bad_page);
                if (k0 + kPagedStage > min(warp_all, kend) || bad_pages) {
                    uint64_t vis[2] = {sees64(k0), sees64(k0 + 64)};
                    if (bad_pages) {
                        if (lane == 0) set_status(a.status, MEDUSA_DEV_BAD_PAGE);
                        for (int e = 0; e < boxes; ++e)
                            if ((bad_pages >> e) & 1u) {
                                const int at = e << box_log2, to = at + (1 << box_log2);
                                vis[0] &= ~(bits_below(to) & ~bits_below(at));
                                vis[1] &= ~(bits_below(to - 64) & ~bits_below(at - 64));
                            }
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t v = (uint32_t)(vis[w >> 1] >> (32 * (w & 1)));
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[32 * w + e] = (v >> e) & 1u ? x[32 * w + e] : -INFINITY;
                    }
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mx[i] = max3f(x[i], x[i + 4], x[i + 8]);
#pragma unroll
                    for (int e = 12; e + 4 < kPagedStage; e += 8) mx[i] = max3f(mx[i], x[i + e], x[i + e + 4]);
                    mx[i] = fmaxf(mx[i], x[i + kPagedStage - 4]);
                }
                const float cm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * row_scale;
                bool grew = false;
                float alpha = 1.f;
                if (cm > m_run + kRescaleLog2) {  // m_run = -inf: the first visible key
                    alpha = exp2f(m_run - cm);
                    m_run = cm;
                    l_run *= alpha;
                    grew = true;
                }
                const float mu = m_run == -INFINITY ? 0.f : m_run;
                // past 2^16 the scores are rounded before the difference, as the maximum
                // was: the fused form keeps bits of the product that the maximum lost,
                // and the largest weight would leave 1
                float sc = row_scale;
                if (__any_sync(0xffffffffu, fabsf(mu) > 65536.f)) {
#pragma unroll
                    for (int e = 0; e < kPagedStage; ++e) x[e] *= row_scale;
                    sc = 1.f;
                }
                if (__any_sync(0xffffffffu, grew && use > 0)) {
                    dead = !wait_or_fail(bar_o + side, (use - 1) & 1, a.wait_polls, failed);
                    if (dead) break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < DH; c += 32) {
                        float ov[32];
                        tc::tmem_ld32(t_o + c, ov);
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] *= alpha;
                        tc::tmem_st32(t_o + c, ov);
                    }
                }
                const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-mu, -mu);
                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // the product begins with the first half
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 y = __ffma2_rn(make_float2(x[64 * c + 2 * e], x[64 * c + 2 * e + 1]), sc2, nm2);
                        const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
                        // Rounded to bf16 for the product only, whose operands are of one
                        // 16-bit type, at most 2^-8 of a weight; the sum adds the fp32
                        // weights.
                        pk[e] = pack_weights<false>(p0, p1);
                        ls[e & 1] = __fadd2_rn(ls[e & 1], make_float2(p0, p1));
                    }
                    tc::tmem_st32u(t_s + 32 * c, pk);
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    tc::mbar_arrive(bar_p + 2 * side + c);
                }
                l_run += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
            } else {
                tc::fence_before_sync();
                tc::mbar_arrive(bar_p + 2 * side);
                tc::mbar_arrive(bar_p + 2 * side + 1);
            }
        }
        // ---- the last product, then the row
        if (!dead && use > 0) dead = !wait_or_fail(bar_o + side, (use - 1) & 1, a.wait_polls, failed);
        tc::fence_after_sync();
        // what V's infinities and NaNs add to 32 columns of the row, from the cache
        auto add_not_finite = [&](int c0, float (&ov)[32]) {
            const bf16 *q_row = static_cast<const bf16 *>(a.q) + row_at(r, m - r * G) * DH;
#pragma unroll 1
            for (int j = j_masked; j < nsub; ++j) {
                if (turns && (j & 1) != side) continue;
#pragma unroll 1
                for (int key = 0; key < kPagedStage; ++key) {
                    if (!((bad_keys[4 * (j - j_masked) + (key >> 5)] >> (key & 31)) & 1u)) continue;
                    const int slot = first_key(j) + key;
                    if (!((sees64(slot & ~63) >> (slot & 63)) & 1ull)) continue;
                    const int page = a.map.page_of(b, slot);
                    if (!a.map.good(page)) continue;
                    const size_t at = (a.map.row(page, slot) * a.Hkv + gs) * DH;
                    const bf16 *kr = static_cast<const bf16 *>(a.kp) + at;
                    const bf16 *vr = static_cast<const bf16 *>(a.vp) + at;
                    float s = 0.f;
#pragma unroll 1
                    for (int c = 0; c < DH; ++c) s = fmaf(__bfloat162float(q_row[c]), __bfloat162float(kr[c]), s);
                    const float p = exp2f(s * row_scale - m_run);
                    if (p == 0.f) continue;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float v = __bfloat162float(vr[c0 + c]);
                        if (!isfinite(v)) ov[c] += p * v;
                    }
                }
            }
        };
        const bool odd_v = *reinterpret_cast<volatile int *>(bad_v) != 0;
        float *join = reinterpret_cast<float *>(sm) + t * L::LD;
        float2 *join_ml = reinterpret_cast<float2 *>(sm + 128 * L::LD * 4) + t;
        const bool none = use == 0;  // no stage was this half's
        if (split) {
            // B's half goes through shared memory: every product has read its operands
            asm volatile("barrier.cta.sync 1, 256;\n" ::: "memory");
            if (side == 1 && !dead && rows_live && !none) {
#pragma unroll 1
                for (int c = 0; c < DH; c += 32) {
                    float ov[32];
                    tc::tmem_ld32(t_o + c, ov);
                    if (odd_v && live) add_not_finite(c, ov);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4 *>(join + c + e) = make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                }
            }
            if (side == 1) *join_ml = make_float2(m_run, l_run);
            asm volatile("barrier.cta.sync 1, 256;\n" ::: "memory");
            dead = __any_sync(0xffffffffu, dead || *failed);  // the other half's wait as well
        }
        if (dead) {
            publish_nothing();
        } else if (rows_live && !(split && side)) {
            // weights of the halves: 2^(m - top)
            float fa = 1.f, fb = 0.f, top = m_run, l = l_run;
            if (split) {
                const float mb = join_ml->x, lb = join_ml->y;
                top = fmaxf(m_run, mb);
                const float mu = top == -INFINITY ? 0.f : top;
                fa = exp2f(m_run - mu);
                fb = exp2f(mb - mu);
                // (also with a factor of 0: a row of NaN scores has m = -inf, l = NaN)
                l = fa * l_run + fb * lb;
            }
            const float inv = !direct ? 1.f : l == 0.f ? 0.f : 1.f / l;
            fa *= inv;
            fb *= inv;
            // Rows go out through shared memory, whole rows of bf16 or halves of fp32 at a
            // time: stored by their threads they took 10700 cycles a CTA (of 81000 for 32
            // stages), and Q read by them 8200.  The place: the side's Q tile, whose last
            // product is done, or (halves) one behind what they were joined in.
            unsigned char *stage = sm + (split ? 3 : side) * L::TILE + (warp & 3) * 32 * DH * 2;
            auto piece = [&](int row, int c) {
                return reinterpret_cast<uint4 *>(stage + row * DH * 2 + ((c ^ (row & 7)) << 4));
            };
            const int passes = direct || CLUSTER ? 1 : 2, wide = DH / passes;  // columns a pass
#pragma unroll 1
            for (int pass = 0; pass < passes; ++pass) {
#pragma unroll 1
                for (int c = pass * wide; c < (pass + 1) * wide; c += 32) {
                    float ov[32];
                    if (none) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = 0.f;
                    } else {
                        tc::tmem_ld32(t_o + c, ov);
                    }
                    if (odd_v && live) add_not_finite(c, ov);
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] *= fa;
                    if (fb != 0.f) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 o = *reinterpret_cast<const float4 *>(join + c + e);
                            ov[e] = fmaf(fb, o.x, ov[e]);
                            ov[e + 1] = fmaf(fb, o.y, ov[e + 1]);
                            ov[e + 2] = fmaf(fb, o.z, ov[e + 2]);
                            ov[e + 3] = fmaf(fb, o.w, ov[e + 3]);
                        }
                    }
                    if (CLUSTER) {
                        float *dst = part_o + t * L::LD + c;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(dst + e) = make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                    } else if (direct) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *piece(lane, (c + e) / 8) =
                                make_uint4(pack_weights<false>(ov[e], ov[e + 1]), pack_weights<false>(ov[e + 2], ov[e + 3]),
                                           pack_weights<false>(ov[e + 4], ov[e + 5]), pack_weights<false>(ov[e + 6], ov[e + 7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *piece(lane, (c - pass * wide + e) / 4) =
                                make_uint4(__float_as_uint(ov[e]), __float_as_uint(ov[e + 1]), __float_as_uint(ov[e + 2]),
                                           __float_as_uint(ov[e + 3]));
                    }
                }
                if (CLUSTER) continue;
                __syncwarp();
                if (direct)
                    for_rows(row_at, 1, a.H - G + 1, [&](int i, int c, long long row) {
                        const uint4 y = *piece(i, c);
                        if (mw + i < M) *reinterpret_cast<uint4 *>(static_cast<bf16 *>(a.out) + row * DH + c * 8) = y;
                    });
                else
                    for_rows(part_at, R, 1 - (long long)(G - 1) * R, [&](int i, int c, long long row) {
                        const uint4 y = *piece(i, c);
                        if (mw + i < M) *reinterpret_cast<uint4 *>(a.part_o + row * DH + pass * wide + c * 4) = y;
                    });
                __syncwarp();
            }
            if (CLUSTER)
                part_ml[t] = make_float2(top, l);
            else if (live && !direct)
                a.part_ml[part_at(r, m - r * G)] = make_float2(top, l);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && *failed) set_status(a.status, MEDUSA_DEV_TIMEOUT);
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
    if constexpr (CLUSTER) join_cluster();
}

// A pool as [Hkv dh / 64][rows][64] for boxes of `box` rows (all of a head's columns
// where a box is a whole stage), 128-byte swizzle, zeros past the rows.
bool encode_pool(CUtensorMap *map, const void *pool, const CacheAttnArgs &a, int dh) {
    EncodeTiled fn = tensor_map_encoder();
    if (!fn) return false;
    const uint32_t box_rows = a.map.shift >= 7 ? 128u : 1u << a.map.shift;
    const cuuint64_t cols = (cuuint64_t)a.Hkv * dh;
    const cuuint64_t dims[3] = {64, (cuuint64_t)a.map.n_pages << a.map.shift, cols / 64};
    const cuuint64_t strides[2] = {cols * 2, 128};
    const cuuint32_t box[3] = {64, box_rows, box_rows == 128 ? (cuuint32_t)dh / 64 : 1u};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(pool), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of a row tile
int units_of(const CacheAttnArgs &a) { return a.pair ? (a.Hkv + 1) / 2 : a.Hkv; }

template <int DH>
cudaError_t launch(const PagedMaps &maps, const CacheAttnArgs &a, cudaStream_t stream) {
    auto kern = a.starts    ? paged_attn_tc_kernel<DH, true, kTiles>
                : a.pair    ? paged_attn_tc_kernel<DH, false, kPair>
                : a.cluster ? paged_attn_tc_kernel<DH, false, kCluster>
                            : paged_attn_tc_kernel<DH, false, kTiles>;
    constexpr int smem = PagedSmem<DH>::TOTAL;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e) return e;
    const dim3 grid(units_of(a) * a.row_tiles, a.ranges ? a.ranges : a.ns, a.ranges ? 1 : a.B);
    if (a.cluster)
        return launch_pdl_cluster(kern, grid, dim3(kThreads), dim3(1, a.ns, 1), (size_t)smem, stream, maps, a);
    return launch_pdl(kern, grid, dim3(kThreads), (size_t)smem, stream, maps, a);
}

}  // namespace

int paged_cluster_slots(int dh, int size) {
    static std::atomic<int> known[64][2][kClusterRanges + 1];  // one more than the count
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::atomic<int> &k = known[dev][dh == 128][size];
    if (int x = k.load(std::memory_order_relaxed)) return x - 1;
    auto kern = dh == 128 ? paged_attn_tc_kernel<128, false, kCluster> : paged_attn_tc_kernel<64, false, kCluster>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = dh == 128 ? PagedSmem<128>::TOTAL : PagedSmem<64>::TOTAL;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = attr.val.clusterDim.z = 1;
    attr.val.clusterDim.y = size;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes) ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) {
        cudaGetLastError();
        return 0;
    }
    k.store(n + 1, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_paged_attention_tc(const CacheAttnArgs &a, int dh, cudaStream_t stream) {
    PagedMaps maps;
    maps.by_g = Divisor(a.H / a.Hkv);
    maps.by_units = Divisor(units_of(a));
    if (!encode_pool(&maps.k, a.kp, a, dh) || !encode_pool(&maps.v, a.vp, a, dh)) {
        set_last_error("tensor maps of the pools could not be made (cuTensorMapEncodeTiled failed)");
        return cudaErrorInvalidValue;
    }
    return dh == 128 ? launch<128>(maps, a, stream) : launch<64>(maps, a, stream);
}

}  // namespace medusa
