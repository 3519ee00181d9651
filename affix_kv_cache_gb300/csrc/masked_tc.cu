// masked_tc.cu -- read-slot attention under a mask on the tensor cores (tcgen05 + TMEM, TMA-fed): bf16, head
// dim 64 or 128, a positive scale.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4.3 and App. C.1 (attention through the read-slot
// map); ranges, caps and distance biases are this library's (include/acache.h, acache_slot_attention_masked).
//
//   s = scale q.k, capped by c tanh(s / c), biased by -slope |pos - t|; softmax over the row's keys [lo, hi)
//
// One CTA per (request, KV head, query block): two Q tiles A and B of 128 rows, a row being a (query, head of the
// group) pair, so that all heads of a group share one K/V stream and a causal block spans few positions.
//   WG0, WG1   softmax + epilogue of tile A / B, thread r owning row r = TMEM lane r: a tile of scores is read
//              into registers, capped, biased, masked, exponentiated in base 2 against a reference that
//              follows the sums of weights, and written back over the scores as bf16 for the product with V.
//   warp 8     issues the MMAs of both (S = Q K^T from shared memory, O += P V with P from TMEM), A's and B's in turn
//   warps 10-15  TMA producers of a 3-stage K ring and a 2-stage V ring: a tile of 128 consecutive slots is tiled
//              box loads of the pool, any other gather4 loads of four rows each.
// A block left with one Q tile splits its keys between the two chains and merges them at the end.  Where blocks leave SMs idle, a
// cluster of up to 8 CTAs shares a block's keys; each leaves its unnormalised sums, references and sums of weights in shared memory and
// merges D / cs columns of all rows out of its peers'.
// The CTA streams only keys from the first that one of its rows sees to the last: the window [min lo, max hi),
// which need not start at a whole tile.  Inside it a row's range is a bit mask per 32 keys; tiles that every row of a warp sees
// whole skip it.  Blocks run from the last to the first, so that a causal call starts its longest first.
// What a masked key holds cannot reach a row through its score (replaced by -infinity), but 0 x NaN is NaN in
// the product with V: a row whose output is not finite while its sum of weights is, is computed again by its
// warp over its own keys alone.
//
// Measured: causal prompts of 2 x 4,096 (32 heads over 8, d = 128) 241 us, 1,140 TFLOP/s over the keys that rows see;
// block-causal capped point of 16 x 986 rows over 2,624 keys (28 over 4) 502 us, 970 TFLOP/s.  A step of both chains takes
// some 3,500 cycles (capped: 4,100) where its MMAs need 2,150: the MMAs of a chain wait for barriers some 700 cycles a
// tile, a capped softmax (2,700 cycles, two of them at a time) for issue.  Set-up, the first tile's loads and the
// epilogue take 14,000 cycles of a CTA's 60,000.  What was tried: two issuing warps (their MMAs interleave and both chains
// end together), waits merged or tested ahead (slower by 2 to 9 %), polling instead of suspended waits (7 to 9 %), chains
// that take turns (no difference, or 8 % slower), CTAs that stay and take block after block, the next one's Q and
// K loaded under the last's epilogue (uncapped 1 % faster, capped 14 % slower: the store of rows straight to memory and
// a longer loop ate what it hid).
//
// Every mbarrier wait is bounded (acache_wait_budget); a wait that gives up raises a CTA-wide abort flag and
// ACACHE_DEV_TIMEOUT, roles leave their loops, MMAs and loads in flight are waited for (bounded), and TMEM is
// freed before the CTA exits.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "masked.cuh"
#include "ptx.cuh"
#include "q8.cuh"
#include "step.cuh"
#include "tc_attn.cuh"

namespace acache {
namespace {

using namespace ptx;
using bf16 = __nv_bfloat16;

constexpr int kBM = 128;                    // rows of a Q tile
constexpr int kQT = 2;                      // Q tiles to a CTA
constexpr int kBN = 128;                    // keys of a tile
constexpr int kKStages = 3, kVStages = 2;
constexpr float kAgain = -1.f;              // in place of a row's sum of weights
constexpr int kMaxParts = 8;                // CTAs to a block (a portable cluster)
constexpr int kMmaWarp = 8, kProdWarp = 10, kProdPerRing = 3;
constexpr int kThreads = (kProdWarp + 2 * kProdPerRing) * 32;
// Registers: 512 threads x 128 at launch; the softmax warpgroups grow to 208, which hold a tile's scores without spilling,
// the others shrink to 48.  (640 threads leave them 168: 3 to 7 % slower.)
constexpr int kRegLaunch = 65536 / kThreads / 8 * 8, kRegSoftmax = 208, kRegOther = 48;
static_assert(2 * 128 * kRegSoftmax + (kThreads - 256) * kRegOther <= kThreads * kRegLaunch, "register split");
constexpr uint32_t kRegion = kBN * 128;     // 64 columns of a 128-row tile
__host__ __device__ constexpr uint32_t tile_bytes(int D) { return (uint32_t)(D / 64) * kRegion; }
__host__ __device__ constexpr uint32_t smem_bytes(int D) { return tile_bytes(D) * (kQT + kKStages + kVStages) + 1024; }
constexpr uint32_t kTmemCols = 512;         // S_A, S_B, O_A, O_B
__host__ __device__ constexpr uint32_t col_s(int t) { return (uint32_t)t * 128u; }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + (uint32_t)t * 128u; }
// Scores within +-50 need no running maximum: weights e^s between 2e-22 and 6e21 are ordinary float32 and bf16 numbers, and so
// are sums of 2^31 of them.  (Products with V beyond float32 give a row that is not finite, which is computed again.)
constexpr float kBoundedCap = 50.f;
// tanh y / y = 1 + c1 y^2 + c2 y^4 + c3 y^6 within 2^-20.5 of itself up to y = 1/2 (relative minimax fit): there 5.0 x 2^-24
// of the cap, and with the roundings of its operations 8, less than the plain form's 11.  (A level of one term
// less up to y = 1/4 made the call slower: most tiles hold a larger score.)
constexpr double kTanhHalf[4] = {1, -0.33328159, 0.1320536, -0.04475064};
constexpr long long kDrainBudget = 1LL << 31, kLandBudget = 1LL << 21;   // cycles: the abort path's own waits

// Log2 units by which partial sums are scaled down where they are joined: each may lie close below 2^128 (a last tile
// whose scores jump by 100 and more raises no reference), and up to 16 of them are added.
constexpr float kSpare = 8.f;

struct MaskParams {
    CUtensorMap tm_q;     // fixed: 4-D [B][n_q][Hq][d], box {64, g, qpt, 1}; ragged: 3-D [total_q][Hq][d], box {64, g, qpt}
    CUtensorMap tm_o;     // output, laid out as tm_q
    CUtensorMap tm_kg;    // 2-D pool rows [num_slots * Hkv][d], box {64, 1} (gather4)
    CUtensorMap tm_vg;
    CUtensorMap tm_kb;    // 3-D pool [num_slots][Hkv][d], box {64, 1, 128} (consecutive slots)
    CUtensorMap tm_vb;
    const bf16 *q, *k_cache, *v_cache;
    bf16* out;
    const int32_t *read_slot, *q_start, *kv_start, *row_range, *q_pos;
    const float* slopes;
    int32_t* dev_status;
    int64_t num_slots;
    int n_rows, total_q, T_len, Hq, Hkv, g;
    int qpt;              // queries of a tile: floor(128 / g)
    int drop, wide;       // wide: a cap above kWideCap
    float scale_log2;     // > 0
    float cap_in;         // 2 log2e scale / softcap: 2^(cap_in q.k) = e^(2 s / softcap)
    float cap_log2;       // softcap log2e
    float cap_near;       // |q.k| of a score of half the cap ...
    float cap_k[4];       // ... up to which the capped score in log2 units is q.k times this polynomial in (q.k)^2
    long long budget;
    int cs;               // CTAs (a cluster) to a block, each with a part of its window
};

struct MaskCtl {
    uint64_t q_full;
    uint64_t k_full[kKStages], k_empty[kKStages];
    uint64_t v_full[kVStages + 1], v_empty[kVStages + 1];   // + the stage in the free Q buffer (split keys)
    uint64_t s_full[kQT], p_half[kQT], p_full[kQT];
    uint64_t drain[kQT];  // chain t's MMAs are complete
    uint64_t fin;         // ... and all of them, on every path
    uint32_t tmem_base;
    int abort;
    int unlanded;         // abort path: some load issued before the abort may not have landed
    int split_ok;
    int win_lo[8], win_hi[8];
    float missing[8];             // (split clusters) by softmax warp: a wait gave up
    float split_m[kBM], split_l[kBM];
};

static_assert(kKStages == 3 && kVStages == 2, "ring sizes 2 and 3");
ACACHE_DEVFN int ring_lap(int e, int n) { return n == 2 ? (e >> 1) : e / 3; }
ACACHE_DEVFN int ring_stage(int e, int n) { return e - ring_lap(e, n) * n; }

// Ring entry e is the e-th tile loaded; chain t reads its i-th tile from entry(t, i).  Unsplit: every chain
// reads every tile.  Split: chain 0 tiles [0, n0), chain 1 the rest, entries alternating.
struct KeySchedule {
    bool split;
    int n_kv, n0;
    ACACHE_DEVFN int n_tiles(int t) const { return split ? (t == 0 ? n0 : n_kv - n0) : n_kv; }
    ACACHE_DEVFN int tile(int t, int i) const { return (split && t == 1) ? n0 + i : i; }
    ACACHE_DEVFN int entry(int t, int i) const {
        if (!split) return i;
        const int n1 = n_kv - n0;
        return i < n1 ? 2 * i + t : n1 + i;
    }
    ACACHE_DEVFN int entry_tile(int e) const {
        if (!split) return e;
        const int n1 = n_kv - n0;
        if (e < 2 * n1) return (e & 1) ? n0 + (e >> 1) : (e >> 1);
        return e - n1;
    }
};

// Bounded wait that also leaves early once another role has aborted.  The hardware's suspending wait returns after a time
// of its own, some microseconds: budgets below that are polled.
constexpr long long kPatient = 1LL << 16;
ACACHE_DEVFN bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* dev_status, long long budget) {
    if (budget >= kPatient ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (budget >= kPatient ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > budget) {
            *abort_flag = 1;
            flag(dev_status, ACACHE_DEV_TIMEOUT);
            return false;
        }
    }
}

ACACHE_DEVFN void st_shared_f32(uint32_t addr, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory"); }
// bits [max(n, 0), 32), none from 32 on (the instruction clamps its shift)
ACACHE_DEVFN uint32_t bits_from(int n) {
    uint32_t r;
    asm("shl.b32 %0, 0xffffffff, %1;" : "=r"(r) : "r"(max(n, 0)));
    return r;
}
// kCap: scores are capped; kBounded: by so little that they need no maximum (then there is no bias); kParts: a
// cluster of CTAs shares a block's keys.
template <int D, bool kCap, bool kBounded, bool kBias, bool kParts>
__global__ void __launch_bounds__(kThreads, 1)
masked_tc_kernel(const __grid_constant__ MaskParams p) {
    constexpr uint32_t kTileBytes = tile_bytes(D);
    constexpr int kHalves = D / 64;                    // 64-column regions of a tile
    extern __shared__ uint8_t dsm[];
    __shared__ MaskCtl ctl;
    const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
    auto sQ = [&](int t) { return base + kTileBytes * (uint32_t)t; };
    auto sK = [&](int s) { return base + kTileBytes * (uint32_t)(kQT + s); };
    auto sV = [&](int s) { return base + kTileBytes * (uint32_t)(kQT + kKStages + s); };
    const int hk = kParts ? (int)blockIdx.x / p.cs : (int)blockIdx.x, rank = kParts ? (int)blockIdx.x % p.cs : 0, b = (int)blockIdx.y, qb = (int)(gridDim.z - 1 - blockIdx.z);
    int n_rows = p.n_rows, T_len = p.T_len;
    int64_t qbase = (int64_t)b * p.n_rows, kbase = (int64_t)b * p.T_len;
    if (p.q_start) {
        qbase = p.q_start[b];
        kbase = p.kv_start[b];
        n_rows = q8_count(p.q_start, b);
        T_len = q8_count(p.kv_start, b);
        if (n_rows != 0 && q8_bad_lengths(n_rows, p.n_rows, T_len, p.T_len, qbase, p.total_q, kbase)) {
            if (threadIdx.x == 0 && qb == 0 && hk == 0) flag(p.dev_status, ACACHE_DEV_BAD_LENGTH);
            return;
        }
    }
    const int qpt = p.qpt;
    const int q0 = qb * kQT * qpt;
    if (q0 >= n_rows) return;
    const int n_qt = q0 + qpt < n_rows ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
    volatile int* abort_flag = &ctl.abort;
    int32_t* dev_status = p.dev_status;
    const long long budget = p.budget;

    // Row `at` of Q tile `t`: its query of the request and its keys [lo, hi) (lo = hi = 0: none, or no row).
    auto row_keys = [&](int t, int at, int& lo, int& hi) -> bool {
        const int qi = q0 + t * qpt + at / p.g;
        lo = hi = 0;
        if (at >= qpt * p.g || qi >= n_rows) return false;
        hi = T_len;
        if (p.row_range) {
            lo = max(p.row_range[2 * (qbase + qi)], 0);
            hi = min(p.row_range[2 * (qbase + qi) + 1], T_len);
        }
        if (lo >= hi) lo = hi = 0;
        return true;
    };
    if (wg < kQT) {
        int lo, hi;
        row_keys(wg, threadIdx.x & 127, lo, hi);
        const int a = __reduce_min_sync(0xffffffffu, lo < hi ? lo : 0x7fffffff), z = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            ctl.win_lo[warp] = a;
            ctl.win_hi[warp] = z;
        }
    }
    if (threadIdx.x == 0) {
        mbar_init(&ctl.q_full, 1);
        // stages fill with one arrival per producer warp of the ring, and are free with the MMAs of the last chain that
        // reads them
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(&ctl.k_full[s], kProdPerRing);
            mbar_init(&ctl.k_empty[s], 1);
        }
        for (int s = 0; s < kVStages + 1; ++s) {
            mbar_init(&ctl.v_full[s], kProdPerRing);
            mbar_init(&ctl.v_empty[s], 1);
        }
        for (int t = 0; t < kQT; ++t) {
            mbar_init(&ctl.s_full[t], 1);
            mbar_init(&ctl.p_half[t], 128);
            mbar_init(&ctl.p_full[t], 128);
            mbar_init(&ctl.drain[t], 1);
        }
        mbar_init(&ctl.fin, 1);
        ctl.abort = 0;
        ctl.unlanded = 0;
        ctl.split_ok = 1;
        fence_mbar_init();
        mbar_arrive_expect_tx(&ctl.q_full, (uint32_t)(n_qt * kHalves * 128 * p.g * qpt));
        for (int t = 0; t < n_qt; ++t)
            for (int x = 0; x < kHalves; ++x) {
                if (p.q_start) tma_load_3d(sQ(t) + x * kRegion, &p.tm_q, 64 * x, hk * p.g, (int)qbase + q0 + t * qpt, &ctl.q_full);
                else tma_load_4d(sQ(t) + x * kRegion, &p.tm_q, 64 * x, hk * p.g, q0 + t * qpt, b, &ctl.q_full);
            }
    }
    // Rows of a Q tile that no (query, head) pair fills are zeros: scores out of what lay there could send their warp the
    // long ways through a cap or a raised reference (measured: an otherwise equal call took 720 us for 574).
    const int n_fill = (kBM - qpt * p.g) * 8;              // 16-byte pieces of a region
    for (int x = threadIdx.x; x < kQT * kHalves * n_fill; x += kThreads)
        *reinterpret_cast<uint4*>(dsm + (base - smem_u32(dsm)) + (x / n_fill) * kRegion + qpt * p.g * 128 + (x % n_fill) * 16) =
            make_uint4(0, 0, 0, 0);
    if (n_fill > 0) fence_proxy_async_smem();
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The window of keys that the CTA streams.
    int w_lo = 0x7fffffff, w_hi = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        w_lo = min(w_lo, ctl.win_lo[x]);
        w_hi = max(w_hi, ctl.win_hi[x]);
    }
    if (w_lo > w_hi) w_lo = w_hi = 0;
    int T_win = w_hi - w_lo;
    if constexpr (kParts) {                            // ... or this CTA's part of them, whole tiles
        const int n_all = (T_win + kBN - 1) / kBN, j0 = n_all * rank / p.cs, j1 = n_all * (rank + 1) / p.cs;
        w_lo += j0 * kBN;
        T_win = max(min(T_win - j0 * kBN, (j1 - j0) * kBN), 0);
    }
    const int n_kv = (T_win + kBN - 1) / kBN;
    const int32_t* rs = p.read_slot + kbase + w_lo;
    const bool split = n_qt == 1 && n_kv >= 2;
    const int n_ch = split ? 2 : n_qt;
    const KeySchedule ks{split, n_kv, split ? (n_kv + 1) / 2 : n_kv};
    const int n_vst = split ? kVStages + 1 : kVStages;
    // (split clusters) what a CTA leaves of its part: sums in sK(0), sK(1) / sV(0), sV(1), [column / 4][row] of 4; m and l in sK(2)
    auto part_o = [&](int t) { return t == 0 ? sK(0) : sV(0); };
    auto part_m = [&](int t) { return sK(2) + 1024u * (uint32_t)t; };
    auto part_l = [&](int t) { return sK(2) + 1024u * (uint32_t)t + 512u; };
    auto sVs = [&](int s) { return s < kVStages ? sV(s) : sQ(1); };
    const uint32_t tmem = ctl.tmem_base;

    if (wg >= 2) {
        setmaxnreg_dec<kRegOther>();
        if (warp >= kProdWarp) {
            // -------------------------------------------------------------- TMA producers
            if (warp == kProdWarp && lane == 0) {
                tma_prefetch_desc(&p.tm_o);
                tma_prefetch_desc(&p.tm_kg);
                tma_prefetch_desc(&p.tm_vg);
                tma_prefetch_desc(&p.tm_kb);
                tma_prefetch_desc(&p.tm_vb);
            }
            const bool flagger = warp == kProdWarp;
            const bool is_v = warp >= kProdWarp + kProdPerRing;
            const int pi = warp - kProdWarp - (is_v ? kProdPerRing : 0);
            const int nst = is_v ? n_vst : kKStages;
            uint64_t* full = is_v ? ctl.v_full : ctl.k_full;
            uint64_t* empty = is_v ? ctl.v_empty : ctl.k_empty;
            const CUtensorMap* tm_g = is_v ? &p.tm_vg : &p.tm_kg;
            const CUtensorMap* tm_b = is_v ? &p.tm_vb : &p.tm_kb;
            const bool leader = pi == 0 && lane == 0;
            const int oob_row = (int)(p.num_slots * p.Hkv);
            // this lane's gather x of a tile: 4-row group x / kHalves, column region x % kHalves
            const int x = kProdPerRing * lane + pi;
            const bool gathers = x < 32 * kHalves;
            const int grp = x / kHalves, half = x % kHalves;
            // Tile j, resolved one entry ahead: lane l reads the slots of keys 4 l .. 4 l + 3; whether the tile's 128
            // slots are consecutive, its first slot, and the pool rows of this lane's gather.  A slot outside
            // the pool, a discarded key and a place behind the window read zeros.
            auto resolve = [&](int j, int (&rows)[4], int& slot0) -> bool {
                int sl[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int t = j * kBN + 4 * lane + u;
                    sl[u] = -1;
                    if (j < n_kv && t < T_win) {
                        const int slot = __ldg(rs + t);
                        if (slot >= 0 && slot < p.num_slots) sl[u] = slot;
                        else if (flagger && !(p.drop && slot == ACACHE_SLOT_NONE)) flag(dev_status, ACACHE_DEV_BAD_SLOT);
                    }
                }
                bool run = sl[0] >= 0 && sl[1] == sl[0] + 1 && sl[2] == sl[0] + 2 && sl[3] == sl[0] + 3;
                const int after = __shfl_down_sync(0xffffffffu, sl[0], 1);
                if (lane < 31) run = run && after == sl[0] + 4;
                slot0 = __shfl_sync(0xffffffffu, sl[0], 0);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int sv = __shfl_sync(0xffffffffu, sl[u], grp & 31);
                    rows[u] = (gathers && sv >= 0) ? sv * p.Hkv + hk : oob_row;
                }
                return __all_sync(0xffffffffu, run);
            };
            int next[4], next_slot0;
            bool next_box = resolve(n_kv > 0 ? ks.entry_tile(0) : 0, next, next_slot0);
            int armed = -1;
            for (int e = 0; e < n_kv; ++e) {
                const int s = ring_stage(e, nst);
                const uint32_t dst = is_v ? sVs(s) : sK(s);
                int rows[4] = {next[0], next[1], next[2], next[3]};
                const int slot0 = next_slot0;
                const bool box = next_box;
                next_box = resolve(e + 1 < n_kv ? ks.entry_tile(e + 1) : n_kv, next, next_slot0);
                if (e >= nst &&
                    !__all_sync(0xffffffffu, wait_bar(&empty[s], (ring_lap(e, nst) - 1) & 1, abort_flag, dev_status, budget)))
                    break;
                // one arrival per warp of the ring, also where the first warp loads alone: no warp can then fall
                // two phases behind a stage's barrier
                if (leader) mbar_arrive_expect_tx(&full[s], kTileBytes);
                else if (lane == 0) mbar_arrive(&full[s]);
                armed = e;
                __syncwarp();
                if (box) {
                    if (leader) {
#pragma unroll
                        for (int h = 0; h < kHalves; ++h) tma_load_3d(dst + h * kRegion, tm_b, 64 * h, hk, slot0, &full[s]);
                    }
                } else if (gathers) {
                    tma_gather4(dst + (uint32_t)half * kRegion + (uint32_t)grp * 512u, tm_g, half * 64, rows[0], rows[1], rows[2],
                                rows[3], &full[s]);
                }
            }
            if (*abort_flag && armed >= 0) {
                bool landed = true;
                for (int e = max(0, armed - nst + 1); e <= armed; ++e)
                    landed = mbar_wait(&full[ring_stage(e, nst)], (uint32_t)ring_lap(e, nst) & 1u, kLandBudget) && landed;
                if (!__all_sync(0xffffffffu, landed) && lane == 0) ctl.unlanded = 1;
            }
        } else {
            // ------------------------------------------------------------------ MMA issuer
            // One thread issues both chains' MMAs, A's and B's in turn: PV(i) in two halves of the tile as the softmax
            // publishes them, then S(i + 1).  A chain's MMAs then run as one burst, and the chains fall into
            // step, one in its softmax while the other's MMAs run.  (Two issuing threads interleaved their MMAs: both
            // chains' bursts took twice as long and ended together, and neither softmax overlapped an MMA.)
            // The whole warp walks the steps, so addresses and descriptors stay in uniform registers, and one lane
            // issues (one lane alone took 80 to 100 cycles to issue an MMA of 64).
            if (warp == kMmaWarp) {
                const bool leader = elect_one();
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                const int nk = __shfl_sync(0xffffffffu, n_kv, 0);
                const bool two = __shfl_sync(0xffffffffu, n_ch, 0) == 2, halved = __shfl_sync(0xffffffffu, (int)split, 0) != 0;
                const KeySchedule us{halved, nk, halved ? (nk + 1) / 2 : nk};
                const int vst = halved ? kVStages + 1 : kVStages;
                constexpr uint32_t idS = idesc_bf16(kBM, kBN, false, false);
                constexpr uint32_t idO = idesc_bf16(kBM, D, false, true);
                auto wait = [&](uint64_t* bar, int phase) {
                    return __all_sync(0xffffffffu, wait_bar(bar, (uint32_t)phase & 1u, abort_flag, dev_status, budget));
                };
                auto issue_s = [&](int t, int e) -> bool {
                    const int st = e % kKStages;
                    if (!wait(&ctl.k_full[st], e / kKStages)) return false;
                    tc_fence_after();
                    const uint64_t dq = sdesc_sw128(sQ(halved ? 0 : t), 16, 1024);
                    const uint64_t dk = sdesc_sw128(sK(st), 16, 1024);
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint64_t ko = ((uint64_t)(k >> 2) * kRegion + (uint64_t)(k & 3) * 32u) >> 4;
                            umma_ss(tm + col_s(t), dq + ko, dk + ko, idS, k > 0);
                        }
                        umma_commit(&ctl.s_full[t]);
                        if (halved || !two || t == 1) umma_commit(&ctl.k_empty[st]);
                    }
                    return true;
                };
                // (also without a key: the Q tiles have landed before the CTA goes on)
                bool ok = wait(&ctl.q_full, 0);
                if (ok && nk > 0) ok = issue_s(0, us.entry(0, 0));
                if (ok && nk > 0 && two) ok = issue_s(1, us.entry(1, 0));
                const int steps = us.n_tiles(0) * (two ? 2 : 1);    // chain 0 has as many tiles as chain 1, or one more
                for (int it = 0; ok && it < steps; ++it) {
                    const int t = two ? it & 1 : 0, i = two ? it >> 1 : it;
                    const int nt = us.n_tiles(t);
                    if (i >= nt) continue;
                    const int e = us.entry(t, i), st = ring_stage(e, vst);
                    ok = wait(&ctl.v_full[st], ring_lap(e, vst)) && wait(&ctl.p_half[t], i);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dv = sdesc_sw128(sVs(st), kRegion, 1024);
                    const uint32_t d_o = tm + col_o(t), d_p = tm + col_s(t);
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) umma_ts(d_o, d_p + k * 8, dv + (uint64_t)(k * 2048 / 16), idO, (i > 0 || k > 0));
                    }
                    ok = wait(&ctl.p_full[t], i);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 4; k < 8; ++k) umma_ts(d_o, d_p + k * 8, dv + (uint64_t)(k * 2048 / 16), idO, 1);
                        if (halved || !two || t == 1) umma_commit(&ctl.v_empty[st]);
                        if (i + 1 == nt) umma_commit(&ctl.drain[t]);    // the chain's last
                    }
                    if (i + 1 < nt) ok = issue_s(t, us.entry(t, i + 1));
                }
                // no MMA may still run when TMEM is released
                if (leader) umma_commit(&ctl.fin);
                mbar_wait(&ctl.fin, 0, kDrainBudget);
            }
            __syncwarp();
        }
        if constexpr (kParts) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        setmaxnreg_inc<kRegSoftmax>();
        if (wg < n_ch) {
        // ------------------------------------------------------------------ softmax + epilogue
        const int t = wg;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int r = threadIdx.x & 127;
        const int rt = split ? 0 : t;                      // (with split keys both chains work on tile A's rows)
        int a_lo, a_hi;
        const bool mine = row_keys(rt, r, a_lo, a_hi);
        a_lo -= w_lo;                                      // from the window's start
        a_hi -= w_lo;
        float slope = 0.f;
        int64_t away = 0;                                  // the row's position from the window's start
        if (kBias && mine) {
            slope = p.slopes[hk * p.g + r % p.g] * kLog2e;
            away = (int64_t)p.q_pos[qbase + q0 + rt * qpt + r / p.g] - w_lo;
        }
        const int nt = ks.n_tiles(t);
        float m_used = kBounded ? 0.f : -INFINITY, l_sum = 0.f;
        int up = 0;                                        // powers of two by which the next tile raises the reference
        bool lost = false, saw = false, ok = true;         // saw: the row sees a key
        for (int i = 0; i < nt; ++i) {
            const int j = ks.tile(t, i);
            // the row's keys of the tile, one bit each, before the wait for its scores
            uint32_t see[4];
            const int f_lo = a_lo - j * kBN, f_hi = a_hi - j * kBN;
            bool whole = f_lo <= 0 && f_hi >= kBN;         // (a row that is none does not count)
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) see[cc] = bits_from(f_lo - 32 * cc) & ~bits_from(f_hi - 32 * cc);
            if (p.drop) {
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    const int tk = j * kBN + cc * 32 + lane;
                    const uint32_t gone = __ballot_sync(0xffffffffu, tk < T_win && rs[tk] == ACACHE_SLOT_NONE);
                    see[cc] &= ~gone;
                    whole = whole && gone == 0u;
                }
            }
            saw = saw || (see[0] | see[1] | see[2] | see[3]) != 0u;
            whole = __all_sync(0xffffffffu, whole || !mine);
            ok = __all_sync(0xffffffffu, wait_bar(&ctl.s_full[t], i & 1, abort_flag, dev_status, budget));
            if (!ok) break;
            tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) tmem_ld32(lane_base + col_s(t) + cc * 32, v[cc]);
            tmem_ld_wait();
            if constexpr (kCap) {
                // |s| up to half the cap in the whole warp: s times a polynomial in s^2, two elements to an instruction
                float am[4];
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    am[cc] = 0.f;
#pragma unroll
                    for (int x = 0; x < 32; x += 2)
                        am[cc] = max3abs(am[cc], __uint_as_float(v[cc][x]), __uint_as_float(v[cc][x + 1]));
                }
                if (!__any_sync(0xffffffffu, max3f(am[0], am[1], fmaxf(am[2], am[3])) > p.cap_near)) {
                    const uint64_t k0 = f2pack(p.cap_k[0], p.cap_k[0]), k1 = f2pack(p.cap_k[1], p.cap_k[1]),
                                   k2 = f2pack(p.cap_k[2], p.cap_k[2]), k3 = f2pack(p.cap_k[3], p.cap_k[3]);
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            const uint64_t d = f2pack(__uint_as_float(v[cc][x]), __uint_as_float(v[cc][x + 1])), z = f2mul(d, d);
                            float y0, y1;
                            f2unpack(f2mul(d, f2fma(f2fma(f2fma(k3, z, k2), z, k1), z, k0)), y0, y1);
                            v[cc][x] = __float_as_uint(y0);
                            v[cc][x + 1] = __float_as_uint(y1);
                        }
                } else if (p.wide) {
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            v[cc][x] = __float_as_uint(capped_wide(__uint_as_float(v[cc][x]), p.cap_in, p.cap_log2, p.scale_log2));
                } else {
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            v[cc][x] = __float_as_uint(capped(__uint_as_float(v[cc][x]), p.cap_in, p.cap_log2));
                }
            }
            if constexpr (kBias) {
                // -slope |d - x| for key x of the tile, d = position - tile start: linear on either side
                const int64_t d = away - j * kBN;
                const float c = kCap ? 1.f : p.scale_log2;
                if (__any_sync(0xffffffffu, d > 0 && d < kBN - 1)) {
                    const float df = (float)d;
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            v[cc][x] = __float_as_uint(fmaf(__uint_as_float(v[cc][x]), c, -slope * fabsf(df - (float)(32 * cc + x))));
                } else {
                    const float sg = d > 0 ? slope : -slope, b0 = -sg * (float)d;
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            v[cc][x] = __float_as_uint(fmaf(__uint_as_float(v[cc][x]), c, fmaf(sg, (float)(32 * cc + x), b0)));
                }
            }
            if (!whole) {
#pragma unroll
                for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (!((see[cc] >> x) & 1u)) v[cc][x] = __float_as_uint(-INFINITY);
            }
            // from here on scores count in log2 units with the factor c
            const float c = (kCap || kBias) ? 1.f : p.scale_log2;
            if constexpr (!kBounded) {
                // The first tile that a row sees something of sets its reference, its maximum there.  Later tiles take
                // the reference as it stands; where a tile's weights sum to more than 2^8, the next one raises it.
                // (Under a bias by distance scores grow by more from tile to tile than weights have room for: there every
                // tile's maximum is found, and the reference raised by it before the weights are.)
                float alpha = 1.f;
                bool raise = false;
                if (kBias || __any_sync(0xffffffffu, m_used == -INFINITY)) {
                    float mx[4];
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) {
                        mx[cc] = max3f(__uint_as_float(v[cc][0]), __uint_as_float(v[cc][1]), __uint_as_float(v[cc][2]));
#pragma unroll
                        for (int x = 3; x < 31; x += 2)
                            mx[cc] = max3f(mx[cc], __uint_as_float(v[cc][x]), __uint_as_float(v[cc][x + 1]));
                        mx[cc] = fmaxf(mx[cc], __uint_as_float(v[cc][31]));
                    }
                    const float mt = max3f(mx[0], mx[1], fmaxf(mx[2], mx[3])) * c;
                    if (m_used == -INFINITY) {
                        m_used = mt;
                        // (what a row that has seen no key has in O so far: zeros, or what masked rows of V made of them)
                    } else if (kBias && mt > m_used + 8.f) {
                        alpha = fast_exp2(m_used - mt);
                        m_used = mt;
                        raise = true;
                    }
                }
                if (!kBias && up > 0) {
                    alpha = __uint_as_float((uint32_t)(127 - up) << 23);
                    m_used += (float)up;
                    raise = true;
                }
                if (__any_sync(0xffffffffu, raise)) {
                    l_sum *= alpha;
                    // S(j) completed after the product before it: O is final up to there; 8 columns at a time
#pragma unroll 1
                    for (int q = 0; q < D / 8; ++q) {
                        uint32_t o[8];
                        tmem_ld8(lane_base + col_o(t) + q * 8, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                        tmem_st8(lane_base + col_o(t) + q * 8, o);
                    }
                    tmem_st_wait();
                }
            }
            // a row that has seen no key exponentiates against 0 (every score is -infinity)
            const float ms = m_used == -INFINITY ? 0.f : m_used;
            const uint64_t c2 = f2pack(c, c), nm2 = f2pack(-ms, -ms);
            uint64_t ls2[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                uint32_t pk[16];
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    float x0, x1;
                    const uint64_t two_s = f2pack(__uint_as_float(v[cc][x]), __uint_as_float(v[cc][x + 1]));
                    f2unpack(kBounded ? two_s : (kCap || kBias) ? f2add(two_s, nm2) : f2fma(two_s, c2, nm2), x0, x1);
                    const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                    ls2[(x >> 1) & 1] = f2add(ls2[(x >> 1) & 1], f2pack(p0, p1));
                    // the weights' one rounding: bf16, the type of V (the sum takes them unrounded)
                    __nv_bfloat162 two = __floats2bfloat162_rn(p0, p1);
                    pk[x >> 1] = *reinterpret_cast<uint32_t*>(&two);
                }
                tmem_st16(lane_base + col_s(t) + cc * 16, pk);
                if (cc == 1) {
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&ctl.p_half[t]);
                }
            }
            float l0, l1, l2, l3;
            f2unpack(ls2[0], l0, l1);
            f2unpack(ls2[1], l2, l3);
            const float sum = (l0 + l1) + (l2 + l3);
            l_sum += sum;
            if constexpr (!kBounded && !kBias) {
                // (sums of 2^127 and beyond: the reference was that far off; such a row is computed again)
                up = sum > 256.f ? min((int)(__float_as_uint(sum) >> 23) - 127, 126) : 0;
                lost = lost || sum == INFINITY;
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&ctl.p_full[t]);
        }
        if (ok && nt > 0) ok = __all_sync(0xffffffffu, wait_bar(&ctl.drain[t], 0, abort_flag, dev_status, budget) && !*abort_flag);
        // (without a key the rows wait for the Q tiles, whose place they are stored from)
        if (ok && nt == 0) ok = __all_sync(0xffffffffu, wait_bar(&ctl.q_full, 0, abort_flag, dev_status, budget));
        // The reference of a row that sees no key is -infinity; of one that sees some, be their scores all -infinity (then
        // its sum of 0 makes it 0 / 0), it is a number.
        m_used = saw ? fmaxf(m_used, -3.4e38f) : -INFINITY;
        // Split keys: chain B's maximum and sum go to chain A, which merges the two and stores the rows.
        float w_a = 1.f, w_b = 0.f;
        if (split) {
            if (t == 1) {
                ctl.split_m[r] = m_used;
                ctl.split_l[r] = lost ? -1.f : l_sum;
                if (!ok) ctl.split_ok = 0;
            }
            named_barrier_sync<1>(2 * kBM);
            if (t == 1) {
                ok = false;
            } else if (ok) {
                ok = ctl.split_ok && __all_sync(0xffffffffu, wait_bar(&ctl.drain[1], 0, abort_flag, dev_status, budget));
                const float mb = ctl.split_m[r], lb = ctl.split_l[r];
                const float m = fmaxf(m_used, mb) + kSpare;
                w_a = m_used == -INFINITY ? 0.f : fast_exp2(m_used - m);
                w_b = mb == -INFINITY ? 0.f : fast_exp2(mb - m);
                // (a sum that is NaN stays: its weight 0 times NaN)
                l_sum = l_sum * w_a + lb * w_b;
                lost = lost || lb == -1.f;
                m_used = m;
            }
        }
        if constexpr (kParts) {
            // A part of the keys: the sums of weighted V as they are, the reference and the sum of weights (kAgain: the row has to
            // be computed again) into shared memory, where K and V were once every MMA is done.
            if (ok && n_kv > 0 && n_ch == 2) ok = __all_sync(0xffffffffu, wait_bar(&ctl.drain[1 - t], 0, abort_flag, dev_status, budget));
            if (!split || t == 0) {
                bool bad = lost;
                if (ok && n_kv > 0) {
                    tc_fence_after();
                    float chk = 0.f;
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        tmem_ld32(lane_base + col_o(t) + cc * 32, o);
                        tmem_ld_wait();
                        if (split) {
                            uint32_t ob[32];
                            tmem_ld32(lane_base + col_o(1) + cc * 32, ob);
                            tmem_ld_wait();
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                o[x] = __float_as_uint(fmaf(__uint_as_float(o[x]), w_a, __uint_as_float(ob[x]) * w_b));
                        }
#pragma unroll
                        for (int x = 0; x < 32; ++x) chk = fmaf(__uint_as_float(o[x]), 0.f, chk);
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            st_shared_v4(part_o(t) + (uint32_t)((8 * cc + x) * kBM + r) * 16u, o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                    }
                    bad = bad || (chk != chk && l_sum == l_sum);
                }
                const bool sees = m_used != -INFINITY && mine;
                if (ok) {                              // (then no load is in flight either)
                    st_shared_f32(part_m(t) + 4u * r, sees ? m_used : -INFINITY);
                    st_shared_f32(part_l(t) + 4u * r, !sees ? 0.f : bad ? kAgain : l_sum);
                }
                if (lane == 0) ctl.missing[warp] = ok ? 0.f : 1.f;
            }
        } else {
        const bool writer = !split || t == 0;
        const uint32_t stage = sQ(t);
        bool fix = false;
        const bool boxed = !(p.q_start && q0 + (t + 1) * qpt > n_rows);   // else a box would reach the next request's rows
        const int64_t row_at = ((qbase + q0 + rt * qpt + r / p.g) * p.Hq + hk * p.g + r % p.g) * D;
        if (ok) {
            tc_fence_after();
            const float inv_l = 1.f / l_sum;
            const bool none = m_used == -INFINITY;         // no key: zeros, whatever the accumulator holds
            float chk = 0.f;                               // NaN once a column is not finite
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                tmem_ld32(lane_base + col_o(t) + cc * 32, o);
                tmem_ld_wait();
                if (split) {
                    uint32_t ob[32];
                    tmem_ld32(lane_base + col_o(1) + cc * 32, ob);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        o[x] = __float_as_uint(fmaf(__uint_as_float(o[x]), w_a, __uint_as_float(ob[x]) * w_b));
                }
                uint32_t pkd[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float y0 = none ? 0.f : __uint_as_float(o[2 * x]) * inv_l, y1 = none ? 0.f : __uint_as_float(o[2 * x + 1]) * inv_l;
                    chk = fmaf(y0, 0.f, fmaf(y1, 0.f, chk));
                    __nv_bfloat162 two = __floats2bfloat162_rn(y0, y1);
                    pkd[x] = *reinterpret_cast<uint32_t*>(&two);
                }
                // 16-byte chunk k of row r: region k / 8, swizzled position (k % 8) ^ (r % 8)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int k = 4 * cc + x;
                    st_shared_v4(stage + (uint32_t)(k >> 3) * kRegion + (uint32_t)r * 128u + ((uint32_t)((k & 7) ^ (r & 7)) << 4),
                                 pkd[4 * x], pkd[4 * x + 1], pkd[4 * x + 2], pkd[4 * x + 3]);
                }
            }
            fix = mine && (lost || (chk != chk && l_sum == l_sum));
        }
        if (writer) {
            fence_proxy_async_smem();
            // the rows leave as a box when all of them are right; every thread of the warpgroup arrives
            const bool clean = t == 0 ? named_barrier_and<2>(kBM, ok && boxed && !fix) : named_barrier_and<3>(kBM, ok && boxed && !fix);
            if (clean) {
                if (r == 0) {
#pragma unroll
                    for (int x = 0; x < kHalves; ++x) {
                        if (p.q_start) tma_store_3d(&p.tm_o, stage + x * kRegion, 64 * x, hk * p.g, (int)qbase + q0 + t * qpt);
                        else tma_store_4d(&p.tm_o, stage + x * kRegion, 64 * x, hk * p.g, q0 + t * qpt, b);
                    }
                    bulk_commit_group();
                    bulk_wait_group_read0();
                }
            } else if (ok) {                               // (uniform over the warp)
                if (mine && !fix) {
#pragma unroll
                    for (int k = 0; k < D / 8; ++k) {
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                     : "r"(stage + (uint32_t)(k >> 3) * kRegion + (uint32_t)r * 128u + ((uint32_t)((k & 7) ^ (r & 7)) << 4))
                                     : "memory");
                        reinterpret_cast<uint4*>(p.out + row_at)[k] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                for (uint32_t todo = __ballot_sync(0xffffffffu, fix); todo; todo &= todo - 1) {
                    const int l0 = __ffs(todo) - 1;
                    const int64_t at = __shfl_sync(0xffffffffu, row_at, l0);
                    masked_row<bf16, D>(MaskedPool<bf16>{p.k_cache, p.v_cache, rs, p.num_slots, p.Hkv, p.drop, p.wide != 0, p.scale_log2, kCap ? p.cap_in : 0.f,
                                                         p.cap_log2, 0.f},
                                  p.q + at, p.out + at, __shfl_sync(0xffffffffu, a_lo, l0), __shfl_sync(0xffffffffu, a_hi, l0), hk,
                                  __shfl_sync(0xffffffffu, slope, l0), __shfl_sync(0xffffffffu, away, l0), lane);
                }
            }
        }
        }
        }
        if constexpr (kParts) {
            // ---- the rows from their parts: each CTA of the cluster merges D / cs columns of all of them
            cluster_sync();
            if (wg < n_qt) {
                const int t = wg, r = threadIdx.x & 127;
                int lo, hi;
                const bool mine = row_keys(t, r, lo, hi);
                float w[kMaxParts], m = -INFINITY, l = 0.f;
                bool again = false, missing = false;
#pragma unroll
                for (int c = 0; c < kMaxParts; ++c) {
                    w[c] = c < p.cs ? ld_cluster_f32(mapa_shared(part_m(t) + 4u * r, (uint32_t)c)) : -INFINITY;
                    m = fmaxf(m, w[c]);
                }
                m += kSpare;
#pragma unroll
                for (int c = 0; c < kMaxParts; ++c) {
                    const float lc = c < p.cs ? ld_cluster_f32(mapa_shared(part_l(t) + 4u * r, (uint32_t)c)) : 0.f;
                    // (a part in which the row sees no key, and a part that is none: no weight, and its sums are not looked at)
                    w[c] = w[c] == -INFINITY ? 0.f : fast_exp2(w[c] - m);
                    again = again || lc == kAgain;
                    // (a wait gave up: the row stays unwritten)
                    missing = missing || (c < p.cs && ld_cluster_f32(mapa_shared(smem_u32(&ctl.missing[warp]), (uint32_t)c)) != 0.f);
                    l = fmaf(w[c], lc, l);
                }
                const bool none = m == -INFINITY;
                const float inv_l = 1.f / l;
                const int per = D / p.cs;
                const int64_t row_at = ((qbase + q0 + t * qpt + r / p.g) * p.Hq + hk * p.g + r % p.g) * D;
                for (int x = rank * per; x < (rank + 1) * per; x += 8) {
                    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < kMaxParts; ++c) {
                        if (c >= p.cs) continue;
                        const uint32_t from = mapa_shared(part_o(t) + (uint32_t)((x >> 2) * kBM + r) * 16u, (uint32_t)c);
                        const float4 u = ld_cluster_v4(from), v = ld_cluster_v4(from + kBM * 16u);
                        if (w[c] > 0.f) {
                            y[0] = fmaf(w[c], u.x, y[0]), y[1] = fmaf(w[c], u.y, y[1]), y[2] = fmaf(w[c], u.z, y[2]), y[3] = fmaf(w[c], u.w, y[3]);
                            y[4] = fmaf(w[c], v.x, y[4]), y[5] = fmaf(w[c], v.y, y[5]), y[6] = fmaf(w[c], v.z, y[6]), y[7] = fmaf(w[c], v.w, y[7]);
                        }
                    }
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        __nv_bfloat162 two = __floats2bfloat162_rn(none ? 0.f : y[2 * e] * inv_l, none ? 0.f : y[2 * e + 1] * inv_l);
                        o[e] = *reinterpret_cast<uint32_t*>(&two);
                    }
                    if (mine && !again && !missing) *reinterpret_cast<uint4*>(p.out + row_at + x) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                if (rank == 0) {
                    float slope = 0.f;
                    int64_t pos = 0;
                    if (kBias && mine) {
                        slope = p.slopes[hk * p.g + r % p.g] * kLog2e;
                        pos = p.q_pos[qbase + q0 + t * qpt + r / p.g];
                    }
                    __syncwarp();
                    for (uint32_t todo = __ballot_sync(0xffffffffu, mine && again && !missing); todo; todo &= todo - 1) {
                        const int l0 = __ffs(todo) - 1;
                        const int64_t at = __shfl_sync(0xffffffffu, row_at, l0);
                        masked_row<bf16, D>(MaskedPool<bf16>{p.k_cache, p.v_cache, p.read_slot + kbase, p.num_slots, p.Hkv, p.drop, p.wide != 0,
                                                             p.scale_log2, kCap ? p.cap_in : 0.f, p.cap_log2, 0.f},
                                      p.q + at, p.out + at, __shfl_sync(0xffffffffu, lo, l0), __shfl_sync(0xffffffffu, hi, l0), hk,
                                      __shfl_sync(0xffffffffu, slope, l0), __shfl_sync(0xffffffffu, pos, l0), lane);
                    }
                }
            }
            cluster_sync();                            // no CTA leaves while another reads its shared memory
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag) {
        if (threadIdx.x == 0 && !mbar_wait(&ctl.q_full, 0, kLandBudget)) ctl.unlanded = 1;
        __syncthreads();
        settle_after_abort(ctl.unlanded != 0);
    }
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool kCap, bool kBounded, bool kBias, bool kParts>
int launch(const MaskParams& prm, dim3 grid, cudaStream_t stream) {
    auto kern = masked_tc_kernel<D, kCap, kBounded, kBias, kParts>;
    static std::atomic<int> prepared[64];             // per device: the launch is allowed for
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    if (!prepared[dev].load(std::memory_order_acquire)) {
        cudaFuncAttributes fa;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(D)) != cudaSuccess ||
            cudaFuncGetAttributes(&fa, kern) != cudaSuccess) {
            (void)cudaGetLastError();
            return ACACHE_ERR_CUDA;
        }
        if (fa.numRegs < kRegLaunch) return ACACHE_ERR_UNSUPPORTED;   // the register split assumes the launch allocation
        prepared[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(D);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)prm.cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kParts ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, prm) != cudaSuccess) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    return launch_status();
}

// Clusters of `cs` CTAs that the current device holds at once (0: unknown); every form of the kernel takes an SM to a CTA.
int clusters_at_once(int cs) {
    static std::atomic<int> known[64][kMaxParts + 1];  // 1 + the number
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return 0;
    }
    int n = known[dev][cs].load(std::memory_order_relaxed);
    if (n == 0) {
        auto kern = masked_tc_kernel<128, false, false, false, true>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)cs);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem_bytes(128);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)cs;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(128)) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        known[dev][cs].store(++n, std::memory_order_relaxed);
    }
    return n - 1;
}

template <int D, bool kParts>
int dispatch(const MaskParams& prm, bool cap, bool bounded, bool bias, dim3 grid, cudaStream_t stream) {
    if (cap && bias) return launch<D, true, false, true, kParts>(prm, grid, stream);
    if (cap) return bounded ? launch<D, true, true, false, kParts>(prm, grid, stream) : launch<D, true, false, false, kParts>(prm, grid, stream);
    return bias ? launch<D, false, false, true, kParts>(prm, grid, stream) : launch<D, false, false, false, kParts>(prm, grid, stream);
}

}  // namespace

bool masked_tc_supported(const MaskedAttn& c) {
    return c.a.dtype == ACACHE_BF16 && c.a.scale > 0.f && c.a.hq / c.a.hkv <= kBM && c.num_slots > 0;
}

int launch_masked_tc(const MaskedAttn& c) {
    const int d = c.a.d, g = c.a.hq / c.a.hkv;
    MaskParams prm{};
    prm.qpt = kBM / g;
    const int64_t n_qb = (c.n_q + 2LL * prm.qpt - 1) / (2LL * prm.qpt);
    if (n_qb > 65535) return ACACHE_ERR_INVALID_ARG;
    const uint64_t dq4[4] = {(uint64_t)d, (uint64_t)c.a.hq, (uint64_t)c.n_q, (uint64_t)c.B};
    const uint64_t dq3[3] = {(uint64_t)d, (uint64_t)c.a.hq, (uint64_t)c.total_q};
    const uint32_t bq[4] = {64u, (uint32_t)g, (uint32_t)prm.qpt, 1u};
    const uint64_t d2[2] = {(uint64_t)d, (uint64_t)c.num_slots * c.a.hkv};
    const uint64_t d3[3] = {(uint64_t)d, (uint64_t)c.a.hkv, (uint64_t)c.num_slots};
    const uint64_t* dq = c.q_start ? dq3 : dq4;
    const int rank = c.q_start ? 3 : 4;
    if (!make_map_box(&prm.tm_q, c.q, rank, dq, bq) || !make_map_box(&prm.tm_o, c.out, rank, dq, bq) ||
        !make_map(&prm.tm_kg, c.k_cache, 2, d2, 1, 1) || !make_map(&prm.tm_vg, c.v_cache, 2, d2, 1, 1) ||
        !make_map(&prm.tm_kb, c.k_cache, 3, d3, 2, kBN) || !make_map(&prm.tm_vb, c.v_cache, 3, d3, 2, kBN))
        return ACACHE_ERR_CUDA;
    prm.q = (const bf16*)c.q;
    prm.k_cache = (const bf16*)c.k_cache;
    prm.v_cache = (const bf16*)c.v_cache;
    prm.out = (bf16*)c.out;
    prm.read_slot = c.read_slot;
    prm.q_start = c.q_start;
    prm.kv_start = c.kv_start;
    prm.row_range = c.mask.row_range;
    prm.q_pos = c.mask.q_pos;
    prm.slopes = c.mask.slopes;
    prm.dev_status = c.dev_status;
    prm.num_slots = c.num_slots;
    prm.n_rows = c.n_q;
    prm.total_q = c.total_q;
    prm.T_len = c.T_len;
    prm.Hq = c.a.hq;
    prm.Hkv = c.a.hkv;
    prm.g = g;
    prm.drop = c.mask.drop_none != 0;
    prm.scale_log2 = c.a.scale * kLog2e;
    const bool cap = c.mask.softcap > 0.f;
    if (cap) {
        prm.cap_in = 2.f * kLog2e * (c.a.scale / c.mask.softcap);
        prm.cap_log2 = c.mask.softcap * kLog2e;
        prm.wide = c.mask.softcap > kWideCap;
        const double y = (double)c.a.scale / c.mask.softcap;         // of q.k = 1
        double k = prm.scale_log2;
        prm.cap_near = (float)std::min(0.5 / y, 1e18);
        for (int i = 0; i < 4; ++i, k *= y * y) {
            prm.cap_k[i] = (float)(k * kTanhHalf[i]);
            if (!(k > 1e-36 && k < 1e36)) prm.cap_near = -1.f;   // a cap far from the scale: not this way
        }
    }
    prm.budget = wait_budget();
    // Blocks that leave SMs idle are split over clusters, as many as run at once, with more than two and a half tiles of keys to
    // a CTA.  us, 28 heads over 4, 32 rows, causal over 3,260 keys: 3 requests 58 whole, 29 in 8 parts; 16 requests 60, 48
    // in 2.  33 rows of 8 heads over 1, 8,000 keys: 115, 33 in 8.  A merge takes some 5 us: 64 rows over 1,408 keys 31, 29 in 2,
    // 23 in 4; 200 rows over 600 keys 21, 23 in 2.
    const int64_t blocks = n_qb * c.B * c.a.hkv, tiles = (c.T_len + kBN - 1) / kBN;
    prm.cs = 1;
    for (int cs = 2; cs <= kMaxParts && 5LL * cs < 2 * tiles && cs * blocks <= sm_count(); cs *= 2)
        if (blocks <= clusters_at_once(cs)) prm.cs = cs;
    const dim3 grid((unsigned)(c.a.hkv * prm.cs), (unsigned)c.B, (unsigned)n_qb);
    const bool bias = c.mask.slopes != nullptr;
    const bool bounded = cap && !bias && c.mask.softcap <= kBoundedCap;
    if (prm.cs > 1)
        return d == 64 ? dispatch<64, true>(prm, cap, bounded, bias, grid, c.stream) : dispatch<128, true>(prm, cap, bounded, bias, grid, c.stream);
    return d == 64 ? dispatch<64, false>(prm, cap, bounded, bias, grid, c.stream) : dispatch<128, false>(prm, cap, bounded, bias, grid, c.stream);
}

}  // namespace acache
