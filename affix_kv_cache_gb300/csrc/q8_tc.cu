// q8_tc.cu -- read-slot attention over an 8-bit pool on the tensor cores (tcgen05 + TMEM): bf16
// queries and outputs, head dim 64 or 128.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4.3 and App. C.1 (attention that
// reads every logical key through the per-request read-slot map); the 8-bit pool is this
// library's.
//
// Mathematics.  out = softmax(scale q . k) v with k = 2^ek kc, v = 2^ev vc, codes kc and vc in e4m3.
//   * S: the keys' codes are an operand as they lie in the pool.  A bf16 query row has 8
//     significant bits, twice e4m3's 4: scaled by a power of two so that its largest element lies in
//     [128, 256), q' = hi + lo with hi = q' cut to 4 bits and lo = e4m3(q' - hi) is exact for elements
//     within 2^-9 of the largest and off by some 2^-17 of the largest below.  S = hi kc + lo kc: two
//     8-bit MMA passes at twice the bf16 rate, so no key is ever converted and the K ring takes
//     half the shared memory.  2^ek multiplies S per key (float32), the row's power of two joins the
//     softmax scale.
//   * O: bf16 P (as in the 16-bit kernels) times V in bf16: 2^(ev - 32) vc has 4 significant bits, so
//     the conversion is exact; the factor 2^32 goes into the final 1/l.
//
// Work.  Rows are (query, query head of the KV head's group) pairs, packed, so a group shares one
// pass over the keys; a CTA takes up to 256 of them (two 128-row tiles A and B) and the keys of one
// (request, KV head).  512 threads, one CTA per SM:
//   WG0, WG1  softmax + epilogue of chain A / B, thread r owns row r (= TMEM lane r): first it turns
//             its query row into hi and lo; then per key tile it reads S from TMEM, multiplies by the
//             keys' factors, exponentiates in base 2 against a lazily raised maximum and writes P
//             over S, 64 keys a step.  A chain has two S buffers of 64 keys: the MMA of the next step
//             runs under the softmax of this one.
//   WG2       warps 8 and 9 issue the MMAs of chain A / B; warps 10 and 11 fill the K ring by TMA (a
//             tile of consecutive slots as one box, any other as 32 gather4 loads) and the ring of the
//             keys' factors.
//   WG3       V: each thread reads 16-byte pieces of pool rows into registers two tiles ahead,
//             converts them to bf16 and writes the V ring.  Through registers instead of a raw ring:
//             the converted tile is the only copy in shared memory.
//   A CTA with one row tile (few rows: decoding) splits its keys between the chains and merges
//   them at the end.  When there are few blocks the key range is also split over a cluster of cs
//   CTAs, whose partial (maximum, sum, O) are merged through distributed shared memory, in rank order.
//
// What bounds it.  16 requests x 986 rows x 2,624 keys, 28 heads over 4, d = 128: 555 us, 1,070 TFLOP/s, 0.55 of the
// measured bf16 rate.  A step of 64 keys takes both chains some 1,800 cycles; their MMAs alone take 1,280
// (2 x 385 for S, whose 64-key MMAs read 6 KB of shared memory, 48 cycles, for 32 cycles of products, and
// 2 x 257 for PV).  No pipe is full (ALU 0.38, FMA 0.27, MUFU 0.21); what comes nearest is shared memory: the
// MMAs' operands, the keys' factors (every softmax warp reads all of them), V's tiles and K's take some
// 1,700 of the 1,800 cycles by count, so two softmax warps per scheduler cannot cover their waits, and
// whatever a softmax warp waits for on its own account shows -- a barrier for the keys' factors cost 7 %,
// per-lane arrivals 1 %.  A block costs some 15,000 cycles besides its steps (launch and set-up 4,000, the
// query terms 6,000, first S 2,000, drain and epilogue 4,000).  Slower were: S of 128 keys at a time, which needs
// only 512 cycles, into one buffer (683 us where this form takes 555); the chains taking turns (+2 to 5 %);
// four softmax warpgroups (+13 %); V's codes through a raw ring in shared memory; the keys' factors read before
// S is waited for (+20 %); waits that poll instead of suspending (+2 to 7 %).  As fast: one S buffer, issued again as
// soon as it is read, with two of P beside it, and the factors in bf16 (559 us).
//
// Every mbarrier wait is bounded; a wait that gives up raises a CTA-wide abort flag and
// ACACHE_DEV_TIMEOUT, roles leave their loops, MMAs in flight are drained, TMA loads issued before
// it are waited for (bounded), TMEM is freed, the cluster barriers are reached on every path, and
// no output row is written that its steps have not all reached.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "q8_tc.cuh"

namespace acache {
namespace {

using namespace q8;

constexpr int kBM = 128;                    // rows per tile (TMEM lanes)
constexpr int kQT = 2;                      // row tiles per CTA
constexpr int kBN = 128;                    // keys per tile (ring entry)
constexpr int kStep = 64;                   // keys per step (half a tile): one S buffer of a chain
constexpr int kMmaWarp = 8;
constexpr int kProdWarp = 10, kProd = 2;    // K producer warps
constexpr int kConvWarp = 12, kConv = 4;    // V converter warps
constexpr int kThreads = 512;
// Registers per thread of the warpgroups, 512 x 128 in all.  The producers of a call with discarded keys carry
// their masks: with 56 they spill, and a long ragged batch takes 76 us instead of 72.
constexpr int kRegSoftmax = 168;
template <bool kDrop>
constexpr int kRegIssue = kDrop ? 64 : 56;
template <bool kDrop>
constexpr int kRegConv = kDrop ? 112 : 120;
constexpr int kRegSum = 2 * kRegSoftmax + kRegIssue<true> + kRegConv<true>;
static_assert(kRegSum == 2 * kRegSoftmax + kRegIssue<false> + kRegConv<false> && 128 * kRegSum <= kThreads * 128, "register split");
constexpr uint32_t kTmemCols = 512;         // two S buffers of 64 columns per chain, O_A, O_B
__host__ __device__ constexpr uint32_t col_s(int t) { return (uint32_t)t * 128u; }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + (uint32_t)t * 128u; }
// log2 units a row's maximum may grow before O and the sum are rescaled.  bf16 and float32 have the
// same exponents, so P up to 2^40 costs no precision, and the sums stay far inside float32.
constexpr float kRescaleThreshold = 40.0f;
constexpr int kVShift = 32;                 // V is carried times 2^-32
constexpr int kFSt = 8;                     // ring of the keys' factors (see the K producers)
constexpr int kMaxCluster = 8;

template <int D>
struct Geo {
    static constexpr uint32_t kQPart = kBM * D;            // one term of a query tile
    static constexpr uint32_t kKTile = kBN * D;            // e4m3
    static constexpr uint32_t kVTile = kBN * D * 2;        // bf16
    static constexpr uint32_t kRegion = kBN * 128;         // 64 bf16 columns of a V tile
    static constexpr int kKSt = D == 128 ? 3 : 4, kVSt = D == 128 ? 3 : 4;
    static constexpr uint32_t kRing = 2 * kQT * kQPart;    // offset of the K ring
    static constexpr uint32_t kBytes = kRing + kKSt * kKTile + kVSt * kVTile + 1024;
    static_assert(kKSt * kKTile + kVSt * kVTile >= kQT * kBM * D * 4u, "partial O reuses the rings");
};

struct Q8Params {
    CUtensorMap tm_k;      // 2-D pool rows [num_slots*Hkv][d], box {d, 1} (gather4)
    CUtensorMap tm_kbox;   // 3-D pool [num_slots][Hkv][d], box {d, 1, 128} (consecutive slots)
    const bf16* q;
    const uint8_t* v_cache;
    const uint8_t* kv_scale;
    const int32_t *read_slot, *q_start, *kv_start;
    bf16* out;
    int32_t* dev_status;
    int64_t num_slots;
    int oob_row;           // a pool row outside the tensor (reads zeros)
    int n_q, total_q, T_len, Hq, Hkv, g;
    int cs, part;          // CTAs per cluster; key tiles per part
    float scale_log2;
    long long budget;      // cycles a pipeline wait may take before it gives up
};

template <int D>
struct Ctl {
    uint64_t q_full;
    uint64_t k_full[Geo<D>::kKSt], k_empty[Geo<D>::kKSt];
    uint64_t v_full[Geo<D>::kVSt], v_empty[Geo<D>::kVSt];
    uint64_t s_full[kQT][2], p_full[kQT][2];   // by step parity
    uint64_t pv_done[kQT];             // phase u: PV of step u is complete
    uint64_t drain[kQT];
    uint32_t tmem_base;
    int abort, unlanded;
    uint32_t drop[kFSt][4];            // discarded keys, 32 per word
    float part_m[kQT * kBM], part_l[kQT * kBM];
    float failed;                      // this CTA gave up (read by the other ranks)
    __align__(16) float factor[kFSt][kBN];
};

// Chain t's i-th key tile comes through ring entry entry(t, i).  One row tile: chain 0 reads
// tiles [0, n0), chain 1 the rest, entries alternating.
struct Schedule {
    bool split;
    int n_kv, n0;
    ACACHE_DEVFN int n_tiles(int t) const { return split ? (t == 0 ? n0 : n_kv - n0) : n_kv; }
    // steps (half tiles) of chain t; `last` = keys of the part's last tile: 64 or fewer leave its
    // second half out
    ACACHE_DEVFN int n_steps(int t, int last) const {
        return 2 * n_tiles(t) - (last <= kStep && (!split || t == 1) ? 1 : 0);
    }
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

// Four e4m3 codes -> bf16 pairs times f2.  A code's exponent and significand bits moved into a
// bf16's lowest exponent bits make code * 2^-120 (subnormal codes included: bf16 subnormals); f2
// holds 2^(120 + ev - 32) twice.
ACACHE_DEVFN void codes_to_bf16(uint32_t w, uint32_t f2, uint32_t& lo, uint32_t& hi) {
    const uint32_t x = __byte_perm(w, 0u, 0x1404), y = __byte_perm(w, 0u, 0x3424);
    const uint32_t a = ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
    const uint32_t b = ((y >> 4) & 0x07f007f0u) | (y & 0x80008000u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(f2));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(f2));
}

template <int D, bool kDrop>
__global__ void __launch_bounds__(kThreads, 1)
q8_attn_kernel(const __grid_constant__ Q8Params p) {
    using G = Geo<D>;
    extern __shared__ uint8_t dsm[];
    __shared__ Ctl<D> ctl;
    const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
    uint8_t* base_ptr = dsm + (base - smem_u32(dsm));
    auto sQ = [&](int t) { return base + 2u * G::kQPart * (uint32_t)t; };          // hi, then lo
    auto sK = [&](int s) { return base + G::kRing + G::kKTile * (uint32_t)s; };
    auto sV = [&](int s) { return base + G::kRing + G::kKTile * G::kKSt + G::kVTile * (uint32_t)s; };
    const int cr = p.cs == 1 ? 0 : (int)(blockIdx.x % (unsigned)p.cs);
    const int hk = p.cs == 1 ? (int)blockIdx.x : (int)(blockIdx.x / (unsigned)p.cs);
    const int b = (int)blockIdx.y;
    int n_q = p.n_q, T_len = p.T_len;
    int64_t qbase = (int64_t)b * p.n_q, kbase = (int64_t)b * p.T_len;
    if (p.q_start) {
        qbase = p.q_start[b];
        kbase = p.kv_start[b];
        n_q = q8_count(p.q_start, b);
        T_len = q8_count(p.kv_start, b);
        if (n_q != 0 && q8_bad_lengths(n_q, p.n_q, T_len, p.T_len, qbase, p.total_q, kbase)) {
            if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.z == 0) flag(p.dev_status, ACACHE_DEV_BAD_LENGTH);
            return;
        }
    }
    const int64_t row0 = (int64_t)blockIdx.z * (kQT * kBM), all_rows = (int64_t)n_q * p.g;
    if (row0 >= all_rows) return;
    const int n_rows = (int)min((int64_t)(kQT * kBM), all_rows - row0);
    const int n_qt = n_rows > kBM ? 2 : 1;
    const int n_all = (T_len + kBN - 1) / kBN;
    const int cs = (n_all + p.part - 1) / p.part;              // parts of this request's keys (<= p.cs)
    if (cr >= cs) return;
    const int kt0 = (int)((int64_t)cr * n_all / cs);
    const int n_kv = (int)((int64_t)(cr + 1) * n_all / cs) - kt0;      // >= 1
    const bool split = n_qt == 1 && n_kv >= 2;
    const int n_ch = split ? 2 : n_qt;
    const Schedule sch{split, n_kv, split ? (n_kv + 1) / 2 : n_kv};
    const int last_keys = min(kBN, T_len - (kt0 + n_kv - 1) * kBN);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
    volatile int* abort_flag = &ctl.abort;
    int32_t* dev_status = p.dev_status;
    const long long budget = p.budget;

    // Softmax warps: chain t, row r of its tile (= TMEM lane), the row of the block it works on, and that
    // row's element offset in q and out.  The query rows are on their way during the set-up.  (Rows past
    // the block read the block's first row; warps past it leave theirs unwritten: what they hold
    // only reaches output rows that are never read.)
    const int t = wg, r = threadIdx.x & 127;
    const int row_of = split ? r : t * kBM + r;
    const bool live = t < n_ch && row_of < n_rows;
    const bool warp_live = __any_sync(0xffffffffu, live);
    const uint32_t q_at = sQ(t & 1) + (uint32_t)((warp & 3) * 32 * D);
    int64_t off = 0;
    if (wg < 2) {
        const uint32_t pr = (uint32_t)row0 + (row_of < n_rows ? row_of : 0), i = pr / (uint32_t)p.g;   // (below 2^24)
        off = ((qbase + i) * p.Hq + (int64_t)hk * p.g + (pr - i * (uint32_t)p.g)) * D;
        if (warp_live) query_load<D>(p.q, off, q_at, q_at + G::kQPart, lane);
    }
    if (threadIdx.x == 32 * (kMmaWarp + 1)) {
        const int readers = split ? 1 : n_qt;
        mbar_init(&ctl.q_full, 4u * n_qt);
        for (int s = 0; s < G::kKSt; ++s) {
            mbar_init(&ctl.k_full[s], 1 + kProd);       // the bytes, and each producer's factors
            mbar_init(&ctl.k_empty[s], readers);
        }
        for (int s = 0; s < G::kVSt; ++s) {
            mbar_init(&ctl.v_full[s], kConv);
            mbar_init(&ctl.v_empty[s], readers);
        }
        for (int t = 0; t < kQT; ++t) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(&ctl.s_full[t][h], 1);
                mbar_init(&ctl.p_full[t][h], 4);
            }
            mbar_init(&ctl.pv_done[t], 1);
            mbar_init(&ctl.drain[t], 1);
        }
        ctl.abort = 0;
        ctl.unlanded = 0;
        ctl.failed = 0.f;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;

    if (wg == 3) {
        setmaxnreg_dec<kRegConv<kDrop>>();
        // ------------------------------------------------------------------ V converters
        constexpr int CPR = D / 16;                  // 16-byte pieces per pool row
        constexpr int RPI = 32 / CPR;                // rows per warp load
        constexpr int NI = 32 / RPI;                 // loads per tile and lane
        const int w = warp - kConvWarp;
        // Lane -> piece c of row rr of a load.  The eight lanes of a shared-memory phase hold four
        // pieces of one 64-column region in two neighbouring rows: their swizzled chunks differ.
        const int c = (lane & 3) | (D == 128 ? (lane >> 4) << 2 : 0), rr = (lane >> 2) & (RPI - 1);
        // Loads are issued a tile or two before their values are looked at: nothing is computed from
        // a value in the step that loads it.
        auto slot_of = [&](int e) -> int {           // slot of this lane's key (32 w + lane) of entry e
            int s = -1;
            if (e < n_kv) {
                const int t = (kt0 + sch.entry_tile(e)) * kBN + 32 * w + lane;
                if (t < T_len) s = p.read_slot[kbase + t];
            }
            return s;
        };
        uint4 dat[2][NI];
        uint32_t sc[2];                              // V's scale byte of this lane's key; 256: no row
        // All shuffles before all loads: between two loads, a shuffle would wait for the first one.
        // A key without a row reads the pool's first row, with factor 0.
        const uint8_t* v_lane = p.v_cache + (int64_t)hk * D + c * 16;
        auto issue = [&](int slot, uint4 (&d)[NI], uint32_t& f) {
            const bool in = slot >= 0 && slot < p.num_slots;
            const int sl = in ? slot : 0;
            int s[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) s[i] = __shfl_sync(0xffffffffu, sl, i * RPI + rr);
            f = 256u;
            if (in) f = p.kv_scale[((int64_t)sl * p.Hkv + hk) * 2 + 1];
#pragma unroll
            for (int i = 0; i < NI; ++i)
                asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(d[i].x), "=r"(d[i].y), "=r"(d[i].z), "=r"(d[i].w)
                             : "l"(v_lane + (int64_t)s[i] * ((int64_t)p.Hkv * D)));
        };
        auto convert = [&](uint32_t dst, const uint4 (&d)[NI], uint32_t f) {
            // 2^(120 + ev - 32) as bf16, twice; a byte above the largest is NaN
            uint32_t g2 = f > 255u ? 0u : f > kQ8MaxByte ? 0x7fffu : (f + 120u - kVShift) << 7;
            g2 |= g2 << 16;
            const uint32_t at = dst + (uint32_t)(32 * w + rr) * 128u + ((uint32_t)c >> 2) * G::kRegion;
            uint32_t f2[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) f2[i] = __shfl_sync(0xffffffffu, g2, i * RPI + rr);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                uint32_t o[8];
                codes_to_bf16(d[i].x, f2[i], o[0], o[1]);
                codes_to_bf16(d[i].y, f2[i], o[2], o[3]);
                codes_to_bf16(d[i].z, f2[i], o[4], o[5]);
                codes_to_bf16(d[i].w, f2[i], o[6], o[7]);
                // chunks 2c and 2c + 1 (of the region) of the row
                const uint32_t a0 = at + i * RPI * 128u + (((2u * c & 7u) ^ ((uint32_t)(i * RPI + rr) & 7u)) << 4);
                st_shared_v4(a0, o[0], o[1], o[2], o[3]);
                st_shared_v4(a0 ^ 16u, o[4], o[5], o[6], o[7]);
            }
        };
        const int s0 = slot_of(0), s1 = slot_of(1);
        int s_next = slot_of(2);
        grid_dependency_wait();                      // store-then-attend: the pool is written now
        issue(s0, dat[0], sc[0]);
        issue(s1, dat[1], sc[1]);
        bool ok = true;
        for (int e0 = 0; ok && e0 < n_kv; e0 += 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int e = e0 + u;
                if (!ok || e >= n_kv) break;
                const int s = e % G::kVSt;
                if (e >= G::kVSt)
                    ok = __all_sync(0xffffffffu, wait_bar<true>(&ctl.v_empty[s], ((e / G::kVSt) - 1) & 1, abort_flag,
                                                          dev_status, budget));
                if (!ok) break;
                convert(sV(s), dat[u], sc[u]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.v_full[s]);
                if (e + 2 < n_kv) issue(s_next, dat[u], sc[u]);
                s_next = slot_of(e + 3);
            }
        }
        __syncwarp();
        if (cs > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else if (wg == 2) {
        setmaxnreg_dec<kRegIssue<kDrop>>();
        if (warp >= kProdWarp) {
            // -------------------------------------------------------------- K producers
            const int pi = warp - kProdWarp;
            const bool leader = pi == 0 && lane == 0;
            if (leader) {
                tma_prefetch_desc(&p.tm_k);
                tma_prefetch_desc(&p.tm_kbox);
            }
            // Lane l reads the slots of keys 4l .. 4l+3; lanes below 16 gather keys 4x .. 4x+3 with
            // x = 16 pi + lane and look up their factors.  128 consecutive slots are one box load.
            // Slots are loaded two entries ahead and scales one.
            const int x = 16 * pi + (lane & 15);
            auto load_slots = [&](int e, int (&raw)[4]) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    raw[u] = -1;
                    if (e < n_kv) {
                        const int t = (kt0 + sch.entry_tile(e)) * kBN + 4 * lane + u;
                        if (t < T_len) raw[u] = p.read_slot[kbase + t];
                    }
                }
            };
            auto resolve = [&](int e, const int (&raw)[4], int (&rows)[4], int& slot0, uint32_t& gone) -> bool {
                int sl[4];
                const int left = T_len - (kt0 + sch.entry_tile(e)) * kBN - 4 * lane;   // keys from the lane's first on
                gone = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool in = raw[u] >= 0 && raw[u] < p.num_slots;
                    sl[u] = in ? raw[u] : -1;
                    if (kDrop && raw[u] == ACACHE_SLOT_NONE) gone |= 1u << u;
                    else if (!in && u < left && pi == 0) flag(dev_status, ACACHE_DEV_BAD_SLOT);
                }
                bool run = sl[0] >= 0 && sl[1] == sl[0] + 1 && sl[2] == sl[0] + 2 && sl[3] == sl[0] + 3;
                const int after = __shfl_down_sync(0xffffffffu, sl[0], 1);
                if (lane < 31) run = run && after == sl[0] + 4;
                slot0 = __shfl_sync(0xffffffffu, sl[0], 0);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int s = __shfl_sync(0xffffffffu, sl[u], x);
                    rows[u] = s >= 0 ? s * p.Hkv + hk : p.oob_row;
                }
                if constexpr (kDrop) {                 // eight lanes' keys make a word
                    gone <<= 4 * (lane & 7);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) gone |= __shfl_xor_sync(0xffffffffu, gone, o);
                }
                return __all_sync(0xffffffffu, run);
            };
            auto load_scales = [&](const int (&rows)[4], uint32_t (&sc)[4]) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    sc[u] = 127u;                      // a zero row: any finite factor
                    if (rows[u] != p.oob_row) sc[u] = p.kv_scale[(int64_t)rows[u] * 2];
                }
            };
            int raw[4], rows[4], slot0;
            uint32_t sc[4], gone;
            load_slots(0, raw);
            bool box = resolve(0, raw, rows, slot0, gone);
            load_slots(1, raw);
            grid_dependency_wait();
            load_scales(rows, sc);
            int armed = -1;
            for (int e = 0; e < n_kv; ++e) {
                const int s = e % G::kKSt, fs = e % kFSt;
                if (e >= G::kKSt && !__all_sync(0xffffffffu, wait_bar<true>(&ctl.k_empty[s], ((e / G::kKSt) - 1) & 1,
                                                                       abort_flag, dev_status, budget)))
                    break;
                if (leader) mbar_arrive_expect_tx(&ctl.k_full[s], G::kKTile);
                armed = e;
                __syncwarp();
                if (box) {
                    if (leader) tma_load_3d(sK(s), &p.tm_kbox, 0, hk, slot0, &ctl.k_full[s]);
                } else if (lane < 16) {
                    tma_gather4(sK(s) + (uint32_t)x * (4u * D), &p.tm_k, 0, rows[0], rows[1], rows[2], rows[3],
                                &ctl.k_full[s]);
                }
                // The factors' ring: a chain's S of a step is issued only after its softmax has written
                // the P two steps before; so once entry e - kKSt is free (the wait above), the
                // factors of that chain's entries before it have been read, and with split keys those
                // of the other chain's up to two entries earlier: kFSt > kKSt + 3 entries suffice.
                if (lane < 16)
                    *reinterpret_cast<float4*>(&ctl.factor[fs][4 * x]) =
                        make_float4(q8_factor(sc[0]), q8_factor(sc[1]), q8_factor(sc[2]), q8_factor(sc[3]));
                if (kDrop && pi == 0 && (lane & 7) == 0) ctl.drop[fs][lane >> 3] = gone;
                // Both warps arrive for every entry, so neither can get a phase ahead of the other.  The
                // softmax reads the factors on the strength of S: its MMAs are issued after this arrival
                // was seen, so their completion comes after these writes.  (With a barrier of the
                // factors' own, the wait for it cost 7 % of a long call.)
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.k_full[s]);
                if (e + 1 < n_kv) {
                    box = resolve(e + 1, raw, rows, slot0, gone);
                    load_scales(rows, sc);
                    load_slots(e + 2, raw);
                }
            }
            // Abort: the loads this warp issued land before the CTA exits (see tc_attn.cu)
            if (*abort_flag && armed >= 0) {
                bool landed = true;
                for (int e = max(0, armed - G::kKSt + 1); e <= armed; ++e)
                    landed = mbar_wait(&ctl.k_full[e % G::kKSt], (uint32_t)(e / G::kKSt) & 1u, kLandBudget) && landed;
                if (!__all_sync(0xffffffffu, landed) && lane == 0) ctl.unlanded = 1;
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------------ MMA issuers
            // The whole warp walks the steps, so addresses and descriptors stay in uniform registers, and
            // one lane issues.
            const int t = __shfl_sync(0xffffffffu, warp, 0) - kMmaWarp;         // chain
            if (t < n_ch) {
                const bool leader = elect_one();
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                constexpr uint32_t idS = idesc_e4m3(kBM, kStep);
                const uint32_t idO = idesc_bf16(kBM, D, false, true);
                const uint32_t d_s = tm + col_s(t), d_o = tm + col_o(t);
                const uint64_t dq = sdesc_rows<D>(sQ(split ? 0 : t));
                const int n_st = sch.n_steps(t, last_keys);
                auto wait = [&](uint64_t* bar, int phase) {
                    return __all_sync(0xffffffffu, wait_bar(bar, (uint32_t)phase & 1u, abort_flag, dev_status, budget));
                };
                // step u: half u & 1 of the chain's tile u / 2, into S buffer u & 1
                auto issue_s = [&](int u) -> bool {
                    const int e = sch.entry(t, u >> 1), h = u & 1;
                    if (h == 0 && !wait(&ctl.k_full[e % G::kKSt], e / G::kKSt)) return false;
                    tc_fence_after();
                    const uint64_t dk = sdesc_rows<D>(sK(e % G::kKSt) + (uint32_t)(h * kStep * D));
                    if (leader) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)                // hi, lo
#pragma unroll
                            for (int k = 0; k < D / 32; ++k)
                                umma_ss_f8(d_s + h * kStep, dq + (uint64_t)((x * G::kQPart + k * 32) >> 4),
                                           dk + (uint64_t)(k * 32 >> 4), idS, x > 0 || k > 0);
                        umma_commit(&ctl.s_full[t][h]);
                        if (h == 1 || u + 1 == n_st) umma_commit(&ctl.k_empty[e % G::kKSt]);
                    }
                    return true;
                };
                bool ok = wait(&ctl.q_full, 0);
                for (int u = 0; ok && u < 2 && u < n_st; ++u) ok = issue_s(u);
                // PV of step u once its P is in TMEM, then S of step u + 2 into the buffer P came from
                // (MMAs of one thread run in issue order); S of step u + 1 is there already, so the
                // softmax never waits for it.
                for (int u = 0; ok && u < n_st; ++u) {
                    const int e = sch.entry(t, u >> 1), h = u & 1;
                    ok = (h == 1 || wait(&ctl.v_full[e % G::kVSt], e / G::kVSt)) && wait(&ctl.p_full[t][h], u >> 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dv = sdesc_sw128(sV(e % G::kVSt) + (uint32_t)(h * kStep * 128), G::kRegion, 1024);
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < kStep / 16; ++k)
                            umma_ts(d_o, d_s + h * kStep + k * 8, dv + (uint64_t)(k * 2048 / 16), idO, (u > 0 || k > 0));
                        umma_commit(&ctl.pv_done[t]);
                    }
                    if (u + 2 < n_st) ok = issue_s(u + 2);
                    if (leader && (h == 1 || u + 1 == n_st)) umma_commit(&ctl.v_empty[e % G::kVSt]);
                }
                // no MMA may still run when TMEM is released
                if (leader) umma_commit(&ctl.drain[t]);
                mbar_wait(&ctl.drain[t], 0, kDrainBudget);
            }
            __syncwarp();
        }
        if (cs > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        setmaxnreg_inc<kRegSoftmax>();
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float c_row = p.scale_log2;
        if (t < n_ch) {
            if (warp_live) c_row = query_terms<D>(q_at, q_at + G::kQPart, lane, p.scale_log2);
            // a split block's chain B converted into the free query buffer: it needs the rows' factors
            if (!(split && t == 1)) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.q_full);
            }
        }
        bool ok = t < n_ch;
        float m_used = -INFINITY, l_sum = 0.f;
        if (t < n_ch) {
            // ---------------------------------------------------------------- softmax
            const int n_st = sch.n_steps(t, last_keys);
            for (int u = 0; u < n_st; ++u) {
                const int e = sch.entry(t, u >> 1), h = u & 1, fs = e % kFSt;
                ok = __all_sync(0xffffffffu, wait_bar(&ctl.s_full[t][h], (u >> 1) & 1, abort_flag, dev_status, budget));
                if (!ok) break;
                tc_fence_after();
                if (!warp_live) {
                    // rows past the block: whatever P holds only reaches rows that are never read
                    if (lane == 0) mbar_arrive(&ctl.p_full[t][h]);
                    continue;
                }
                const uint32_t s_at = lane_base + col_s(t) + (uint32_t)(h * kStep);
                uint32_t v[2][32];
                tmem_ld32(s_at, v[0]);
                tmem_ld32(s_at + 32, v[1]);
                // the keys' factors
                uint32_t f[kStep / 4][4];
#pragma unroll
                for (int x = 0; x < kStep / 4; ++x)
                    ld_shared_v4(smem_u32(&ctl.factor[fs][0]) + (uint32_t)(h * kStep + 4 * x) * 4u, f[x]);
                tmem_ld_wait();
                // logits in units of c_row: S times the keys' factors
#pragma unroll
                for (int x = 0; x < kStep; x += 2) {
                    float a, bb;
                    f2unpack(f2mul(f2pack(__uint_as_float(v[x >> 5][x & 31]), __uint_as_float(v[x >> 5][(x & 31) + 1])),
                                   f2pack(__uint_as_float(f[x >> 2][x & 3]), __uint_as_float(f[x >> 2][(x & 3) + 1]))), a, bb);
                    v[x >> 5][x & 31] = __float_as_uint(a);
                    v[x >> 5][(x & 31) + 1] = __float_as_uint(bb);
                }
                const int valid = T_len - (kt0 + sch.tile(t, u >> 1)) * kBN - h * kStep;
                if (valid < kStep) {
#pragma unroll
                    for (int x = 0; x < kStep; ++x)
                        if (x >= valid) v[x >> 5][x & 31] = __float_as_uint(-INFINITY);
                }
                if constexpr (kDrop) {
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        const uint32_t gone = ctl.drop[fs][2 * h + cc];
                        if (gone) {
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if ((gone >> x) & 1u) v[cc][x] = __float_as_uint(-INFINITY);
                        }
                    }
                }
                auto row_max = [&]() {
                    float mx[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t* y = &v[q >> 1][(q & 1) * 16];
                        mx[q] = max3f(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]));
#pragma unroll
                        for (int x = 3; x < 15; x += 2) mx[q] = max3f(mx[q], __uint_as_float(y[x]), __uint_as_float(y[x + 1]));
                        mx[q] = fmaxf(mx[q], __uint_as_float(y[15]));
                    }
                    return max3f(mx[0], mx[1], fmaxf(mx[2], mx[3])) * c_row;
                };
                // P of the step against m_used, over S; returns its sum
                auto exponentiate = [&]() {
                    // a row whose keys so far were all discarded exponentiates against 0
                    const float ms = (kDrop && m_used == -INFINITY) ? 0.f : m_used;
                    const uint64_t c2 = f2pack(c_row, c_row), nm2 = f2pack(-ms, -ms);
                    uint64_t ls2[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        uint32_t pk[16];
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            float x0, x1;
                            f2unpack(f2fma(f2pack(__uint_as_float(v[cc][x]), __uint_as_float(v[cc][x + 1])), c2, nm2), x0, x1);
                            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                            ls2[(x >> 1) & 1] = f2add(ls2[(x >> 1) & 1], f2pack(p0, p1));
                            __nv_bfloat162 two = __floats2bfloat162_rn(p0, p1);
                            pk[x >> 1] = *reinterpret_cast<uint32_t*>(&two);
                        }
                        tmem_st16(s_at + cc * 16, pk);
                    }
                    float l0, l1, l2, l3;
                    f2unpack(ls2[0], l0, l1);
                    f2unpack(ls2[1], l2, l3);
                    return (l0 + l1) + (l2 + l3);
                };
                // P is taken against the maximum so far while this step's is found; only where that has
                // grown past the threshold are O and the sum rescaled and P taken again.
                if (u == 0) m_used = row_max();
                float sum = exponentiate();
                const float mt = row_max();
                const bool grown = mt > m_used + kRescaleThreshold;
                if (__any_sync(0xffffffffu, grown)) {
                    const float alpha = grown ? fast_exp2(m_used - mt) : 1.f;
                    if (grown) m_used = mt;
                    if (u > 0) {
                        // O holds the steps before this one once PV of the last is complete
                        ok = __all_sync(0xffffffffu, wait_bar(&ctl.pv_done[t], (u - 1) & 1, abort_flag, dev_status, budget));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 8; ++q) {
                            uint32_t o[8];
                            tmem_ld8(lane_base + col_o(t) + q * 8, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                            tmem_st8(lane_base + col_o(t) + q * 8, o);
                        }
                        l_sum *= alpha;
                    }
                    sum = exponentiate();
                }
                l_sum += sum;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full[t][h]);
            }
            // An issuer that gave up commits its drain too: only without an abort do all the steps stand behind it.
            if (ok)
                ok = __all_sync(0xffffffffu, wait_bar(&ctl.drain[t], 0, abort_flag, dev_status, budget) && !*abort_flag);
        }
        // Split keys: chain A merges the two partial states (weight 0 for a chain without keys)
        float w_a = 1.f, w_b = 0.f;
        if (split) {
            if (t == 1) {
                ctl.part_m[kBM + r] = m_used;
                ctl.part_l[kBM + r] = l_sum;
            }
            if (!ok) ctl.failed = 1.f;
            named_barrier_sync<1>(2 * kBM);
            ok = ok && ctl.failed == 0.f;
            if (t == 1) {
                ok = false;                                // chain A carries the rows from here
            } else if (ok) {
                ok = __all_sync(0xffffffffu, wait_bar(&ctl.drain[1], 0, abort_flag, dev_status, budget));
                const float mb = ctl.part_m[kBM + r], lb = ctl.part_l[kBM + r];
                const float m = fmaxf(m_used, mb);
                w_a = m_used == -INFINITY ? 0.f : fast_exp2(m_used - m);
                w_b = mb == -INFINITY ? 0.f : fast_exp2(mb - m);
                l_sum = l_sum * w_a + lb * w_b;
                m_used = m;
            }
        }
        auto load_o = [&](int cc, uint32_t (&o)[32]) {
            uint32_t ob[32];
            tmem_ld32(lane_base + col_o(t) + cc * 32, o);
            if (split) tmem_ld32(lane_base + col_o(1) + cc * 32, ob);
            tmem_ld_wait();
            if (split) {
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    o[x] = __float_as_uint(fmaf(__uint_as_float(o[x]), w_a, __uint_as_float(ob[x]) * w_b));
            }
        };
        constexpr float kUnshift = 4294967296.f;           // 2^kVShift
        if (cs == 1) {
            if (ok) {
                tc_fence_after();
                // A lane writes its row, a 32-byte sector at a time where the output's address allows.  (Half
                // sectors: 570 us where this takes 555; whole rows per warp through shared memory: 562.)
                const float inv = l_sum == 0.f ? 0.f : kUnshift / l_sum;
                const bool write = (split ? r : t * kBM + r) < n_rows, wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
                uint4* to = reinterpret_cast<uint4*>(p.out + off);
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    load_o(cc, o);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t k[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float a = __uint_as_float(o[16 * x + 2 * y]) * inv, d = __uint_as_float(o[16 * x + 2 * y + 1]) * inv;
                            __nv_bfloat162 two = __floats2bfloat162_rn(a, d);
                            k[y] = *reinterpret_cast<uint32_t*>(&two);
                        }
                        if (!write) continue;
                        if (wide) {
                            st_global_v8(to + cc * 4 + x * 2, k);
                        } else {
                            to[cc * 4 + x * 2] = make_uint4(k[0], k[1], k[2], k[3]);
                            to[cc * 4 + x * 2 + 1] = make_uint4(k[4], k[5], k[6], k[7]);
                        }
                    }
                }
            }
        } else {
            // partial of this part: the rings are free once both chains' MMAs are complete
            if (!split && n_ch == 2 && ok)
                ok = __all_sync(0xffffffffu, wait_bar(&ctl.drain[t ^ 1], 0, abort_flag, dev_status, budget));
            if (t < n_qt) {
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        load_o(cc, o);
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            *reinterpret_cast<uint4*>(base_ptr + G::kRing + part_off<D>(t * kBM + r, cc * 8 + x)) =
                                make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                    }
                    ctl.part_m[t * kBM + r] = m_used;
                    ctl.part_l[t * kBM + r] = l_sum;
                } else {
                    ctl.failed = 1.f;
                }
            }
            cluster_sync();
            // A lane finalises (row, 4-column) items, a warp 32 neighbouring ones, so that a load takes whole lines
            // of the other SM's shared memory (16 columns to a lane, lanes on 16 different rows: 12 us for 256
            // rows from four ranks).  Eight items' and ranks' loads are in flight.  Every value loaded is used,
            // so none is still on its way when the ranks part.
            const uint32_t m_a = smem_u32(&ctl.part_m[0]), l_a = smem_u32(&ctl.part_l[0]), f_a = smem_u32(&ctl.failed);
            float lost = 0.f;
#pragma unroll
            for (int w = 0; w < kMaxCluster; ++w)
                if (w < cs) lost += ld_cluster_f32(mapa_shared(f_a, w));
            constexpr int kItems = D / 4;                  // per row
            const int n_items = lost == 0.f ? n_rows * kItems : 0;
            auto finalise = [&](auto ranks) {
                constexpr int W = decltype(ranks)::value, N = kMaxCluster / W;
                const int step = 32 * cs * 2 * (kBM / 32);
#pragma unroll 1
                for (int it = 32 * (cr + cs * warp) + lane; it < n_items; it += N * step) {
                    float mw[N][W], lw[N][W];
                    float4 f[N][W];
#pragma unroll
                    for (int n = 0; n < N; ++n)
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            mw[n][w] = -INFINITY;
                            lw[n][w] = 0.f;
                            f[n][w] = make_float4(0.f, 0.f, 0.f, 0.f);
                            const int at = it + n * step, rr = at / kItems;
                            if (w < cs && at < n_items) {
                                mw[n][w] = ld_cluster_f32(mapa_shared(m_a + 4u * rr, w));
                                lw[n][w] = ld_cluster_f32(mapa_shared(l_a + 4u * rr, w));
                                f[n][w] = ld_cluster_v4(mapa_shared(base + G::kRing + part_off<D>(rr, at % kItems), w));
                            }
                        }
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int at = it + n * step, rr = at / kItems;
                        float M = -INFINITY, L = 0.f;
#pragma unroll
                        for (int w = 0; w < W; ++w) M = fmaxf(M, mw[n][w]);
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            const bool none = mw[n][w] == -INFINITY && lw[n][w] == 0.f;        // no key in this part
                            const float e = none ? 0.f : fast_exp2(mw[n][w] - M);
                            L = fmaf(e, lw[n][w], L);
                            acc.x = none ? acc.x : fmaf(e, f[n][w].x, acc.x);
                            acc.y = none ? acc.y : fmaf(e, f[n][w].y, acc.y);
                            acc.z = none ? acc.z : fmaf(e, f[n][w].z, acc.z);
                            acc.w = none ? acc.w : fmaf(e, f[n][w].w, acc.w);
                        }
                        const float inv = L == 0.f ? 0.f : kUnshift / L;
                        const uint32_t pr = (uint32_t)(row0 + rr), i = pr / (uint32_t)p.g;
                        __nv_bfloat162 a2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
                        if (at < n_items) {
                            bf16* o = p.out + ((qbase + i) * p.Hq + (int64_t)hk * p.g + (pr - i * (uint32_t)p.g)) * D + at % kItems * 4;
                            *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<uint32_t*>(&a2), *reinterpret_cast<uint32_t*>(&b2));
                        }
                    }
                }
            };
            if (cs <= 2) finalise(std::integral_constant<int, 2>{});
            else if (cs <= 4) finalise(std::integral_constant<int, 4>{});
            else finalise(std::integral_constant<int, 8>{});
            __syncwarp();
            cluster_sync();        // no CTA may leave while another still reads its shared memory
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag) settle_after_abort(ctl.unlanded != 0);
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Per device and variant: 0 = not prepared yet, 1 = ready, otherwise the status to return.
// Preparing twice is harmless, so a race between threads only repeats the work.
std::atomic<int> g_prepared[4][64];

template <int D, bool kDrop>
int prepare() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    std::atomic<int>& st = g_prepared[(D == 128 ? 2 : 0) + (kDrop ? 1 : 0)][dev];
    const int known = st.load(std::memory_order_acquire);
    if (known) return known == 1 ? ACACHE_OK : known;
    auto kern = q8_attn_kernel<D, kDrop>;
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kBytes) != cudaSuccess ||
        cudaFuncGetAttributes(&fa, kern) != cudaSuccess) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;   // not cached: a later call may succeed
    }
    // the register split assumes the launch allocation; refuse to launch otherwise
    const int rc = fa.numRegs * kThreads < 128 * kRegSum ? ACACHE_ERR_UNSUPPORTED
                                                                                                 : ACACHE_OK;
    st.store(rc == ACACHE_OK ? 1 : rc, std::memory_order_release);
    return rc;
}

template <int D, bool kDrop>
int launch(const Q8Params& prm, dim3 grid, cudaStream_t stream, bool pdl) {
    auto kern = q8_attn_kernel<D, kDrop>;
    if (int rc = prepare<D, kDrop>()) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Geo<D>::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned na = 0;
    if (prm.cs > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = (unsigned)prm.cs;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    if (pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    if (cudaLaunchKernelEx(&cfg, kern, prm) != cudaSuccess) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    return launch_status();
}

// CTAs of the kernel that run at once in clusters of cs: a cluster stays within a group of SMs, and the groups are
// no multiples of most sizes (152 SMs hold 152, 144 and 120 CTAs in clusters of 2, 4 and 8).
std::atomic<int> g_slots[kMaxCluster + 1][64];
int cluster_slots(int cs) {
    int dev = 0;
    if (cs == 1 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sm_count();
    std::atomic<int>& known = g_slots[cs][dev];
    int n = known.load(std::memory_order_relaxed);
    if (n) return n;
    n = sm_count();
    if (prepare<128, false>() == ACACHE_OK) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)cs;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)cs);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Geo<128>::kBytes;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, q8_attn_kernel<128, false>, &cfg) == cudaSuccess && clusters > 0)
            n = clusters * cs;
        else
            (void)cudaGetLastError();
    }
    known.store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace

bool q8_tc_supported(const AttnArgs& a) {
    return a.dtype == ACACHE_BF16 && a.scale > 0.f;
}

int launch_q8_tc_attention(const Q8Attn& c) {
    const int d = c.a.d, hkv = c.a.hkv, g = c.a.hq / hkv;
    const int64_t n_rb = ((int64_t)c.n_q * g + kQT * kBM - 1) / (kQT * kBM);
    Q8Params prm{};
    const uint64_t rows[2] = {(uint64_t)d, (uint64_t)(c.num_slots * hkv)};
    const uint64_t pool[3] = {(uint64_t)d, (uint64_t)hkv, (uint64_t)c.num_slots};
    const uint32_t one[2] = {(uint32_t)d, 1}, box[3] = {(uint32_t)d, 1, kBN};
    if (!make_map_u8(&prm.tm_k, c.k_cache, 2, rows, one) || !make_map_u8(&prm.tm_kbox, c.k_cache, 3, pool, box))
        return ACACHE_ERR_CUDA;
    prm.q = (const bf16*)c.q;
    prm.v_cache = c.v_cache;
    prm.kv_scale = c.kv_scale;
    prm.read_slot = c.read_slot;
    prm.q_start = c.q_start;
    prm.kv_start = c.kv_start;
    prm.out = (bf16*)c.out;
    prm.dev_status = c.dev_status;
    prm.num_slots = c.num_slots;
    prm.oob_row = (int)(c.num_slots * hkv) + (c.num_slots == 0);
    prm.n_q = c.n_q;
    prm.total_q = c.total_q;
    prm.T_len = c.T_len;
    prm.Hq = c.a.hq;
    prm.Hkv = hkv;
    prm.g = g;
    prm.scale_log2 = c.a.scale * kLog2e;
    prm.budget = wait_budget();
    // Parts of the key range: waves x what a CTA takes, in thirds of a key tile against two row tiles (1.9 us at
    // d = 128; against one, two thirds of that).  A CTA costs 16 (12) besides its keys, a cluster's merge 11 (7).
    // (Measured for 1, 2, 4 and 8 parts: 600 rows x 3000 keys, 8 heads over 2: 56, 41, 29 and 42 us; 300 x 700,
    // 4 heads: 23, 23, 21, 21; 200 x 500, 2 requests, 32 heads over 8: 21, 23, 35, 35; 100 x 2000, 16 heads:
    // 31, 25, 19, 29.)
    const int n_all = (c.T_len + kBN - 1) / kBN;
    const int64_t units = (int64_t)c.B * hkv * n_rb;
    const bool two = (int64_t)c.n_q * g > kBM;
    prm.cs = 1;
    int64_t best = 0;
    for (int cs = 1; cs <= kMaxCluster && cs <= n_all; ++cs) {
        const int64_t slots = cluster_slots(cs);
        const int64_t cta = (two ? 3 : 2) * ((n_all + cs - 1) / cs) + (two ? 16 : 12) + (cs == 1 ? 0 : two ? 11 : 7);
        const int64_t est = (units * cs + slots - 1) / slots * cta;
        if (cs == 1 || est < best) {
            best = est;
            prm.cs = cs;
        }
    }
    prm.part = (n_all + prm.cs - 1) / prm.cs;
    const dim3 grid((unsigned)(hkv * prm.cs), (unsigned)c.B, (unsigned)n_rb);
    if (d == 128)
        return c.drop_none ? launch<128, true>(prm, grid, c.stream, c.after_store)
                           : launch<128, false>(prm, grid, c.stream, c.after_store);
    return c.drop_none ? launch<64, true>(prm, grid, c.stream, c.after_store)
                       : launch<64, false>(prm, grid, c.stream, c.after_store);
}

}  // namespace acache
