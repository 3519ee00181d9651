// q8_decode.cu -- read-slot attention over an 8-bit pool for few query rows per (request, KV head): the
// block-decode step and single tokens.  bf16 queries and outputs, head dim 64 or 128, tcgen05 + TMEM.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4.3, App. C.1 and Sec. 5 (block length
// 32); the 8-bit pool is this library's.
//
// Memory-bound: each (request, KV head) streams its keys' and values' codes once, 256 bytes a key
// (d = 128), against at most 64 packed rows (queries x heads of the group).
//   * S as in q8_tc.cu: hi and lo of the query rows times the codes as they lie in the pool.
//   * O: P times V's codes converted to f16 (exact, one instruction for two).  Their power of two goes
//     into the exponent instead: P = 2^(s + ev - m) with m the running maximum of s + ev, so P
//     V is right whatever the rows' scales are, P never exceeds 2^15 and keys down to 2^-27 of the
//     largest weighted one count (f16 subnormals); the sum adds P 2^-ev in float32.  Each thread has 32 or 64
//     keys of a tile, so this costs less than scaling 128 x d values would.
//   * Up to 32 (64) rows are replicated 4 (2) times over the 128 TMEM lanes, each replica taking a
//     quarter (half) of every tile's keys, so that the four softmax warps share a tile's
//     exponentials; P buffers whose other columns stay zero let one MMA add every replica's keys
//     into its own O rows.  S and P are double-buffered.
//   * The key range is split over a cluster of up to 8 CTAs when that fills the SMs better; partial
//     (maximum, sum, O) of all replicas and ranks are merged through distributed shared memory in a
//     fixed order -- no workspace, no second launch.
//
// Warps (416 threads, 1 CTA per SM): 0-3 softmax; 4-7 bring V's codes and convert them; 8-11 bring K's
// codes and the keys' factors; 12 issues every MMA.  The codes come by 16-byte cp.async, a warp taking
// 32 keys of every tile: a gather4 takes its warp some 90 cycles to issue for four rows (measured),
// a cp.async instruction a tenth of that for as many; and pool addresses need no tensor maps.
// TMEM (512 columns): S0 [0,128)  S1 [128,256)  O [256,384)  P0 [384,448)  P1 [448,512).
//
// Every mbarrier wait is bounded (see q8_tc.cu).
#include <atomic>

#include "q8_tc.cuh"

namespace acache {
namespace {

using namespace q8;

constexpr int kBM = 128, kBN = 128;
constexpr int kThreads = 416;
constexpr int kVWarp = 4, kKWarp = 8, kMmaWarp = 12;
constexpr int kKSt = 4, kKLag = 2;          // K ring; an entry is announced kKLag entries after its loads
constexpr int kRSt = 3;                     // V's codes (each warp's rows are its own)
constexpr int kVSt = 2;                     // V in f16
constexpr int kFSt = 8;                     // factors
constexpr int kMaxCluster = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS0 = 0, kColO = 256, kColP0 = 384;
constexpr float kPHead = 3.0f;              // P of the used maximum is 2^3 ...
constexpr float kRescaleThreshold = 12.0f;  // ... and never above 2^15

template <int D>
struct Geo {
    static constexpr uint32_t kQPart = kBM * D;
    static constexpr uint32_t kTile = kBN * D;             // codes of K or of V
    static constexpr uint32_t kVTile = kBN * D * 2;        // V in f16
    static constexpr uint32_t kRegion = kBN * 128;         // 64 columns of it
    static constexpr uint32_t kRing = 2 * kQPart;
    static constexpr uint32_t kRRing = kRing + kKSt * kTile;
    static constexpr uint32_t kVRing = kRRing + kRSt * kTile;
    static constexpr uint32_t kBytes = kVRing + kVSt * kVTile + 1024;
    static_assert(kKSt * kTile >= kBM * D * 4u, "partial O reuses the K ring");
    static_assert(kVSt * kVTile >= 64 * D * 4u, "and the merged rows V's");
};

struct DecParams {
    const bf16* q;
    const uint8_t *k_cache, *v_cache, *kv_scale;
    const int32_t *read_slot, *q_start, *kv_start;
    bf16* out;
    int32_t* dev_status;
    int64_t num_slots;
    int n_q, T_len, Hq, Hkv, g;
    int cs, part;                   // CTAs per cluster; key tiles per part
    float scale_log2;
    long long budget;
};

struct Ctl {
    uint64_t q_full;
    uint64_t k_full[kKSt], k_empty[kKSt];
    uint64_t v_full[kVSt], v_empty[kVSt];
    uint64_t f_full[kFSt];
    uint64_t s_full[2], p_full[2];
    uint64_t pv_done, drain;
    uint32_t tmem_base;
    int abort;
    float failed;
    uint32_t drop[kFSt][4];
    float part_m[kBM], part_l[kBM];         // per lane
    float row_m[64], row_l[64];             // per row, replicas merged
    float c_row[64];
    __align__(16) float fk[kFSt][kBN];      // 2^ek
    __align__(16) float ev[kFSt][kBN];      // ev
    __align__(16) float rv[kFSt][kBN];      // 2^-ev
};

constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int D, int REP, bool kDrop>
__global__ void __launch_bounds__(kThreads, 1)
q8_decode_kernel(const __grid_constant__ DecParams p) {
    using G = Geo<D>;
    constexpr int GL = kBM / REP;                    // lanes per replica
    constexpr int NC = 4 / REP;                      // 32-key chunks of a thread
    extern __shared__ uint8_t dsm[];
    __shared__ Ctl ctl;
    const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
    const uint32_t sQ = base;
    auto sK = [&](int s) { return base + G::kRing + G::kTile * (uint32_t)s; };
    auto sR = [&](int s) { return base + G::kRRing + G::kTile * (uint32_t)s; };
    auto sV = [&](int s) { return base + G::kVRing + G::kVTile * (uint32_t)s; };
    const int cr = p.cs == 1 ? 0 : (int)(blockIdx.x % (unsigned)p.cs);
    const int hk = p.cs == 1 ? (int)blockIdx.x : (int)(blockIdx.x / (unsigned)p.cs);
    const int b = (int)blockIdx.y;
    int n_q = p.n_q, T_len = p.T_len;
    int64_t qbase = (int64_t)b * p.n_q, kbase = (int64_t)b * p.T_len;
    if (p.q_start) {
        qbase = p.q_start[b];
        kbase = p.kv_start[b];
        n_q = (int)(p.q_start[b + 1] - qbase);
        T_len = (int)(p.kv_start[b + 1] - kbase);
        if (n_q != 0 && (n_q < 0 || n_q > p.n_q || T_len < 1 || T_len > p.T_len)) {
            if (threadIdx.x == 0 && blockIdx.x == 0) flag(p.dev_status, ACACHE_DEV_BAD_LENGTH);
            return;
        }
    }
    const int n_rows = n_q * p.g;                    // <= GL
    if (n_rows == 0) return;
    const int n_all = (T_len + kBN - 1) / kBN;
    const int cs = (n_all + p.part - 1) / p.part;    // parts of this request's keys (<= p.cs)
    if (cr >= cs) return;
    const int kt0 = (int)((int64_t)cr * n_all / cs);
    const int n_kv = (int)((int64_t)(cr + 1) * n_all / cs) - kt0;      // >= 1
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &ctl.abort;
    int32_t* dev_status = p.dev_status;
    const long long budget = p.budget;

    // K and V warps: lane l looks after key 32 w + l of every tile.  The maps are not written by a store
    // this launch may overlap: the first slots are on their way during the set-up.
    const int w = warp & 3;
    auto slot_of = [&](int e) -> int {
        const int t = (kt0 + e) * kBN + 32 * w + lane;
        int s = kNoKey;
        if (e < n_kv && t < T_len) s = p.read_slot[kbase + t];
        return s;
    };
    int s_cur = kNoKey, s_next = kNoKey;
    if (warp >= kVWarp && warp < kMmaWarp) {
        s_cur = slot_of(0);
        s_next = slot_of(1);
    }
    if (threadIdx.x == 0) {
        mbar_init(&ctl.q_full, 4);
        for (int s = 0; s < kKSt; ++s) {
            mbar_init(&ctl.k_full[s], 4);
            mbar_init(&ctl.k_empty[s], 1);
        }
        for (int s = 0; s < kVSt; ++s) {
            mbar_init(&ctl.v_full[s], 4);
            mbar_init(&ctl.v_empty[s], 1);
        }
        for (int s = 0; s < kFSt; ++s) mbar_init(&ctl.f_full[s], 4);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&ctl.s_full[t], 1);
            mbar_init(&ctl.p_full[t], 4);
        }
        mbar_init(&ctl.pv_done, 1);
        mbar_init(&ctl.drain, 1);
        ctl.abort = 0;
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
    // Pieces of a row (16 bytes), rows per warp instruction, instructions per tile of a K or V warp.
    constexpr int CPR = D / 16, RPI = 32 / CPR, NI = 32 / RPI;

    if (warp >= kKWarp && warp < kMmaWarp) {
        // ---------------------------------------------------------------------- K
        const int c = lane % CPR, rr = lane / CPR;
        const uint8_t* src = p.k_cache + (int64_t)hk * D + c * 16;
        const int64_t row_bytes = (int64_t)p.Hkv * D;
        auto scale_of = [&](int s) -> uint32_t {
            uint32_t two = 127u | 127u << 8;             // a zero row: factor 1
            if (s >= 0 && s < p.num_slots) two = reinterpret_cast<const uint16_t*>(p.kv_scale)[(int64_t)s * p.Hkv + hk];
            return two;
        };
        grid_dependency_wait();                          // store-then-attend: the pool is written now
        uint32_t sc = scale_of(s_cur);
        int e = 0;
        for (; e < n_kv; ++e) {
            const int s = e % kKSt, fs = e % kFSt;
            if (e >= kKSt && !__all_sync(0xffffffffu, wait_bar(&ctl.k_empty[s], ((e / kKSt) - 1) & 1, abort_flag, dev_status, budget)))
                break;
            const bool in = s_cur >= 0 && s_cur < p.num_slots;
            const bool none = kDrop && s_cur == ACACHE_SLOT_NONE;
            if (!in && !none && s_cur != kNoKey) flag(dev_status, ACACHE_DEV_BAD_SLOT);
            const int sl = in ? s_cur : -1;
            int row[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) row[i] = __shfl_sync(0xffffffffu, sl, i * RPI + rr);
            const uint32_t dst = sK(s) + (uint32_t)(32 * w * D);
#pragma unroll
            for (int i = 0; i < NI; ++i)                 // (a key without a row is filled with zeros)
                cp_async16(dst + row_chunk<D>((uint32_t)(i * RPI + rr), (uint32_t)c), src + max(row[i], 0) * row_bytes,
                           row[i] >= 0 ? 16u : 0u);
            cp_async_commit();
            // The factors.  S of an entry is issued after the softmax of the entry two before it wrote P,
            // so with entry e - kKSt free the oldest factors in use are those of e - kKSt - 1.
            static_assert(kFSt > kKSt + 1, "factor ring");
            {
                const uint32_t v = sc >> 8, y = max(v, (uint32_t)(kQ8MinExp + 127));
                ctl.fk[fs][32 * w + lane] = q8_factor(sc & 0xffu);
                ctl.ev[fs][32 * w + lane] = v > kQ8MaxByte ? __uint_as_float(0x7fffffffu) : (float)((int)y - 127);
                ctl.rv[fs][32 * w + lane] = __uint_as_float((254u - min(y, kQ8MaxByte)) << 23);
                if constexpr (kDrop) {
                    const uint32_t gone = __ballot_sync(0xffffffffu, none);
                    if (lane == 0) ctl.drop[fs][w] = gone;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.f_full[fs]);
            s_cur = s_next;
            sc = scale_of(s_cur);
            s_next = slot_of(e + 2);
            if (e >= kKLag) {
                cp_async_wait<kKLag>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.k_full[(e - kKLag) % kKSt]);
            }
        }
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (e == n_kv && lane == 0)
            for (int x = max(0, n_kv - kKLag); x < n_kv; ++x) mbar_arrive(&ctl.k_full[x % kKSt]);
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------------- MMA issuer
        // S(0), S(1), then per tile j: PV(j) once P(j) is in TMEM, then S(j+2) into the buffer P(j)'s
        // scores came from.  MMAs of one thread run in issue order: S(j+2) complete implies PV(j)
        // complete, so the softmax of tile j+2 may overwrite P buffer j % 2.
        if (lane == 0) {
            constexpr uint32_t idS = idesc_e4m3(kBM, kBN), idO = idesc_f16(kBM, D, true);
            const uint64_t dq = sdesc_rows<D>(sQ);
            auto issue_s = [&](int j) -> bool {
                if (!wait_bar(&ctl.k_full[j % kKSt], (j / kKSt) & 1, abort_flag, dev_status, budget)) return false;
                tc_fence_after();
                const uint64_t dk = sdesc_rows<D>(sK(j % kKSt));
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        umma_ss_f8(tmem + kColS0 + (uint32_t)(j & 1) * 128u, dq + (uint64_t)((h * G::kQPart + k * 32) >> 4),
                                   dk + (uint64_t)(k * 32 >> 4), idS, h > 0 || k > 0);
                umma_commit(&ctl.s_full[j & 1]);
                umma_commit(&ctl.k_empty[j % kKSt]);
                return true;
            };
            bool ok = wait_bar(&ctl.q_full, 0, abort_flag, dev_status, budget);
            for (int j = 0; ok && j < 2 && j < n_kv; ++j) ok = issue_s(j);
            for (int j = 0; ok && j < n_kv; ++j) {
                ok = wait_bar(&ctl.v_full[j % kVSt], (j / kVSt) & 1, abort_flag, dev_status, budget) &&
                     wait_bar(&ctl.p_full[j & 1], (j >> 1) & 1, abort_flag, dev_status, budget);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dv = sdesc_sw128(sV(j % kVSt), G::kRegion, 1024);
                const uint32_t a_p = tmem + kColP0 + (uint32_t)(j & 1) * 64u;
#pragma unroll
                for (int k = 0; k < kBN / 16; ++k)
                    umma_ts(tmem + kColO, a_p + k * 8, dv + (uint64_t)(k * 2048 / 16), idO, (j > 0 || k > 0));
                umma_commit(&ctl.v_empty[j % kVSt]);
                umma_commit(&ctl.pv_done);
                if (j + 2 < n_kv) ok = issue_s(j + 2);
            }
            umma_commit(&ctl.drain);
            mbar_wait(&ctl.drain, 0, kDrainBudget);
        }
        __syncwarp();
    } else if (warp >= kVWarp) {
        // ---------------------------------------------------------------------- V
        // A warp's 32 rows of a tile arrive in rows of D bytes, two tiles ahead; it converts what it
        // brought, so nobody else waits for them.
        const int lc = lane % CPR, lr = lane / CPR;
        const uint8_t* vsrc = p.v_cache + (int64_t)hk * D + lc * 16;
        const int64_t row_bytes = (int64_t)p.Hkv * D;
        auto bring = [&](int e, int slot) {
            const int sl = (slot >= 0 && slot < p.num_slots) ? slot : -1;
            int row[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) row[i] = __shfl_sync(0xffffffffu, sl, i * RPI + lr);
            const uint32_t dst = sR(e % kRSt) + (uint32_t)((32 * w + lr) * D + lc * 16);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                cp_async16(dst + (uint32_t)(i * RPI * D), vsrc + max(row[i], 0) * row_bytes, row[i] >= 0 ? 16u : 0u);
        };
        // Conversion: 16-byte piece c of rows r0, r0 + RPI, ...  The eight lanes of a shared-memory phase take
        // four pieces of one 64-column region from each of two neighbouring rows (the f16 tile is
        // swizzled), so neither side meets in a bank.
        const int q = lane >> 3, k = lane & 7;
        const int c = D == 128 ? k : (k & 3);
        const int r0 = 32 * w + (D == 128 ? (q & 2) + ((k >> 2) ^ (q & 1)) : 2 * q + (k >> 2));
        grid_dependency_wait();
        bring(0, s_cur);
        cp_async_commit();
        if (n_kv > 1) bring(1, s_next);
        cp_async_commit();
        s_next = slot_of(2);
        for (int e = 0; e < n_kv; ++e) {
            const int s = e % kVSt, rs = e % kRSt;
            if (e + 2 < n_kv) bring(e + 2, s_next);
            cp_async_commit();
            s_next = slot_of(e + 3);
            cp_async_wait<2>();
            __syncwarp();
            if (e >= kVSt && !__all_sync(0xffffffffu, wait_bar(&ctl.v_empty[s], ((e / kVSt) - 1) & 1, abort_flag, dev_status, budget)))
                break;
            const uint32_t src = sR(rs) + (uint32_t)(r0 * D + c * 16);
            const uint32_t dst = sV(s) + (uint32_t)r0 * 128u + ((uint32_t)c >> 2) * G::kRegion;
#pragma unroll
            for (int i0 = 0; i0 < NI; i0 += 4) {
                uint32_t d[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) ld_shared_v4(src + (uint32_t)((i0 + i) * RPI * D), d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t o[8];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o[2 * y]) : "h"((unsigned short)(d[i][y] & 0xffffu)));
                        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o[2 * y + 1]) : "h"((unsigned short)(d[i][y] >> 16)));
                    }
                    const uint32_t r8 = (uint32_t)(r0 + (i0 + i) * RPI) & 7u;
                    const uint32_t a0 = dst + (uint32_t)((i0 + i) * RPI) * 128u + (((2u * c & 7u) ^ r8) << 4);
                    st_shared_v4(a0, o[0], o[1], o[2], o[3]);
                    st_shared_v4(a0 ^ 16u, o[4], o[5], o[6], o[7]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.v_full[s]);
        }
        cp_async_wait<0>();
    } else {
        // ---------------------------------------------------------------------- softmax
        const int rep = warp / (4 / REP);                 // replica = key group of this warp
        const int kb = rep * (kBN / REP);                 // first key of the group in a tile
        const int r = threadIdx.x;                        // TMEM lane
        const int row = r % GL;                           // row of the block
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        const bool warp_live = (warp * 32) % GL < n_rows;
        // Each warp converts a quarter of the rows for every replica.  (Lanes past the rows, and warps past
        // them, hold what they like: it stays in their rows.)
        {
            constexpr int NR = GL / 4;
            const int f0 = warp * NR;
            const int64_t o = [&] {
                const int pr = f0 + (lane & (NR - 1)) < n_rows ? f0 + (lane & (NR - 1)) : 0, i = pr / p.g;
                return ((qbase + i) * p.Hq + (int64_t)hk * p.g + (pr - i * p.g)) * D;
            }();
            if (f0 < n_rows)
                query_terms<D, NR, REP>(p.q, o, sQ + (uint32_t)(f0 * D), sQ + G::kQPart + (uint32_t)(f0 * D), (uint32_t)(GL * D),
                                        lane, p.scale_log2, n_rows - f0, &ctl.c_row[f0]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.q_full);
        }
        {   // P starts as zeros: columns outside this warp's key group are never written
            uint32_t z[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0u;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) tmem_st32(lane_base + kColP0 + cc * 32, z);
            tmem_st_wait();
        }
        float m_used = -INFINITY, l_sum = 0.f;
        bool ok = __all_sync(0xffffffffu, wait_bar(&ctl.q_full, 0, abort_flag, dev_status, budget));
        const float c_row = ctl.c_row[row];
        for (int j = 0; ok && j < n_kv; ++j) {
            const int sb = j & 1, fs = j % kFSt;
            ok = __all_sync(0xffffffffu, wait_bar(&ctl.f_full[fs], (j / kFSt) & 1, abort_flag, dev_status, budget) &&
                                             wait_bar(&ctl.s_full[sb], (j >> 1) & 1, abort_flag, dev_status, budget));
            if (!ok) break;
            tc_fence_after();
            if (!warp_live) {
                if (lane == 0) mbar_arrive(&ctl.p_full[sb]);
                continue;
            }
            uint32_t v[NC][32];
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) tmem_ld32(lane_base + kColS0 + sb * 128 + kb + cc * 32, v[cc]);
            tmem_ld_wait();
            // t = s + ev in log2 units
            const uint64_t c2 = f2pack(c_row, c_row);
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&ctl.fk[fs][kb + cc * 32 + i]);
                    const float4 e = *reinterpret_cast<const float4*>(&ctl.ev[fs][kb + cc * 32 + i]);
                    float t0, t1;
                    f2unpack(f2fma(f2mul(f2pack(__uint_as_float(v[cc][i]), __uint_as_float(v[cc][i + 1])), f2pack(f.x, f.y)),
                                   c2, f2pack(e.x, e.y)), t0, t1);
                    v[cc][i] = __float_as_uint(t0);
                    v[cc][i + 1] = __float_as_uint(t1);
                    f2unpack(f2fma(f2mul(f2pack(__uint_as_float(v[cc][i + 2]), __uint_as_float(v[cc][i + 3])), f2pack(f.z, f.w)),
                                   c2, f2pack(e.z, e.w)), t0, t1);
                    v[cc][i + 2] = __float_as_uint(t0);
                    v[cc][i + 3] = __float_as_uint(t1);
                }
            const int valid = T_len - (kt0 + j) * kBN - kb;       // keys of the group in range
            if (valid < kBN / REP) {
#pragma unroll
                for (int cc = 0; cc < NC; ++cc)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (cc * 32 + i >= valid) v[cc][i] = __float_as_uint(-INFINITY);
            }
            if constexpr (kDrop) {
#pragma unroll
                for (int cc = 0; cc < NC; ++cc) {
                    const uint32_t gone = ctl.drop[fs][kb / 32 + cc];
                    if (gone) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if ((gone >> i) & 1u) v[cc][i] = __float_as_uint(-INFINITY);
                    }
                }
            }
            float mt = 0.f;
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) {
                float mx[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t* y = &v[cc][q * 16];
                    mx[q] = max3f(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]));
#pragma unroll
                    for (int i = 3; i < 15; i += 2) mx[q] = max3f(mx[q], __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
                    mx[q] = fmaxf(mx[q], __uint_as_float(y[15]));
                }
                // (no -inf to start from: a row of NaN stays NaN)
                mt = cc == 0 ? fmaxf(mx[0], mx[1]) : max3f(mt, mx[0], mx[1]);
            }
            float alpha = 1.f;
            bool resc = false;
            if (j == 0) {
                m_used = mt;
            } else if (row < n_rows && mt > m_used + kRescaleThreshold) {
                alpha = fast_exp2(m_used - mt);   // 0 while no key of the group was there
                m_used = mt;
                resc = true;
            }
            if (__any_sync(0xffffffffu, resc)) {
                // O holds tiles 0..j-1 once PV(j-1) is complete
                ok = __all_sync(0xffffffffu, wait_bar(&ctl.pv_done, (j - 1) & 1, abort_flag, dev_status, budget));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    tmem_ld32(lane_base + kColO + q * 32, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    tmem_st32(lane_base + kColO + q * 32, o);
                }
                tmem_st_wait();
            }
            // a group without a key so far exponentiates against 0 (every value is -inf)
            const float ms = m_used == -INFINITY ? 0.f : m_used - kPHead;
            const uint64_t nm2 = f2pack(-ms, -ms);
            uint64_t ls2[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 rv = *reinterpret_cast<const float4*>(&ctl.rv[fs][kb + cc * 32 + i]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x0, x1;
                        f2unpack(f2add(f2pack(__uint_as_float(v[cc][i + 2 * h]), __uint_as_float(v[cc][i + 2 * h + 1])), nm2), x0, x1);
                        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                        ls2[h] = f2fma(f2pack(p0, p1), h ? f2pack(rv.z, rv.w) : f2pack(rv.x, rv.y), ls2[h]);
                        // f16 keeps 11 bits, so P is rounded finer than bf16 would
                        __half2 two = __floats2half2_rn(p0, p1);
                        pk[i / 2 + h] = *reinterpret_cast<uint32_t*>(&two);
                    }
                }
                tmem_st16(lane_base + kColP0 + sb * 64 + kb / 2 + cc * 16, pk);
            }
            float l0, l1, l2, l3;
            f2unpack(ls2[0], l0, l1);
            f2unpack(ls2[1], l2, l3);
            l_sum = l_sum * alpha + ((l0 + l1) + (l2 + l3));
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.p_full[sb]);
        }
        if (ok) ok = __all_sync(0xffffffffu, wait_bar(&ctl.drain, 0, abort_flag, dev_status, budget));
        if (!ok) {
            ctl.failed = 1.f;
        } else if (warp_live) {
            // this lane's partial, over the free ring
            tc_fence_after();
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                tmem_ld32(lane_base + kColO + cc * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int y = 0; y < 8; ++y)
                    st_shared_v4(base + G::kRing + part_off<D>(r, cc * 8 + y), o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
            }
        }
        ctl.part_m[r] = m_used;
        ctl.part_l[r] = l_sum;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);

    // -------------------------------------------------------------------------- merge
    // First the replicas of each row (replica x at lane x GL + r), a thread taking 4 columns.
    bool all = ctl.failed == 0.f;
    const bool split = cs > 1;
    const uint32_t rows_at = base + G::kVRing;               // merged rows of this part, f32
    if (all)
        for (int it = (int)threadIdx.x; it < n_rows * (D / 4); it += kThreads) {
            const int r = it / (D / 4), c4 = it % (D / 4);
            float m[REP], M = -INFINITY;
#pragma unroll
            for (int x = 0; x < REP; ++x) {
                m[x] = ctl.part_m[x * GL + r];
                M = fmaxf(M, m[x]);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float L = 0.f;
#pragma unroll
            for (int x = 0; x < REP; ++x) {
                const float lv = ctl.part_l[x * GL + r];
                if (m[x] == -INFINITY && lv == 0.f) continue;        // no key in this partial
                const float e = fast_exp2(m[x] - M);
                uint32_t f[4];
                ld_shared_v4(base + G::kRing + part_off<D>(x * GL + r, c4), f);
                L = fmaf(e, lv, L);
                acc.x = fmaf(e, __uint_as_float(f[0]), acc.x);
                acc.y = fmaf(e, __uint_as_float(f[1]), acc.y);
                acc.z = fmaf(e, __uint_as_float(f[2]), acc.z);
                acc.w = fmaf(e, __uint_as_float(f[3]), acc.w);
            }
            if (split) {
                if (c4 == 0) {
                    ctl.row_m[r] = M;
                    ctl.row_l[r] = L;
                }
                st_shared_v4(rows_at + (uint32_t)(it * 16), __float_as_uint(acc.x), __float_as_uint(acc.y),
                             __float_as_uint(acc.z), __float_as_uint(acc.w));
            } else {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                const int i = r / p.g;
                bf16* o = p.out + ((qbase + i) * p.Hq + (int64_t)hk * p.g + (r - i * p.g)) * D + c4 * 4;
                __nv_bfloat162 a2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<uint32_t*>(&a2), *reinterpret_cast<uint32_t*>(&b2));
            }
        }
    if (!split) return;
    // Then the parts: rank x finalises the (row, 4-column) items x, x + cs, ...
    __syncwarp();
    cluster_sync();
    const uint32_t m_a = smem_u32(&ctl.row_m[0]), l_a = smem_u32(&ctl.row_l[0]), f_a = smem_u32(&ctl.failed);
    all = true;
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x)
        if (x < cs) all = all && ld_cluster_f32(mapa_shared(f_a, x)) == 0.f;
    if (all)
        for (int it = cr + cs * (int)threadIdx.x; it < n_rows * (D / 4); it += cs * kThreads) {
            const int r = it / (D / 4), c4 = it % (D / 4);
            float m[kMaxCluster], l[kMaxCluster], M = -INFINITY;
            float4 o[kMaxCluster];
#pragma unroll
            for (int x = 0; x < kMaxCluster; ++x) {
                m[x] = -INFINITY;
                l[x] = 0.f;
                if (x < cs) {
                    m[x] = ld_cluster_f32(mapa_shared(m_a + 4u * r, x));
                    l[x] = ld_cluster_f32(mapa_shared(l_a + 4u * r, x));
                    o[x] = ld_cluster_v4(mapa_shared(rows_at + (uint32_t)(it * 16), x));
                }
            }
#pragma unroll
            for (int x = 0; x < kMaxCluster; ++x) M = fmaxf(M, m[x]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float L = 0.f;
#pragma unroll
            for (int x = 0; x < kMaxCluster; ++x) {
                if (m[x] == -INFINITY && l[x] == 0.f) continue;      // no key in this part
                const float e = fast_exp2(m[x] - M);
                L = fmaf(e, l[x], L);
                acc.x = fmaf(e, o[x].x, acc.x);
                acc.y = fmaf(e, o[x].y, acc.y);
                acc.z = fmaf(e, o[x].z, acc.z);
                acc.w = fmaf(e, o[x].w, acc.w);
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int i = r / p.g;
            bf16* o2 = p.out + ((qbase + i) * p.Hq + (int64_t)hk * p.g + (r - i * p.g)) * D + c4 * 4;
            __nv_bfloat162 a2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2*>(o2) = make_uint2(*reinterpret_cast<uint32_t*>(&a2), *reinterpret_cast<uint32_t*>(&b2));
        }
    __syncwarp();
    cluster_sync();                // no CTA may leave while another still reads its shared memory
}

std::atomic<int> g_prepared[8][64];   // see q8_tc.cu

template <int D, int REP, bool kDrop>
int launch(const DecParams& prm, dim3 grid, cudaStream_t stream, bool pdl) {
    auto kern = q8_decode_kernel<D, REP, kDrop>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    std::atomic<int>& st = g_prepared[(D == 128 ? 4 : 0) + (REP == 4 ? 2 : 0) + (kDrop ? 1 : 0)][dev];
    if (!st.load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kBytes) != cudaSuccess) {
            (void)cudaGetLastError();
            return ACACHE_ERR_CUDA;
        }
        st.store(1, std::memory_order_release);
    }
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

template <int D>
int dispatch(const DecParams& prm, int rep, bool drop, dim3 grid, cudaStream_t stream, bool pdl) {
    if (rep == 4)
        return drop ? launch<D, 4, true>(prm, grid, stream, pdl) : launch<D, 4, false>(prm, grid, stream, pdl);
    return drop ? launch<D, 2, true>(prm, grid, stream, pdl) : launch<D, 2, false>(prm, grid, stream, pdl);
}

}  // namespace

bool q8_decode_supported(const AttnArgs& a, int n_q) {
    return q8_tc_supported(a) && (int64_t)n_q * (a.hq / a.hkv) <= 64;
}

int launch_q8_decode_attention(const Q8Attn& c) {
    const int d = c.a.d, hkv = c.a.hkv, g = c.a.hq / hkv;
    if (c.B > 65535 || (int64_t)hkv * kMaxCluster > 0x7fffffff) return ACACHE_ERR_INVALID_ARG;
    DecParams prm{};
    prm.k_cache = c.k_cache;
    prm.v_cache = c.v_cache;
    prm.q = (const bf16*)c.q;
    prm.kv_scale = c.kv_scale;
    prm.read_slot = c.read_slot;
    prm.q_start = c.q_start;
    prm.kv_start = c.kv_start;
    prm.out = (bf16*)c.out;
    prm.dev_status = c.dev_status;
    prm.num_slots = c.num_slots;
    prm.n_q = c.n_q;
    prm.T_len = c.T_len;
    prm.Hq = c.a.hq;
    prm.Hkv = hkv;
    prm.g = g;
    prm.scale_log2 = c.a.scale * kLog2e;
    prm.budget = wait_budget();
    // Parts of the key range: waves x (tiles per part + the fixed cost of a CTA and of a merge)
    const int n_all = (c.T_len + kBN - 1) / kBN;
    const int64_t units = (int64_t)c.B * hkv, nsm = sm_count();
    prm.cs = 1;
    int64_t best = 0;
    for (int cs = 1; cs <= kMaxCluster && cs <= n_all; cs *= 2) {
        const int64_t est = ((units * cs + nsm - 1) / nsm) * ((n_all + cs - 1) / cs + 6 + (cs > 1 ? 2 : 0));
        if (cs == 1 || est < best) {
            best = est;
            prm.cs = cs;
        }
    }
    prm.part = (n_all + prm.cs - 1) / prm.cs;
    const dim3 grid((unsigned)(hkv * prm.cs), (unsigned)c.B, 1);
    const int rep = (int64_t)c.n_q * g <= 32 ? 4 : 2;
    return d == 128 ? dispatch<128>(prm, rep, c.drop_none, grid, c.stream, c.after_store)
                    : dispatch<64>(prm, rep, c.drop_none, grid, c.stream, c.after_store);
}

}  // namespace acache
