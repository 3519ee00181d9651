// q8_decode.cu -- read-slot attention over an 8-bit pool for few query rows per (request, KV head): the
// block-decode step and single tokens.  bf16 queries and outputs, head dim 64 or 128.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4.3, App. C.1 and Sec. 5 (block length
// 32); the 8-bit pool is this library's.
//
// Memory-bound: each (request, KV head) streams its keys' and values' codes once, 256 bytes a key
// (d = 128), against at most 32 packed rows (queries x heads of the group).  What limits it is how many
// bytes are in flight and what a CTA costs besides its keys.  So a warp owns 8, 16 or 32 rows and works
// alone: it brings 16 keys at a time into its own three-stage ring by cp.async, two chunks ahead of the
// one it works on, and no barrier stands between a load and its use; two to four CTAs of four warps
// to an SM.
//   * S^T = kc q', m16n8k16 f16 products of 16 keys x 8 rows.  A bf16 query row divided by a power of two so
//     that its largest element lies in [128, 256) is f16 exactly down to 2^-22 of the largest (and off by
//     at most 2^-32 of it below); codes are f16 exactly, one instruction for two.  The contraction
//     order over d is free, so a thread's 16-byte piece of a key row is its operand as it lies.
//     (m16n8k32 e4m3 products are carried out as f16 ones here, and convert both operands every time.
//     Loading the operands straight into registers, a chunk ahead, was slower than the ring: the loads
//     of one chunk waited for those of the last.  S of rows x keys wastes half of an operand on 8 rows.)
//   * O^T = V^T P^T, V's codes converted to f16 likewise.  The order of its rows (the columns of O) is
//     free too: thread group g takes the 16 bytes of columns 16 g .. 16 g + 15 of four keys, and byte j
//     of two neighbouring keys is an operand.  P^T becomes one by an 8 x 8 transposition.
//   * V's power of two goes into the exponent: P = 2^(s + ev - m) with m the running maximum of
//     s + ev, so P V is right whatever the rows' scales are, P never exceeds 2^15 and keys down to 2^-27
//     of the largest weighted one count (f16 subnormals); the sum adds P 2^-ev in float32.
// The warps of a CTA, the CTAs of a cluster (up to 8, where that fills the SMs better) share the keys; partial
// (maximum, sum, O) are merged in a fixed order through (distributed) shared memory.
//
// Measured: 8 requests x 32 rows x 4,480 keys (32 heads, d = 128) 86 us with their store, 0.21 of the rate at which the
// pool's bytes could be read: bound by the latency between the products of a chunk (32 rows take 8 warps to an SM;
// a warp waits for fixed latencies in half of its cycles, the tensor pipe is busy in 0.42 of them); 48 single tokens of
// 1 to 16,000 keys (32 heads over 8) 54 us, 0.41: the longest request's parts, 2,000 keys each, take most of that; 16 tokens
// over 4,000 keys each 26.5 us, 0.60: launch, the first loads and the merges, some 7 us, stand beside 16 us of reading.
//
// The register-operand products run at a quarter of tcgen05's rate, which few rows do not need: 128 keys
// against 16 rows are 525 cycles of an SM's matrix pipes, and reading them at the memory's rate takes
// 1400.  The tcgen05 form of this kernel (rows replicated over the 128 TMEM lanes, f16 V through shared
// memory) took 2300 cycles a tile of 128 keys, 1600 of them its M = 128 products of mostly unused rows.  (With the keys
// as the 128 rows of S^T and the query rows as its columns nothing would be unused: not built.)
#include <algorithm>
#include <atomic>

#include "q8_tc.cuh"

namespace acache {
namespace {

using namespace q8;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kChunk = 16;                  // keys a warp takes at a time
constexpr int kSt = 3;                      // chunks in a warp's ring
constexpr int kMaxCluster = 8;
// CTAs to an SM for NB groups of 8 rows to a warp (registers: 32 NB of O and what one chunk needs)
__host__ __device__ constexpr int ctas_per_sm(int NB) { return NB == 1 ? 4 : NB == 2 ? 3 : 2; }
constexpr float kPHead = 3.0f;              // P of the used maximum is 2^3 ...
constexpr float kRescaleThreshold = 12.0f;  // ... and never above 2^15
constexpr float kNoMax = -1e38f;            // maximum before any key; a key that takes no part lies below it
constexpr uint32_t kNoEv = 0xff610000u;     // bf16 -2.99e38: its ev
constexpr uint32_t kZeroEv = 0xc2480000u;   // bf16 -50: ev of a row of zeros
static_assert(kQ8MinExp == -50, "kZeroEv");

struct DecParams {
    const bf16* q;
    const uint8_t *k_cache, *v_cache, *kv_scale;
    const int32_t *read_slot, *q_start, *kv_start;
    bf16* out;
    int32_t* dev_status;
    int64_t num_slots;
    int n_q, total_q, T_len, Hq, Hkv, g;
    int cs, part;                   // CTAs per cluster; chunks per part
    int drop;
    float scale_log2;
};

// NR: rows of a warp
template <int D, int NR>
struct Smem {
    alignas(128) uint8_t q[NR * D * 2];             // query rows in f16
    union {
        alignas(128) uint8_t ring[kWarps][kSt][2][kChunk * D];      // codes of K and V, a warp's own
        alignas(16) float o[kWarps][NR * D];                        // partials
    };
    float m[kWarps][NR], l[kWarps][NR];
    float row_m[NR], row_l[NR];                     // merged over the CTA's warps
    float c_row[NR];
};

ACACHE_DEVFN void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// NR query rows -> f16, by one warp: lane i brings the element offset of row i; row i goes to `at` + i 2 D
// bytes and its factor (scale_log2 times the power of two it was divided by; NaN for a row that is not
// finite, which is carried as zeros) to c_row[i].
template <int D, int NR>
ACACHE_DEVFN void query_rows(const bf16* q, int64_t off, uint32_t at, int lane, float scale_log2, float* c_row) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, NI = NR / RPI;
    const int row = lane / LPR, pc = lane % LPR;
    uint4 w[NI];
    int64_t o[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) o[i] = __shfl_sync(0xffffffffu, off, i * RPI + row);
#pragma unroll
    for (int i = 0; i < NI; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(q + o[i]) + pc);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t top = __vmaxu2(__vmaxu2(x[0] & 0x7fff7fffu, x[1] & 0x7fff7fffu), __vmaxu2(x[2] & 0x7fff7fffu, x[3] & 0x7fff7fffu));
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int s = LPR / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
        const uint32_t E = max(top >> 7, 8u);                    // biased exponent of the row's largest
        const bool finite = E != 255u;
        const float up = __uint_as_float((261u - E) << 23);      // 2^(134 - E): largest in [128, 256)
        if (pc == 0) c_row[i * RPI + row] = finite ? scale_log2 * __uint_as_float((E - 7u) << 23) : __uint_as_float(0x7fffffffu);
        uint32_t h[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            __half2 two = __floats2half2_rn(__uint_as_float(x[y] << 16) * up, __uint_as_float(x[y] & 0xffff0000u) * up);
            h[y] = finite ? *reinterpret_cast<uint32_t*>(&two) : 0u;
        }
        // (odd rows have their 16-byte pieces exchanged in pairs: see the operand's reads)
        st_shared_v4(at + (uint32_t)((i * RPI + row) * 2 * D + (pc ^ (row & 1)) * 16), h[0], h[1], h[2], h[3]);
    }
}
ACACHE_DEVFN void ld_words(uint32_t addr, uint32_t (&r)[4]) { ld_shared_v4(addr, r); }
ACACHE_DEVFN void ld_words(uint32_t addr, uint32_t (&r)[2]) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
// Position of 16-byte piece c of row r in a chunk: a K operand is read by four lanes a row from two
// neighbouring rows at a time, a V operand by two lanes a row from every other row.
template <int D> ACACHE_DEVFN uint32_t k_piece(uint32_t r, uint32_t c) { return r * D + ((D == 128 ? c ^ ((r & 1u) << 2) : c) << 4); }
template <int D> ACACHE_DEVFN uint32_t v_piece(uint32_t r, uint32_t c) {
    return r * D + ((D == 128 ? c ^ (((r >> 1) & 3u) << 1) : c ^ ((r >> 1) & 3u)) << 4);
}
// four codes -> f16 pairs
ACACHE_DEVFN void to_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

// NB: groups of 8 rows.  The warps share the block's rows and split its keys.
template <int D, int NB>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NB))
q8_decode_kernel(const DecParams p) {
    constexpr int NR = 8 * NB;
    constexpr int H = D / 64;                        // 16-byte pieces of a key row per thread
    constexpr int NV = D / 8;                        // bytes of a value row per thread
    extern __shared__ __align__(128) uint8_t raw_smem[];
    Smem<D, NR>& sm = *reinterpret_cast<Smem<D, NR>*>(raw_smem);
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
            if (threadIdx.x == 0 && blockIdx.x == 0) flag(p.dev_status, ACACHE_DEV_BAD_LENGTH);
            return;
        }
    }
    const int n_rows = n_q * p.g;                    // <= NR
    if (n_rows == 0) return;
    const int n_ch = (T_len + kChunk - 1) / kChunk;
    const int cs = (n_ch + p.part - 1) / p.part;     // parts of this request's keys (<= p.cs)
    if (cr >= cs) return;
    const int ch0 = (int)((int64_t)cr * n_ch / cs), ch1 = (int)((int64_t)(cr + 1) * n_ch / cs);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;           // fragment coordinates

    // lanes 0-15 look after the keys of a chunk (16-31 repeat them)
    auto slot_of = [&](int ch) -> int {
        const int key = ch * kChunk + (lane & 15);
        int s = -1;
        if (ch < ch1 && key < T_len) s = p.read_slot[kbase + key];
        return s;
    };
    // slots of the chunk at hand and the two after it (the maps are not written by a store)
    int s0 = slot_of(ch0 + warp), s1 = slot_of(ch0 + warp + kWarps), s2 = slot_of(ch0 + warp + 2 * kWarps);
    {   // query rows: 8 to a warp
        constexpr int NC = 8;
        const int f0 = warp * NC;
        if (f0 < NR) {
            const int pr = f0 + (lane & (NC - 1)) < n_rows ? f0 + (lane & (NC - 1)) : 0, i = pr / p.g;
            const int64_t off = ((qbase + i) * p.Hq + (int64_t)hk * p.g + (pr - i * p.g)) * D;
            query_rows<D, NC>(p.q, off, smem_u32(&sm.q[f0 * D * 2]), lane, p.scale_log2, &sm.c_row[f0]);
        }
    }
    const uint32_t row_bytes = (uint32_t)p.Hkv * D;
    constexpr int CPR = D / 16, RPI = 32 / CPR, NI = kChunk / RPI;      // pieces a row, rows an instruction
    const uint32_t rr = (uint32_t)(lane / CPR), pc = (uint32_t)(lane % CPR);
    const uint8_t* ksrc = p.k_cache + (int64_t)hk * D + pc * 16;
    const uint8_t* vsrc = p.v_cache + (int64_t)hk * D + pc * 16;
    const uint32_t ring = smem_u32(&sm.ring[warp][0][0][0]);
    // 2^ek as bf16 with ev as bf16 above it, of this lane's key; past: it lies behind the request's last
    auto factors = [&](int slot, uint32_t sc, bool past) -> uint32_t {
        if (slot >= 0 && slot < p.num_slots) {
            const uint32_t k = sc & 0xffu, v = sc >> 8;
            const uint32_t ev = v > kQ8MaxByte ? 0x7fff0000u
                                               : __float_as_uint((float)((int)max(v, (uint32_t)(kQ8MinExp + 127)) - 127));
            return (k > kQ8MaxByte ? 0x7fffu : k << 7) | (ev & 0xffff0000u);
        }
        if (past || (p.drop && slot == ACACHE_SLOT_NONE)) return kNoEv;
        // outside the pool: a zero row that counts, with the exponent a stored one has (a larger one would raise
        // the maximum of s + ev over the rows that hold something, and their P would lose its bits)
        return 0x3f80u | kZeroEv;
    };
    auto load_scale = [&](int slot) -> uint32_t {
        uint32_t sc = 0;
        if (slot >= 0 && slot < p.num_slots) sc = reinterpret_cast<const uint16_t*>(p.kv_scale)[(int64_t)slot * p.Hkv + hk];
        return sc;
    };
    auto bring = [&](int slot, uint32_t stage) {     // all shuffles before all loads
        const int sl = (slot >= 0 && slot < p.num_slots) ? slot : -1;
        int r[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) r[i] = __shfl_sync(0xffffffffu, sl, i * RPI + rr);
#pragma unroll
        for (int i = 0; i < NI; ++i) {               // (a key without a row is zeros)
            const uint64_t at = (uint64_t)(uint32_t)max(r[i], 0) * row_bytes;
            const uint32_t bytes = r[i] >= 0 ? 16u : 0u, row = (uint32_t)(i * RPI) + rr;
            cp_async16(stage + k_piece<D>(row, pc), ksrc + at, bytes);
            cp_async16(stage + kChunk * D + v_piece<D>(row, pc), vsrc + at, bytes);
        }
    };
    grid_dependency_wait();                          // store-then-attend: the pool is written now
    bring(s0, ring);
    cp_async_commit();
    bring(s1, ring + 2 * kChunk * D);
    cp_async_commit();
    uint32_t sc0 = load_scale(s0), sc1 = load_scale(s1), sc2 = 0;
    __syncthreads();                                 // the query terms are there
    // the query operand: row g of group b, half x of the thread's piece h (NB = 4 reads it as it goes)
    auto load_q = [&](int b, int h, int x, uint32_t (&r)[4]) {
        ld_shared_v4(smem_u32(&sm.q[0]) + (uint32_t)((8 * b + g) * 2 * D + (t + 4 * h) * 32 + ((x ^ (g & 1)) * 16)), r);
    };
    constexpr bool kQRegs = NB <= 2;
    uint32_t qf[kQRegs ? NB : 1][H][2][4];
    if constexpr (kQRegs) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int x = 0; x < 2; ++x) load_q(b, h, x, qf[b][h][x]);
    }
    float c[NB][2], m[NB][2], l[NB][2];              // of rows 2t, 2t + 1 of each group
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            c[b][x] = sm.c_row[8 * b + 2 * t + x];
            m[b][x] = kNoMax;
            l[b][x] = 0.f;
        }
    // O^T: o[j][b][0..3] = columns NV g + 2 j (rows 2t, 2t + 1 of group b) and NV g + 2 j + 1 (the same rows)
    float o[NV / 2][NB][4];
#pragma unroll
    for (int j = 0; j < NV / 2; ++j)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[j][b][x] = 0.f;
    bool any = false;                                // a key of this lane's takes part
    uint32_t at = 0, at2 = 2;                        // stages of the chunk at hand and of the one to bring
    for (int ch = ch0 + warp; ch < ch1; ch += kWarps) {
        bring(s2, ring + at2 * (2 * kChunk * D));
        cp_async_commit();
        sc2 = load_scale(s2);
        const bool past = ch * kChunk + (lane & 15) >= T_len;
        const uint32_t fe_own = factors(s0, sc0, past);
        any = any || fe_own != kNoEv;
        if (!past && (s0 < 0 || s0 >= p.num_slots) && !(p.drop && s0 == ACACHE_SLOT_NONE))
            flag(p.dev_status, ACACHE_DEV_BAD_SLOT);
        s0 = s1;
        s1 = s2;
        sc0 = sc1;
        sc1 = sc2;
        s2 = slot_of(ch + 3 * kWarps);
        uint32_t fe[2];                              // of keys g and g + 8
#pragma unroll
        for (int x = 0; x < 2; ++x) fe[x] = __shfl_sync(0xffffffffu, fe_own, g + 8 * x);
        cp_async_wait<2>();
        __syncwarp();
        const uint32_t kat = ring + at * (2 * kChunk * D), vat = kat + kChunk * D;
        at2 = at;
        at = at == kSt - 1 ? 0 : at + 1;
        constexpr int CH = NB == 1 ? 4 : NB == 2 ? 2 : 1;      // chains of products per result: four in all
        float s[NB][CH][4];
#pragma unroll
        for (int i = 0; i < NB * CH * 4; ++i) s[i / (CH * 4)][i / 4 % CH][i % 4] = 0.f;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            uint32_t kf[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) ld_shared_v4(kat + k_piece<D>((uint32_t)(8 * n + g), (uint32_t)(t + 4 * h)), kf[n]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t a[2][4], qr[NB][4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {        // four elements of the piece to a product
                    to_f16(kf[0][2 * x + y], a[y][0], a[y][2]);
                    to_f16(kf[1][2 * x + y], a[y][1], a[y][3]);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (!kQRegs) {
                        load_q(b, h, x, qr[b]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) qr[b][i] = qf[b][h][x][i];
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        mma_f16(s[b][(2 * x + y) % CH], a[y][0], a[y][1], a[y][2], a[y][3], qr[b][2 * y], qr[b][2 * y + 1]);
                }
            }
        }
        uint32_t vf[4][NV / 4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t key = (uint32_t)(2 * t + (x & 1) + 8 * (x >> 1));
            ld_words(vat + (D == 128 ? v_piece<D>(key, (uint32_t)g) : v_piece<D>(key, (uint32_t)g >> 1) + 8u * (g & 1)), vf[x]);
        }
        // u = s + ev in log2 units, u[b][2 k + x]: key g + 8 k, row 2t + x of group b
        float ev[2], rv[2], u[NB][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float fk = __uint_as_float(fe[k] << 16);
            ev[k] = __uint_as_float(fe[k] & 0xffff0000u);
            rv[k] = fast_exp2(fminf(-ev[k], 126.f));             // (finite where the key takes no part)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float d = s[b][0][2 * k + x];
#pragma unroll
                    for (int i = 1; i < CH; ++i) d += s[b][i][2 * k + x];
                    u[b][2 * k + x] = fmaf(d * fk, c[b][x], ev[k]);
                }
        }
        bool grow = false;                           // (a maximum that is NaN -- every key of the row so far -- is left alone)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int x = 0; x < 2; ++x) grow = grow || fmaxf(u[b][x], u[b][2 + x]) > m[b][x] + kRescaleThreshold;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float al[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float top = fmaxf(u[b][x], u[b][2 + x]);
#pragma unroll
                    for (int i = 4; i < 32; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));   // over the chunk's keys
                    const float mn = top > m[b][x] + kRescaleThreshold ? top : m[b][x];
                    al[x] = fast_exp2(m[b][x] - mn);
                    l[b][x] *= al[x];
                    m[b][x] = mn;
                }
#pragma unroll
                for (int j = 0; j < NV / 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[j][b][i] *= al[i & 1];
            }
        }
        uint32_t pb[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float pr[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    pr[x] = fast_exp2(u[b][2 * k + x] - (m[b][x] - kPHead));
                    l[b][x] = fmaf(pr[x], rv[k], l[b][x]);
                }
                // f16 keeps 11 bits, so P is rounded finer than bf16 would
                const __half2 w = __floats2half2_rn(pr[0], pr[1]);
                asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pb[b][k]) : "r"(*reinterpret_cast<const uint32_t*>(&w)));
            }
#pragma unroll
        for (int y = 0; y < NV / 4; ++y) {
            // bytes 4y .. 4y + 3 of the four keys, two keys to an operand
            uint32_t a[4][2];
            to_f16(__byte_perm(vf[0][y], vf[1][y], 0x5140), a[0][0], a[1][0]);
            to_f16(__byte_perm(vf[0][y], vf[1][y], 0x7362), a[2][0], a[3][0]);
            to_f16(__byte_perm(vf[2][y], vf[3][y], 0x5140), a[0][1], a[1][1]);
            to_f16(__byte_perm(vf[2][y], vf[3][y], 0x7362), a[2][1], a[3][1]);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    mma_f16(o[2 * y + x][b], a[2 * x][0], a[2 * x + 1][0], a[2 * x][1], a[2 * x + 1][1], pb[b][0], pb[b][1]);
        }
        __syncwarp();                                // the next chunk but two lands in this stage
    }
    cp_async_wait<0>();
    any = __any_sync(0xffffffffu, any);
    __syncthreads();                                 // the partials go over the rings
    // -------------------------------------------------------------------------- merge
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) l[b][x] += __shfl_xor_sync(0xffffffffu, l[b][x], i);
            if (g == 0) {
                sm.m[warp][8 * b + 2 * t + x] = m[b][x];
                sm.l[warp][8 * b + 2 * t + x] = any ? l[b][x] : 0.f;   // (a row that is not finite: NaN even so)
            }
        }
    // float4 slot of a row, moved by row and by thread group so that the lanes spread over the banks
    auto slot4 = [&](int r, int q4) { return r * D + 4 * (((q4 ^ (q4 / (NV / 4) & (NV / 4 - 1))) + (r & 7) * 2) & (D / 4 - 1)); };
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x)                  // row 2t + x of group b, columns NV g ...
#pragma unroll
            for (int j = 0; j < NV / 4; ++j)
                *reinterpret_cast<float4*>(&sm.o[warp][slot4(8 * b + 2 * t + x, g * (NV / 4) + j)]) =
                    make_float4(o[2 * j][b][x], o[2 * j][b][2 + x], o[2 * j + 1][b][x], o[2 * j + 1][b][2 + x]);
    __syncthreads();
    // First the warps, a thread taking 4 columns of a row.
    const bool split = cs > 1;
    for (int it = (int)threadIdx.x; it < n_rows * (D / 4); it += kThreads) {
        const int r = it / (D / 4), q4 = it % (D / 4);
        float m[kWarps], M = kNoMax;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            m[x] = sm.m[x][r];
            M = fmaxf(M, m[x]);
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float lv = sm.l[x][r];
            if (lv == 0.f) continue;                             // no key in this partial
            const float e = fast_exp2(m[x] - M);
            const float4 f = *reinterpret_cast<const float4*>(&sm.o[x][slot4(r, q4)]);
            L = fmaf(e, lv, L);
            acc.x = fmaf(e, f.x, acc.x);
            acc.y = fmaf(e, f.y, acc.y);
            acc.z = fmaf(e, f.z, acc.z);
            acc.w = fmaf(e, f.w, acc.w);
        }
        if (split) {
            if (q4 == 0) {
                sm.row_m[r] = M;
                sm.row_l[r] = L;
            }
            *reinterpret_cast<float4*>(&sm.o[0][slot4(r, q4)]) = acc;      // (only this thread reads or writes it)
        } else {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int i = r / p.g;
            bf16* dst = p.out + ((qbase + i) * p.Hq + (int64_t)hk * p.g + (r - i * p.g)) * D + q4 * 4;
            __nv_bfloat162 a2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<uint32_t*>(&a2), *reinterpret_cast<uint32_t*>(&b2));
        }
    }
    if (!split) return;
    // Then the parts: a warp finalises 32 neighbouring (row, 4-column) items at a time, so that a load takes whole
    // lines of the other SM's shared memory.
    __syncwarp();
    cluster_sync();
    const uint32_t m_a = smem_u32(&sm.row_m[0]), l_a = smem_u32(&sm.row_l[0]);
    for (int it = 32 * (cr + cs * warp) + lane; it < n_rows * (D / 4); it += cs * kThreads) {
        const int r = it / (D / 4), q4 = it % (D / 4);
        const uint32_t at = smem_u32(&sm.o[0][slot4(r, q4)]);
        float m[kMaxCluster], l[kMaxCluster], M = kNoMax;
        float4 f[kMaxCluster];
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) {
            m[x] = kNoMax;
            l[x] = 0.f;
            f[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x < cs) {
                m[x] = ld_cluster_f32(mapa_shared(m_a + 4u * r, x));
                l[x] = ld_cluster_f32(mapa_shared(l_a + 4u * r, x));
                f[x] = ld_cluster_v4(mapa_shared(at, x));
            }
        }
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) M = fmaxf(M, m[x]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) {
            // (no key in this part: nothing to add; but every value loaded is used, so none is still on its way when
            // the ranks part)
            const bool none = l[x] == 0.f;
            const float e = fast_exp2(m[x] - M);
            L = none ? L : fmaf(e, l[x], L);
            acc.x = none ? acc.x : fmaf(e, f[x].x, acc.x);
            acc.y = none ? acc.y : fmaf(e, f[x].y, acc.y);
            acc.z = none ? acc.z : fmaf(e, f[x].z, acc.z);
            acc.w = none ? acc.w : fmaf(e, f[x].w, acc.w);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int i = r / p.g;
        bf16* dst = p.out + ((qbase + i) * p.Hq + (int64_t)hk * p.g + (r - i * p.g)) * D + q4 * 4;
        __nv_bfloat162 a2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<uint32_t*>(&a2), *reinterpret_cast<uint32_t*>(&b2));
    }
    __syncwarp();
    cluster_sync();                // no CTA may leave while another still reads its shared memory
}

std::atomic<int> g_prepared[6][64];   // the kernel's shared memory is allowed for, per device and variant

template <int D, int NB>
int launch(const DecParams& prm, dim3 grid, cudaStream_t stream, bool pdl) {
    auto kern = q8_decode_kernel<D, NB>;
    constexpr int smem = (int)sizeof(Smem<D, 8 * NB>);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    std::atomic<int>& st = g_prepared[(D == 128 ? 3 : 0) + NB / 2][dev];
    if (!st.load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
            (void)cudaGetLastError();
            return ACACHE_ERR_CUDA;
        }
        st.store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
int dispatch(const DecParams& prm, int rows, dim3 grid, cudaStream_t stream, bool pdl) {
    if (rows <= 8) return launch<D, 1>(prm, grid, stream, pdl);
    if (rows <= 16) return launch<D, 2>(prm, grid, stream, pdl);
    return launch<D, 4>(prm, grid, stream, pdl);
}

}  // namespace

// 64 rows in two such groups took longer than the tcgen05 kernel except for the shortest calls: 8 requests x 64
// rows x 4480 keys (32 heads) 162 us against 118, 64 x 16000 (8 heads) 64 against 38, 64 x 500 (4 heads) 15 against 19.
bool q8_decode_supported(const AttnArgs& a, int n_q) {
    return q8_tc_supported(a) && (int64_t)n_q * (a.hq / a.hkv) <= 32;
}

int launch_q8_decode_attention(const Q8Attn& c) {
    const int d = c.a.d, hkv = c.a.hkv, g = c.a.hq / hkv;
    DecParams prm{};
    prm.q = (const bf16*)c.q;
    prm.k_cache = c.k_cache;
    prm.v_cache = c.v_cache;
    prm.kv_scale = c.kv_scale;
    prm.read_slot = c.read_slot;
    prm.q_start = c.q_start;
    prm.kv_start = c.kv_start;
    prm.out = (bf16*)c.out;
    prm.dev_status = c.dev_status;
    prm.num_slots = c.num_slots;
    prm.n_q = c.n_q;
    prm.total_q = c.total_q;
    prm.T_len = c.T_len;
    prm.Hq = c.a.hq;
    prm.Hkv = hkv;
    prm.g = g;
    prm.drop = c.drop_none;
    prm.scale_log2 = c.a.scale * kLog2e;
    // Parts of the key range, in chunks of a warp: kFix is what a CTA costs besides its keys, kMerge a merge
    // over the cluster.  A fixed batch runs in waves of equal CTAs.  Of a ragged batch the host knows the
    // longest request only: parts until that one no longer outlasts the others, taken as an eighth as
    // long.
    constexpr int kFix = 6, kMerge = 2;
    const int rows = c.n_q * g;
    const int n_ch = (c.T_len + kChunk - 1) / kChunk;
    const int64_t units = (int64_t)c.B * hkv, slots = (int64_t)sm_count() * ctas_per_sm(rows <= 8 ? 1 : rows <= 16 ? 2 : 4);
    prm.cs = 1;
    int64_t best = 0;
    for (int cs = 1; cs <= kMaxCluster && cs <= n_ch; ++cs) {
        const int64_t per = (n_ch + cs * kWarps - 1) / (cs * kWarps) + kFix + (cs > 1 ? kMerge : 0);
        int64_t est = ((units * cs + slots - 1) / slots) * per;
        if (c.q_start) est = std::max(per, (units * (n_ch / (8 * kWarps) + kFix + (cs > 1 ? kMerge : 0)) + slots - 1) / slots);
        if (cs == 1 || est < best) {
            best = est;
            prm.cs = cs;
        }
    }
    prm.part = (n_ch + prm.cs - 1) / prm.cs;
    const dim3 grid((unsigned)(hkv * prm.cs), (unsigned)c.B, 1);
    return d == 128 ? dispatch<128>(prm, rows, grid, c.stream, c.after_store)
                    : dispatch<64>(prm, rows, grid, c.stream, c.after_store);
}

}  // namespace acache
