// masked_decode.cu -- read-slot attention under a mask for few query rows per (request, KV head): single tokens
// and short blocks.  bf16, head dim 64 or 128, a positive scale, at most 32 rows (queries x heads of a group).
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4.3, App. C.1 and Sec. 5 (block decoding); the masks are
// this library's (include/acache.h, acache_slot_attention_masked).
//
// Memory-bound: a (request, KV head) streams the keys and values of its window (from the first key that one of
// its rows sees to the last) once, 512 bytes a key at d = 128, against 8, 16 or 32 rows.  Every warp works alone: it brings
// 16 keys at a time into its own three-stage ring by cp.async, two chunks ahead, with no barrier between a
// load and its use; the warps of a CTA and the CTAs of a cluster share the window's chunks.
//   * S^T = K q', m16n8k16 products of 16 keys x 8 rows.  The contraction order over d is free, so a thread's 16-byte
//     piece of a key row is its operand as it lies.
//   * O^T = V^T P^T: V by transposing matrix loads, P^T by an 8 x 8 transposition in registers.
// Partial (maximum, sum, O) are merged in a fixed order through (distributed) shared memory.  A masked key's score
// is replaced by -infinity; a row that met a masked V which is not finite is computed again over its own keys.
//
// Measured: 8 single tokens over windows of 4,096 of 8,000 keys (32 heads over 8, capped) 29.7 us on the device, 0.67 of the copy
// bandwidth: 64 units in 4 parts fill 0.84 of the 304 places for a CTA, and launch, the chain range -> slot ->
// row and the merges take some 7 us; 16 over 4,000 keys 50.5 us, 0.76; one over 8,000 14.3 us in 16 parts (21.5 in 8); a decode
// block of 4 x 32 rows over 4,480 keys (32 heads over 32) 80.6 us, 0.54.  Two warps to a CTA and four CTAs to an SM: the same for
// these, 38 us for the one token.
#include <algorithm>
#include <atomic>

#include "masked.cuh"
#include "ptx.cuh"
#include "q8.cuh"
#include "step.cuh"

namespace acache {
namespace {

using namespace ptx;
using bf16 = __nv_bfloat16;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kChunk = 16;                  // keys a warp takes at a time
constexpr int kSt = 3;                      // chunks in a warp's ring
constexpr int kMaxCluster = 16;             // (above 8: not on every GPU, but on the one this is for)
constexpr int kCtasPerSm = 2;
constexpr float kRescaleThreshold = 8.0f;   // log2 units: weights stay below 2^8

struct DecParams {
    const bf16 *q, *k_cache, *v_cache;
    bf16* out;
    const int32_t *read_slot, *q_start, *kv_start, *row_range, *q_pos;
    const float* slopes;
    int32_t* dev_status;
    int64_t num_slots;
    int n_q, total_q, T_len, Hq, Hkv, g, cs, drop, wide;
    float scale_log2, cap_in, cap_log2;     // cap_in = 0: no cap
};

template <int D, int NR>
struct Smem {
    static constexpr int kRow = D + 4;      // floats of a partial row: the lanes of a store spread over the banks
    alignas(128) uint8_t q[NR * D * 2];
    union {
        alignas(128) uint8_t ring[kWarps][kSt][2][kChunk * D * 2];
        alignas(16) float o[kWarps][NR * kRow];
    };
    float m[kWarps][NR], l[kWarps][NR];
    float row_m[NR], row_l[NR];             // merged over the CTA's warps
    int lo[NR], hi[NR];                     // keys of a row, from the window's start
    float slope[NR];                        // in log2 units
    int64_t pos[NR];
    int win[2];
};

ACACHE_DEVFN void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
ACACHE_DEVFN void ld4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
ACACHE_DEVFN void ldmatrix_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Byte of 16-byte piece c of row r in a chunk: a K operand is read by four lanes a row from two neighbouring rows at
// a time, a V operand one piece from eight rows.
template <int D> ACACHE_DEVFN uint32_t k_piece(uint32_t r, uint32_t c) { return r * (2 * D) + ((c ^ ((r & 1u) << 2)) << 4); }
template <int D> ACACHE_DEVFN uint32_t v_piece(uint32_t r, uint32_t c) { return r * (2 * D) + ((c ^ (r & 7u)) << 4); }

// NB: groups of 8 rows.
template <int D, int NB>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
masked_decode_kernel(const DecParams p) {
    constexpr int NR = 8 * NB, H = D / 32;          // H: pieces of a key row per thread
    extern __shared__ __align__(128) uint8_t raw_smem[];
    using S = Smem<D, NR>;
    S& sm = *reinterpret_cast<S*>(raw_smem);
    const int cs = p.cs;
    const int cr = cs == 1 ? 0 : (int)(blockIdx.x % (unsigned)cs);
    const int hk = cs == 1 ? (int)blockIdx.x : (int)(blockIdx.x / (unsigned)cs);
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;           // fragment coordinates
    if (warp == 0) {                                 // lane i: row i
        int lo = 0, hi = 0;
        const int i = lane / p.g;
        if (lane < n_rows) {
            hi = T_len;
            if (p.row_range) {
                lo = max(p.row_range[2 * (qbase + i)], 0);
                hi = min(p.row_range[2 * (qbase + i) + 1], T_len);
            }
            if (lo >= hi) lo = hi = 0;
        }
        const int a = __reduce_min_sync(0xffffffffu, lo < hi ? lo : 0x7fffffff), z = __reduce_max_sync(0xffffffffu, hi);
        const int w = z > 0 ? a : 0;
        if (lane == 0) {
            sm.win[0] = w;
            sm.win[1] = z;
        }
        if (lane < NR) {
            sm.lo[lane] = lo - w;
            sm.hi[lane] = hi - w;
            const bool biased = p.slopes && lane < n_rows;
            sm.slope[lane] = biased ? p.slopes[hk * p.g + lane % p.g] * kLog2e : 0.f;
            sm.pos[lane] = biased ? (int64_t)p.q_pos[qbase + i] - w : 0;
        }
    }
    // query rows, 16 bytes a thread at a time (rows that are none: zeros); odd rows have their pieces exchanged in pairs
    for (int x = threadIdx.x; x < NR * (D / 8); x += kThreads) {
        const int row = x / (D / 8), pc = x % (D / 8);
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (row < n_rows) {
            const int i = row / p.g;
            w = __ldg(reinterpret_cast<const uint4*>(p.q + ((qbase + i) * p.Hq + (int64_t)hk * p.g + (row - i * p.g)) * D) + pc);
        }
        *reinterpret_cast<uint4*>(&sm.q[k_piece<D>((uint32_t)row, (uint32_t)pc)]) = w;
    }
    __syncthreads();
    const int w_lo = sm.win[0], T_win = sm.win[1] - w_lo;
    const int n_ch = (T_win + kChunk - 1) / kChunk;
    const int ch0 = (int)((int64_t)cr * n_ch / cs), ch1 = (int)((int64_t)(cr + 1) * n_ch / cs);
    const int32_t* rs = p.read_slot + kbase + w_lo;
    // lanes 0-15 look after the keys of a chunk (16-31 repeat them); -1: none, or a discarded key; -2: outside the pool
    auto slot_of = [&](int ch) -> int {
        const int key = ch * kChunk + (lane & 15);
        int s = -1;
        if (ch < ch1 && key < T_win) {
            s = rs[key];
            if (s < 0 || s >= p.num_slots) {
                const bool dropped = p.drop && s == ACACHE_SLOT_NONE;
                if (!dropped) flag(p.dev_status, ACACHE_DEV_BAD_SLOT);
                s = dropped ? -1 : -2;
            }
        }
        return s;
    };
    const uint64_t row_bytes = (uint64_t)p.Hkv * D * 2;
    constexpr int CPR = D / 8, RPI = 32 / CPR, NI = kChunk / RPI;      // pieces a row, rows an instruction
    const uint32_t rr = (uint32_t)(lane / CPR), pc = (uint32_t)(lane % CPR);
    const uint8_t* ksrc = reinterpret_cast<const uint8_t*>(p.k_cache + (int64_t)hk * D) + pc * 16;
    const uint8_t* vsrc = reinterpret_cast<const uint8_t*>(p.v_cache + (int64_t)hk * D) + pc * 16;
    const uint32_t ring = smem_u32(&sm.ring[warp][0][0][0]);
    constexpr uint32_t kMat = kChunk * D * 2;
    auto bring = [&](int slot, uint32_t stage) {     // all shuffles before all loads
        int r[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) r[i] = __shfl_sync(0xffffffffu, slot, i * RPI + rr);
#pragma unroll
        for (int i = 0; i < NI; ++i) {               // (a key without a row is zeros)
            const uint64_t at = (uint64_t)(uint32_t)max(r[i], 0) * row_bytes;
            const uint32_t bytes = r[i] >= 0 ? 16u : 0u, row = (uint32_t)(i * RPI) + rr;
            cp_async16(stage + k_piece<D>(row, pc), ksrc + at, bytes);
            cp_async16(stage + kMat + v_piece<D>(row, pc), vsrc + at, bytes);
        }
    };
    int s0 = slot_of(ch0 + warp), s1 = slot_of(ch0 + warp + kWarps), s2 = slot_of(ch0 + warp + 2 * kWarps);
    bring(s0, ring);
    cp_async_commit();
    bring(s1, ring + 2 * kMat);
    cp_async_commit();
    // the query operand: row g of group b, the thread's piece h
    auto load_q = [&](int b, int h, uint32_t (&r)[4]) {
        ld4(smem_u32(&sm.q[0]) + k_piece<D>((uint32_t)(8 * b + g), (uint32_t)(t + 4 * h)), r);
    };
    constexpr bool kQRegs = NB == 1;
    uint32_t qf[kQRegs ? NB : 1][H][4];
    if constexpr (kQRegs) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < H; ++h) load_q(b, h, qf[b][h]);
    }
    // of rows 2 t, 2 t + 1 of each group: running maximum and sum, and the keys they see
    float m[NB][2], l[NB][2];
    int lo[NB][2], hi[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            m[b][x] = -INFINITY;
            l[b][x] = 0.f;
            lo[b][x] = sm.lo[8 * b + 2 * t + x];
            hi[b][x] = sm.hi[8 * b + 2 * t + x];
        }
    // O^T: o[j][b] = columns 16 j + g (rows 2 t, 2 t + 1 of group b) and 16 j + g + 8 (the same rows)
    float o[D / 16][NB][4];
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[j][b][x] = 0.f;
    uint32_t saw = 0;                                // bit 2 b + x: row 2 t + x of group b sees a key
    uint32_t at = 0, at2 = 2;                        // stages of the chunk at hand and of the one to bring
    for (int ch = ch0 + warp; ch < ch1; ch += kWarps) {
        bring(s2, ring + at2 * (2 * kMat));
        cp_async_commit();
        const bool there = s0 != -1;
        const uint32_t have = __ballot_sync(0xffffffffu, there);
        s0 = s1;
        s1 = s2;
        s2 = slot_of(ch + 3 * kWarps);
        cp_async_wait<2>();
        __syncwarp();
        const uint32_t kat = ring + at * (2 * kMat), vat = kat + kMat;
        at2 = at;
        at = at == kSt - 1 ? 0 : at + 1;
        constexpr int CH = NB == 1 ? 4 : NB == 2 ? 2 : 1;      // chains of products per result
        float s[NB][CH][4];
#pragma unroll
        for (int i = 0; i < NB * CH * 4; ++i) s[i / (CH * 4)][i / 4 % CH][i % 4] = 0.f;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            uint32_t kf[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) ld4(kat + k_piece<D>((uint32_t)(8 * n + g), (uint32_t)(t + 4 * h)), kf[n]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t qr[4];
                if constexpr (kQRegs) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) qr[i] = qf[b][h][i];
                } else {
                    load_q(b, h, qr);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y)          // four elements of the piece to a product
                    mma_bf16(s[b][(2 * h + y) % CH], kf[0][2 * y], kf[1][2 * y], kf[0][2 * y + 1], kf[1][2 * y + 1], qr[2 * y], qr[2 * y + 1]);
            }
        }
        // u[b][2 k + x]: key g + 8 k, row 2 t + x of group b, in log2 units
        float u[NB][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int key = ch * kChunk + g + 8 * k;
            const bool in = (have >> (g + 8 * k)) & 1u;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float d = s[b][0][2 * k + x];
#pragma unroll
                    for (int i = 1; i < CH; ++i) d += s[b][i][2 * k + x];
                    float y = p.cap_in > 0.f ? (p.wide ? capped_wide(d, p.cap_in, p.cap_log2, p.scale_log2) : capped(d, p.cap_in, p.cap_log2)) : d * p.scale_log2;
                    if (p.slopes) y = fmaf(-sm.slope[8 * b + 2 * t + x], fabsf((float)(sm.pos[8 * b + 2 * t + x] - key)), y);
                    const bool see = in && key >= lo[b][x] && key < hi[b][x];
                    saw |= (uint32_t)see << (2 * b + x);
                    u[b][2 * k + x] = see ? y : -INFINITY;
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
                    const bool up = top > m[b][x] + kRescaleThreshold;
                    al[x] = up ? fast_exp2(m[b][x] - top) : 1.f;
                    l[b][x] *= al[x];
                    if (up) m[b][x] = top;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[j][b][i] *= al[i & 1];
            }
        }
        uint32_t pb[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float ms[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) ms[x] = m[b][x] == -INFINITY ? 0.f : m[b][x];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float pr[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    pr[x] = fast_exp2(u[b][2 * k + x] - ms[x]);
                    l[b][x] += pr[x];
                }
                // the weights' one rounding: bf16, the type of V (the sum takes them unrounded)
                const __nv_bfloat162 w = __floats2bfloat162_rn(pr[0], pr[1]);
                asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pb[b][k]) : "r"(*reinterpret_cast<const uint32_t*>(&w)));
            }
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            // matrices of 8 keys x 8 columns: (keys 0-7, columns 16 j), (0-7, + 8), (8-15, 16 j), (8-15, + 8), transposed
            uint32_t a[4];
            const uint32_t key = (uint32_t)((lane & 7) + 8 * (lane >> 4)), col = (uint32_t)(2 * j + ((lane >> 3) & 1));
            ldmatrix_trans(vat + v_piece<D>(key, col), a);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma_bf16(o[j][b], a[0], a[1], a[2], a[3], pb[b][0], pb[b][1]);
        }
        __syncwarp();                                // the next chunk but two lands in this stage
    }
    cp_async_wait<0>();
    // The maximum of a row that sees no key stays -infinity; of one that sees some, be their scores all -infinity (then its
    // sum of 0 makes it 0 / 0), it is a number.
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) saw |= __shfl_xor_sync(0xffffffffu, saw, i);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if ((saw >> (2 * b + x)) & 1u) m[b][x] = fmaxf(m[b][x], -3.4e38f);
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
                sm.l[warp][8 * b + 2 * t + x] = l[b][x];
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    sm.o[warp][(8 * b + 2 * t + x) * S::kRow + 16 * j + 8 * y + g] = o[j][b][2 * y + x];
        }
    __syncthreads();
    // A merged row's 4 columns at a time; a warp takes 32 neighbouring items.  Rows whose output is not finite while their sum
    // is are computed again.
    auto finish = [&](int it, bool in, const float4& acc, float M, float L) {
        const int r = in ? it / (D / 4) : 0, q4 = it % (D / 4), i = r / p.g;
        const int64_t row_at = ((qbase + i) * p.Hq + (int64_t)hk * p.g + (r - i * p.g)) * D;
        const float inv = 1.f / L;
        const bool none = M == -INFINITY;            // no key: zeros
        const float y0 = none ? 0.f : acc.x * inv, y1 = none ? 0.f : acc.y * inv, y2 = none ? 0.f : acc.z * inv, y3 = none ? 0.f : acc.w * inv;
        const float chk = fmaf(y0, 0.f, fmaf(y1, 0.f, fmaf(y2, 0.f, y3 * 0.f)));
        if (in) {
            __nv_bfloat162 a2 = __floats2bfloat162_rn(y0, y1), b2 = __floats2bfloat162_rn(y2, y3);
            *reinterpret_cast<uint2*>(p.out + row_at + q4 * 4) = make_uint2(*reinterpret_cast<uint32_t*>(&a2), *reinterpret_cast<uint32_t*>(&b2));
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, in && chk != chk && L == L);
        if (bad) {
            __syncwarp();
#pragma unroll 1
            for (int part = 0; part < 32; part += D / 4) {
                if (!((bad >> part) & (D == 128 ? 0xffffffffu : 0xffffu))) continue;
                const int rw = __shfl_sync(0xffffffffu, r, part);
                const int64_t ra = __shfl_sync(0xffffffffu, row_at, part);
                masked_row<bf16, D>(MaskedPool<bf16>{p.k_cache, p.v_cache, rs, p.num_slots, p.Hkv, p.drop, p.wide != 0, p.scale_log2, p.cap_in, p.cap_log2, 0.f},
                              p.q + ra, p.out + ra, sm.lo[rw], sm.hi[rw], hk, sm.slope[rw], sm.pos[rw], lane);
            }
        }
    };
    // First the warps of the CTA.
    const bool split = cs > 1;
    for (int it0 = 32 * warp; it0 < n_rows * (D / 4); it0 += kThreads) {
        const int it = it0 + lane;
        const bool in = it < n_rows * (D / 4);
        const int r = in ? it / (D / 4) : 0, q4 = it % (D / 4);
        float mw[kWarps], M = -INFINITY;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            mw[x] = sm.m[x][r];
            M = fmaxf(M, mw[x]);
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float lv = sm.l[x][r];
            if (lv == 0.f) continue;                             // no key in this partial
            const float e = fast_exp2(mw[x] - M);
            const float4 f = *reinterpret_cast<const float4*>(&sm.o[x][r * S::kRow + 4 * q4]);
            L = fmaf(e, lv, L);
            acc.x = fmaf(e, f.x, acc.x);
            acc.y = fmaf(e, f.y, acc.y);
            acc.z = fmaf(e, f.z, acc.z);
            acc.w = fmaf(e, f.w, acc.w);
        }
        if (!split) {
            finish(it, in, acc, M, L);
        } else if (in) {
            if (q4 == 0) {
                sm.row_m[r] = M;
                sm.row_l[r] = L;
            }
            *reinterpret_cast<float4*>(&sm.o[0][r * S::kRow + 4 * q4]) = acc;      // (only this thread reads or writes it)
        }
    }
    if (!split) return;
    // Then the parts: a load takes whole lines of the other SM's shared memory.
    cluster_sync();
    const uint32_t m_a = smem_u32(&sm.row_m[0]), l_a = smem_u32(&sm.row_l[0]);
    for (int it0 = 32 * (cr + cs * warp); it0 < n_rows * (D / 4); it0 += cs * kThreads) {
        const int it = it0 + lane;
        const bool in = it < n_rows * (D / 4);
        const int r = in ? it / (D / 4) : 0, q4 = it % (D / 4);
        const uint32_t at4 = smem_u32(&sm.o[0][r * S::kRow + 4 * q4]);
        float mc[kMaxCluster], lc[kMaxCluster], M = -INFINITY;
        float4 f[kMaxCluster];
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) {
            mc[x] = -INFINITY;
            lc[x] = 0.f;
            f[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x < cs) {
                mc[x] = ld_cluster_f32(mapa_shared(m_a + 4u * r, x));
                lc[x] = ld_cluster_f32(mapa_shared(l_a + 4u * r, x));
                f[x] = ld_cluster_v4(mapa_shared(at4, x));
            }
        }
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) M = fmaxf(M, mc[x]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int x = 0; x < kMaxCluster; ++x) {
            // (no key in this part: nothing to add; but every value loaded is used, so none is still on its way when
            // the ranks part)
            const bool none = lc[x] == 0.f;
            const float e = fast_exp2(mc[x] - M);
            L = none ? L : fmaf(e, lc[x], L);
            acc.x = none ? acc.x : fmaf(e, f[x].x, acc.x);
            acc.y = none ? acc.y : fmaf(e, f[x].y, acc.y);
            acc.z = none ? acc.z : fmaf(e, f[x].z, acc.z);
            acc.w = none ? acc.w : fmaf(e, f[x].w, acc.w);
        }
        finish(it, in, acc, M, L);
    }
    cluster_sync();                // no CTA may leave while another still reads its shared memory
}

std::atomic<int> g_clusters[6][kMaxCluster + 1][64];   // per variant, size and device: 1 + the clusters that run at once

// Clusters of `cs` CTAs of a variant that the device holds at once.  A cluster stays within a group of SMs, whose places the
// larger sizes leave unused (of 304: 296 in use at 4 to a cluster, 288 at 8, 247 at 13, 196 at 14); 0: the size cannot be launched.
template <int D, int NB>
int clusters_at_once(cudaLaunchConfig_t cfg, cudaLaunchAttribute attr, int cs, int dev) {
    std::atomic<int>& known = g_clusters[(D == 128 ? 3 : 0) + NB / 2][cs][dev];
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
        cfg.gridDim = dim3((unsigned)cs);
        attr.val.clusterDim.x = (unsigned)cs;
        cfg.attrs = &attr;
        if (cudaOccupancyMaxActiveClusters(&n, masked_decode_kernel<D, NB>, &cfg) != cudaSuccess || n < 0) {
            (void)cudaGetLastError();
            n = 0;
        }
        known.store(++n, std::memory_order_relaxed);
    }
    return n - 1;
}

template <int D, int NB>
int launch(DecParams prm, const MaskedAttn& c) {
    auto kern = masked_decode_kernel<D, NB>;
    constexpr int smem = (int)sizeof(Smem<D, 8 * NB>);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    static std::atomic<int> prepared[64];             // the kernel's shared memory and clusters are allowed for, per device
    if (!prepared[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            (void)cudaGetLastError();
            return ACACHE_ERR_CUDA;
        }
        prepared[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // Parts of the key range, in chunks of a warp: kFix is what a CTA costs besides its keys, kMerge a merge
    // over the cluster.  A fixed batch runs in waves of as many clusters as run at once.  Of a ragged batch the host knows
    // the longest request only: its time, or that of the waves of all of them with an eighth of its keys each, whichever is
    // longer.  us, single tokens of 32 heads over 8, as chosen here and with the best and the worst of 1 to 16 parts.  Lengths
    // even over their logarithm: 16 requests up to 2,000 keys 16.7 (16.7, 54.7), up to 8,000 34.7 (34.7, 143), 32 up to 8,000
    // 68.9 (68.9, 144).  Even up to 8,000: 16 requests 81.9 (78.4, 147).  All 8,000: 4 requests 42.2 (30.1, 144), 16 107 (96.3, 163).
    // All but one short: 32 requests up to 16,000 keys 77.6 (51.6, 282), the furthest that was found.
    constexpr int kFix = 6, kMerge = 2;
    const int n_ch = (c.T_len + kChunk - 1) / kChunk;
    const int64_t units = (int64_t)c.B * prm.Hkv;
    prm.cs = 1;
    int64_t best = 0;
    for (int cs = 1; cs <= kMaxCluster && cs <= n_ch; ++cs) {
        int64_t clusters = clusters_at_once<D, NB>(cfg, attr[0], cs, dev);
        if (clusters == 0) {
            if (cs > 1) continue;
            clusters = (int64_t)sm_count() * kCtasPerSm;
        }
        const int64_t waves = (units + clusters - 1) / clusters;
        auto takes = [&](int64_t chunks) { return (chunks + cs * kWarps - 1) / (cs * kWarps) + kFix + (cs > 1 ? kMerge : 0); };
        const int64_t est = c.q_start ? std::max(takes(n_ch), waves * takes(n_ch / 8)) : waves * takes(n_ch);
        if (cs == 1 || est < best) {
            best = est;
            prm.cs = cs;
        }
    }
    cfg.gridDim = dim3((unsigned)(prm.Hkv * prm.cs), (unsigned)c.B, 1);
    attr[0].val.clusterDim.x = (unsigned)prm.cs;
    cfg.numAttrs = prm.cs > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, prm) != cudaSuccess) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    return launch_status();
}

template <int D>
int dispatch(const DecParams& prm, const MaskedAttn& c) {
    const int rows = c.n_q * prm.g;
    if (rows <= 8) return launch<D, 1>(prm, c);
    if (rows <= 16) return launch<D, 2>(prm, c);
    return launch<D, 4>(prm, c);
}

}  // namespace

bool masked_decode_supported(const MaskedAttn& c) {
    return c.a.dtype == ACACHE_BF16 && c.a.scale > 0.f && (int64_t)c.n_q * (c.a.hq / c.a.hkv) <= 32;
}

int launch_masked_decode(const MaskedAttn& c) {
    const int hkv = c.a.hkv, g = c.a.hq / hkv;
    DecParams prm{};
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
    prm.n_q = c.n_q;
    prm.total_q = c.total_q;
    prm.T_len = c.T_len;
    prm.Hq = c.a.hq;
    prm.Hkv = hkv;
    prm.g = g;
    prm.drop = c.mask.drop_none != 0;
    prm.scale_log2 = c.a.scale * kLog2e;
    if (c.mask.softcap > 0.f) {
        prm.cap_in = 2.f * kLog2e * (c.a.scale / c.mask.softcap);
        prm.cap_log2 = c.mask.softcap * kLog2e;
        prm.wide = c.mask.softcap > kWideCap;
    }
    return c.a.d == 128 ? dispatch<128>(prm, c) : dispatch<64>(prm, c);
}

}  // namespace acache
