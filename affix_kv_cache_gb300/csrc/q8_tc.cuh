// q8_tc.cuh -- what the two tensor-core kernels over an 8-bit pool share: bounded waits, the 8-bit MMA
// with its descriptors, and the two-term form of the query rows.
#pragma once

#include "q8.cuh"
#include "ptx.cuh"
#include "tc_attn.cuh"

namespace acache {
namespace q8 {

using namespace ptx;
using bf16 = __nv_bfloat16;

constexpr int kNoKey = INT32_MIN;           // read-slot entry of a key past the request's last
constexpr long long kDrainBudget = 1LL << 31, kLandBudget = 1LL << 21;   // cycles, abort path

// Bounded wait for a phase.  A try that finds the phase incomplete suspends the warp for some 90 cycles;
// what it issues between tries is taken from the working warps' slots.  kSlack: the waiter runs a
// ring's depth ahead, so it sleeps between tries instead.
template <bool kSlack = false>
ACACHE_DEVFN bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* dev_status,
                           long long budget) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (kSlack) __nanosleep(100);
        if (mbar_try_wait(bar, parity)) return true;
        if (!kSlack) {
            if (mbar_try_wait(bar, parity)) return true;
            if (mbar_try_wait(bar, parity)) return true;
        }
        if (*abort_flag) return false;
        if (clock64() - t0 > budget) {
            *abort_flag = 1;
            flag(dev_status, ACACHE_DEV_TIMEOUT);
            return false;
        }
    }
}

ACACHE_DEVFN uint64_t f2mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
ACACHE_DEVFN void ld_shared_v4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
ACACHE_DEVFN void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
ACACHE_DEVFN uint64_t f2sub(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// D[tmem] (+)= A[smem desc] * B[smem desc], 8-bit float inputs, fp32 accumulate
ACACHE_DEVFN void umma_ss_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same with A in TMEM (four elements to a 32-bit column)
ACACHE_DEVFN void umma_ts_f8(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// e4m3 A and B (format 0), fp32 D, K-major operands
constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// K-major descriptor of a tile whose rows are D bytes (one swizzle span of 128 or 64 bytes)
template <int D>
ACACHE_DEVFN uint64_t sdesc_rows(uint32_t addr) {
    uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)1 << 16;
    d |= (uint64_t)((8u * D) >> 4) << 32;                    // next 8 rows
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(D == 128 ? 2 : 4) << 61;                 // 128- or 64-byte swizzle
    return d;
}
// byte offset of 16-byte chunk c of row r in such a tile
template <int D>
ACACHE_DEVFN uint32_t row_chunk(uint32_t r, uint32_t c) {
    return r * D + ((D == 128 ? c ^ (r & 7u) : c ^ ((r >> 1) & 3u)) << 4);
}
// float4 slot q of row r in the partial-O area
template <int D>
ACACHE_DEVFN uint32_t part_off(int r, int q) { return (uint32_t)r * (D * 4u) + (uint32_t)((q ^ (r & (D / 4 - 1))) << 4); }

// 32 query rows -> two e4m3 terms each, by one warp, in two steps.  Lane i brings the element offset of row i;
// `hi` and `lo` are the shared-memory addresses of row 0's terms (rows of D bytes, swizzled, row 0 a
// multiple of 8).
// First the rows land by cp.async where their terms will be, the first half of a row in its row of hi, the
// second in its row of lo: LPR lanes to a row, so the loads are whole rows.
template <int D>
ACACHE_DEVFN void query_load(const bf16* q, int64_t off, uint32_t hi, uint32_t lo, int lane) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, NI = 32 / RPI;
    const uint32_t pc = (uint32_t)(lane % LPR), row = (uint32_t)(lane / LPR);
    const uint32_t at = (pc >= LPR / 2 ? lo : hi) + (pc % (LPR / 2)) * 16u + row * D;
#pragma unroll 4
    for (int it = 0; it < NI; ++it) {
        const int64_t o = __shfl_sync(0xffffffffu, off, it * RPI + row);
        cp_async16(at + (uint32_t)(it * RPI * D), q + o + pc * 8, 16);
    }
    cp_async_commit();
}
// Then the terms, in place.  c_row[i] receives the factor of row i: its logits are S times the keys' factors
// times it (scale_log2 times the power of two the row was divided by; NaN for a row that is not finite,
// which is carried as zeros).  GR groups of rows at a time keep the chain load - maximum - convert -
// subtract - convert of several rows in flight.  The scaled elements are carried in f16: exact down to
// 2^-22 of the row's largest, below that off by less than the low term's own last place.
template <int D>
ACACHE_DEVFN void query_terms(uint32_t hi, uint32_t lo, int lane, float scale_log2, float* c_row) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, NI = 32 / RPI, GR = 4;
    const uint32_t pc = (uint32_t)(lane % LPR), row = (uint32_t)(lane / LPR);
    const uint32_t at = (pc >= LPR / 2 ? lo : hi) + (pc % (LPR / 2)) * 16u + row * D;
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll 1
    for (int g = 0; g < NI / GR; ++g) {
        uint32_t w[GR][4], top[GR];
#pragma unroll
        for (int u = 0; u < GR; ++u) ld_shared_v4(at + (uint32_t)((g * GR + u) * RPI * D), w[u]);
#pragma unroll
        for (int u = 0; u < GR; ++u) {
            top[u] = __vmaxu2(__vmaxu2(w[u][0] & 0x7fff7fffu, w[u][1] & 0x7fff7fffu),
                              __vmaxu2(w[u][2] & 0x7fff7fffu, w[u][3] & 0x7fff7fffu));
            top[u] = max(top[u] & 0xffffu, top[u] >> 16);
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < GR; ++u) top[u] = max(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
#pragma unroll
        for (int u = 0; u < GR; ++u) {
            const uint32_t r = (uint32_t)((g * GR + u) * RPI) + row;
            const uint32_t E = max(top[u] >> 7, 8u);              // biased exponent of the row's largest
            const bool finite = E != 255u;
            const uint32_t keep = finite ? 0xffffffffu : 0u;
            const uint32_t up2 = (261u - E) << 7 | (261u - E) << 23;              // 2^(134 - E) in bf16: largest in [128, 256)
            if (pc == 0) c_row[r] = finite ? scale_log2 * __uint_as_float((E - 7u) << 23) : __uint_as_float(0x7fffffffu);
            uint32_t h[2], l[2];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint32_t x, f, back;
                unsigned short t;
                asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w[u][y] & keep), "r"(up2));
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f) : "f"(__uint_as_float(x & 0xffff0000u)), "f"(__uint_as_float(x << 16)));
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(t) : "r"(f));
                h[y >> 1] = (y & 1) ? h[y >> 1] | (uint32_t)t << 16 : t;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(t));
                asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(f) : "r"(f), "r"(back));
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(t) : "r"(f));
                l[y >> 1] = (y & 1) ? l[y >> 1] | (uint32_t)t << 16 : t;
            }
            // (the shuffles ordered the rows' reads before these writes)
            const uint32_t o = row_chunk<D>(r, pc >> 1) + (pc & 1u) * 8u;
            st_shared_v2(hi + o, h[0], h[1]);
            st_shared_v2(lo + o, l[0], l[1]);
        }
    }
}

}  // namespace q8
}  // namespace acache
