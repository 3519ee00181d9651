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

constexpr long long kDrainBudget = 1LL << 31, kLandBudget = 1LL << 21;   // cycles, abort path

// Bounded wait for a phase.  A try that finds the phase incomplete suspends the warp until it completes, for
// some 7,900 cycles at most (whatever limit it is given), so a loop of tries takes nothing from the
// working warps.  kPolls (the rings' producers, which run ahead): a budget below that is kept by polling.
constexpr long long kTryCycles = 1 << 13;
template <bool kPolls = false>
ACACHE_DEVFN bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* dev_status,
                           long long budget) {
    const bool poll = kPolls && budget < kTryCycles;
    if (!poll && mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
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
// 32 bytes to a 32-byte aligned address
ACACHE_DEVFN void st_global_v8(void* to, const uint32_t (&k)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(k[0]), "r"(k[1]), "r"(k[2]), "r"(k[3]),
                 "r"(k[4]), "r"(k[5]), "r"(k[6]), "r"(k[7])
                 : "memory");
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

// 32 query rows -> two e4m3 terms each, by one warp, in two steps.  `hi` and `lo` are the shared-memory
// addresses of row 0's terms (rows of D bytes, swizzled, row 0 a multiple of 8).
// First the rows land by cp.async where their terms will be, the first half of a row in its row of hi, the
// second in its row of lo.  Lane i brings the element offset of row i; D / 8 lanes to a row, so the loads
// are whole rows.
template <int D>
ACACHE_DEVFN void query_load(const bf16* q, int64_t off, uint32_t hi, uint32_t lo, int lane) {
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    const uint32_t pc = (uint32_t)(lane % LPR), row = (uint32_t)(lane / LPR);
    const uint32_t to = pc >= LPR / 2 ? lo : hi;
#pragma unroll 4
    for (int it = 0; it < 32 / RPI; ++it) {
        const uint32_t r = (uint32_t)(it * RPI) + row;
        const int64_t o = __shfl_sync(0xffffffffu, off, (int)r);
        cp_async16(to + row_chunk<D>(r, pc % (LPR / 2)), q + o + pc * 8, 16);
    }
    cp_async_commit();
}
// Two pairs of bf16, each below 2^-111, to the four e4m3 codes of 2^120 times them, cut to e4m3's last place:
// a bf16 of that range has e4m3's exponent (or its subnormal form) 4 bits higher.
ACACHE_DEVFN uint32_t cut_codes(uint32_t a, uint32_t b) {
    uint32_t m, s;
    asm("prmt.b32 %0, %1, %2, 0x6420;" : "=r"(m) : "r"(a >> 4), "r"(b >> 4));
    asm("prmt.b32 %0, %1, %2, 0x7531;" : "=r"(s) : "r"(a), "r"(b));
    return (m & 0x7f7f7f7fu) | (s & 0x80808080u);
}
// Then the terms, in place, row `lane` by its lane: whole rows pass through its registers, so the row's
// largest needs no exchange.  Returns the row's factor: its logits are S times the keys' factors times it
// (scale_log2 times the power of two the row was divided by).  A row that is not finite has NaN for all its
// terms, so that S is NaN, and 1 for its factor: a discarded key, masked after S, must stay out.  The factor
// stays a normal number: a logit that the raise would change is below 2^-60, and 0 times a masked key's
// -infinity would be NaN.
// hi is q' cut to 4 significant bits and lo the rest, rounded to e4m3's subnormal step where it is longer.
template <int D>
ACACHE_DEVFN float query_terms(uint32_t hi, uint32_t lo, int lane, float scale_log2) {
    constexpr int NC = D / 8;                                 // 16-byte pieces of a bf16 row
    cp_async_wait<0>();
    __syncwarp();                                             // (a row's pieces came by several lanes' copies)
    uint32_t w[NC][4], top = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        ld_shared_v4((c < NC / 2 ? hi : lo) + row_chunk<D>(lane, c % (NC / 2)), w[c]);
#pragma unroll
        for (int y = 0; y < 4; ++y) top = __vmaxu2(top, w[c][y] & 0x7fff7fffu);
    }
    top = max(top & 0xffffu, top >> 16);
    const uint32_t E = max(top >> 7, 8u);                     // biased exponent of the row's largest
    const bool finite = E != 255u;
    const uint32_t nan2 = finite ? 0u : 0x7fff7fffu;
    const uint32_t up2 = (261u - E) << 7 | (261u - E) << 23;  // 2^(134 - E), twice: the largest goes to [128, 256)
    constexpr uint32_t kDown2 = 0x03800380u;                  // 2^-120, twice
#pragma unroll
    for (int c = 0; c < NC; c += 2) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int y = 0; y < 8; y += 2) {
            uint32_t x[2], r[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t v = w[c + (y >> 2)][(y & 3) + j] | nan2;
                asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x[j]) : "r"(v), "r"(up2));
                asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x[j]) : "r"(x[j]), "r"(kDown2));
                asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r[j]) : "r"(x[j]), "r"(x[j] & 0xfff0fff0u));
            }
            h[y >> 1] = cut_codes(x[0], x[1]);
            l[y >> 1] = cut_codes(r[0] + 0x00080008u, r[1] + 0x00080008u);
        }
        const uint32_t o = row_chunk<D>(lane, c >> 1);
        st_shared_v4(hi + o, h[0], h[1], h[2], h[3]);
        st_shared_v4(lo + o, l[0], l[1], l[2], l[3]);
    }
    return finite ? fmaxf(scale_log2 * __uint_as_float((E - 7u) << 23), 0x1p-126f) : 1.f;
}

}  // namespace q8
}  // namespace acache
