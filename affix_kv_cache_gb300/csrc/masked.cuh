// masked.cuh -- what the tensor-core kernels of attention under a mask share: the capped score, and a row computed
// over its own keys alone.
#pragma once

#include "common.cuh"

namespace acache {

// max(|a|, |b|, |c|)
ACACHE_DEVFN float max3abs(float a, float b, float c) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
ACACHE_DEVFN uint64_t f2mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
ACACHE_DEVFN float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// c tanh(s / c) in log2 units from the product q.k: tanh y = 1 - 2 / (1 + e^2y), within 11 x 2^-24 c of it
// (infinities of e^2y give the limits).  cap_in = 2 log2e scale / c, cap_log2 = c log2e.
// In units of 2^-24 c, with E = e^2y: 16 |y| E / (1 + E)^2 from the four roundings of the exponent, 8 E / (1 + E)^2 from exp2
// (2^-22 of itself), 2 / (1 + E) from the sum, 4 / (1 + E) from the reciprocal (2^-23 of itself), 3 |tanh y| from the last
// product and the two of cap_log2.  Their sum is largest at y = -1.08: 10.1.
ACACHE_DEVFN float capped(float dot, float cap_in, float cap_log2) {
    return fmaf(-2.f * cap_log2, fast_rcp(1.f + fast_exp2(dot * cap_in)), cap_log2);
}
// The same within 2^-19 of itself, for large caps (2^-20 below y = 1/4; from there on as above, worst at y = -1/4 with
// 7.3 x 2^-24 c of c / 4.08): below y = 1/4 by y - y^3/3 + 2 y^5/15 - 17 y^7/315 (what follows is
// below 62/2835 y^9), with the score itself for y: next to a cap near the end of float32 cap_in has few bits or none.
ACACHE_DEVFN float capped_wide(float dot, float cap_in, float cap_log2, float scale_log2) {
    const float y = dot * (cap_in * 0.34657359f), z = y * y;        // ln2 / 2
    const float near = dot * scale_log2 * fmaf(z, fmaf(z, fmaf(z, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
    return fabsf(y) < 0.25f ? near : capped(dot, cap_in, cap_log2);
}
// Up to here the plain form is off by at most 2^-11.6, a sixth of a weight's rounding to bf16.
constexpr float kWideCap = 512.f;

template <typename T>
struct MaskedPool {
    const T *k_cache, *v_cache;
    const int32_t* read_slot;       // of the request, from the first of the keys counted below
    int64_t num_slots;
    int hkv, drop;
    bool wide;                      // a cap above kWideCap
    float scale_log2, cap_in, cap_log2;   // cap_in = 0: no cap
    float scale;                    // float32 rows: cap_in is the cap itself, and tanh the library's
};

// One row over its own keys [lo, hi), by a warp: for rows whose product with V met a masked key that is not
// finite (0 x NaN is NaN).  pos counts as the keys do.
template <typename T, int D>
ACACHE_DEVFN void masked_row(const MaskedPool<T>& p, const T* q, T* out, int lo, int hi, int hk, float slope_log2, int64_t pos,
                             int lane) {
    constexpr int kPer = D / 32;
    float m = -INFINITY, l = 0.f, acc[kPer];
    bool any = false;
#pragma unroll
    for (int x = 0; x < kPer; ++x) acc[x] = 0.f;
#pragma unroll 1
    for (int t0 = lo; t0 < hi; t0 += 32) {
        const int t = t0 + lane;
        float s = -INFINITY;
        int64_t at = -1;
        if (t < hi) {
            const int slot = p.read_slot[t];
            if (!(p.drop && slot == ACACHE_SLOT_NONE)) {
                float dot = 0.f;
                any = true;
                if (slot >= 0 && slot < p.num_slots) {
                    at = ((int64_t)slot * p.hkv + hk) * D;
#pragma unroll 4
                    for (int c = 0; c < D; ++c) dot = fmaf(to_f32(q[c]), to_f32(p.k_cache[at + c]), dot);
                }
                if (p.scale != 0.f || p.scale_log2 == 0.f)
                    s = p.cap_in > 0.f ? p.cap_in * tanhf(dot * p.scale / p.cap_in) * kLog2e : dot * p.scale * kLog2e;
                else
                    s = p.cap_in > 0.f ? (p.wide ? capped_wide(dot, p.cap_in, p.cap_log2, p.scale_log2) : capped(dot, p.cap_in, p.cap_log2)) : dot * p.scale_log2;
                if (slope_log2 != 0.f) s = fmaf(-slope_log2, fabsf((float)(pos - t)), s);
            }
        }
        const float m_new = fmaxf(m, warp_max(s)), m_ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = fast_exp2(m - m_ref), w = fast_exp2(s - m_ref);
        l = l * alpha + warp_sum(w);
#pragma unroll
        for (int x = 0; x < kPer; ++x) acc[x] *= alpha;
#pragma unroll 1
        for (int u = 0; u < min(32, hi - t0); ++u) {
            const float wu = __shfl_sync(0xffffffffu, w, u);
            const int64_t au = __shfl_sync(0xffffffffu, at, u);
            if (au < 0) continue;              // a key that takes no part, or a zero value row
#pragma unroll
            for (int x = 0; x < kPer; ++x) acc[x] = fmaf(wu, to_f32(p.v_cache[au + lane + 32 * x]), acc[x]);
        }
        m = m_new;
    }
    any = __any_sync(0xffffffffu, any);
#pragma unroll
    for (int x = 0; x < kPer; ++x) out[lane + 32 * x] = from_f32<T>(any ? acc[x] / l : 0.f);
}

}  // namespace acache
