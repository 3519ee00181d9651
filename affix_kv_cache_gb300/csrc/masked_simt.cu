// masked_simt.cu -- read-slot attention under a mask on CUDA cores: float32, and bf16 with a scale that is
// not positive.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4.3 and App. C.1 (attention through the read-slot
// map); the masks are this library's (include/acache.h, acache_slot_attention_masked).
//
// One warp per (row, query head): the lanes take 32 keys of the row's range at a time, one key each, for
// the logits; the warp keeps the running maximum and sum of the softmax, and each lane accumulates d / 32
// columns of the output.  Keys outside the range are not touched.
#include "q8.cuh"
#include "step.cuh"

namespace acache {
namespace {

constexpr int kWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
masked_simt_kernel(const MaskedAttn p) {
    constexpr int kPer = D / 32;
    __shared__ float qs[kWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hq = p.a.hq, g = hq / p.a.hkv;
    const int64_t gw = (int64_t)blockIdx.x * kWarps + warp;
    if (gw >= (int64_t)p.B * p.n_q * hq) return;
    const int h = (int)(gw % hq), hk = h / g;
    const int i = (int)(gw / hq % p.n_q), b = (int)(gw / hq / p.n_q);
    int T_len = p.T_len;
    int64_t qrow = (int64_t)b * p.n_q + i, kbase = (int64_t)b * p.T_len;
    if (p.q_start) {
        const int64_t q0 = p.q_start[b];
        kbase = p.kv_start[b];
        const int n = q8_count(p.q_start, b);
        T_len = q8_count(p.kv_start, b);
        if (n != 0 && q8_bad_lengths(n, p.n_q, T_len, p.T_len, q0, p.total_q, kbase)) {
            if (i == 0 && h == 0 && lane == 0) flag(p.dev_status, ACACHE_DEV_BAD_LENGTH);
            return;
        }
        if (i >= n) return;
        qrow = q0 + i;
    }
    int lo = 0, hi = T_len;
    if (p.mask.row_range) {
        lo = max(p.mask.row_range[2 * qrow], 0);
        hi = min(p.mask.row_range[2 * qrow + 1], T_len);
    }
    const float slope = p.mask.slopes ? p.mask.slopes[h] : 0.f;
    const int pos = p.mask.slopes ? p.mask.q_pos[qrow] : 0;
    const float cap = p.mask.softcap;
    const T* q = (const T*)p.q + (qrow * hq + h) * D;
    for (int c = lane; c < D; c += 32) qs[warp][c] = to_f32(q[c]);
    __syncwarp();
    const T *kc = (const T*)p.k_cache, *vc = (const T*)p.v_cache;
    float m = -INFINITY, l = 0.f, acc[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) acc[x] = 0.f;
    for (int t0 = lo; t0 < hi; t0 += 32) {
        const int t = t0 + lane;
        float s = -INFINITY;
        int64_t at = -1;                       // the key's row; -1: a zero row, or none
        if (t < hi) {
            const int32_t slot = p.read_slot[kbase + t];
            if (!(p.mask.drop_none && slot == ACACHE_SLOT_NONE)) {
                float dot = 0.f;
                if (slot >= 0 && slot < p.num_slots) {
                    at = ((int64_t)slot * p.a.hkv + hk) * D;
#pragma unroll 8
                    for (int c = 0; c < D; ++c) dot = fmaf(qs[warp][c], to_f32(kc[at + c]), dot);
                } else {
                    flag(p.dev_status, ACACHE_DEV_BAD_SLOT);
                }
                s = dot * p.a.scale;
                if (cap > 0.f) s = cap * tanhf(s / cap);
                if (p.mask.slopes) s = fmaf(-slope, fabsf((float)(pos - (int64_t)t)), s);
                s *= kLog2e;
            }
        }
        const float m_new = fmaxf(m, warp_max(s));
        // while no key has taken part (m_new = -inf) exponentiate against 0
        const float m_ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = fast_exp2(m - m_ref), w = fast_exp2(s - m_ref);
        l = l * alpha + warp_sum(w);
#pragma unroll
        for (int x = 0; x < kPer; ++x) acc[x] *= alpha;
        for (int u = 0; u < min(32, hi - t0); ++u) {
            const float wu = __shfl_sync(0xffffffffu, w, u);
            const int64_t au = __shfl_sync(0xffffffffu, at, u);
            if (au < 0) continue;              // a key that takes no part, or a zero value row
#pragma unroll
            for (int x = 0; x < kPer; ++x) acc[x] = fmaf(wu, to_f32(vc[au + lane + 32 * x]), acc[x]);
        }
        m = m_new;
    }
    const float inv = l == 0.f && m == -INFINITY ? 0.f : 1.f / l;
    T* out = (T*)p.out + (qrow * hq + h) * D;
#pragma unroll
    for (int x = 0; x < kPer; ++x) out[lane + 32 * x] = from_f32<T>(acc[x] * inv);
}

template <typename T, int D>
int launch(const MaskedAttn& c) {
    const int64_t blocks = ((int64_t)c.B * c.n_q * c.a.hq + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return ACACHE_ERR_INVALID_ARG;
    masked_simt_kernel<T, D><<<(unsigned)blocks, kWarps * 32, 0, c.stream>>>(c);
    return launch_status();
}

}  // namespace

int launch_masked_simt(const MaskedAttn& c) {
    if (c.a.dtype == ACACHE_F32) return c.a.d == 64 ? launch<float, 64>(c) : launch<float, 128>(c);
    return c.a.d == 64 ? launch<__nv_bfloat16, 64>(c) : launch<__nv_bfloat16, 128>(c);
}

}  // namespace acache
