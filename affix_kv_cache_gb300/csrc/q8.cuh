// q8.cuh -- the 8-bit KV pool: number format, key source and launch declarations.
//
// A pool row is one (slot, KV head) of K or of V: d e4m3 codes and one biased power-of-two
// exponent s in kv_scale[slot][head][K or V]; element i stands for code_i * 2^(s - 127).
// The block of tokens that shares a scale is one slot, because a store writes single slots
// anywhere in the pool: a scale shared with neighbouring slots would have to be raised, and
// their codes rewritten, while other requests read them.  A power of two costs a floating code
// no precision, and makes scaling, reading back (4 significant bits fit bf16) and storing a
// read-back row again exact in value.
#pragma once

#include <cuda_fp8.h>

#include "attn.cuh"

namespace acache {

// Exponents a store writes: 2^kQ8MinExp .. 2^kQ8MaxExp.  The attention carries V times 2^-32 in
// bf16 and accumulates in float32; in this range neither under- nor overflows.
constexpr int kQ8MinExp = -50, kQ8MaxExp = 38;
constexpr uint32_t kQ8MaxByte = kQ8MaxExp + 127;   // larger bytes read as NaN
constexpr uint32_t kQ8Poison = 255;                // row with a value that is not finite, or too large

// Smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8 is the largest e4m3 value) from the bits of
// amax >= 0: adding 2^21 - 1 carries into the exponent exactly when the significand is above
// 1.75.  Clamped from below; kQ8Poison when amax is not finite or needs more than kQ8MaxExp.
ACACHE_DEVFN uint32_t q8_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return kQ8Poison;
    const int s = (int)((amax_bits + 0x1fffffu) >> 23) - 8;     // biased exponent
    if (s > (int)kQ8MaxByte) return kQ8Poison;
    return (uint32_t)max(s, kQ8MinExp + 127);
}
// 2^(s - 127); 0 for s = 0 (a pool set to zero bytes reads as zeros), NaN for poisoned rows.
ACACHE_DEVFN float q8_factor(uint32_t s) { return __uint_as_float(s > kQ8MaxByte ? 0x7fffffffu : s << 23); }

// Two e4m3 codes (low byte first) -> float32.
ACACHE_DEVFN float2 q8_decode2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}
// Nearest e4m3 codes of two floats (ties to even), `a` in the low byte.
ACACHE_DEVFN uint32_t q8_encode2(float a, float b) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Rows or keys of ragged request b, from the offsets.  One behind the other's start is no count, however far: the
// difference of two offsets need not fit 32 bits.  (With a negative start, which is refused too, it may be anything.)
ACACHE_DEVFN int q8_count(const int32_t* start, int b) {
    const int32_t a = start[b], z = start[b + 1];
    return z < a ? -1 : (int)((uint32_t)z - (uint32_t)a);
}
// A ragged request with rows that is not computed: counts outside the call's bounds, or rows outside q.
ACACHE_DEVFN bool q8_bad_lengths(int n_q, int max_q, int T_len, int max_T, int64_t q_at, int total_q, int64_t kv_at) {
    return n_q < 0 || n_q > max_q || T_len < 1 || T_len > max_T || q_at < 0 || q_at + n_q > total_q || kv_at < 0;
}

// The attention over an 8-bit pool as the launchers take it.  q_start / kv_start: ragged batches
// (then n_q and T_len bound the per-request counts and q holds total_q rows), else null.
struct Q8Attn {
    AttnArgs a;
    int B, n_q, T_len, total_q;
    const int32_t *q_start, *kv_start;
    const void* q;
    const int32_t* read_slot;
    const uint8_t *k_cache, *v_cache, *kv_scale;
    int64_t num_slots;
    void* out;
    bool drop_none;
    int32_t* dev_status;
    cudaStream_t stream;
    bool after_store;      // launched behind the store of the same call: may overlap its tail
};

int launch_q8_write(int dtype, int batch, int rows, int hkv, int d, const int32_t* write_slot, const void* k_new,
                    const void* v_new, uint8_t* k_cache, uint8_t* v_cache, uint8_t* kv_scale, int64_t num_slots,
                    int64_t private_begin, int32_t* dev_status, cudaStream_t stream);
int launch_q8_gather(int dtype, int batch, int seq_len, int hkv, int d, const int32_t* read_slot,
                     const uint8_t* k_cache, const uint8_t* v_cache, const uint8_t* kv_scale, int64_t num_slots,
                     void* k_out, void* v_out, int32_t* dev_status, cudaStream_t stream);
int launch_q8_simt_attention(const Q8Attn& c);
// True when the tcgen05 kernel covers the call: bf16 and a positive softmax scale.
bool q8_tc_supported(const AttnArgs& a);
int launch_q8_tc_attention(const Q8Attn& c);
// ... and the one for few rows per (request, KV head): at most 32 packed rows (queries x group).
bool q8_decode_supported(const AttnArgs& a, int n_q);
int launch_q8_decode_attention(const Q8Attn& c);

}  // namespace acache
