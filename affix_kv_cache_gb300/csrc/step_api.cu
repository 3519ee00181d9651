// step_api.cu -- the C ABI's entry points around the attention of a step: rotary descriptors, norm and
// rotation, the store that applies them, attention under a mask, token scores (declared and documented in
// include/acache.h).
#include <math.h>

#include <algorithm>

#include "step.cuh"

using namespace acache;

namespace {

constexpr double kTwoPi = 6.283185307179586476925;
constexpr double kPerTurn = 0x1.45f306dc9c883p-3, kPerTurnLow = -0x1.6b01ec5417056p-57;   // 1 / 2 pi and what it is off by

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

// f / 2 pi modulo one turn, in units of 2^-64 turns.  Below one turn: to the nearest unit, from the quotient in two doubles
// (1 / 2 pi in two as well: within 2^-105 of itself).  Faster: f / 2 pi rounded to 53 bits, and what follows is exact (a
// fraction within 2^-64 of one turn is taken as zero).
bool to_phase(double f, uint64_t* out) {
    if (!(fabs(f) < 1e300)) return false;
    double turns = f / kTwoPi;
    if (fabs(turns) < 1) {
        const double p = f * kPerTurn, rest = fma(f, kPerTurn, -p) + f * kPerTurnLow;
        const double units = ldexp(p, 64), whole = floor(units);          // (p too is below one turn: the largest f gives 1 - 2^-53)
        const uint64_t u = whole < 0 ? 0 - (uint64_t)-whole : (uint64_t)whole;
        *out = u + (uint64_t)(int64_t)floor(units - whole + ldexp(rest, 64) + 0.5);
        return true;
    }
    turns -= floor(turns);
    const double units = ldexp(turns, 64);
    *out = units >= 18446744073709551616.0 ? 0 : (uint64_t)units;
    return true;
}

bool rotary_dim_ok(int rd) { return rd >= 2 && rd <= 128 && rd % 2 == 0; }

// A call's rotation (null: none, then positions are not read).
bool rope_ok(const acache_rope* r, const AttnArgs& a, const int32_t* positions) {
    if (!r) return true;
    return rotary_dim_ok(r->rotary_dim) && r->rotary_dim <= a.d && isfinite(r->amplitude) && positions != nullptr &&
           aligned(positions, 4);
}

// A strided matrix of `heads` heads to a row.
bool rows_ok(const AttnArgs& a, const void* p, int64_t stride, int heads) {
    const int64_t e = a.dtype == ACACHE_F32 ? 4 : 2;
    return p && aligned16(p) && stride >= (int64_t)heads * a.d && stride * e % 16 == 0 && stride < (1LL << 40);
}
int64_t row_bytes(const AttnArgs& a, int heads) { return (int64_t)heads * a.d * (a.dtype == ACACHE_F32 ? 4 : 2); }
// Bytes from the first row of one matrix to the end of its last.
int64_t span(const AttnArgs& a, int64_t rows, int64_t stride, int heads) {
    return (rows - 1) * stride * (a.dtype == ACACHE_F32 ? 4 : 2) + row_bytes(a, heads);
}
// Two matrices lie apart: one behind the other, or with the same stride each in the gaps between the other's rows.  kUnknown:
// their rows are spaced otherwise, and the one begins before the other ends.
enum Apart { kMeet, kApart, kUnknown };
Apart lie(const AttnArgs& a, int64_t rows, const void* x, int64_t sx, int hx, const void* y, int64_t sy, int hy) {
    const uintptr_t x0 = (uintptr_t)x, y0 = (uintptr_t)y;
    if (x0 + span(a, rows, sx, hx) <= y0 || y0 + span(a, rows, sy, hy) <= x0) return kApart;
    if (rows == 1) return kMeet;
    if (sx != sy) return kUnknown;
    const int64_t step = sx * (a.dtype == ACACHE_F32 ? 4 : 2), behind = ((int64_t)(y0 - x0) % step + step) % step;
    return behind >= row_bytes(a, hx) && step - behind >= row_bytes(a, hy) ? kApart : kMeet;
}
// An output is its own input, or lies apart from it.
bool apart(const AttnArgs& a, int64_t rows, const void* in, int64_t si, const void* out, int64_t so, int heads) {
    return in == out ? si == so : lie(a, rows, in, si, heads, out, so, heads) == kApart;
}
// Head counts of one call (items of a row are numbered in 32 bits) and rows whose byte offsets fit 64.
bool sizes_fit(const AttnArgs& a, int64_t rows) {
    return a.hkv <= 1 << 20 && a.hq <= 1 << 20 && rows <= 1LL << 31;
}

int rotate_store(const acache_attn_desc* desc, const acache_rope* rope, int batch, int rows, const int32_t* positions,
                 const int32_t* write_slot, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                 int64_t v_stride, const void* q_weight, const void* k_weight, float eps, void* q_out, void* k_cache,
                 void* v_cache, bool q8, uint8_t* kv_scale, int64_t num_slots, int64_t private_begin, int32_t* dev_status,
                 void* stream) {
    AttnArgs a;
    if (int rc = check_desc(desc, &a)) return rc;
    if (batch < 0 || rows < 0 || num_slots < 0 || private_begin < 0 || private_begin > num_slots || !(eps >= 0.f) || isinf(eps))
        return ACACHE_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0) return ACACHE_OK;
    const int64_t n = (int64_t)batch * rows;
    if (!sizes_fit(a, n) || !rope_ok(rope, a, positions) || !write_slot || !rows_ok(a, k, k_stride, a.hkv) ||
        !rows_ok(a, v, v_stride, a.hkv) || !aligned16(q_weight) || !aligned16(k_weight) || !k_cache || !v_cache ||
        !aligned16(k_cache) || !aligned16(v_cache) || (q8 && (!kv_scale || !aligned(kv_scale, 2))))
        return ACACHE_ERR_INVALID_ARG;
    const int64_t row = (int64_t)a.hq * a.d;
    if (q && (!rows_ok(a, q, q_stride, a.hq) || !rows_ok(a, q_out, row, a.hq) || !apart(a, n, q, q_stride, q_out, row, a.hq)))
        return ACACHE_ERR_INVALID_ARG;
    if (q && (lie(a, n, k, k_stride, a.hkv, q_out, row, a.hq) == kMeet || lie(a, n, v, v_stride, a.hkv, q_out, row, a.hq) == kMeet))
        return ACACHE_ERR_INVALID_ARG;
    RotateCall c{};
    c.a = a;
    c.rope = rope;
    c.rows = n;
    c.positions = positions;
    c.write_slot = write_slot;
    c.q = q;
    c.k = k;
    c.v = v;
    c.q_weight = q_weight;
    c.k_weight = k_weight;
    c.q_stride = q_stride;
    c.k_stride = k_stride;
    c.v_stride = v_stride;
    c.eps = eps;
    c.q_out = q_out;
    c.q_out_stride = row;
    c.k_cache = k_cache;
    c.v_cache = v_cache;
    c.kv_scale = kv_scale;
    c.num_slots = num_slots;
    c.private_begin = private_begin;
    c.dev_status = dev_status;
    c.stream = (cudaStream_t)stream;
    return launch_rotate(c, q8 ? kRotateStoreQ8 : kRotateStore);
}

// What a mask and the geometry of a masked call have to keep to.
bool masked_ok(const AttnArgs& a, const acache_mask* m, int batch, int n_q, int T_len, int64_t num_slots) {
    if (m && (!(m->softcap >= 0.f) || isinf(m->softcap) || (m->slopes && !m->q_pos) || !aligned(m->row_range, 4) ||
              !aligned(m->q_pos, 4) || !aligned(m->slopes, 4)))
        return false;
    // (the capped score's constants have to be numbers)
    if (m && m->softcap > 0.f && (!isfinite(2.f * kLog2e * (a.scale / m->softcap)) || !isfinite(m->softcap * kLog2e))) return false;
    return batch <= 65535 && (int64_t)n_q * (a.hq / a.hkv) <= 65535LL * 64 && T_len <= 0x7fffffff - 1023 &&
           a.hkv <= 1 << 20 && num_slots < 0x7fffffffLL / a.hkv;
}

int attend(const MaskedAttn& c) {
    if (!c.q || !c.read_slot || !c.out || !c.k_cache || !c.v_cache || !aligned16(c.q) || !aligned16(c.out) ||
        !aligned16(c.k_cache) || !aligned16(c.v_cache))
        return ACACHE_ERR_INVALID_ARG;
    if (masked_decode_supported(c)) return launch_masked_decode(c);
    return masked_tc_supported(c) ? launch_masked_tc(c) : launch_masked_simt(c);
}

MaskedAttn masked_call(const AttnArgs& a, const acache_mask* mask, int batch, int n_q, const void* q, int seq_len,
                       const int32_t* read_slot, const void* k_cache, const void* v_cache, int64_t num_slots, void* out,
                       int32_t* dev_status, void* stream) {
    MaskedAttn c{};
    c.a = a;
    if (mask) c.mask = *mask;
    c.B = batch;
    c.n_q = n_q;
    c.T_len = seq_len;
    c.q = q;
    c.read_slot = read_slot;
    c.k_cache = k_cache;
    c.v_cache = v_cache;
    c.num_slots = num_slots;
    c.out = out;
    c.dev_status = dev_status;
    c.stream = (cudaStream_t)stream;
    return c;
}

}  // namespace

extern "C" {

int acache_rope_init_frequencies(acache_rope* out, int rotary_dim, int interleaved, const double* frequencies,
                                 float amplitude) {
    if (!out || !frequencies || !rotary_dim_ok(rotary_dim) || !isfinite(amplitude)) return ACACHE_ERR_INVALID_ARG;
    acache_rope r{};
    r.rotary_dim = rotary_dim;
    r.interleaved = interleaved != 0;
    r.amplitude = amplitude;
    for (int i = 0; i < rotary_dim / 2; ++i)
        if (!to_phase(frequencies[i], &r.phase[i])) return ACACHE_ERR_INVALID_ARG;
    *out = r;
    return ACACHE_OK;
}

int acache_rope_init(acache_rope* out, int rotary_dim, int interleaved, double theta, int scaling, double factor,
                     int64_t trained_len, double turns_low, double turns_high) {
    if (!out || !rotary_dim_ok(rotary_dim) || !(theta > 0) || !isfinite(theta)) return ACACHE_ERR_INVALID_ARG;
    if (scaling < ACACHE_ROPE_NONE || scaling > ACACHE_ROPE_BANDS) return ACACHE_ERR_INVALID_ARG;
    const int rd = rotary_dim;
    const bool by_length = scaling == ACACHE_ROPE_YARN || scaling == ACACHE_ROPE_BANDS;
    if (scaling != ACACHE_ROPE_NONE && (!(factor > 0) || !isfinite(factor))) return ACACHE_ERR_INVALID_ARG;
    if (scaling == ACACHE_ROPE_NTK && rd <= 2) return ACACHE_ERR_INVALID_ARG;
    if (by_length) {
        if (turns_low == 0 && turns_high == 0) {
            turns_low = 1;
            turns_high = scaling == ACACHE_ROPE_YARN ? 32 : 4;
        }
        if (trained_len <= 0 || !(turns_low > 0) || !(turns_high > turns_low) || !isfinite(turns_high))
            return ACACHE_ERR_INVALID_ARG;
    }
    if (scaling == ACACHE_ROPE_YARN && (!(factor > 1) || !(theta > 1))) return ACACHE_ERR_INVALID_ARG;
    const double len = (double)trained_len;
    double base = theta, amplitude = 1;
    if (scaling == ACACHE_ROPE_NTK) base *= pow(factor, (double)rd / (rd - 2));
    int first = 0, last = 0;
    if (scaling == ACACHE_ROPE_YARN) {
        auto pair_at = [&](double turns) { return rd * log(len / (kTwoPi * turns)) / (2 * log(theta)); };
        first = (int)std::max(floor(pair_at(turns_high)), 0.0);
        last = (int)std::min(ceil(pair_at(turns_low)), rd - 1.0);
        amplitude = 0.1 * log(factor) + 1;
    }
    double f[64];
    for (int i = 0; i < rd / 2; ++i) {
        f[i] = pow(base, -2.0 * i / rd);
        double keep = 1;                                  // share of the frequency that is not divided
        if (scaling == ACACHE_ROPE_LINEAR) keep = 0;
        if (scaling == ACACHE_ROPE_YARN)
            keep = i <= first ? 1 : i >= last ? 0 : 1 - (double)(i - first) / (last - first);
        if (scaling == ACACHE_ROPE_BANDS)
            keep = std::min(std::max((f[i] * len / kTwoPi - turns_low) / (turns_high - turns_low), 0.0), 1.0);
        if (keep < 1) f[i] = f[i] * keep + f[i] / factor * (1 - keep);
    }
    return acache_rope_init_frequencies(out, rd, interleaved, f, (float)amplitude);
}

int acache_rotate_qk(const acache_attn_desc* desc, const acache_rope* rope, int64_t rows, const int32_t* positions,
                     const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* q_weight,
                     const void* k_weight, float eps, void* q_out, int64_t q_out_stride, void* k_out,
                     int64_t k_out_stride, void* stream) {
    AttnArgs a;
    if (int rc = check_desc(desc, &a)) return rc;
    if (rows < 0 || !(eps >= 0.f) || isinf(eps)) return ACACHE_ERR_INVALID_ARG;
    if (rows == 0 || (!q && !k)) return ACACHE_OK;
    if (!sizes_fit(a, rows) || !rope_ok(rope, a, positions) || !aligned16(q_weight) || !aligned16(k_weight))
        return ACACHE_ERR_INVALID_ARG;
    if (q && (!rows_ok(a, q, q_stride, a.hq) || !rows_ok(a, q_out, q_out_stride, a.hq) ||
              !apart(a, rows, q, q_stride, q_out, q_out_stride, a.hq)))
        return ACACHE_ERR_INVALID_ARG;
    if (k && (!rows_ok(a, k, k_stride, a.hkv) || !rows_ok(a, k_out, k_out_stride, a.hkv) ||
              !apart(a, rows, k, k_stride, k_out, k_out_stride, a.hkv)))
        return ACACHE_ERR_INVALID_ARG;
    if (q && k && (lie(a, rows, q, q_stride, a.hq, k_out, k_out_stride, a.hkv) == kMeet ||
                   lie(a, rows, k, k_stride, a.hkv, q_out, q_out_stride, a.hq) == kMeet ||
                   lie(a, rows, q_out, q_out_stride, a.hq, k_out, k_out_stride, a.hkv) == kMeet))
        return ACACHE_ERR_INVALID_ARG;
    RotateCall c{};
    c.a = a;
    c.rope = rope;
    c.rows = rows;
    c.positions = positions;
    c.q = q;
    c.k = k;
    c.q_weight = q_weight;
    c.k_weight = k_weight;
    c.q_stride = q_stride;
    c.k_stride = k_stride;
    c.eps = eps;
    c.q_out = q_out;
    c.q_out_stride = q_out_stride;
    c.k_out = k_out;
    c.k_out_stride = k_out_stride;
    c.stream = (cudaStream_t)stream;
    return launch_rotate(c, kRotate);
}

int acache_rotate_store(const acache_attn_desc* desc, const acache_rope* rope, int batch, int rows,
                        const int32_t* positions, const int32_t* write_slot, const void* q, int64_t q_stride,
                        const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q_weight,
                        const void* k_weight, float eps, void* q_out, void* k_cache, void* v_cache, int64_t num_slots,
                        int64_t private_begin, int32_t* dev_status, void* stream) {
    return rotate_store(desc, rope, batch, rows, positions, write_slot, q, q_stride, k, k_stride, v, v_stride, q_weight,
                        k_weight, eps, q_out, k_cache, v_cache, false, nullptr, num_slots, private_begin, dev_status, stream);
}

int acache_rotate_store_q8(const acache_attn_desc* desc, const acache_rope* rope, int batch, int rows,
                           const int32_t* positions, const int32_t* write_slot, const void* q, int64_t q_stride,
                           const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q_weight,
                           const void* k_weight, float eps, void* q_out, void* k_cache, void* v_cache, uint8_t* kv_scale,
                           int64_t num_slots, int64_t private_begin, int32_t* dev_status, void* stream) {
    return rotate_store(desc, rope, batch, rows, positions, write_slot, q, q_stride, k, k_stride, v, v_stride, q_weight,
                        k_weight, eps, q_out, k_cache, v_cache, true, kv_scale, num_slots, private_begin, dev_status, stream);
}

int acache_slot_attention_masked(const acache_attn_desc* desc, const acache_mask* mask, int batch, int n_q, const void* q,
                                 int seq_len, const int32_t* read_slot, const void* k_cache, const void* v_cache,
                                 int64_t num_slots, void* out, int32_t* dev_status, void* stream) {
    AttnArgs a;
    if (int rc = check_desc(desc, &a)) return rc;
    if (batch < 0 || n_q < 0 || seq_len < 0 || num_slots < 0) return ACACHE_ERR_INVALID_ARG;
    if (batch == 0 || n_q == 0) return ACACHE_OK;
    if (seq_len == 0 || !masked_ok(a, mask, batch, n_q, seq_len, num_slots)) return ACACHE_ERR_INVALID_ARG;
    return attend(masked_call(a, mask, batch, n_q, q, seq_len, read_slot, k_cache, v_cache, num_slots, out, dev_status,
                              stream));
}

int acache_slot_attention_masked_varlen(const acache_attn_desc* desc, const acache_mask* mask, int batch,
                                        const int32_t* q_start, int max_q_rows, int total_q_rows, const void* q,
                                        const int32_t* kv_start, int max_seq_len, const int32_t* read_slot,
                                        const void* k_cache, const void* v_cache, int64_t num_slots, void* out,
                                        int32_t* dev_status, void* stream) {
    AttnArgs a;
    if (int rc = check_desc(desc, &a)) return rc;
    if (batch < 0 || max_q_rows < 0 || total_q_rows < 0 || max_seq_len < 0 || num_slots < 0) return ACACHE_ERR_INVALID_ARG;
    if (batch == 0 || max_q_rows == 0 || total_q_rows == 0) return ACACHE_OK;
    if (max_seq_len == 0 || !q_start || !kv_start || !masked_ok(a, mask, batch, max_q_rows, max_seq_len, num_slots))
        return ACACHE_ERR_INVALID_ARG;
    MaskedAttn c = masked_call(a, mask, batch, max_q_rows, q, max_seq_len, read_slot, k_cache, v_cache, num_slots, out,
                               dev_status, stream);
    c.q_start = q_start;
    c.kv_start = kv_start;
    c.total_q = total_q_rows;
    return attend(c);
}

int acache_token_scores(int dtype, int64_t rows, int vocab, const void* logits, int64_t row_stride, float temperature,
                        const int32_t* tokens, float* token_logprob, float* entropy, int k, int32_t* top_tokens,
                        float* top_logprob, int32_t* dev_status, void* stream) {
    if (dtype != ACACHE_F32 && dtype != ACACHE_BF16) return ACACHE_ERR_UNSUPPORTED;
    if (rows < 0 || vocab < 0 || k < 0 || k > ACACHE_MAX_ALTERNATIVES || k > vocab || rows > 0x7fffffffLL / 8)
        return ACACHE_ERR_INVALID_ARG;
    if (!(temperature > 0.f) || !isfinite(1.f / temperature) || !isfinite(temperature)) return ACACHE_ERR_INVALID_ARG;
    if (!isfinite(kLog2e / temperature)) return ACACHE_ERR_INVALID_ARG;
    if (rows == 0) return ACACHE_OK;
    if (vocab == 0 || vocab > 0x7fffffff - 64 || !logits || !aligned(logits, dtype == ACACHE_F32 ? 4 : 2) ||
        (rows > 1 && row_stride < vocab) || row_stride >= (1LL << 40) || row_stride < 0 || (tokens == nullptr) != (token_logprob == nullptr) ||
        (k > 0 && !top_tokens))
        return ACACHE_ERR_INVALID_ARG;
    if (!token_logprob && !entropy && k == 0) return ACACHE_OK;
    const ScoreCall c{dtype, rows, vocab, logits, row_stride, temperature, tokens, token_logprob, entropy, k, top_tokens,
                      top_logprob, dev_status, (cudaStream_t)stream};
    return launch_token_scores(c);
}

}  // extern "C"
