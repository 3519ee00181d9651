// q8_api.cu -- the C ABI's entry points over an 8-bit KV pool: argument validation and dispatch
// (declared and documented in include/acache.h).
#include "q8.cuh"

using namespace acache;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned2(const void* p) { return ((uintptr_t)p & 1u) == 0; }

bool pool_ok(const void* k_cache, const void* v_cache, const void* kv_scale) {
    return k_cache && v_cache && kv_scale && aligned16(k_cache) && aligned16(v_cache) && aligned2(kv_scale);
}

// Head counts whose items (16-byte pieces of a row) and row bytes are numbered in 32 bits.
bool heads_fit(const AttnArgs& a) { return a.hkv <= 1 << 24; }
// What the attention's grids and tensor maps hold (clusters of up to 8 CTAs a head along x), and keys whose indices,
// rounded up to whole tiles and looked up a few tiles ahead, stay in 32 bits.
bool fits(const AttnArgs& a, int batch, int n_q, int T_len, int64_t num_slots) {
    return batch <= 65535 && (int64_t)n_q * (a.hq / a.hkv) <= 65535LL * 64 && heads_fit(a) &&
           T_len <= 0x7fffffff - 1023 && num_slots < 0x7fffffffLL / a.hkv;
}

// Fixed and ragged attention after their own scalar checks (q_start null: fixed).
int attend(const Q8Attn& c) {
    if (!c.q || !c.read_slot || !c.out || !aligned16(c.q) || !aligned16(c.out) ||
        !pool_ok(c.k_cache, c.v_cache, c.kv_scale) || !fits(c.a, c.B, c.n_q, c.T_len, c.num_slots))
        return ACACHE_ERR_INVALID_ARG;
    // (an empty pool: every key is a zero row, and there is no row for a tensor map to start at)
    if (c.num_slots == 0 || !q8_tc_supported(c.a)) return launch_q8_simt_attention(c);
    return q8_decode_supported(c.a, c.n_q) ? launch_q8_decode_attention(c) : launch_q8_tc_attention(c);
}

Q8Attn call(const AttnArgs& a, int batch, int n_q, const void* q, int seq_len, const int32_t* read_slot,
            const void* k_cache, const void* v_cache, const uint8_t* kv_scale, int64_t num_slots, void* out,
            int drop_none, int32_t* dev_status, void* stream) {
    Q8Attn c{};
    c.a = a;
    c.B = batch;
    c.n_q = n_q;
    c.T_len = seq_len;
    c.q = q;
    c.read_slot = read_slot;
    c.k_cache = (const uint8_t*)k_cache;
    c.v_cache = (const uint8_t*)v_cache;
    c.kv_scale = kv_scale;
    c.num_slots = num_slots;
    c.out = out;
    c.drop_none = drop_none != 0;
    c.dev_status = dev_status;
    c.stream = (cudaStream_t)stream;
    return c;
}

}  // namespace

extern "C" {

int acache_write_slots_q8(const acache_attn_desc* desc, int batch, int rows, const int32_t* write_slot,
                          const void* k_new, const void* v_new, void* k_cache, void* v_cache, uint8_t* kv_scale,
                          int64_t num_slots, int64_t private_begin, int32_t* dev_status, void* stream) {
    AttnArgs a;
    if (int rc = check_desc(desc, &a)) return rc;
    if (batch < 0 || rows < 0 || num_slots < 0 || private_begin < 0 || private_begin > num_slots)
        return ACACHE_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0) return ACACHE_OK;
    if (!write_slot || !k_new || !v_new || !aligned16(k_new) || !aligned16(v_new) || !heads_fit(a) ||
        !pool_ok(k_cache, v_cache, kv_scale))
        return ACACHE_ERR_INVALID_ARG;
    return launch_q8_write(a.dtype, batch, rows, a.hkv, a.d, write_slot, k_new, v_new, (uint8_t*)k_cache,
                           (uint8_t*)v_cache, kv_scale, num_slots, private_begin, dev_status, (cudaStream_t)stream);
}

int acache_gather_slots_q8(const acache_attn_desc* desc, int batch, int seq_len, const int32_t* read_slot,
                           const void* k_cache, const void* v_cache, const uint8_t* kv_scale, int64_t num_slots,
                           void* k_out, void* v_out, int32_t* dev_status, void* stream) {
    AttnArgs a;
    if (int rc = check_desc(desc, &a)) return rc;
    if (batch < 0 || seq_len < 0 || num_slots < 0) return ACACHE_ERR_INVALID_ARG;
    if (batch == 0 || seq_len == 0) return ACACHE_OK;
    if (!read_slot || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out) || !heads_fit(a) ||
        !pool_ok(k_cache, v_cache, kv_scale))
        return ACACHE_ERR_INVALID_ARG;
    return launch_q8_gather(a.dtype, batch, seq_len, a.hkv, a.d, read_slot, (const uint8_t*)k_cache,
                            (const uint8_t*)v_cache, kv_scale, num_slots, k_out, v_out, dev_status,
                            (cudaStream_t)stream);
}

int acache_slot_attention_q8(const acache_attn_desc* desc, int batch, int n_q, const void* q, int seq_len,
                             const int32_t* read_slot, const void* k_cache, const void* v_cache,
                             const uint8_t* kv_scale, int64_t num_slots, void* out, int drop_none,
                             int32_t* dev_status, void* stream) {
    AttnArgs a;
    if (int rc = check_desc(desc, &a)) return rc;
    if (batch < 0 || n_q < 0 || seq_len < 0 || num_slots < 0) return ACACHE_ERR_INVALID_ARG;
    if (batch == 0 || n_q == 0) return ACACHE_OK;
    if (seq_len == 0) return ACACHE_ERR_INVALID_ARG;       // a softmax over no keys
    return attend(call(a, batch, n_q, q, seq_len, read_slot, k_cache, v_cache, kv_scale, num_slots, out, drop_none,
                       dev_status, stream));
}

int acache_slot_attention_varlen_q8(const acache_attn_desc* desc, int batch, const int32_t* q_start, int max_q_rows,
                                    int total_q_rows, const void* q, const int32_t* kv_start, int max_seq_len,
                                    const int32_t* read_slot, const void* k_cache, const void* v_cache,
                                    const uint8_t* kv_scale, int64_t num_slots, void* out, int drop_none,
                                    int32_t* dev_status, void* stream) {
    AttnArgs a;
    if (int rc = check_desc(desc, &a)) return rc;
    if (batch < 0 || max_q_rows < 0 || total_q_rows < 0 || max_seq_len < 0 || num_slots < 0)
        return ACACHE_ERR_INVALID_ARG;
    if (batch == 0 || max_q_rows == 0 || total_q_rows == 0) return ACACHE_OK;
    if (max_seq_len == 0) return ACACHE_ERR_INVALID_ARG;   // a softmax over no keys
    if (!q_start || !kv_start) return ACACHE_ERR_INVALID_ARG;
    Q8Attn c = call(a, batch, max_q_rows, q, max_seq_len, read_slot, k_cache, v_cache, kv_scale, num_slots, out,
                    drop_none, dev_status, stream);
    c.q_start = q_start;
    c.kv_start = kv_start;
    c.total_q = total_q_rows;
    return attend(c);
}

int acache_store_attend_q8(const acache_attn_desc* desc, int batch, int rows, const int32_t* write_slot,
                           const void* k_new, const void* v_new, void* k_cache, void* v_cache, uint8_t* kv_scale,
                           int64_t num_slots, int64_t private_begin, int n_q, const void* q, int seq_len,
                           const int32_t* read_slot, void* out, int drop_none, int32_t* dev_status, void* stream) {
    AttnArgs a;
    if (int rc = check_desc(desc, &a)) return rc;
    // both halves are checked before either is launched
    if (batch < 0 || rows < 0 || n_q < 0 || seq_len < 0 || num_slots < 0 || private_begin < 0 ||
        private_begin > num_slots)
        return ACACHE_ERR_INVALID_ARG;
    if (batch == 0) return ACACHE_OK;
    const bool store = rows > 0, attends = n_q > 0;
    if (store && (!write_slot || !k_new || !v_new || !aligned16(k_new) || !aligned16(v_new) || !heads_fit(a)))
        return ACACHE_ERR_INVALID_ARG;
    if (attends && (seq_len == 0 || !q || !read_slot || !out || !aligned16(q) || !aligned16(out) ||
                    !fits(a, batch, n_q, seq_len, num_slots)))
        return ACACHE_ERR_INVALID_ARG;
    if ((store || attends) && !pool_ok(k_cache, v_cache, kv_scale)) return ACACHE_ERR_INVALID_ARG;
    if (store)
        if (int rc = launch_q8_write(a.dtype, batch, rows, a.hkv, a.d, write_slot, k_new, v_new, (uint8_t*)k_cache,
                                     (uint8_t*)v_cache, kv_scale, num_slots, private_begin, dev_status,
                                     (cudaStream_t)stream))
            return rc;
    if (!attends) return ACACHE_OK;
    Q8Attn c = call(a, batch, n_q, q, seq_len, read_slot, k_cache, v_cache, kv_scale, num_slots, out, drop_none,
                    dev_status, stream);
    c.after_store = store;
    return attend(c);
}

}  // extern "C"
