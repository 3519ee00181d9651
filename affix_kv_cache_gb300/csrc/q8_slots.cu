// q8_slots.cu -- the quantising store into an 8-bit KV pool and the read-back.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4.1, 4.3 and App. C.1 (the store
// through the write-side map and the logical KV view); the page keeps a 16-bit cache, the 8-bit
// pool is this library's.
//
// Both are bound by memory.  The store's item is 16 consecutive elements of one (row, head), of K and of
// V: a lane reads an item of each matrix with 16-byte loads, the d/16 lanes of a head agree on the
// largest magnitude with shuffles, and one lane writes the head's two exponents as one 16-bit
// word (16 x 1,205 rows of 32 heads, d = 128: 76 us in bf16, 123 us in float32, 0.92 and 0.95 of the copy bandwidth); a
// thread keeps two items in flight.  The read-back's item is one 16-byte piece of the output.  Items are
// numbered across rows, so every lane has work whatever the head count is; a step of the grid advances
// (row, item) by a constant pair, so the only division is at a thread's start.
#include "q8.cuh"
#include "ptx.cuh"

namespace acache {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;

// 16 elements of T in 16-byte words.
template <typename T> struct Item { uint4 w[sizeof(T)]; };

template <typename T> ACACHE_DEVFN void load_item(Item<T>& it, const T* src) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) it.w[i] = __ldcs(reinterpret_cast<const uint4*>(src) + i);
}
// element pair i (0..7) as float32
template <typename T> ACACHE_DEVFN float2 item_pair(const Item<T>& it, int i);
template <> ACACHE_DEVFN float2 item_pair<float>(const Item<float>& it, int i) {
    const uint4& w = it.w[i >> 1];
    return (i & 1) ? make_float2(__uint_as_float(w.z), __uint_as_float(w.w))
                   : make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
}
template <> ACACHE_DEVFN float2 item_pair<__nv_bfloat16>(const Item<__nv_bfloat16>& it, int i) {
    const uint4& w = it.w[i >> 2];
    const uint32_t v = (i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w;
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// Exponent byte of the head and the 16 codes of this lane's item.
template <typename T, int D>
ACACHE_DEVFN uint32_t quantise_item(const Item<T>& it, uint4& codes) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = item_pair<T>(it, i);
        top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
    }
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t s = q8_scale_byte(top);
    // 2^-e; a poisoned row stores zero codes (its exponent makes every element NaN)
    const float inv = s == kQ8Poison ? 0.f : __uint_as_float((254u - s) << 23);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = item_pair<T>(it, 2 * i), g = item_pair<T>(it, 2 * i + 1);
        c[i] = q8_encode2(f.x * inv, f.y * inv) | q8_encode2(g.x * inv, g.y * inv) << 16;
    }
    codes = s == kQ8Poison ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(c[0], c[1], c[2], c[3]);
    return s;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
q8_write_kernel(const int32_t* __restrict__ write_slot, int64_t nrows, int ipr, int64_t step_r, int step_c,
                const T* __restrict__ k_new, const T* __restrict__ v_new, uint8_t* __restrict__ k_cache,
                uint8_t* __restrict__ v_cache, uint8_t* __restrict__ kv_scale, int64_t num_slots,
                int64_t private_begin, int32_t* dev_status) {
    ptx::grid_launch_dependents();
    int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / ipr;
    int c = (int)(((int64_t)blockIdx.x * kThreads + threadIdx.x) - r * ipr);
    const int lane_in_head = threadIdx.x & (D / 16 - 1);
    // the trip count is the same for every lane of a warp: the shuffles need them all
    while (__any_sync(0xffffffffu, r < nrows)) {
        Item<T> k[kUnroll], v[kUnroll];
        int64_t slot[kUnroll], col[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            slot[u] = -1;
            col[u] = c;
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i) k[u].w[i] = v[u].w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < nrows) {
                const int64_t s = write_slot[r];
                const bool bad = s < 0 || s >= num_slots, shared = !bad && s < private_begin;
                if (c == 0 && (bad || shared)) flag(dev_status, bad ? ACACHE_DEV_BAD_SLOT : ACACHE_DEV_SHARED_WRITE);
                if (!bad && !shared) slot[u] = s;
                load_item<T>(k[u], k_new + (r * ipr + c) * 16);
                load_item<T>(v[u], v_new + (r * ipr + c) * 16);
            }
            r += step_r;
            c += step_c;
            if (c >= ipr) {
                c -= ipr;
                ++r;
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            uint4 ck, cv;
            const uint32_t sk = quantise_item<T, D>(k[u], ck), sv = quantise_item<T, D>(v[u], cv);
            if (slot[u] >= 0) {
                const int64_t item = slot[u] * ipr + col[u];
                reinterpret_cast<uint4*>(k_cache)[item] = ck;
                reinterpret_cast<uint4*>(v_cache)[item] = cv;
                if (lane_in_head == 0) {
                    reinterpret_cast<uint16_t*>(kv_scale)[item / (D / 16)] = (uint16_t)(sk | sv << 8);
                    if (sk == kQ8Poison || sv == kQ8Poison) flag(dev_status, ACACHE_DEV_BAD_VALUE);
                }
            }
        }
    }
}

// One 16-byte piece of the output: 4 float32 or 8 bf16 from as many codes, so that the lanes of a warp
// write whole lines (with 16 codes to a lane, as in the store, a lane's pieces of the output are 32
// or 64 bytes apart from the next lane's: twice the time).  One piece at a time: few registers, so all the
// warps an SM holds are there to keep loads in flight, and what they write stays close together: 26.4 us
// for 8 x 4,480 rows of 8 heads (d = 64, float32, 147 MB written: 0.86 of the copy bandwidth) and 119 us for 32 heads
// (d = 128, bf16, 587 MB: 0.80); with four pieces at a time 1.2 to 1.3 times that.
template <typename T> struct Piece;
template <> struct Piece<float> {
    using Codes = uint32_t;
    ACACHE_DEVFN static uint4 make(uint32_t c, float f) {
        const float2 a = q8_decode2(c & 0xffffu), b = q8_decode2(c >> 16);
        return make_uint4(__float_as_uint(a.x * f), __float_as_uint(a.y * f), __float_as_uint(b.x * f), __float_as_uint(b.y * f));
    }
};
template <> struct Piece<__nv_bfloat16> {
    using Codes = uint2;
    ACACHE_DEVFN static uint32_t pair(uint32_t two, float f) {
        const float2 a = q8_decode2(two);
        __nv_bfloat162 x = __floats2bfloat162_rn(a.x * f, a.y * f);
        return *reinterpret_cast<uint32_t*>(&x);
    }
    ACACHE_DEVFN static uint4 make(uint2 c, float f) {
        return make_uint4(pair(c.x & 0xffffu, f), pair(c.x >> 16, f), pair(c.y & 0xffffu, f), pair(c.y >> 16, f));
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
q8_gather_kernel(const int32_t* __restrict__ read_slot, int64_t nrows, int ipr, int64_t step_r, int step_c,
                 const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
                 const uint8_t* __restrict__ kv_scale, int64_t num_slots, T* __restrict__ k_out,
                 T* __restrict__ v_out, int32_t* dev_status) {
    using Codes = typename Piece<T>::Codes;
    constexpr int kPer = D / (int)sizeof(Codes);     // pieces of a head
    int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / ipr;
    int c = (int)(((int64_t)blockIdx.x * kThreads + threadIdx.x) - r * ipr);
    while (r < nrows) {
        const int64_t s = read_slot[r];
        if (s >= 0 && s < num_slots) {
            const int64_t src = s * ipr + c, dst = r * ipr + c;
            const Codes k = __ldg(reinterpret_cast<const Codes*>(k_cache) + src), v = __ldg(reinterpret_cast<const Codes*>(v_cache) + src);
            const uint32_t s2 = __ldg(reinterpret_cast<const uint16_t*>(kv_scale) + src / kPer);
            __stcs(reinterpret_cast<uint4*>(k_out) + dst, Piece<T>::make(k, q8_factor(s2 & 0xffu)));
            __stcs(reinterpret_cast<uint4*>(v_out) + dst, Piece<T>::make(v, q8_factor(s2 >> 8)));
        } else if (c == 0) {
            flag(dev_status, ACACHE_DEV_BAD_SLOT);
        }
        r += step_r;
        c += step_c;
        if (c >= ipr) {
            c -= ipr;
            ++r;
        }
    }
}

struct Shape {
    unsigned grid;
    int ipr;
    int64_t step_r;
    int step_c;
};
Shape item_shape(int64_t nrows, int ipr, int unroll) {
    Shape s;
    s.ipr = ipr;
    const int64_t items = nrows * s.ipr;
    int64_t want = (items + kThreads * unroll - 1) / (kThreads * unroll);
    const int64_t cap = (int64_t)sm_count() * 8;      // 8 resident CTAs of 256 threads per SM
    if (want > cap) want = cap;
    s.grid = (unsigned)(want < 1 ? 1 : want);
    const int64_t step = (int64_t)s.grid * kThreads;
    s.step_r = step / s.ipr;
    s.step_c = (int)(step - s.step_r * s.ipr);
    return s;
}

}  // namespace

#define ACACHE_Q8_DISPATCH(dtype, d, ...)                                                                     \
    do {                                                                                                      \
        if ((dtype) == ACACHE_F32 && (d) == 64) { using T = float; constexpr int D = 64; __VA_ARGS__; }       \
        else if ((dtype) == ACACHE_F32 && (d) == 128) { using T = float; constexpr int D = 128; __VA_ARGS__; } \
        else if ((dtype) == ACACHE_BF16 && (d) == 64) { using T = __nv_bfloat16; constexpr int D = 64; __VA_ARGS__; } \
        else if ((dtype) == ACACHE_BF16 && (d) == 128) { using T = __nv_bfloat16; constexpr int D = 128; __VA_ARGS__; } \
        else return ACACHE_ERR_UNSUPPORTED;                                                                   \
    } while (0)

int launch_q8_write(int dtype, int batch, int rows, int hkv, int d, const int32_t* write_slot, const void* k_new,
                    const void* v_new, uint8_t* k_cache, uint8_t* v_cache, uint8_t* kv_scale, int64_t num_slots,
                    int64_t private_begin, int32_t* dev_status, cudaStream_t stream) {
    const int64_t nrows = (int64_t)batch * rows;
    if (nrows == 0) return ACACHE_OK;
    const Shape s = item_shape(nrows, hkv * (d / 16), kUnroll);
    ACACHE_Q8_DISPATCH(dtype, d, {
        q8_write_kernel<T, D><<<s.grid, kThreads, 0, stream>>>(write_slot, nrows, s.ipr, s.step_r, s.step_c,
                                                               (const T*)k_new, (const T*)v_new, k_cache, v_cache,
                                                               kv_scale, num_slots, private_begin, dev_status);
        return launch_status();
    });
}

int launch_q8_gather(int dtype, int batch, int seq_len, int hkv, int d, const int32_t* read_slot,
                     const uint8_t* k_cache, const uint8_t* v_cache, const uint8_t* kv_scale, int64_t num_slots,
                     void* k_out, void* v_out, int32_t* dev_status, cudaStream_t stream) {
    const int64_t nrows = (int64_t)batch * seq_len;
    if (nrows == 0) return ACACHE_OK;
    const Shape s = item_shape(nrows, hkv * (d / (dtype == ACACHE_F32 ? 4 : 8)), 1);
    ACACHE_Q8_DISPATCH(dtype, d, {
        q8_gather_kernel<T, D><<<s.grid, kThreads, 0, stream>>>(read_slot, nrows, s.ipr, s.step_r, s.step_c, k_cache,
                                                                v_cache, kv_scale, num_slots, (T*)k_out, (T*)v_out,
                                                                dev_status);
        return launch_status();
    });
}

}  // namespace acache
