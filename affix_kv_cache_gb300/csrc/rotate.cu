// rotate.cu -- per-head norm and rotary position of query and key rows: alone, and on the way into a
// 16-bit / float32 or an 8-bit pool.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4 and App. C.1 (the cache is kept after
// the rotation, and a recompute point stores its rows through the write-side map); norm, rotation and
// the 8-bit pool are this library's.
//
//   x' = x / sqrt(mean x^2 + eps) * w,   (a, b) -> A (a cos - b sin, a sin + b cos),   angle = p f_i
//
// Bound by memory: every element is read once and written once.  The item is one head of one row, taken
// by d / (16-byte piece * 2) lanes with two pieces each, placed so that a pair's two elements lie in the same
// lane: pieces i and i + r/2 of the rotated part (half layout), or neighbours in a piece (interleaved).  Sums of
// squares and 8-bit scales go over the item's lanes by shuffles.  The angles of a row serve all of its heads: a
// CTA takes a few rows, computes their cosines and sines once into shared memory, and its items read them
// from there.  The angle is exact modulo one turn: position times a frequency held in 2^-64 turns, in
// integers; only what is left within half a turn becomes a float.
#include <algorithm>

#include "q8.cuh"
#include "ptx.cuh"
#include "step.cuh"

namespace acache {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;                 // rows of a CTA

// How a head's pairs lie: in two pieces of a lane, inside a piece, or anywhere (half layout whose half is
// no whole number of pieces: through shared memory).
enum Layout { kHalfPieces = 0, kPairs = 1, kHalfAny = 2 };

struct RotateParams {
    const void *q, *k, *v;
    const void *q_weight, *k_weight;
    void *q_out, *k_out;                    // k_out: rows, or the pool of keys
    void* v_out;                            // the pool of values
    uint8_t* kv_scale;
    const int32_t *positions, *write_slot;
    int64_t rows, q_stride, k_stride, v_stride, q_out_stride, k_out_stride, num_slots, private_begin;
    int32_t* dev_status;
    int nq, nk, heads;                      // query heads, KV heads of the call's items; all items of a row
    int hkv;
    int rows_per_cta, heads_per_cta;
    int half;                               // pairs
    float eps, amplitude;
    uint64_t phase[64];
};

template <typename T> struct Word;          // a 16-byte piece
template <> struct Word<float> {
    static constexpr int kN = 4;
    ACACHE_DEVFN static void unpack(const uint4& w, float (&x)[4]) {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
    ACACHE_DEVFN static uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <> struct Word<__nv_bfloat16> {
    static constexpr int kN = 8;
    ACACHE_DEVFN static void unpack(const uint4& w, float (&x)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    ACACHE_DEVFN static uint4 pack(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 two = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<uint32_t*>(&two);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// N codes of e4m3 of x * inv
ACACHE_DEVFN void store_codes(uint8_t* at, const float (&x)[8], float inv) {
    const uint32_t a = q8_encode2(x[0] * inv, x[1] * inv) | q8_encode2(x[2] * inv, x[3] * inv) << 16;
    const uint32_t b = q8_encode2(x[4] * inv, x[5] * inv) | q8_encode2(x[6] * inv, x[7] * inv) << 16;
    *reinterpret_cast<uint2*>(at) = make_uint2(a, b);
}
ACACHE_DEVFN void store_codes(uint8_t* at, const float (&x)[4], float inv) {
    *reinterpret_cast<uint32_t*>(at) = q8_encode2(x[0] * inv, x[1] * inv) | q8_encode2(x[2] * inv, x[3] * inv) << 16;
}

template <typename T, int D, int kMode, int kLayout>
__global__ void __launch_bounds__(kThreads)
rotate_kernel(const __grid_constant__ RotateParams p) {
    using W = Word<T>;
    constexpr int N = W::kN, LPH = D / (2 * N), G = kThreads / LPH;   // elements a piece, lanes a head, heads at a time
    __shared__ __align__(16) float s_cos[kMaxRows][64], s_sin[kMaxRows][64], s_w[2][D];
    __shared__ float s_head[kLayout == kHalfAny ? G * D : 1];
    if (kMode != kRotate) ptx::grid_launch_dependents();
    const int64_t row0 = (int64_t)blockIdx.x * p.rows_per_cta;
    const int n_rows = (int)min((int64_t)p.rows_per_cta, p.rows - row0);
    const int h0 = (int)blockIdx.y * p.heads_per_cta, n_heads = min(p.heads_per_cta, p.heads - h0);
    const bool normed = p.q_weight || p.k_weight;
    if (normed)
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            const T* w = (const T*)(i < D ? p.q_weight : p.k_weight);
            s_w[i / D][i % D] = w ? to_f32(w[i % D]) : 1.f;
        }
    for (int i = threadIdx.x; i < n_rows * p.half; i += kThreads) {
        const int r = i / p.half, f = i - r * p.half;
        const uint64_t turn = (uint64_t)(int64_t)p.positions[row0 + r] * p.phase[f];
        // half turns in [-1, 1)
        float s, c;
        sincospif((float)(int64_t)turn * 0x1p-63f, &s, &c);
        s_cos[r][f] = c * p.amplitude;
        s_sin[r][f] = s * p.amplitude;
    }
    __syncthreads();
    const int grp = threadIdx.x / LPH, j = threadIdx.x % LPH;
    // the lane's two pieces of a head
    const int hp = kLayout == kHalfPieces ? p.half / N : 0;            // pieces in the first half
    const int pa = kLayout == kHalfPieces && j >= hp ? hp + j : j;
    const int pb = kLayout == kHalfPieces ? (j < hp ? j + hp : LPH + j) : j + LPH;
    const bool turns = kLayout == kHalfPieces && j < hp;
    const int n_items = n_rows * n_heads;
    // (the trip count is the same for every lane of a CTA: the shuffles need them all)
    for (int it0 = 0; it0 < n_items; it0 += G) {
        const int it = it0 + grp;
        const bool live = it < n_items;
        const int r = live ? it / n_heads : 0, h = h0 + (live ? it - r * n_heads : 0);
        const int64_t row = row0 + r;
        const int kind = h < p.nq ? 0 : h < p.nq + p.nk ? 1 : 2;     // query, key or value head
        const int hh = h - (kind == 0 ? 0 : kind == 1 ? p.nq : p.nq + p.nk);
        const T* src = kind == 0 ? (const T*)p.q + row * p.q_stride : kind == 1 ? (const T*)p.k + row * p.k_stride
                                                                                : (const T*)p.v + row * p.v_stride;
        uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
        int64_t slot = 0;
        bool stores = live;
        if (live) {
            const uint4* at = reinterpret_cast<const uint4*>(src + (int64_t)hh * D);
            wa = __ldcs(at + pa);
            wb = __ldcs(at + pb);
            if (kMode != kRotate && kind != 0) {
                slot = p.write_slot[row];
                const bool bad = slot < 0 || slot >= p.num_slots, shared = !bad && slot < p.private_begin;
                stores = !bad && !shared;
                if (!stores && kind == 1 && hh == 0 && j == 0) flag(p.dev_status, bad ? ACACHE_DEV_BAD_SLOT : ACACHE_DEV_SHARED_WRITE);
            }
        }
        float a[N], b[N];
        W::unpack(wa, a);
        W::unpack(wb, b);
        if (normed) {
            float ss = 0.f;
#pragma unroll
            for (int x = 0; x < N; ++x) ss = fmaf(a[x], a[x], fmaf(b[x], b[x], ss));
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (kind == 0 ? p.q_weight != nullptr : kind == 1 && p.k_weight != nullptr) {
                const float f = 1.f / sqrtf(fmaf(ss, 1.f / D, p.eps));
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    a[x] = a[x] * f * s_w[kind][pa * N + x];
                    b[x] = b[x] * f * s_w[kind][pb * N + x];
                }
            }
        }
        if (kLayout == kHalfAny) {
            // partners may lie with other lanes: the head through shared memory
            __syncwarp();
#pragma unroll
            for (int x = 0; x < N; ++x) {
                s_head[grp * D + pa * N + x] = a[x];
                s_head[grp * D + pb * N + x] = b[x];
            }
            __syncwarp();
            if (kind != 2) {
                auto turn = [&](int e, float v) {
                    if (e >= 2 * p.half) return v;
                    const bool lo = e < p.half;
                    const int i = lo ? e : e - p.half;
                    const float w = s_head[grp * D + (lo ? e + p.half : i)], c = s_cos[r][i], s = s_sin[r][i];
                    return lo ? fmaf(v, c, -w * s) : fmaf(w, s, v * c);
                };
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    a[x] = turn(pa * N + x, a[x]);
                    b[x] = turn(pb * N + x, b[x]);
                }
            }
        } else if (kLayout == kHalfPieces) {
            if (turns && kind != 2) {
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    const float c = s_cos[r][j * N + x], s = s_sin[r][j * N + x], lo = a[x], hi = b[x];
                    a[x] = fmaf(lo, c, -hi * s);
                    b[x] = fmaf(lo, s, hi * c);
                }
            }
        } else if (kind != 2) {
            auto turn = [&](int i, float& lo, float& hi) {
                if (i >= p.half) return;
                const float c = s_cos[r][i], s = s_sin[r][i], x = lo, y = hi;
                lo = fmaf(x, c, -y * s);
                hi = fmaf(x, s, y * c);
            };
#pragma unroll
            for (int x = 0; x < N; x += 2) {
                turn((pa * N + x) / 2, a[x], a[x + 1]);
                turn((pb * N + x) / 2, b[x], b[x + 1]);
            }
        }
        if (kMode == kRotateStoreQ8) {
            uint32_t top = 0;
#pragma unroll
            for (int x = 0; x < N; ++x)
                top = max(top, max(__float_as_uint(a[x]) & 0x7fffffffu, __float_as_uint(b[x]) & 0x7fffffffu));
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (kind != 0 && stores) {
                const uint32_t s = q8_scale_byte(top);
                const int64_t item = slot * p.hkv + hh;
                uint8_t* to = (uint8_t*)(kind == 1 ? p.k_out : p.v_out) + item * D;
                // 2^-e; a poisoned row stores zero codes (its exponent makes every element NaN)
                const float inv = s == kQ8Poison ? 0.f : __uint_as_float((254u - s) << 23);
                if (s == kQ8Poison) {
#pragma unroll
                    for (int x = 0; x < N; ++x) a[x] = b[x] = 0.f;
                }
                store_codes(to + pa * N, a, inv);
                store_codes(to + pb * N, b, inv);
                if (j == 0) {
                    p.kv_scale[2 * item + (kind - 1)] = (uint8_t)s;
                    if (s == kQ8Poison) flag(p.dev_status, ACACHE_DEV_BAD_VALUE);
                }
                continue;
            }
        }
        if (!stores || (kMode == kRotateStoreQ8 && kind != 0)) continue;
        T* to = kind == 0 ? (T*)p.q_out + row * p.q_out_stride
                          : kMode == kRotate ? (T*)p.k_out + row * p.k_out_stride
                                             : (T*)(kind == 1 ? p.k_out : p.v_out) + slot * p.hkv * D;
        uint4* at = reinterpret_cast<uint4*>(to + (int64_t)hh * D);
        at[pa] = kind == 2 ? wa : W::pack(a);
        at[pb] = kind == 2 ? wb : W::pack(b);
    }
}

template <typename T, int D, int kMode>
int launch_layout(const RotateParams& p, Layout layout, dim3 grid, cudaStream_t stream) {
    switch (layout) {
        case kHalfPieces: rotate_kernel<T, D, kMode, kHalfPieces><<<grid, kThreads, 0, stream>>>(p); break;
        case kPairs: rotate_kernel<T, D, kMode, kPairs><<<grid, kThreads, 0, stream>>>(p); break;
        default: rotate_kernel<T, D, kMode, kHalfAny><<<grid, kThreads, 0, stream>>>(p); break;
    }
    return launch_status();
}

template <typename T, int D>
int launch_mode(const RotateParams& p, RotateMode mode, Layout layout, dim3 grid, cudaStream_t stream) {
    switch (mode) {
        case kRotate: return launch_layout<T, D, kRotate>(p, layout, grid, stream);
        case kRotateStore: return launch_layout<T, D, kRotateStore>(p, layout, grid, stream);
        default: return launch_layout<T, D, kRotateStoreQ8>(p, layout, grid, stream);
    }
}

}  // namespace

int launch_rotate(const RotateCall& c, RotateMode mode) {
    RotateParams p{};
    const int d = c.a.d, n = c.a.dtype == ACACHE_F32 ? 4 : 8;
    p.q = c.q;
    p.k = c.k;
    p.v = c.v;
    p.q_weight = c.q ? c.q_weight : nullptr;
    p.k_weight = c.k ? c.k_weight : nullptr;
    p.q_out = c.q_out;
    p.k_out = mode == kRotate ? c.k_out : c.k_cache;
    p.v_out = c.v_cache;
    p.kv_scale = c.kv_scale;
    p.positions = c.positions;
    p.write_slot = c.write_slot;
    p.rows = c.rows;
    p.q_stride = c.q_stride;
    p.k_stride = c.k_stride;
    p.v_stride = c.v_stride;
    p.q_out_stride = c.q_out_stride;
    p.k_out_stride = c.k_out_stride;
    p.num_slots = c.num_slots;
    p.private_begin = c.private_begin;
    p.dev_status = c.dev_status;
    p.hkv = c.a.hkv;
    p.nq = c.q ? c.a.hq : 0;
    p.nk = c.k ? c.a.hkv : 0;
    p.heads = p.nq + p.nk + (mode == kRotate ? 0 : c.a.hkv);
    p.eps = c.eps;
    Layout layout = kPairs;
    if (c.rope) {
        p.half = c.rope->rotary_dim / 2;
        p.amplitude = c.rope->amplitude;
        for (int i = 0; i < p.half; ++i) p.phase[i] = c.rope->phase[i];
        layout = c.rope->interleaved ? kPairs : p.half % n == 0 ? kHalfPieces : kHalfAny;
    }
    // Rows of a CTA: as many as leave every SM a few CTAs; with few rows their heads are spread.
    const int g = kThreads / (d / (2 * n));
    const int64_t want = 4LL * sm_count();
    p.rows_per_cta = (int)std::min<int64_t>(kMaxRows, std::max<int64_t>(1, c.rows / want));
    p.heads_per_cta = p.heads;
    const int64_t blocks = (c.rows + p.rows_per_cta - 1) / p.rows_per_cta;
    if (blocks < want) {
        const int64_t parts = std::min<int64_t>((p.heads + g - 1) / g, (want + blocks - 1) / blocks);
        p.heads_per_cta = (int)((p.heads + parts - 1) / parts);
    }
    // (an item's number within a CTA: rows_per_cta * heads <= 8 * 3 * 2^20)
    const dim3 grid((unsigned)blocks, (unsigned)((p.heads + p.heads_per_cta - 1) / p.heads_per_cta));
    if (blocks > 0x7fffffffLL || grid.y > 65535) return ACACHE_ERR_INVALID_ARG;
    if (c.a.dtype == ACACHE_F32)
        return d == 64 ? launch_mode<float, 64>(p, mode, layout, grid, c.stream) : launch_mode<float, 128>(p, mode, layout, grid, c.stream);
    return d == 64 ? launch_mode<__nv_bfloat16, 64>(p, mode, layout, grid, c.stream)
                   : launch_mode<__nv_bfloat16, 128>(p, mode, layout, grid, c.stream);
}

}  // namespace acache
