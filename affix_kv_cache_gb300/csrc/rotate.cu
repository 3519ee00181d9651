// rotate.cu -- per-head norm and rotary position of query and key rows: alone, and on the way into a
// 16-bit / float32 or an 8-bit pool.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4 and App. C.1 (the cache is kept after
// the rotation, and a recompute point stores its rows through the write-side map); norm, rotation and
// the 8-bit pool are this library's.
//
//   x' = x / sqrt(mean x^2 + eps) * w,   (a, b) -> A (a cos - b sin, a sin + b cos),   angle = p f_i
//
// Bound by memory: every element is read once and written once.  A warp takes a row (or with few rows a part of its
// heads), several heads at a time with d / (16-byte piece * 2) lanes to a head and two pieces to a lane, placed so that a pair's two
// elements lie in the same lane: pieces i and i + r/2 of the rotated part (half layout), or neighbours in a piece
// (interleaved).  Sums of squares and 8-bit scales go over a head's lanes by shuffles.  The angles of a row serve all of
// its heads: the warp computes their cosines and sines once, into shared memory, while the first heads are on their way.  An
// angle is exact modulo one turn: position times a frequency held in 2^-64 turns, in integers; only what is
// left within an eighth of a turn becomes a float.
// Measured (bf16, d = 128): 16 x 1,562 rows of 28 + 4 heads, half of each rotated, 68 us, 0.88 of the copy bandwidth; the normed
// store of 16 x 1,205 rows 66 us, 0.79 (latency: a warp loads two steps of a row, turns them and only then loads again; issue is
// active 47 % of the time, and most stalls wait for loads); 8,191 rows into an 8-bit pool with their read-back 48 us, 0.72 (the
// same).  float32: 138 us, 0.87, and 133 us, 0.79.  With the angles read from shared memory for every head 92 and 72 us (LDS
// wavefronts); a CTA to 8 rows behind one barrier 80 and 78 us.
#include <algorithm>

#include "q8.cuh"
#include "ptx.cuh"
#include "step.cuh"

namespace acache {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnroll = 2;                  // heads a lane has in flight
constexpr int kCtas = 3;                    // CTAs to an SM

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
    int nq, nk, hkv;                        // heads of the queries and keys that the call has; of the pool
    int q_steps, kv_steps, steps;           // of a row: of HPW heads each
    int parts, steps_per_part;              // of a row, for a warp each
    int half;                               // pairs
    float eps, amplitude;
    uint64_t phase[64];
};

template <int K> struct Kind { static constexpr int value = K; };

template <typename T> struct Word;          // a 16-byte piece, as pairs of float32
template <> struct Word<float> {
    static constexpr int kN = 4;
    ACACHE_DEVFN static void unpack(const uint4& w, uint64_t (&x)[2]) {
        x[0] = (uint64_t)w.y << 32 | w.x, x[1] = (uint64_t)w.w << 32 | w.z;
    }
    ACACHE_DEVFN static uint4 pack(const uint64_t (&x)[2]) {
        return make_uint4((uint32_t)x[0], (uint32_t)(x[0] >> 32), (uint32_t)x[1], (uint32_t)(x[1] >> 32));
    }
};
template <> struct Word<__nv_bfloat16> {
    static constexpr int kN = 8;
    ACACHE_DEVFN static void unpack(const uint4& w, uint64_t (&x)[4]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2pack(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    }
    ACACHE_DEVFN static uint4 pack(const uint64_t (&x)[4]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2unpack(x[i], a, b);
            __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
            u[i] = *reinterpret_cast<uint32_t*>(&two);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
ACACHE_DEVFN uint64_t f2mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// P pairs of floats from shared memory, 16 bytes at a time
template <int P>
ACACHE_DEVFN void pairs_at(const float* at, uint64_t (&x)[P]) {
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(at + 2 * i);
        x[i] = v.x;
        x[i + 1] = v.y;
    }
}

// The weights of a piece of N elements.
template <int N, int D>
ACACHE_DEVFN void weights_at(const float* w, int piece, uint64_t (&x)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(w + i * (D / N * 4) + piece * 4);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
    }
}

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
__global__ void __launch_bounds__(kThreads, kCtas)
rotate_kernel(const __grid_constant__ RotateParams p) {
    using W = Word<T>;
    constexpr int N = W::kN, P = N / 2, LPH = D / (2 * N), HPW = 32 / LPH;   // elements and pairs a piece, lanes a head, heads a warp
    __shared__ __align__(16) float s_cos[kWarps][64], s_sin[kWarps][64];   // of a warp's row
    __shared__ __align__(16) float s_w[2][D];                              // 4 elements of each piece after 4 of each (no bank conflicts)
    __shared__ float s_head[kLayout == kHalfAny ? kWarps * HPW * D : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPH, j = lane % LPH;
    // the lane's two pieces of a head
    const int hp = kLayout == kHalfPieces ? p.half / N : 0;            // pieces in the first half
    const int pa = kLayout == kHalfPieces && j >= hp ? hp + j : j;
    const int pb = kLayout == kHalfPieces ? (j < hp ? j + hp : LPH + j) : j + LPH;
    const bool turns = kLayout == kHalfPieces && j < hp;
    const bool normed = p.q_weight || p.k_weight;
    // Unit u: part u % parts of row u / parts.  A row's steps take HPW heads each: first the queries', then the keys', then
    // the values'.
    const int64_t n_units = p.rows * p.parts, n_warps = (int64_t)gridDim.x * kWarps;
    int64_t u = (int64_t)blockIdx.x * kWarps + warp;
    int64_t row = u / p.parts;
    int32_t pos = 0, slot = 0;
    auto look_up = [&]() {                  // the row's position and slot, a unit ahead
        if (u < n_units) {
            if (p.half) pos = p.positions[row];
            if (kMode != kRotate) slot = p.write_slot[row];
        }
    };
    look_up();
    if (normed) {
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            const T* w = (const T*)(i < D ? p.q_weight : p.k_weight);
            const int e = i % D;
            s_w[i / D][(e % N) / 4 * (D / N * 4) + e / N * 4 + e % 4] = w ? to_f32(w[e]) : 1.f;
        }
        __syncthreads();
    }
    float* const t_cos = s_cos[warp];
    float* const t_sin = s_sin[warp];
    while (u < n_units) {
        const int64_t at_row = row;
        const int32_t at_pos = pos, at_slot = slot;
        const int i0 = (int)(u - row * p.parts) * p.steps_per_part, i1 = min(p.steps, i0 + p.steps_per_part);
        u += n_warps;
        row = u / p.parts;
        look_up();
        bool stores = true;                  // the row's keys and values
        if (kMode != kRotate) {
            const bool bad = at_slot < 0 || at_slot >= p.num_slots, shared = !bad && at_slot < p.private_begin;
            stores = !bad && !shared;
            if (!stores && lane == 0 && i0 == 0) flag(p.dev_status, bad ? ACACHE_DEV_BAD_SLOT : ACACHE_DEV_SHARED_WRITE);
        }
        uint64_t rc[P], rs[P];               // cosines and sines: of the lane's pairs; interleaved: of pair x of either piece
        bool table = false;
        // the row's angles, once a first step's heads are on their way
        auto angles = [&]() {
            table = true;
            __syncwarp();
            for (int f = lane; f < p.half; f += 32) {
                // the angle in 2^-64 turns, then quarter turns and what is left, within half of one either way
                const uint64_t turn = (uint64_t)(int64_t)at_pos * p.phase[f];
                const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
                float s, c;
                sincospif((float)(int64_t)(turn - ((uint64_t)quarter << 62)) * 0x1p-63f, &s, &c);
                const float c1 = (quarter & 1u ? s : c) * p.amplitude, s1 = (quarter & 1u ? c : s) * p.amplitude;
                t_cos[f] = quarter == 1u || quarter == 2u ? -c1 : c1;
                t_sin[f] = quarter >= 2u ? -s1 : s1;
            }
            __syncwarp();
            // the lane's, for all heads of the row: the same places of each
            if (kLayout == kHalfPieces && turns) {
                pairs_at<P>(&t_cos[j * N], rc);
                pairs_at<P>(&t_sin[j * N], rs);
            }
            if (kLayout == kPairs) {
#pragma unroll
                for (int x = 0; x < P; ++x) {
                    const int ia = min(pa * P + x, 63), ib = min(pb * P + x, 63);
                    rc[x] = f2pack(t_cos[ia], t_cos[ib]);
                    rs[x] = f2pack(t_sin[ia], t_sin[ib]);
                }
            }
        };
        // norm and rotation of a head
        auto turn_head = [&](uint64_t (&a)[P], uint64_t (&b)[P], const float* w) {
            float f = 1.f;
            if (w) {
                uint64_t ss2 = f2mul(a[0], a[0]), st2 = f2mul(b[0], b[0]);
#pragma unroll
                for (int x = 1; x < P; ++x) {
                    ss2 = f2fma(a[x], a[x], ss2);
                    st2 = f2fma(b[x], b[x], st2);
                }
                float s0, s1;
                f2unpack(f2add(ss2, st2), s0, s1);
                float ss = s0 + s1;
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                f = rsqrtf(fmaf(ss, 1.f / D, p.eps));
                const uint64_t f2 = f2pack(f, f);
                uint64_t wa[P], wb[P];
                weights_at<N, D>(w, pa, wa);
                weights_at<N, D>(w, pb, wb);
#pragma unroll
                for (int x = 0; x < P; ++x) {
                    a[x] = f2mul(f2mul(a[x], f2), wa[x]);
                    b[x] = f2mul(f2mul(b[x], f2), wb[x]);
                }
            }
            if (kLayout == kHalfAny) {
                // partners may lie with other lanes: the head through shared memory
                float* head = &s_head[(warp * HPW + sub) * D];
                __syncwarp();
#pragma unroll
                for (int x = 0; x < P; ++x) {
                    f2unpack(a[x], head[pa * N + 2 * x], head[pa * N + 2 * x + 1]);
                    f2unpack(b[x], head[pb * N + 2 * x], head[pb * N + 2 * x + 1]);
                }
                __syncwarp();
                auto turn = [&](int e) {
                    const float v = head[e];
                    if (e >= 2 * p.half) return v;
                    const bool lo = e < p.half;
                    const int i = lo ? e : e - p.half;
                    const float w = head[lo ? e + p.half : i], c = t_cos[i], s = t_sin[i];
                    return lo ? fmaf(v, c, -w * s) : fmaf(w, s, v * c);
                };
#pragma unroll
                for (int x = 0; x < P; ++x) {
                    a[x] = f2pack(turn(pa * N + 2 * x), turn(pa * N + 2 * x + 1));
                    b[x] = f2pack(turn(pb * N + 2 * x), turn(pb * N + 2 * x + 1));
                }
            } else if (kLayout == kHalfPieces) {
                if (turns) {
                    const uint64_t minus = f2pack(-1.f, -1.f);
#pragma unroll
                    for (int x = 0; x < P; ++x) {
                        const uint64_t lo = a[x], hi = b[x];
                        a[x] = f2fma(lo, rc[x], f2mul(f2mul(hi, minus), rs[x]));
                        b[x] = f2fma(lo, rs[x], f2mul(hi, rc[x]));
                    }
                }
            } else {
#pragma unroll
                for (int x = 0; x < P; ++x) {
                    float ca, cb, sa, sb, lo, hi;
                    f2unpack(rc[x], ca, cb);
                    f2unpack(rs[x], sa, sb);
                    if (pa * P + x < p.half) {                       // (the rotated part may end inside a piece)
                        f2unpack(a[x], lo, hi);
                        a[x] = f2pack(fmaf(lo, ca, -hi * sa), fmaf(lo, sa, hi * ca));
                    }
                    if (pb * P + x < p.half) {
                        f2unpack(b[x], lo, hi);
                        b[x] = f2pack(fmaf(lo, cb, -hi * sb), fmaf(lo, sb, hi * cb));
                    }
                }
            }
        };
        // a head of the 8-bit pool: its codes and exponent
        auto store_q8 = [&](const uint64_t (&a)[P], const uint64_t (&b)[P], uint8_t* pool, int hh, int which, bool live) {
            float fa[N], fb[N];
#pragma unroll
            for (int x = 0; x < P; ++x) {
                f2unpack(a[x], fa[2 * x], fa[2 * x + 1]);
                f2unpack(b[x], fb[2 * x], fb[2 * x + 1]);
            }
            uint32_t top = 0;
#pragma unroll
            for (int x = 0; x < N; ++x)
                top = max(top, max(__float_as_uint(fa[x]) & 0x7fffffffu, __float_as_uint(fb[x]) & 0x7fffffffu));
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (!live) return;
            const uint32_t s = q8_scale_byte(top);
            const int64_t item = (int64_t)at_slot * p.hkv + hh;
            uint8_t* to = pool + item * D;
            // 2^-e; a poisoned row stores zero codes (its exponent makes every element NaN)
            const float inv = s == kQ8Poison ? 0.f : __uint_as_float((254u - s) << 23);
            if (s == kQ8Poison) {
#pragma unroll
                for (int x = 0; x < N; ++x) fa[x] = fb[x] = 0.f;
            }
            store_codes(to + pa * N, fa, inv);
            store_codes(to + pb * N, fb, inv);
            if (j == 0) {
                p.kv_scale[2 * item + which] = (uint8_t)s;
                if (s == kQ8Poison) flag(p.dev_status, ACACHE_DEV_BAD_VALUE);
            }
        };
        // steps [from, to) of one matrix (kKind 0 queries, 1 keys, 2 values) of `heads` heads
        auto run = [&](auto kind, int from, int to, int heads, const T* src, T* dst, const float* w) {
            constexpr int kKind = decltype(kind)::value;
            const uint4* sa = reinterpret_cast<const uint4*>(src) + sub * (D / N) + pa;
            uint4* da = reinterpret_cast<uint4*>(dst) + sub * (D / N) + pa;
            const int ab = pb - pa;
            for (int i = from; i < to; i += kUnroll) {
                uint4 la[kUnroll], lb[kUnroll];
#pragma unroll
                for (int n = 0; n < kUnroll; ++n) {
                    la[n] = lb[n] = make_uint4(0u, 0u, 0u, 0u);
                    if (i + n < to && (i + n) * HPW + sub < heads) {
                        la[n] = __ldcs(sa + (i + n) * 32 * 2);
                        lb[n] = __ldcs(sa + (i + n) * 32 * 2 + ab);
                    }
                }
                if (kKind != 2 && !table) angles();
#pragma unroll
                for (int n = 0; n < kUnroll; ++n) {
                    if (i + n >= to) break;                          // (the same for the whole warp)
                    const bool live = (i + n) * HPW + sub < heads && (kKind == 0 || stores);
                    if (kKind == 2 && kMode != kRotateStoreQ8) {
                        if (live) {
                            da[(i + n) * 32 * 2] = la[n];
                            da[(i + n) * 32 * 2 + ab] = lb[n];
                        }
                        continue;
                    }
                    uint64_t a[P], b[P];
                    W::unpack(la[n], a);
                    W::unpack(lb[n], b);
                    if (kKind != 2) turn_head(a, b, w);
                    if (kKind != 0 && kMode == kRotateStoreQ8) {
                        store_q8(a, b, (uint8_t*)(kKind == 1 ? p.k_out : p.v_out), (i + n) * HPW + sub, kKind - 1, live);
                    } else if (live) {
                        da[(i + n) * 32 * 2] = W::pack(a);
                        da[(i + n) * 32 * 2 + ab] = W::pack(b);
                    }
                }
            }
        };
        const int nq = p.q_steps, nk = p.kv_steps;               // of a matrix
        if (i0 < nq)
            run(Kind<0>{}, i0, min(i1, nq), p.nq, (const T*)p.q + at_row * p.q_stride, (T*)p.q_out + at_row * p.q_out_stride,
                p.q_weight ? s_w[0] : nullptr);
        const int64_t at = kMode == kRotate ? at_row * p.k_out_stride : (int64_t)at_slot * p.hkv * D;
        if (p.nk && i0 < nq + nk && i1 > nq)
            run(Kind<1>{}, max(i0 - nq, 0), min(i1 - nq, nk), p.nk, (const T*)p.k + at_row * p.k_stride, (T*)p.k_out + at,
                p.k_weight ? s_w[1] : nullptr);
        if (kMode != kRotate && i1 > nq + nk)
            run(Kind<2>{}, max(i0 - nq - nk, 0), i1 - nq - nk, p.hkv, (const T*)p.v + at_row * p.v_stride, (T*)p.v_out + at, nullptr);
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
    p.eps = c.eps;
    Layout layout = kPairs;
    if (c.rope) {
        p.half = c.rope->rotary_dim / 2;
        p.amplitude = c.rope->amplitude;
        for (int i = 0; i < p.half; ++i) p.phase[i] = c.rope->phase[i];
        layout = c.rope->interleaved ? kPairs : p.half % n == 0 ? kHalfPieces : kHalfAny;
    }
    // A warp to a row; with few rows several, down to a step for each.
    const int hpw = 32 / (d / (2 * n));
    p.q_steps = (p.nq + hpw - 1) / hpw;
    p.kv_steps = p.nk ? (p.nk + hpw - 1) / hpw : 0;
    p.steps = p.q_steps + p.kv_steps * (mode == kRotate ? 1 : 2);
    const int64_t slots = (int64_t)sm_count() * kCtas * kWarps;
    p.parts = (int)std::min<int64_t>(p.steps, std::max<int64_t>(1, slots / c.rows));
    p.steps_per_part = (p.steps + p.parts - 1) / p.parts;
    p.parts = (p.steps + p.steps_per_part - 1) / p.steps_per_part;
    const int64_t blocks = std::min<int64_t>((c.rows * p.parts + kWarps - 1) / kWarps, slots / kWarps);
    const dim3 grid((unsigned)blocks);
    if (c.a.dtype == ACACHE_F32)
        return d == 64 ? launch_mode<float, 64>(p, mode, layout, grid, c.stream) : launch_mode<float, 128>(p, mode, layout, grid, c.stream);
    return d == 64 ? launch_mode<__nv_bfloat16, 64>(p, mode, layout, grid, c.stream)
                   : launch_mode<__nv_bfloat16, 128>(p, mode, layout, grid, c.stream);
}

}  // namespace acache
