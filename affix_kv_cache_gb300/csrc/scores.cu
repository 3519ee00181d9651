// scores.cu -- token scores: log probabilities of given tokens, entropy and the likeliest tokens of rows of
// logits, each row read once.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 5 (decoding keeps the masked positions whose likeliest
// token passes a confidence threshold).
//
//   M = max x,  d = (x - M) log2e / temperature,  S = sum 2^d,  U = sum 2^d d
//   log p(t) = (x_t - M) / temperature - ln S,   entropy = ln S - ln2 U / S
//
// Bound by memory.  A row's 16-byte pieces go round the threads of a CTA (or, with few rows, of a cluster);
// every thread keeps its own reference in place of M (within 2^6 of its maximum, so next to nothing cancels between the
// terms of the entropy), S and U.
// The k likeliest: candidates are compared by (value, lower token), all different.  The k-th best of the groups of threads,
// each by its best logit, is a bound that k elements reach, so only threads whose best reaches it are looked at again, a
// warp to the pieces of one, for the elements that do; these -- few more than k -- are ranked by comparing all
// with all.
// Measured: 4,100 rows of 100,003 in bf16 146 us with 5 alternatives (0.82 of the copy bandwidth; 138 without, 200 with 32); 128 rows
// of 126,464 13 us on the device (launch, two dependent loads, five barriers and a merge beside 5 us of
// reading); one row of 32,000 in float32 with 20 alternatives 7.5 us.
#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"
#include "step.cuh"

namespace acache {
namespace {

constexpr int kMaxK = ACACHE_MAX_ALTERNATIVES;
constexpr int kMaxCluster = 8;
constexpr int kList = 1024;                 // candidates of a CTA
constexpr float kNone = -3.402823466e38f;   // maximum before any logit (lowest finite value: as a logit it counts)
constexpr float kLowest = -200.f;           // d from here on down is a weight of zero
constexpr float kHead = 6.f, kFloor = 300.f;   // log2 units: how far a logit may pass the reference; where a floor under it lies
constexpr int kBatch = 4;                   // pieces in flight
// CTAs to an SM: 1,536 threads (40 registers); of 64 and 32 threads 22, as many as their 9 KB of shared memory, most of it the
// list, let in (1,408 and 704 threads)
constexpr int ctas(int nt) { return nt >= 128 ? 1536 / nt : 22; }

struct ScoreParams {
    const void* logits;
    int64_t row_stride;
    const int32_t* tokens;
    float *token_logprob, *entropy, *top_logprob;
    int32_t *top_tokens, *dev_status;
    int vocab, k, cs;
    float to_log2;                          // log2e / temperature
    float half, far_log2, far_ln;           // differences of any two logits: taken of their halves (half = 1/2) where the
                                            // temperature is above 1, as the quotient can be a number where the difference
                                            // is not; log2e / temperature and 1 / temperature over `half`
    float head, floor_gap;                  // kHead and kFloor in logits
    bool far;                               // a weight that counts may lie further than the end of float32 from the largest
};

ACACHE_DEVFN float max_nan(float a, float b) {
    float c;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
    return c;
}
ACACHE_DEVFN uint64_t f2mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <typename T> struct Piece;
template <> struct Piece<float> {
    static constexpr int kN = 4;
    static constexpr uint32_t kNegInf = 0xff800000u;
    ACACHE_DEVFN static float at(const uint4& w, int i) { return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w); }
    ACACHE_DEVFN static float top(const uint4& w) { return fmaxf(fmaxf(at(w, 0), at(w, 1)), fmaxf(at(w, 2), at(w, 3))); }
    template <int B> ACACHE_DEVFN static float top(const uint4 (&w)[B]) {
        float m = top(w[0]);
#pragma unroll
        for (int u = 1; u < B; ++u) m = fmaxf(m, top(w[u]));
        return m;
    }
    // Elements e, e + 1; weights' exponents are bounded from below one by one (far: differences that count may leave float32).
    struct Floor {};
    ACACHE_DEVFN static Floor floor_of(float, float) { return {}; }
    ACACHE_DEVFN static bool bounds(Floor, bool far) { return !far; }
    ACACHE_DEVFN static uint64_t pair(const uint4& w, int e, Floor) { return f2pack(at(w, e), at(w, e + 1)); }
    ACACHE_DEVFN static void bound(float& a, float& b) {
        a = max_nan(a, kLowest);
        b = max_nan(b, kLowest);
    }
    ACACHE_DEVFN static void put(uint4& w, int i, float x) {
        const uint32_t u = __float_as_uint(x);
        if (i == 0) w.x = u;
        if (i == 1) w.y = u;
        if (i == 2) w.z = u;
        if (i == 3) w.w = u;
    }
};
template <> struct Piece<__nv_bfloat16> {
    static constexpr int kN = 8;
    static constexpr uint32_t kNegInf = 0xff80ff80u;
    ACACHE_DEVFN static float at(const uint4& w, int i) {
        const uint32_t v = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
        return __uint_as_float(i & 1 ? v & 0xffff0000u : v << 16);
    }
    ACACHE_DEVFN static float top(const uint4& w) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    template <int B> ACACHE_DEVFN static float top(const uint4 (&w)[B]) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w[0]);
        __nv_bfloat162 m[4] = {h[0], h[1], h[2], h[3]};
#pragma unroll
        for (int i = 4; i < 4 * B; ++i) m[i & 3] = __hmax2(m[i & 3], h[i]);
        m[0] = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
        return fmaxf(__low2float(m[0]), __high2float(m[0]));
    }
    // Elements e, e + 1, raised to a floor below which a weight is zero all the same: two to an instruction.  The floor
    // lies kFloor in log2 units below the reference, and by more than its rounding, at most 1.01 gap + |m| / 42; 0: there
    // is no such bf16 value, or its distance in log2 units (|m| / 42 of kFloor / gap) might leave float32, and a weight
    // of zero times that in the entropy's sum were NaN.
    using Floor = uint32_t;
    ACACHE_DEVFN static Floor floor_of(float m, float gap) {
        const float f = m - gap - fabsf(m) * 0.015625f;
        if (!(f > -3.3e38f) || fabsf(m) > gap * 1e36f) return 0u;
        const uint32_t u = __float_as_uint(f) >> 16;         // (cut: a little more for negative ones, less for others)
        return u | u << 16;
    }
    ACACHE_DEVFN static bool bounds(Floor f, bool) { return f != 0u; }
    ACACHE_DEVFN static uint64_t pair(const uint4& w, int e, Floor f) {
        uint32_t v = e == 0 ? w.x : e == 2 ? w.y : e == 4 ? w.z : w.w;
        const __nv_bfloat162 h = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&f));
        v = *reinterpret_cast<const uint32_t*>(&h);
        return f2pack(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    ACACHE_DEVFN static void bound(float&, float&) {}
    ACACHE_DEVFN static void put(uint4& w, int i, float x) {
        const uint32_t u = __float_as_uint(x) >> 16;        // (the value is one of bf16)
        uint32_t& v = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
        v = i & 1 ? (v & 0xffffu) | u << 16 : (v & 0xffff0000u) | u;
    }
};

// Order of values as whole numbers (-0.0 as +0.0, NaN the lowest), and of candidates: by value, then the lower token; 0 is
// no candidate.
ACACHE_DEVFN uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return x != x ? 1u : (b >> 31) ? ~b : b | 0x80000000u;
}
ACACHE_DEVFN float value_of(uint32_t o) {
    return __uint_as_float(o == 1u ? 0x7fffffffu : (o >> 31) ? o & 0x7fffffffu : ~o);
}
ACACHE_DEVFN uint64_t make_key(float x, int token) { return (uint64_t)order_of(x) << 32 | (uint32_t)~token; }
ACACHE_DEVFN int key_token(uint64_t key) { return (int)~(uint32_t)key; }
ACACHE_DEVFN float key_value(uint64_t key) { return value_of((uint32_t)(key >> 32)); }
ACACHE_DEVFN uint64_t max_key(uint64_t a, uint64_t b) { return a > b ? a : b; }
ACACHE_DEVFN uint64_t warp_max_key(uint64_t key) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
    return (uint64_t)hi << 32 | lo;
}

// Running maximum, sum of weights and of weights times d.
struct Stat {
    float m, s, u;
};
// `b` brought to the maximum m (>= b.m)
ACACHE_DEVFN Stat moved(const Stat& b, float m, const ScoreParams& p) {
    const float dd = max_nan(fmaf(b.m, p.half, -m * p.half) * p.far_log2, kLowest);
    const float a = fast_exp2(dd);
    return Stat{m, b.s * a, (b.u + b.s * dd) * a};
}

template <int NT>
struct Smem {
    alignas(16) float val[NT];              // a thread's best
    alignas(16) float group[NT];
    uint64_t list[kList];
    uint64_t best[kMaxK];                   // of this CTA, in order; 0 behind the last
    int cand[NT];
    uint32_t bound;
    uint64_t wkey[NT / 32];
    Stat part[NT / 32];
    Stat stat;
    int n_list, n_cand;
};

ACACHE_DEVFN uint64_t ld_cluster_u64(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// NT threads to a CTA, cs CTAs (a cluster) to a row; candidates are bounded by kGroups groups of threads.
template <typename T, int NT, int kGroups>
__global__ void __launch_bounds__(NT, ctas(NT))
scores_kernel(const ScoreParams p) {
    using W = Piece<T>;
    constexpr int N = W::kN, kWarps = NT / 32;
    static_assert(kGroups == NT || kGroups == NT / 2);
    __shared__ Smem<NT> sm;
    const int64_t row = blockIdx.x / (unsigned)p.cs;
    const int cr = (int)(blockIdx.x % (unsigned)p.cs);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T* x = (const T*)p.logits + row * p.row_stride;
    const int skip = (int)(((uintptr_t)x & 15u) / sizeof(T));   // elements of the first piece in front of the row
    const uint4* w0 = reinterpret_cast<const uint4*>(x - skip);
    const int64_t end = (int64_t)skip + p.vocab;                // the row is elements [skip, end) of the pieces
    const int n_all = (int)((end + N - 1) / N);
    const int p0 = (int)((int64_t)n_all * cr / p.cs), p1 = (int)((int64_t)n_all * (cr + 1) / p.cs);
    // Piece i, whole or with the elements outside the row at -infinity (they are not read).
    auto whole = [&](int i) { return (i > 0 || skip == 0) && (int64_t)(i + 1) * N <= end; };
    auto load = [&](int i) -> uint4 {
        if (whole(i)) return w0[i];
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int64_t at = (int64_t)i * N + e - skip;
            W::put(w, e, at >= 0 && at < p.vocab ? to_f32(x[at]) : -INFINITY);
        }
        return w;
    };
    // The reference st.m is the maximum of the thread's first batch and rises when a later one is 2^kHead times as
    // likely; the best logit is kept beside it.
    Stat st{kNone, 0.f, 0.f};
    float best = -INFINITY;
    auto note = [&](float m) -> bool {
        best = fmaxf(best, m);
        const bool up = m > st.m + p.head;
        if (up) st = moved(st, m, p);
        return up;
    };
    // One piece, or what there is of it, with every weight's exponent bounded from below on its own.
    auto add = [&](const uint4& w) {
        note(W::top(w));
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = max_nan(fmaf(W::at(w, e), p.half, -st.m * p.half) * p.far_log2, kLowest), q = fast_exp2(d);
            st.s += q;
            st.u = fmaf(q, d, st.u);
        }
    };
    int i = p0 + tid;
    if (i == 0 && skip != 0) {              // a first piece that begins in front of the row
        add(load(i));
        i += NT;
    }
    const int z = whole(n_all - 1) || p1 < n_all ? p1 : p1 - 1;     // pieces from here on are not whole
    typename W::Floor floor = W::floor_of(st.m, p.floor_gap);
    const uint32_t none = W::kNegInf;
    for (; i < z; i += kBatch * NT) {
        uint4 w[kBatch];                    // (behind the last: -infinity, which adds nothing)
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            w[u] = make_uint4(none, none, none, none);
            if (i + u * NT < z) w[u] = __ldg(w0 + i + u * NT);
        }
        if (note(W::top(w))) floor = W::floor_of(st.m, p.floor_gap);
        if (!W::bounds(floor, p.far)) {            // (a maximum near the lowest value, or far beyond the temperature, or next to
                                            // nothing beside it)
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (i + u * NT < z) add(w[u]);
        } else {
            const uint64_t nm = f2pack(-st.m, -st.m), c2 = f2pack(p.to_log2, p.to_log2);
            uint64_t s2 = f2pack(0.f, 0.f), u2 = s2;
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    float d0, d1;
                    f2unpack(f2mul(f2add(W::pair(w[u], e, floor), nm), c2), d0, d1);
                    W::bound(d0, d1);
                    const uint64_t q2 = f2pack(fast_exp2(d0), fast_exp2(d1));
                    s2 = f2add(s2, q2);
                    u2 = f2fma(q2, f2pack(d0, d1), u2);
                }
            float a0, a1;
            f2unpack(s2, a0, a1);
            st.s += a0 + a1;
            f2unpack(u2, a0, a1);
            st.u += a0 + a1;
        }
    }
    // a last piece that ends behind the row, by the thread whose turn it is
    if (z < p1 && (z - p0) % NT == tid && (z > 0 || skip == 0)) add(load(z));
    // ---- the CTA's maximum, S and U
    {
        float m = warp_max(st.m);
        Stat t = moved(st, m, p);
        t.s = warp_sum(t.s);
        t.u = warp_sum(t.u);
        if (lane == 0) sm.part[warp] = t;
        sm.val[tid] = best;
        if (tid == 0) {
            sm.n_list = sm.n_cand = 0;
            sm.bound = order_of(-INFINITY);
        }
        if (tid < kMaxK) sm.best[tid] = 0ull;
    }
    __syncthreads();
    if (warp == 0) {
        Stat t = lane < kWarps ? sm.part[lane] : Stat{kNone, 0.f, 0.f};
        const float m = warp_max(t.m);
        t = moved(t, m, p);
        t.s = warp_sum(t.s);
        t.u = warp_sum(t.u);
        if (lane == 0) sm.stat = Stat{m, t.s, t.u};
    }
    if (p.k > 0) {
        // ---- candidates.  A bound that k elements reach: the k-th best of the groups of threads, each by its best.
        float mine = best;
        if constexpr (kGroups < NT) {
            if (tid < kGroups) sm.group[tid] = mine = fmaxf(best, sm.val[tid + kGroups]);
            __syncthreads();
        }
        const float* group = kGroups < NT ? sm.group : sm.val;
        if (tid < kGroups) {
            int reach = 0;
#pragma unroll 8
            for (int q = 0; q < kGroups; q += 4) {
                const float4 v = *reinterpret_cast<const float4*>(group + q);
                reach += (v.x >= mine) + (v.y >= mine) + (v.z >= mine) + (v.w >= mine);
            }
            if (reach >= p.k) atomicMax(&sm.bound, order_of(mine));
        }
        __syncthreads();
        const float bound = value_of(sm.bound);
        const bool any = bound == -INFINITY;                 // (then NaN may be among them too)
        if (any || best >= bound) sm.cand[atomicAdd(&sm.n_cand, 1)] = tid;
        __syncthreads();
        // Threads whose best reaches the bound: their pieces are looked at again, a warp to a thread's.
        const int n_cand = sm.n_cand;
        auto candidates = [&](float from, auto&& see) {
            for (int c = warp; c < n_cand; c += kWarps)
                for (int q = p0 + sm.cand[c] + lane * NT; q < p1; q += 32 * NT) {
                    const uint4 w = load(q);
                    if (W::top(w) < from) continue;
#pragma unroll
                    for (int e = 0; e < N; ++e) see(W::at(w, e), q * N + e - skip);
                }
        };
        auto append = [&](float x, int at) {
            if (at < 0 || at >= p.vocab) return;
            const int n = atomicAdd(&sm.n_list, 1);
            if (n < kList) sm.list[n] = make_key(x, at);
        };
        candidates(bound, [&](float x, int at) { if (any || x >= bound) append(x, at); });
        __syncthreads();
        int n = sm.n_list;
        if (n > kList) {
            // More than the list holds, as where most logits are one and the same: those above the bound, then
            // those at it from the front.
            __syncthreads();
            if (tid == 0) sm.n_list = 0;
            __syncthreads();
            candidates(bound, [&](float x, int at) { if (x > bound) append(x, at); });
            __syncthreads();
            const int above = sm.n_list;
            __syncthreads();
            if (above + 32 * N + kMaxK > kList) {            // one after the other
                uint64_t last = ~0ull;
                for (int r = 0; r < p.k; ++r) {
                    uint64_t top = 0;
                    candidates(bound, [&](float x, int at) {
                        const uint64_t c = at >= 0 && at < p.vocab && (any || x >= bound) ? make_key(x, at) : 0ull;
                        if (c < last) top = max_key(top, c);
                    });
                    top = warp_max_key(top);
                    if (lane == 0) sm.wkey[warp] = top;
                    __syncthreads();
#pragma unroll
                    for (int q = 0; q < kWarps; ++q) top = max_key(top, sm.wkey[q]);
                    last = top;
                    if (tid == 0) sm.best[r] = top;
                    __syncthreads();
                }
                n = 0;
            } else {
                for (int nan = 0; nan < (any ? 2 : 1); ++nan)
                    for (int q0 = p0; q0 < p1; q0 += 32) {
                        if (warp != 0) break;
                        int have = lane == 0 ? *(volatile int*)&sm.n_list : 0;
                        have = __shfl_sync(0xffffffffu, have, 0);
                        if (have >= above + p.k) break;
                        if (q0 + lane < p1) {
                            const uint4 w = load(q0 + lane);
#pragma unroll
                            for (int e = 0; e < N; ++e) {
                                const float x = W::at(w, e);
                                if (nan ? x != x : x == bound) append(x, (q0 + lane) * N + e - skip);
                            }
                        }
                        __syncwarp();
                    }
                __syncthreads();
                n = sm.n_list;
            }
        }
        for (int a = tid; a < n; a += NT) {
            const uint64_t c = sm.list[a];
            int above = 0;
            for (int q = 0; q < n; ++q) above += sm.list[q] > c;
            if (above < p.k) sm.best[above] = c;
        }
    }
    __syncthreads();
    // ---- the row's from its CTAs'
    Stat all = sm.stat;
    uint64_t mine = 0;                      // this thread's alternative, tid-th in order
    if (p.cs == 1) {
        if (tid < p.k) mine = sm.best[tid];
    } else {
        ptx::cluster_sync();
        if (cr == 0) {
            // every CTA's alternatives into one list, then each to its place
            for (int a = tid; a < p.cs * p.k; a += NT)
                sm.list[a] = ld_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sm.best[a % p.k]), (uint32_t)(a / p.k)));
            const uint32_t at = ptx::smem_u32(&sm.stat);
            Stat t{kNone, 0.f, 0.f};
            if (lane < p.cs) {
                const uint32_t a = ptx::mapa_shared(at, (uint32_t)lane);
                t = Stat{ptx::ld_cluster_f32(a), ptx::ld_cluster_f32(a + 4), ptx::ld_cluster_f32(a + 8)};
            }
            const float m = warp_max(t.m);
            t = moved(t, m, p);
            all = Stat{m, warp_sum(t.s), warp_sum(t.u)};
            __syncthreads();
            for (int a = tid; a < p.cs * p.k; a += NT) {
                const uint64_t c = sm.list[a];
                int above = 0;
                for (int q = 0; q < p.cs * p.k; ++q) above += sm.list[q] > c;
                if (c && above < p.k) sm.best[above] = c;    // (its own alternatives are in the list)
            }
            __syncthreads();
            if (tid < p.k) mine = sm.best[tid];
        }
        ptx::cluster_sync();                // no CTA may leave while another still reads its shared memory
        if (cr != 0) return;
    }
    if (warp != 0) return;
    const float ln_s = logf(all.s);
    auto logprob = [&](float v) { return fmaf(v, p.half, -all.m * p.half) * p.far_ln - ln_s; };
    if (lane == 0) {
        if (all.s != all.s) flag(p.dev_status, ACACHE_DEV_NAN);
        if (p.entropy) p.entropy[row] = ln_s - 0.693147180559945f * (all.u / all.s);
        if (p.tokens) {
            const int t = p.tokens[row];
            if (t >= 0 && t < p.vocab) p.token_logprob[row] = logprob(to_f32(x[t]));
            else flag(p.dev_status, ACACHE_DEV_BAD_TOKEN);
        }
    }
    if (lane < p.k) {
        p.top_tokens[row * p.k + lane] = key_token(mine);
        if (p.top_logprob) p.top_logprob[row * p.k + lane] = logprob(key_value(mine));
    }
}

template <typename T, int NT, int kGroups = NT == 32 ? 32 : NT / 2>
int launch(const ScoreParams& p, int64_t rows, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.cs));
    cfg.blockDim = dim3(NT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cs > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, scores_kernel<T, NT, kGroups>, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    return launch_status();
}

template <typename T>
int dispatch(ScoreParams& p, int64_t rows, cudaStream_t stream) {
    const int64_t pieces = ((int64_t)p.vocab * sizeof(T) + 15) / 16;
    p.cs = 1;
    // A row's phases behind its loads (sums, candidates, their order) wait, so that CTAs of fewer threads, more of them to an
    // SM, are the faster the shorter the rows -- where there are rows to fill the SMs with.  bf16, one alternative, us: 16,400 rows
    // of 2,000: 40 of 64 threads, 58 of 128, 101 of 256; of 8,000: 74, 78, 117; of 16,000: 120, 113, 154; of 32,000: 214, 185, 223;
    // 4,100 of 50,000: 121, 99, 97.  300 of 8,000: 13, 10.9.  With many alternatives 64 threads need 64 groups
    // (20 of 2,000: 89, with 32 groups 103; one: 44, with 32 groups 40).
    if (pieces <= 128) return launch<T, 32>(p, rows, stream);
    if (pieces <= 1024 && rows > (int64_t)ctas(128) * sm_count())
        return p.k <= 8 ? launch<T, 64, 32>(p, rows, stream) : launch<T, 64, 64>(p, rows, stream);
    if (pieces <= 1024 || (pieces <= 4096 && rows > (int64_t)ctas(256) * sm_count())) return launch<T, 128>(p, rows, stream);
    // rows that leave SMs idle are split over a cluster, in one wave and with four pieces a thread at least
    p.cs = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxCluster, 4LL * sm_count() / rows, pieces / (4 * 256)}));
    return launch<T, 256>(p, rows, stream);
}

}  // namespace

int launch_token_scores(const ScoreCall& c) {
    ScoreParams p{};
    p.logits = c.logits;
    p.row_stride = c.row_stride;
    p.tokens = c.tokens;
    p.token_logprob = c.token_logprob;
    p.entropy = c.entropy;
    p.top_logprob = c.top_logprob;
    p.top_tokens = c.top_tokens;
    p.dev_status = c.dev_status;
    p.vocab = c.vocab;
    p.k = c.k;
    p.to_log2 = kLog2e / c.temperature;
    p.half = c.temperature > 1.f ? 0.5f : 1.f;
    p.far_log2 = (float)((double)kLog2e / c.temperature / p.half);
    p.far_ln = (float)(1.0 / c.temperature / p.half);
    p.head = kHead / p.to_log2;
    p.floor_gap = kFloor / p.to_log2;
    p.far = p.floor_gap > 1.7e38f;
    return c.dtype == ACACHE_F32 ? dispatch<float>(p, c.rows, c.stream) : dispatch<__nv_bfloat16>(p, c.rows, c.stream);
}

}  // namespace acache
