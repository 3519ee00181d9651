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
// every thread keeps its own running maximum, S and U, raised when a batch of pieces holds more.  Both
// terms of the entropy are >= 0, so nothing cancels.
// The k likeliest: candidates are compared by (value, lower token), all different.  A thread's best piece is
// remembered by the way; the k threads with the best elements hold all of the row's k best (each
// other thread's best is below k elements), so only their pieces are looked at again, against the k-th
// best of the threads.
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
constexpr int kBatch = 4;                   // pieces in flight

struct ScoreParams {
    const void* logits;
    int64_t row_stride;
    const int32_t* tokens;
    float *token_logprob, *entropy, *top_logprob;
    int32_t *top_tokens, *dev_status;
    int vocab, k, cs;
    float to_log2, to_ln;                   // log2e / temperature, 1 / temperature
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
    ACACHE_DEVFN static float at(const uint4& w, int i) { return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w); }
    ACACHE_DEVFN static float top(const uint4& w) { return fmaxf(fmaxf(at(w, 0), at(w, 1)), fmaxf(at(w, 2), at(w, 3))); }
    template <int B> ACACHE_DEVFN static float top(const uint4 (&w)[B]) {
        float m = top(w[0]);
#pragma unroll
        for (int u = 1; u < B; ++u) m = fmaxf(m, top(w[u]));
        return m;
    }
    // Elements e, e + 1; weights' exponents are bounded from below one by one.
    struct Floor {};
    ACACHE_DEVFN static Floor floor_of(float, float) { return {}; }
    ACACHE_DEVFN static bool bounds(Floor) { return true; }
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
    // lies 300 in log2 units below the maximum, and by more than its rounding; 0: there is no such bf16 value.
    using Floor = uint32_t;
    ACACHE_DEVFN static Floor floor_of(float m, float to_log2) {
        const float f = m - 300.f / to_log2 - fabsf(m) * 0.015625f;
        if (!(f > -3.3e38f)) return 0u;
        const uint32_t u = __float_as_uint(f) >> 16;         // (cut: a little more for negative ones, less for others)
        return u | u << 16;
    }
    ACACHE_DEVFN static bool bounds(Floor f) { return f != 0u; }
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

// Order of candidates: by value, then the lower token; 0 is no candidate, NaN the lowest.
ACACHE_DEVFN uint64_t make_key(float x, int token) {
    const uint32_t b = __float_as_uint(x + 0.f);             // -0.0 counts as +0.0
    const uint32_t o = x != x ? 1u : (b >> 31) ? ~b : b | 0x80000000u;
    return (uint64_t)o << 32 | (uint32_t)~token;
}
ACACHE_DEVFN int key_token(uint64_t key) { return (int)~(uint32_t)key; }
ACACHE_DEVFN float key_value(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o == 1u ? 0x7fffffffu : (o >> 31) ? o & 0x7fffffffu : ~o);
}
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
ACACHE_DEVFN Stat moved(const Stat& b, float m, float to_log2) {
    const float dd = max_nan((b.m - m) * to_log2, kLowest);
    const float a = fast_exp2(dd);
    return Stat{m, b.s * a, (b.u + b.s * dd) * a};
}

template <int NT>
struct Smem {
    uint64_t keys[NT];
    uint64_t list[kList];
    uint64_t best[kMaxK];                   // of this CTA, in order; 0 behind the last
    int cand[kMaxK];
    uint64_t threshold;
    uint64_t wkey[NT / 32];
    Stat part[NT / 32];
    Stat stat;
    int n_list;
};

ACACHE_DEVFN uint64_t ld_cluster_u64(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// NT threads to a CTA, cs CTAs (a cluster) to a row.
template <typename T, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 5 : 1)
scores_kernel(const ScoreParams p) {
    using W = Piece<T>;
    constexpr int N = W::kN, kWarps = NT / 32;
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
    auto key_of = [&](const uint4& w, int i, int e) -> uint64_t {
        const int64_t at = (int64_t)i * N + e - skip;
        return at >= 0 && at < p.vocab ? make_key(W::at(w, e), (int)at) : 0ull;
    };
    Stat st{kNone, 0.f, 0.f};
    int best_piece = -1;
    // One piece, or what there is of it, with every weight's exponent bounded from below on its own.
    auto add = [&](const uint4& w, int i) {
        const float m = W::top(w);
        if (m > st.m) {
            st = moved(st, m, p.to_log2);
            best_piece = i;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = max_nan((W::at(w, e) - st.m) * p.to_log2, kLowest), q = fast_exp2(d);
            st.s += q;
            st.u = fmaf(q, d, st.u);
        }
    };
    int i = p0 + tid;
    if (i < p1 && !whole(i)) {              // a first piece that begins in front of the row
        add(load(i), i);
        i += NT;
    }
    const int z = whole(n_all - 1) || p1 < n_all ? p1 : p1 - 1;     // pieces from here on are not whole
    typename W::Floor floor = W::floor_of(st.m, p.to_log2);
    for (; i + (kBatch - 1) * NT < z; i += kBatch * NT) {
        uint4 w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) w[u] = __ldg(w0 + i + u * NT);
        const float m = W::top(w);
        if (m > st.m) {
            st = moved(st, m, p.to_log2);
            floor = W::floor_of(m, p.to_log2);
#pragma unroll
            for (int u = kBatch - 1; u >= 0; --u)
                if (W::top(w[u]) == m) best_piece = i + u * NT;
        }
        if (!W::bounds(floor)) {            // (a maximum near the lowest value)
#pragma unroll
            for (int u = 0; u < kBatch; ++u) add(w[u], i + u * NT);
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
    for (; i < p1; i += NT) add(load(i), i);
    // ---- the CTA's maximum, S and U
    {
        float m = warp_max(st.m);
        Stat t = moved(st, m, p.to_log2);
        t.s = warp_sum(t.s);
        t.u = warp_sum(t.u);
        if (lane == 0) sm.part[warp] = t;
        if (tid == 0) sm.n_list = 0;
        if (tid < kMaxK) sm.best[tid] = 0ull;
    }
    // ---- candidates
    uint64_t key = 0;
    if (p.k > 0) {
        if (best_piece >= 0) {
            const uint4 w = load(best_piece);
#pragma unroll
            for (int e = N - 1; e >= 0; --e)
                if (W::at(w, e) == st.m) key = key_of(w, best_piece, e);
        } else {                            // nothing above the lowest value: each element as it is
            for (int q = p0 + tid; q < p1; q += NT) {
                const uint4 w = load(q);
#pragma unroll
                for (int e = 0; e < N; ++e) key = max_key(key, key_of(w, q, e));
            }
        }
        if (p.k == 1) {
            key = warp_max_key(key);
            if (lane == 0) sm.wkey[warp] = key;
        } else {
            sm.keys[tid] = key;
        }
    }
    __syncthreads();
    if (warp == 0) {
        Stat t = lane < kWarps ? sm.part[lane] : Stat{kNone, 0.f, 0.f};
        const float m = warp_max(t.m);
        t = moved(t, m, p.to_log2);
        t.s = warp_sum(t.s);
        t.u = warp_sum(t.u);
        if (lane == 0) sm.stat = Stat{m, t.s, t.u};
        if (p.k == 1) {
            const uint64_t top = warp_max_key(lane < kWarps ? sm.wkey[lane] : 0ull);
            if (lane == 0) sm.best[0] = top;
        } else if (p.k > 1) {
            // the k best threads, one after the other
            uint64_t mine[kWarps], top = 0, last = 0;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) {
                mine[q] = sm.keys[32 * q + lane];
                top = max_key(top, mine[q]);
            }
            for (int r = 0; r < p.k; ++r) {
                last = warp_max_key(top);
                if (top == last && last) {
                    top = 0;
                    int from = 0;
#pragma unroll
                    for (int q = 0; q < kWarps; ++q) {
                        if (mine[q] == last) {
                            from = 32 * q + lane;
                            mine[q] = 0;
                        }
                        top = max_key(top, mine[q]);
                    }
                    sm.cand[r] = from;
                }
                if (lane == 0 && !last) sm.cand[r] = -1;
            }
            if (lane == 0) sm.threshold = last;
        }
    }
    __syncthreads();
    if (p.k > 1) {
        const uint64_t least = max_key(sm.threshold, 1);
        const int per = (p1 - p0 + NT - 1) / NT;                // pieces of a thread, at most
        auto candidates = [&](auto&& see) {
            for (int64_t it = tid; it < (int64_t)p.k * per; it += NT) {
                const int from = sm.cand[it / per], q = p0 + from + (int)(it % per) * NT;
                if (from < 0 || q >= p1) continue;
                const uint4 w = load(q);
#pragma unroll
                for (int e = 0; e < N; ++e) see(key_of(w, q, e));
            }
        };
        candidates([&](uint64_t c) {
            if (c >= least) {
                const int at = atomicAdd(&sm.n_list, 1);
                if (at < kList) sm.list[at] = c;
            }
        });
        __syncthreads();
        const int n = sm.n_list;
        if (n <= kList) {
            for (int a = tid; a < n; a += NT) {
                const uint64_t c = sm.list[a];
                int above = 0;
                for (int q = 0; q < n; ++q) above += sm.list[q] > c;
                if (above < p.k) sm.best[above] = c;
            }
        } else {                            // more than the list holds: one after the other
            uint64_t last = ~0ull;
            for (int r = 0; r < p.k; ++r) {
                uint64_t top = 0;
                candidates([&](uint64_t c) { if (c < last) top = max_key(top, c); });
                top = warp_max_key(top);
                if (lane == 0) sm.wkey[warp] = top;
                __syncthreads();
#pragma unroll
                for (int q = 0; q < kWarps; ++q) top = max_key(top, sm.wkey[q]);
                last = top;
                if (tid == 0) sm.best[r] = top;
                __syncthreads();
            }
        }
        __syncthreads();
    }
    // ---- the row's from its CTAs'
    Stat all = sm.stat;
    uint64_t mine = 0;                      // this thread's alternative, tid-th in order
    if (p.cs == 1) {
        if (tid < p.k) mine = sm.best[tid];
    } else {
        ptx::cluster_sync();
        if (cr == 0 && warp == 0) {
            const uint32_t at = ptx::smem_u32(&sm.stat);
            Stat t{kNone, 0.f, 0.f};
            if (lane < p.cs) {
                const uint32_t a = ptx::mapa_shared(at, (uint32_t)lane);
                t = Stat{ptx::ld_cluster_f32(a), ptx::ld_cluster_f32(a + 4), ptx::ld_cluster_f32(a + 8)};
            }
            const float m = warp_max(t.m);
            t = moved(t, m, p.to_log2);
            all = Stat{m, warp_sum(t.s), warp_sum(t.u)};
            uint64_t c[kMaxCluster];        // lane's of each CTA
#pragma unroll
            for (int q = 0; q < kMaxCluster; ++q)
                c[q] = q < p.cs && lane < p.k ? ld_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sm.best[lane]), (uint32_t)q)) : 0ull;
            for (int r = 0; r < p.k; ++r) {
                uint64_t top = 0;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q) top = max_key(top, c[q]);
                top = warp_max_key(top);
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)
                    if (c[q] == top) c[q] = 0;
                if (lane == r) mine = top;
            }
        }
        ptx::cluster_sync();                // no CTA may leave while another still reads its shared memory
        if (cr != 0) return;
    }
    if (warp != 0) return;
    const float ln_s = logf(all.s);
    auto logprob = [&](float v) { return (v - all.m) * p.to_ln - ln_s; };
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

template <typename T, int NT>
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
    if (cudaLaunchKernelEx(&cfg, scores_kernel<T, NT>, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    return launch_status();
}

template <typename T>
int dispatch(ScoreParams& p, int64_t rows, cudaStream_t stream) {
    const int64_t pieces = ((int64_t)p.vocab * sizeof(T) + 15) / 16;
    p.cs = 1;
    if (pieces <= 128) return launch<T, 32>(p, rows, stream);
    if (pieces <= 1024) return launch<T, 128>(p, rows, stream);
    // rows that leave SMs idle are split over a cluster, four pieces a thread at least
    while (p.cs < kMaxCluster && rows * p.cs < 4LL * sm_count() && pieces >= 4LL * 256 * 2 * p.cs) p.cs *= 2;
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
    p.to_ln = 1.f / c.temperature;
    return c.dtype == ACACHE_F32 ? dispatch<float>(p, c.rows, c.stream) : dispatch<__nv_bfloat16>(p, c.rows, c.stream);
}

}  // namespace acache
