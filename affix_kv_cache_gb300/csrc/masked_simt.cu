// masked_simt.cu -- read-slot attention under a mask on CUDA cores: float32, and bf16 with a scale that is
// not positive, groups of more than 128 heads or an empty pool.
//
// Page: "Affix Cache for Diffusion Large Language Models", Sec. 4.3 and App. C.1 (attention through the read-slot
// map); the masks are this library's (include/acache.h, acache_slot_attention_masked).
//
// One CTA per 64 rows (query, head of the group) of a (request, KV head) and per part of the keys of its window
// (from the first that one of its rows sees to the last): tiles of 64 keys go to shared memory in float32, S = Q K^T
// and O += P V run as 4 x 4 and 4 x d/16 register tiles, and the softmax keeps a running maximum and sum per row
// in base 2.  Bound by FFMA issue and the shared-memory reads that feed it.  With at most 32 or 16 rows a CTA takes that
// many with as many fewer threads; when there are few blocks the window is split over a cluster of up to 8 CTAs, which
// merge their partial (maximum, sum, O) through distributed shared memory in rank order.  A masked key's score is
// replaced by -infinity; a row that met a masked V which is not finite (0 x NaN is NaN) is computed again by a
// warp over its own keys.
// Measured, float32, d = 128: causal 2 x 300 rows over 800 keys (32 heads over 8, capped) 262 us; 4 x 32 over 1,400 (32 heads)
// 233 us.  A single token over 8,000 keys takes 410 us out of memory: 12 of 16 rows are padding and no load is under way during the
// products.
#include <cfloat>

#include <algorithm>
#include <atomic>

#include "masked.cuh"
#include "ptx.cuh"
#include "q8.cuh"
#include "step.cuh"

namespace acache {
namespace {

constexpr int kBN = 64;                     // keys per tile; 4 threads to a row
constexpr int kMaxCluster = 8;

struct SimtParams {
    const void *q, *k_cache, *v_cache;
    void* out;
    const int32_t *read_slot, *q_start, *kv_start, *row_range, *q_pos;
    const float* slopes;
    int32_t* dev_status;
    int64_t num_slots;
    int n_q, total_q, T_len, Hq, Hkv, g, cs, drop;
    float scale, softcap;
};

template <int D, int kBM>
struct SimtSmem {
    float q[D][kBM];          // transposed; the partial O of a split window afterwards
    float k[D][kBN];          // transposed
    float v[kBN][D];
    union {
        float p[kBN][kBM];    // transposed
        float ml[2][kBM];     // maximum and sum of a split window afterwards
    };
    int row[kBN];             // pool row, or -1 (zero row), or -2 (no key)
    int pos[kBM];             // of a row
    float slope[kBM];
    uint32_t again[2];        // rows to compute again, a bit each
    int win[2];
};
// two CTAs to an SM (228 KB, of which a CTA takes 1 KB more than it asks for)
static_assert(2 * (sizeof(SimtSmem<128, 64>) + 1024) <= 228 * 1024, "shared memory of two CTAs");

template <typename T, int D, int kBM>
__global__ void __launch_bounds__(4 * kBM)
masked_simt_kernel(const SimtParams p) {
    constexpr int kThreads = 4 * kBM, kWarps = kThreads / 32;
    constexpr int N = 16 / (int)sizeof(T), PPT = kBN * (D / N) / kThreads;   // elements of a 16-byte piece, pieces a thread loads
    extern __shared__ __align__(16) uint8_t raw[];
    SimtSmem<D, kBM>& sm = *reinterpret_cast<SimtSmem<D, kBM>*>(raw);
    constexpr int NC = D / 64;                          // 4-column chunks of O per thread
    const int cs = p.cs;
    const int cr = (int)(blockIdx.x % (unsigned)cs), hk = (int)(blockIdx.x / (unsigned)cs);
    const int b = (int)blockIdx.y, zb = (int)(gridDim.z - 1 - blockIdx.z);   // (the last rows, with most keys, first)
    int n_q = p.n_q, T_len = p.T_len;
    int64_t qbase = (int64_t)b * p.n_q, kbase = (int64_t)b * p.T_len;
    if (p.q_start) {
        qbase = p.q_start[b];
        kbase = p.kv_start[b];
        n_q = q8_count(p.q_start, b);
        T_len = q8_count(p.kv_start, b);
        if (n_q != 0 && q8_bad_lengths(n_q, p.n_q, T_len, p.T_len, qbase, p.total_q, kbase)) {
            if (threadIdx.x == 0 && blockIdx.x == 0 && zb == 0) flag(p.dev_status, ACACHE_DEV_BAD_LENGTH);
            return;
        }
    }
    const int64_t r0 = (int64_t)zb * kBM, n_rows = (int64_t)n_q * p.g;
    if (r0 >= n_rows) return;
    const int rows = (int)min((int64_t)kBM, n_rows - r0);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, warp = tid >> 5, lane = tid & 31;
    auto q_off = [&](int r) {                           // element offset of packed row r0 + r
        const int64_t i = (r0 + r) / p.g;
        return ((qbase + i) * p.Hq + (int64_t)hk * p.g + (r0 + r - i * p.g)) * D;
    };
    // The keys [lo, hi) of packed row r0 + r (lo = hi = 0: none, or no row), and the window that holds all rows'.
    auto row_keys = [&](int r, int& lo, int& hi) {
        lo = hi = 0;
        if (r >= rows) return;
        const int64_t i = qbase + (r0 + r) / p.g;
        hi = T_len;
        if (p.row_range) {
            lo = max(p.row_range[2 * i], 0);
            hi = min(p.row_range[2 * i + 1], T_len);
        }
        if (lo >= hi) lo = hi = 0;
    };
    if (tid == 0) {
        sm.win[0] = 0x7fffffff;
        sm.win[1] = 0;
        sm.again[0] = sm.again[1] = 0u;
    }
    __syncthreads();
    if (tid < kBM) {
        int lo, hi;
        row_keys(tid, lo, hi);
        if (lo < hi) {
            atomicMin(&sm.win[0], lo);
            atomicMax(&sm.win[1], hi);
        }
        const int64_t i = (r0 + tid) / p.g;
        const bool biased = p.slopes && tid < rows;
        sm.slope[tid] = biased ? p.slopes[hk * p.g + (int)(r0 + tid - i * p.g)] : 0.f;
        sm.pos[tid] = biased ? p.q_pos[qbase + i] : 0;
    }
    for (int x = tid; x < kBM * D; x += kThreads) {
        const int r = x / D, c = x % D;
        sm.q[c][r] = r < rows ? to_f32(((const T*)p.q)[q_off(r) + c]) : 0.f;
    }
    __syncthreads();
    const int w_lo = sm.win[1] > 0 ? sm.win[0] : 0, T_win = sm.win[1] - w_lo;
    const int32_t* rs = p.read_slot + kbase + w_lo;
    const int n_all = (T_win + kBN - 1) / kBN;
    const int j0 = (int)((int64_t)cr * n_all / cs), j1 = (int)((int64_t)(cr + 1) * n_all / cs);
    int lo[4], hi[4];
    float m[4], l[4], acc[4][NC * 4];
    uint32_t saw = 0;                                   // bit y: row 4 ty + y sees a key of this thread's columns
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        row_keys(4 * ty + y, lo[y], hi[y]);
        lo[y] -= w_lo;
        hi[y] -= w_lo;
        m[y] = -INFINITY;
        l[y] = 0.f;
#pragma unroll
        for (int x = 0; x < NC * 4; ++x) acc[y][x] = 0.f;
    }
    // slots of a tile's keys, looked up a tile ahead
    int row = -2;
    auto look_up = [&](int j) {
        const int t = j * kBN + tid;
        row = -2;
        if (j < j1 && tid < kBN && t < T_win) {
            const int64_t s = rs[t];
            if (s >= 0 && s < p.num_slots) {
                row = (int)(s * p.Hkv + hk);
            } else if (!(p.drop && s == ACACHE_SLOT_NONE)) {
                row = -1;
                flag(p.dev_status, ACACHE_DEV_BAD_SLOT);
            }
        }
    };
    look_up(j0);
    for (int j = j0; j < j1; ++j) {
        __syncthreads();                                // the last tile has been read
        if (tid < kBN) sm.row[tid] = row;
        look_up(j + 1);
        __syncthreads();
        {
            // K: consecutive lanes take consecutive keys, so the transposed stores do not conflict
            const int key = tid & (kBN - 1);
            const int64_t kr = sm.row[key];
#pragma unroll 4
            for (int it = 0; it < PPT; ++it) {
                const int c = (tid / kBN) * PPT + it;
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (kr >= 0) w = *reinterpret_cast<const uint4*>((const T*)p.k_cache + kr * D + c * N);
                const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
                for (int i = 0; i < N; ++i) sm.k[c * N + i][key] = to_f32(e[i]);
            }
#pragma unroll 4
            for (int it = 0; it < PPT; ++it) {
                const int x = it * kThreads + tid, vk = x / (D / N), c = x % (D / N);
                const int64_t vr = sm.row[vk];
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (vr >= 0) w = *reinterpret_cast<const uint4*>((const T*)p.v_cache + vr * D + c * N);
                const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
                for (int i = 0; i < N; i += 4)
                    *reinterpret_cast<float4*>(&sm.v[vk][c * N + i]) = make_float4(to_f32(e[i]), to_f32(e[i + 1]), to_f32(e[i + 2]), to_f32(e[i + 3]));
            }
        }
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 8
        for (int c = 0; c < D; ++c) {
            const float4 qv = *reinterpret_cast<const float4*>(&sm.q[c][4 * ty]);
            const float4 kv = *reinterpret_cast<const float4*>(&sm.k[c][4 * tx]);
            const float qa[4] = {qv.x, qv.y, qv.z, qv.w}, ka[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[y][x] = fmaf(qa[y], ka[x], s[y][x]);
        }
        bool there[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) there[x] = sm.row[4 * tx + x] != -2;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            float mt = -INFINITY;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int t = j * kBN + 4 * tx + x;
                const bool see = there[x] && t >= lo[y] && t < hi[y];
                saw |= (uint32_t)see << y;
                float v = s[y][x] * p.scale;
                if (p.softcap > 0.f) v = p.softcap * tanhf(v / p.softcap);
                if (p.slopes) v = fmaf(-sm.slope[4 * ty + y], fabsf((float)((int64_t)sm.pos[4 * ty + y] - w_lo - t)), v);
                s[y][x] = see ? v * kLog2e : -INFINITY;
                mt = fmaxf(mt, s[y][x]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
            const float mn = fmaxf(m[y], mt);
            const float ref = mn == -INFINITY ? 0.f : mn;      // no key so far: exponentiate against 0
            const float alpha = fast_exp2(m[y] - ref);
            m[y] = mn;
            float lt = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[y][x] = fast_exp2(s[y][x] - ref);
                lt += s[y][x];
            }
            l[y] = l[y] * alpha + lt;                           // this lane's share of the row's sum
#pragma unroll
            for (int x = 0; x < NC * 4; ++x) acc[y][x] *= alpha;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
            *reinterpret_cast<float4*>(&sm.p[4 * tx + x][4 * ty]) = make_float4(s[0][x], s[1][x], s[2][x], s[3][x]);
        __syncwarp();                                           // a warp reads only rows it wrote
#pragma unroll 4
        for (int t = 0; t < kBN; ++t) {
            const float4 pv = *reinterpret_cast<const float4*>(&sm.p[t][4 * ty]);
            const float pa[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const float4 vv = *reinterpret_cast<const float4*>(&sm.v[t][n * 64 + 4 * tx]);
                const float va[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[y][n * 4 + x] = fmaf(pa[y], va[x], acc[y][n * 4 + x]);
            }
        }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            l[y] += __shfl_xor_sync(0xffffffffu, l[y], o);
            saw |= __shfl_xor_sync(0xffffffffu, saw, o);
        }
        // A row has a maximum if it has a key, be its score -infinity: then a sum of 0 is 0 / 0, not an empty row.
        if ((saw >> y) & 1u) m[y] = fmaxf(m[y], -FLT_MAX);
    }
    // 4 columns of row r, and whether the row has to be computed again
    auto put = [&](int r, int col, const float4& o, float M, float L) {
        const bool none = M == -INFINITY;                       // no key: zeros, whatever was added with weight 0
        const float inv = 1.f / L;
        const float y[4] = {none ? 0.f : o.x * inv, none ? 0.f : o.y * inv, none ? 0.f : o.z * inv, none ? 0.f : o.w * inv};
        T* to = (T*)p.out + q_off(r) + col;
        float chk = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            to[x] = from_f32<T>(y[x]);
            chk = fmaf(y[x], 0.f, chk);
        }
        if (chk != chk && L == L) atomicOr(&sm.again[r >> 5], 1u << (r & 31));
    };
    auto again = [&](int first, int step) {                     // rows first, first + step, ... of this CTA, a warp to each
        __syncthreads();
        for (int r = first + step * warp; r < rows; r += step * kWarps)
            if ((sm.again[r >> 5] >> (r & 31)) & 1u) {
                const int64_t at = q_off(r);
                int lo, hi;
                row_keys(r, lo, hi);
                masked_row<T, D>(MaskedPool<T>{(const T*)p.k_cache, (const T*)p.v_cache, rs, p.num_slots, p.Hkv, p.drop, false, p.scale * kLog2e,
                                               p.softcap, 0.f, p.scale},
                                 (const T*)p.q + at, (T*)p.out + at, lo - w_lo, hi - w_lo, hk, sm.slope[r] * kLog2e,
                                 (int64_t)sm.pos[r] - w_lo, lane);
            }
    };
    if (cs == 1) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int r = 4 * ty + y;
            if (r >= rows) continue;
#pragma unroll
            for (int n = 0; n < NC; ++n)
                put(r, n * 64 + 4 * tx, make_float4(acc[y][n * 4], acc[y][n * 4 + 1], acc[y][n * 4 + 2], acc[y][n * 4 + 3]), m[y], l[y]);
        }
        again(0, 1);
        return;
    }
    // merge the parts: rank w finalises rows w, w + cs, ...
    __syncthreads();
    float* part = &sm.q[0][0];                                  // [row][D]
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const int r = 4 * ty + y;
        if (tx == 0) {
            sm.ml[0][r] = m[y];
            sm.ml[1][r] = l[y];
        }
#pragma unroll
        for (int n = 0; n < NC; ++n)
            *reinterpret_cast<float4*>(part + r * D + n * 64 + 4 * tx) =
                make_float4(acc[y][n * 4], acc[y][n * 4 + 1], acc[y][n * 4 + 2], acc[y][n * 4 + 3]);
    }
    ptx::cluster_sync();
    const uint32_t m_a = ptx::smem_u32(&sm.ml[0][0]), l_a = ptx::smem_u32(&sm.ml[1][0]), o_a = ptx::smem_u32(part);
    for (int x = tid; x < ((rows - cr + cs - 1) / cs) * (D / 4); x += kThreads) {
        const int r = cr + (x / (D / 4)) * cs, c = x % (D / 4);
        float pm[kMaxCluster], pl[kMaxCluster], M = -INFINITY, L = 0.f;
        float4 po[kMaxCluster], O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kMaxCluster; ++w) {                 // all ranks' loads in flight
            pm[w] = -INFINITY;
            pl[w] = 0.f;
            po[w] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (w < cs) {
                pm[w] = ptx::ld_cluster_f32(ptx::mapa_shared(m_a + 4u * r, w));
                pl[w] = ptx::ld_cluster_f32(ptx::mapa_shared(l_a + 4u * r, w));
                po[w] = ptx::ld_cluster_v4(ptx::mapa_shared(o_a + (uint32_t)(r * D + 4 * c) * 4u, w));
            }
        }
#pragma unroll
        for (int w = 0; w < kMaxCluster; ++w) M = fmaxf(M, pm[w]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kMaxCluster; ++w) {
            const float e = fast_exp2(pm[w] - ref);
            L = fmaf(e, pl[w], L);
            O.x = fmaf(e, po[w].x, O.x);
            O.y = fmaf(e, po[w].y, O.y);
            O.z = fmaf(e, po[w].z, O.z);
            O.w = fmaf(e, po[w].w, O.w);
        }
        put(r, 4 * c, O, M, L);
    }
    ptx::cluster_sync();       // no CTA may leave while another still reads its shared memory
    again(cr, cs);
}

// CTAs of a variant that run at once in clusters of cs (a cluster stays within a group of SMs), per device.
std::atomic<int> g_slots[2][2][3][kMaxCluster + 1][64];

template <typename T, int D, int kBM>
int launch(SimtParams prm, const MaskedAttn& c) {
    auto kern = masked_simt_kernel<T, D, kBM>;
    constexpr int smem = (int)sizeof(SimtSmem<D, kBM>);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(4 * kBM);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // Parts of the window, taken as long as the request: waves x (tiles of a part, a CTA's own cost of about one and as
    // much for a merge)
    const int64_t n_rb = ((int64_t)c.n_q * prm.g + kBM - 1) / kBM, units = (int64_t)c.B * prm.Hkv * n_rb;
    if (n_rb > 65535) return ACACHE_ERR_INVALID_ARG;
    const int tiles = (c.T_len + kBN - 1) / kBN;
    int64_t best = 0;
    for (int cs = 1; cs <= kMaxCluster && cs <= tiles; ++cs) {
        std::atomic<int>& known = g_slots[sizeof(T) == 4][D == 128][kBM == 16 ? 0 : kBM == 32 ? 1 : 2][cs][dev];
        int slots = known.load(std::memory_order_relaxed);
        if (!slots) {
            int clusters = 0;
            cfg.gridDim = dim3((unsigned)cs);
            attr[0].val.clusterDim.x = (unsigned)cs;
            if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters < 1) {
                (void)cudaGetLastError();
                clusters = std::max(1, sm_count() / cs);
            }
            slots = clusters * cs;
            known.store(slots, std::memory_order_relaxed);
        }
        const int64_t est = (units * cs + slots - 1) / slots * ((tiles + cs - 1) / cs + 1 + (cs > 1));
        if (cs == 1 || est < best) {
            best = est;
            prm.cs = cs;
        }
    }
    cfg.gridDim = dim3((unsigned)(prm.Hkv * prm.cs), (unsigned)c.B, (unsigned)n_rb);
    attr[0].val.clusterDim.x = (unsigned)prm.cs;
    cfg.numAttrs = prm.cs > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, prm) != cudaSuccess) {
        (void)cudaGetLastError();
        return ACACHE_ERR_CUDA;
    }
    return launch_status();
}

template <typename T, int D>
int launch(const SimtParams& prm, const MaskedAttn& c) {
    const int64_t rows = (int64_t)c.n_q * prm.g;
    return rows <= 16 ? launch<T, D, 16>(prm, c) : rows <= 32 ? launch<T, D, 32>(prm, c) : launch<T, D, 64>(prm, c);
}

}  // namespace

int launch_masked_simt(const MaskedAttn& c) {
    SimtParams prm{};
    prm.q = c.q;
    prm.k_cache = c.k_cache;
    prm.v_cache = c.v_cache;
    prm.out = c.out;
    prm.read_slot = c.read_slot;
    prm.q_start = c.q_start;
    prm.kv_start = c.kv_start;
    prm.row_range = c.mask.row_range;
    prm.q_pos = c.mask.q_pos;
    prm.slopes = c.mask.slopes;
    prm.dev_status = c.dev_status;
    prm.num_slots = c.num_slots;
    prm.n_q = c.n_q;
    prm.total_q = c.total_q;
    prm.T_len = c.T_len;
    prm.Hq = c.a.hq;
    prm.Hkv = c.a.hkv;
    prm.g = c.a.hq / c.a.hkv;
    prm.drop = c.mask.drop_none != 0;
    prm.scale = c.a.scale;
    prm.softcap = c.mask.softcap;
    if (c.a.dtype == ACACHE_F32) return c.a.d == 64 ? launch<float, 64>(prm, c) : launch<float, 128>(prm, c);
    return c.a.d == 64 ? launch<__nv_bfloat16, 64>(prm, c) : launch<__nv_bfloat16, 128>(prm, c);
}

}  // namespace acache
