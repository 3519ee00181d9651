// q8_simt.cu -- read-slot attention over an 8-bit pool on CUDA cores: float32 queries and outputs, and
// calls that the tensor-core kernels do not cover (a softmax scale that is not positive, an empty pool).
// (One pass of a tensor-core product would cut float32 queries and probabilities to 8 or 11 bits.  The codes are
// exact in bf16, so passes over three bf16 terms of the float32 operand would keep them: not built.)
//
// One CTA per 64 packed rows -- (query, query head of the KV head's group), so the heads of a
// group share one pass over the keys -- and per part of the key range: 64-key tiles are decoded to
// float32 in shared memory, S = Q K^T and O += P V run as 4 x 4 and 4 x d/16 register tiles, and
// the softmax keeps a running maximum and sum per row in base 2.  Bound by FFMA issue and the
// shared-memory reads that feed it; at least two CTAs per SM (4 x 589 rows over 1,408 keys, 8 heads, d = 128,
// float32: 478 us, 28 TFLOP/s; 560 with one).  With at most 32 or 16 rows to a (request, KV head) a CTA takes that
// many, with as many fewer threads: the products of 64 rows would be mostly of rows that are not there (8 single
// tokens over 4,000 keys, 32 heads over 8, d = 128, float32: 137 us where they share the keys and 183 where each has its
// own, 265 and 284 in tiles of 64; 4 x 32 rows over 1,408 keys, 8 heads: 45 and 63).  When there are few blocks the key range
// is split over a cluster of up to 8 CTAs, which merge their partial (maximum, sum, O) through
// distributed shared memory in rank order.
#include <cfloat>

#include <algorithm>
#include <atomic>

#include "q8.cuh"
#include "ptx.cuh"

namespace acache {
namespace {

constexpr int kBN = 64;                     // keys per tile; 4 threads to a row
constexpr int kMaxCluster = 8;

struct SimtParams {
    const void* q;
    const uint8_t *k_cache, *v_cache, *kv_scale;
    const int32_t *read_slot, *q_start, *kv_start;
    void* out;
    int32_t* dev_status;
    int64_t num_slots;
    int n_q, total_q, T_len, Hq, Hkv, g, cs;
    bool drop_none;
    float scale_log2;
};

template <int D, int kBM>
struct SimtSmem {
    float q[D][kBM];          // transposed; the partial O of a split key range afterwards
    float k[D][kBN];          // transposed
    float v[kBN][D];
    union {
        float p[kBN][kBM];    // transposed
        float ml[2][kBM];     // maximum and sum of a split key range afterwards
    };
    float ks[kBN], vs[kBN];
    int64_t row[kBN];         // pool row, or -1 (zero row), or -2 (no key)
};
// two CTAs to an SM (228 KB, of which a CTA takes 1 KB more than it asks for)
static_assert(2 * (sizeof(SimtSmem<128, 64>) + 1024) <= 228 * 1024, "shared memory of two CTAs");

template <typename T, int D, int kBM>
__global__ void __launch_bounds__(4 * kBM)
q8_simt_kernel(const SimtParams p) {
    constexpr int kThreads = 4 * kBM;
    extern __shared__ __align__(16) uint8_t raw[];
    SimtSmem<D, kBM>& sm = *reinterpret_cast<SimtSmem<D, kBM>*>(raw);
    constexpr int NC = D / 64;                          // 4-column chunks of O per thread
    const int cr = (int)(blockIdx.x % (unsigned)p.cs), hk = (int)(blockIdx.x / (unsigned)p.cs);
    const int b = (int)blockIdx.y;
    int n_q = p.n_q, T_len = p.T_len;
    int64_t qbase = (int64_t)b * p.n_q, kbase = (int64_t)b * p.T_len;
    if (p.q_start) {
        qbase = p.q_start[b];
        kbase = p.kv_start[b];
        n_q = q8_count(p.q_start, b);
        T_len = q8_count(p.kv_start, b);
        if (n_q != 0 && q8_bad_lengths(n_q, p.n_q, T_len, p.T_len, qbase, p.total_q, kbase)) {
            if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.z == 0) flag(p.dev_status, ACACHE_DEV_BAD_LENGTH);
            return;
        }
    }
    const int64_t r0 = (int64_t)blockIdx.z * kBM, n_rows = (int64_t)n_q * p.g;
    if (r0 >= n_rows) return;
    const int rows = (int)min((int64_t)kBM, n_rows - r0);
    const int n_all = (T_len + kBN - 1) / kBN;
    const int cs = min(p.cs, n_all);                    // ranks past the tiles have nothing to do
    if (cr >= cs) return;
    const int j0 = (int)((int64_t)cr * n_all / cs), j1 = (int)((int64_t)(cr + 1) * n_all / cs);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    auto q_off = [&](int r) {                           // element offset of packed row r0 + r
        const int64_t i = (r0 + r) / p.g;
        return ((qbase + i) * p.Hq + (int64_t)hk * p.g + (r0 + r - i * p.g)) * D;
    };
    for (int x = tid; x < kBM * D; x += kThreads) {
        const int r = x / D, c = x % D;
        sm.q[c][r] = r < rows ? to_f32(((const T*)p.q)[q_off(r) + c]) : 0.f;
    }
    bool any = false;                                   // a key of this thread's columns is there
    float m[4], l[4], acc[4][NC * 4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        m[y] = -INFINITY;
        l[y] = 0.f;
#pragma unroll
        for (int x = 0; x < NC * 4; ++x) acc[y][x] = 0.f;
    }
    // slots and exponents of a tile's keys, looked up a tile ahead
    int64_t row = -2;
    uint32_t two = 0;
    auto look_up = [&](int j) {
        const int t = j * kBN + tid;
        row = -2;
        two = 0;
        if (j < j1 && tid < kBN && t < T_len) {
            const int64_t s = p.read_slot[kbase + t];
            if (s >= 0 && s < p.num_slots) {
                row = s * p.Hkv + hk;
                two = reinterpret_cast<const uint16_t*>(p.kv_scale)[row];
            } else if (!(p.drop_none && s == ACACHE_SLOT_NONE)) {
                row = -1;
                flag(p.dev_status, ACACHE_DEV_BAD_SLOT);
            }
        }
    };
    look_up(j0);
    for (int j = j0; j < j1; ++j) {
        __syncthreads();                                // the last tile has been read
        if (tid < kBN) {
            sm.row[tid] = row;
            sm.ks[tid] = row >= 0 ? q8_factor(two & 0xffu) : 0.f;
            sm.vs[tid] = row >= 0 ? q8_factor(two >> 8) : 0.f;
        }
        look_up(j + 1);
        __syncthreads();
#pragma unroll
        for (int it = 0; it < kBN * D / 16 / kThreads; ++it) {
            const int x = it * kThreads + tid;
            {   // K: consecutive lanes take consecutive keys, so the transposed stores do not conflict
                const int key = x & (kBN - 1), c = x / kBN;
                const int64_t row = sm.row[key];
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (row >= 0) w = *reinterpret_cast<const uint4*>(p.k_cache + row * D + c * 16);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
                const float f = sm.ks[key];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 e = q8_decode2((ww[i >> 1] >> (16 * (i & 1))) & 0xffffu);
                    sm.k[c * 16 + 2 * i][key] = e.x * f;
                    sm.k[c * 16 + 2 * i + 1][key] = e.y * f;
                }
            }
            {   // V
                const int key = x / (D / 16), c = x % (D / 16);
                const int64_t row = sm.row[key];
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (row >= 0) w = *reinterpret_cast<const uint4*>(p.v_cache + row * D + c * 16);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
                const float f = row >= 0 ? sm.vs[key] : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 e = q8_decode2(ww[i] & 0xffffu), h = q8_decode2(ww[i] >> 16);
                    *reinterpret_cast<float4*>(&sm.v[key][c * 16 + 4 * i]) =
                        make_float4(e.x * f, e.y * f, h.x * f, h.y * f);
                }
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
        bool gone[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            gone[x] = sm.row[4 * tx + x] == -2;
            any = any || !gone[x];
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            float mt = -INFINITY;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[y][x] = gone[x] ? -INFINITY : s[y][x] * p.scale_log2;
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
    for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) l[y] += __shfl_xor_sync(0xffffffffu, l[y], o);
    // A row has a maximum if it has a key, be its logit -infinity: then a sum of 0 is 0 / 0, not an empty row.
    any = __any_sync(0xffffffffu, any);
#pragma unroll
    for (int y = 0; y < 4; ++y)
        if (any) m[y] = fmaxf(m[y], -FLT_MAX);
    if (cs == 1) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int r = 4 * ty + y;
            if (r >= rows) continue;
            T* o = (T*)p.out + q_off(r);
            // a row without keys gives zeros (a NaN sum is carried into the output)
            const float inv = m[y] == -INFINITY && l[y] == 0.f ? 0.f : 1.f / l[y];
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[n * 64 + 4 * tx + x] = from_f32<T>(acc[y][n * 4 + x] * inv);
        }
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
        const float inv = M == -INFINITY && L == 0.f ? 0.f : 1.f / L;
        T* o = (T*)p.out + q_off(r) + 4 * c;
        o[0] = from_f32<T>(O.x * inv);
        o[1] = from_f32<T>(O.y * inv);
        o[2] = from_f32<T>(O.z * inv);
        o[3] = from_f32<T>(O.w * inv);
    }
    ptx::cluster_sync();       // no CTA may leave while another still reads its shared memory
}

// CTAs of a variant that run at once in clusters of cs (a cluster stays within a group of SMs), per device.
std::atomic<int> g_slots[2][3][kMaxCluster + 1][64];

template <typename T, int D, int kBM>
int launch(SimtParams prm, const Q8Attn& c) {
    auto kern = q8_simt_kernel<T, D, kBM>;
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
    // Parts of the key range: waves x (tiles of a part, a CTA's own cost of about one and as much for a merge)
    const int64_t n_rb = ((int64_t)c.n_q * prm.g + kBM - 1) / kBM, units = (int64_t)c.B * prm.Hkv * n_rb;
    const int tiles = (c.T_len + kBN - 1) / kBN;
    int64_t best = 0;
    for (int cs = 1; cs <= kMaxCluster && cs <= tiles; ++cs) {
        std::atomic<int>& known = g_slots[D == 128][kBM == 16 ? 0 : kBM == 32 ? 1 : 2][cs][dev];
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
int launch(const SimtParams& prm, const Q8Attn& c) {
    const int64_t rows = (int64_t)c.n_q * prm.g;
    return rows <= 16 ? launch<T, D, 16>(prm, c) : rows <= 32 ? launch<T, D, 32>(prm, c) : launch<T, D, 64>(prm, c);
}

}  // namespace

int launch_q8_simt_attention(const Q8Attn& c) {
    const int g = c.a.hq / c.a.hkv;
    SimtParams prm{};
    prm.q = c.q;
    prm.k_cache = c.k_cache;
    prm.v_cache = c.v_cache;
    prm.kv_scale = c.kv_scale;
    prm.read_slot = c.read_slot;
    prm.q_start = c.q_start;
    prm.kv_start = c.kv_start;
    prm.out = c.out;
    prm.dev_status = c.dev_status;
    prm.num_slots = c.num_slots;
    prm.n_q = c.n_q;
    prm.total_q = c.total_q;
    prm.T_len = c.T_len;
    prm.Hq = c.a.hq;
    prm.Hkv = c.a.hkv;
    prm.g = g;
    prm.drop_none = c.drop_none;
    prm.scale_log2 = c.a.scale * kLog2e;
    if (c.a.dtype == ACACHE_F32) return c.a.d == 64 ? launch<float, 64>(prm, c) : launch<float, 128>(prm, c);
    return c.a.d == 64 ? launch<__nv_bfloat16, 64>(prm, c) : launch<__nv_bfloat16, 128>(prm, c);
}

}  // namespace acache
