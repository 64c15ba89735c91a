// Cross attention of a few rows: single tokens (and up to four rows that read
// one key set: short queries, or the query heads of a group), forward and
// backward.
//
// The formulas are those of cross_attn.cu and cross_bwd.cu.  With so few rows a
// key's bytes take longer than its products, so there is no tensor-core tile to
// fill: D/8 lanes hold a key's row in 16-byte chunks, several keys are under way
// in each group of lanes, and everything is fp32 from the products on (no p or ds
// is rounded).  A mask is read where it is used, without a list of kept keys.
//
// One cluster of CTAs per key set, each with a range of its keys; the ranges
// meet over distributed shared memory in rank order, so a call is one launch
// with no partial sums in memory, and equal calls give equal bits.
//
// Bound by HBM (k, v once; backward dk, dv once) and by launch latency: 24 heads
// of 8 requests over 512 states of 128 dims take 16 us forward and 30 us
// backward, where the tensor-core kernels take 20 and 118.
#include <cooperative_groups.h>

#include "cross_common.cuh"

namespace scope {
namespace op {

namespace cg = cooperative_groups;

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 4;      // most rows of a key set
constexpr int kFewKeys = 2048;   // most keys of a CTA (the backward kernel keeps their p and dp)

template <int D>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct FewRow {
    int b, h, n;
};

__device__ __forceinline__ FewRow few_row(const CrossArgs &a, int bk, int hk, int r)
{
    const RowTile w{a.Bk != a.B ? 0 : bk, hk * a.G, 0, 0};
    FewRow x;
    tile_row(a, w, hk, r, x.b, x.h, x.n);
    return x;
}

// This CTA's key set and range of the set's keys, of `n` in all.
struct FewRange {
    int bk, hk, k0, k1, nk;
};

__device__ __forceinline__ FewRange few_range(const CrossArgs &a, int ranks, int rank, bool all)
{
    FewRange w;
    w.bk = a.by_Hk((int)(blockIdx.x / ranks), w.hk);
    w.nk = keys_of(a, w.bk);
    const int64_t n = all ? a.M : w.nk;
    w.k0 = (int)(n * rank / ranks);
    w.k1 = (int)(n * (rank + 1) / ranks);
    return w;
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(kFewThreads) cross_few_kernel(const __grid_constant__ CrossArgs a)
{
    constexpr int LPR = D / 8, NG = kFewThreads / LPR, U = 4;
    __shared__ float w_o[kFewWarps][R][D], w_m[kFewWarps][R], w_l[kFewWarps][R];
    __shared__ float c_o[R][D], c_m[R], c_l[R];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const FewRange w = few_range(a, ranks, rank, false);
    const int rows = a.heads * a.N;
    const int g = threadIdx.x / LPR, c8 = threadIdx.x % LPR, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *k = static_cast<const T *>(a.k) + w.bk * a.kB + w.hk * a.kH + c8 * 8;
    const T *v = static_cast<const T *>(a.v) + w.bk * a.vB + w.hk * a.vH + c8 * 8;
    const uint8_t *mask = a.mask ? a.mask + w.bk * a.mask_stride : nullptr;
    float q[R][8], o[R][8], m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const FewRow x = few_row(a, w.bk, w.hk, min(r, rows - 1));
        load8(static_cast<const T *>(a.q) + x.b * a.qB + x.h * a.qH + x.n * a.qN + c8 * 8, q[r]);
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[r][i] = 0.f;
    }
    // each step's rows are under way while the one before is worked on
    Raw8<T> kr[U], vr[U];
    bool on[U], next[U];
    auto allowed = [&](int key) { return key < w.k1 && (!mask || mask[key]); };
    auto fetch = [&](Raw8<T> &x, const T *base, int64_t stride, int key, bool ok) {
        x.u = make_uint4(0u, 0u, 0u, 0u);
        if (ok) x.load(base + key * stride);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int key = w.k0 + u * NG + g;
        next[u] = allowed(key);
        fetch(kr[u], k, a.kN, key, next[u]);
        fetch(vr[u], v, a.vN, key, next[u]);
    }
#pragma unroll 1
    for (int k0 = w.k0; k0 < w.k1; k0 += NG * U) {  // uniform for the CTA
        float s[R][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int later = k0 + (U + u) * NG + g;
            float x[8];
            kr[u].values(x);
            on[u] = next[u];
            next[u] = allowed(later);
            fetch(kr[u], k, a.kN, later, next[u]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float d = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) d = fmaf(q[r][i], x[i], d);
                s[r][u] = d;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float mx = m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[r][u] = group_sum<D>(s[r][u]) * a.scale_log2;
                if (!on[u]) s[r][u] = -INFINITY;
                mx = fmaxf(mx, s[r][u]);
            }
            const float ref = mx == -INFINITY ? 0.f : mx, alpha = tc::ex2(m[r] - ref);
            m[r] = mx;
            l[r] *= alpha;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[r][i] *= alpha;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[r][u] = tc::ex2(s[r][u] - ref);
                l[r] += s[r][u];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[8];
            vr[u].values(x);
            fetch(vr[u], v, a.vN, k0 + (U + u) * NG + g, next[u]);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) o[r][i] = fmaf(s[r][u], x[i], o[r][i]);
        }
    }
    // the groups of a warp, then the warps, then the CTAs
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int x = LPR; x < 32; x <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m[r], x), mx = fmaxf(m[r], m2);
            const float ref = mx == -INFINITY ? 0.f : mx, s1 = tc::ex2(m[r] - ref), s2 = tc::ex2(m2 - ref);
            l[r] = l[r] * s1 + __shfl_xor_sync(0xffffffffu, l[r], x) * s2;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[r][i] = o[r][i] * s1 + __shfl_xor_sync(0xffffffffu, o[r][i], x) * s2;
            m[r] = mx;
        }
        if (lane < LPR) {
            store8(&w_o[warp][r][c8 * 8], o[r]);
            if (c8 == 0) {
                w_m[warp][r] = m[r];
                w_l[warp][r] = l[r];
            }
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < R * D; e += kFewThreads) {
        const int r = e / D, d = e % D;
        float mx = -INFINITY, ls = 0.f, os = 0.f;
        for (int x = 0; x < kFewWarps; ++x) mx = fmaxf(mx, w_m[x][r]);
        const float ref = mx == -INFINITY ? 0.f : mx;
        for (int x = 0; x < kFewWarps; ++x) {
            const float s = tc::ex2(w_m[x][r] - ref);
            ls = fmaf(w_l[x][r], s, ls);
            os = fmaf(w_o[x][r][d], s, os);
        }
        c_o[r][d] = os;
        if (d == 0) {
            c_m[r] = mx;
            c_l[r] = ls;
        }
    }
    cluster.sync();
    if (rank == 0)
        for (int e = threadIdx.x; e < rows * D; e += kFewThreads) {
            const int r = e / D, d = e % D;
            float mx = -INFINITY, ls = 0.f, os = 0.f;
            for (int x = 0; x < ranks; ++x) mx = fmaxf(mx, cluster.map_shared_rank(c_m, x)[r]);
            const float ref = mx == -INFINITY ? 0.f : mx;
            for (int x = 0; x < ranks; ++x) {
                const float s = tc::ex2(cluster.map_shared_rank(c_m, x)[r] - ref);
                ls = fmaf(cluster.map_shared_rank(c_l, x)[r], s, ls);
                os = fmaf(cluster.map_shared_rank(&c_o[0][0], x)[e], s, os);
            }
            const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);  // a NaN sum stays one
            const FewRow y = few_row(a, w.bk, w.hk, r);
            T *dst = static_cast<T *>(a.o) + y.b * a.oB + y.h * a.oH + y.n * a.oN + d;
            if constexpr (sizeof(T) == 2) {
                const uint32_t bits = pack2(T(), os * inv, 0.f);
                *reinterpret_cast<uint16_t *>(dst) = (uint16_t)bits;
            }
            if (d == 0 && a.lse)
                a.lse[((int64_t)y.b * a.H + y.h) * a.N + y.n] = ls == 0.f ? -INFINITY : (mx + log2f(ls)) * 0.6931471805599453f;
        }
    cluster.sync();  // nobody leaves while its sums are read
}

// p and dp of the CTA's keys; sums of each warp and of the CTA: p dp k, p k, p dp
// and the keys that are read.
template <int D, int R>
constexpr size_t few_bwd_smem(int keys)
{
    return ((size_t)keys * R * 2 + (size_t)(kFewWarps + 1) * R * (2 * D + 2) + R) * 4;
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(kFewThreads, R == 1 ? 3 : R == 2 ? 2 : 1) cross_few_bwd_kernel(const __grid_constant__ CrossArgs a, int cap)
{
    // with one row the registers of rows under way cost more (CTAs a SM) than they give: 30 us for 35
    constexpr bool kAhead = R > 1;
    constexpr int LPR = D / 8, NG = kFewThreads / LPR, U = 2, S = 2 * D + 2;
    extern __shared__ __align__(16) float few_smem[];
    float2 *pd = reinterpret_cast<float2 *>(few_smem);        // [cap][R]
    float *w_s = few_smem + (size_t)cap * R * 2;              // [warps][R][S]
    float *c_s = w_s + kFewWarps * R * S, *s_D = c_s + R * S;  // [R][S], [R]
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const FewRange w = few_range(a, ranks, rank, true);
    const int rows = a.heads * a.N;
    const int g = threadIdx.x / LPR, c8 = threadIdx.x % LPR, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *k = static_cast<const T *>(a.k) + w.bk * a.kB + w.hk * a.kH + c8 * 8;
    const T *v = static_cast<const T *>(a.v) + w.bk * a.vB + w.hk * a.vH + c8 * 8;
    const uint8_t *mask = a.mask ? a.mask + w.bk * a.mask_stride : nullptr;
    float q[R][8], y[R][8], t[R][8], e[R][8], nl[R], delta[R], count = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const FewRow x = few_row(a, w.bk, w.hk, min(r, rows - 1));
        load8(static_cast<const T *>(a.q) + x.b * a.qB + x.h * a.qH + x.n * a.qN + c8 * 8, q[r]);
        load8(static_cast<const T *>(a.dout) + x.b * a.dB + x.h * a.dH + x.n * a.dN + c8 * 8, y[r]);
        const float lse = a.lse[((int64_t)x.b * a.H + x.h) * a.N + x.n];
        nl[r] = r < rows && lse != -INFINITY ? -lse * 1.4426950408889634f : -INFINITY;  // such a row's p is 0
        delta[r] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t[r][i] = e[r][i] = 0.f;
    }
    Raw8<T> kr[U], vr[U];
    bool next[U];
    auto fetch = [&](int u, int key) {
        next[u] = key < min(w.k1, w.nk) && (!mask || mask[key]);
        kr[u].u = vr[u].u = make_uint4(0u, 0u, 0u, 0u);
        if (next[u]) {
            kr[u].load(k + key * a.kN);
            vr[u].load(v + key * a.vN);
        }
    };
    if constexpr (kAhead) {
#pragma unroll
        for (int u = 0; u < U; ++u) fetch(u, w.k0 + u * NG + g);
    }
#pragma unroll 1
    for (int k0 = w.k0; k0 < w.k1; k0 += NG * U) {  // uniform for the CTA
        if constexpr (!kAhead) {
#pragma unroll
            for (int u = 0; u < U; ++u) fetch(u, k0 + u * NG + g);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = k0 + u * NG + g;
            const bool on = next[u];
            if (on) count += 1.f;
            float x[8], z[8];
            kr[u].values(x);
            vr[u].values(z);
            if constexpr (kAhead) fetch(u, key + U * NG);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float s = 0.f, dp = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s = fmaf(q[r][i], x[i], s);
                    dp = fmaf(y[r][i], z[i], dp);
                }
                s = group_sum<D>(s);
                dp = group_sum<D>(dp);
                // (a row or key that is not there counts nothing, whatever its other side holds)
                const bool some = on && nl[r] != -INFINITY;
                const float p = some ? tc::ex2(fmaf(s, a.scale_log2, nl[r])) : 0.f;
                if (!some) dp = 0.f;
                const float pdp = p * dp;
                delta[r] += pdp;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    t[r][i] = fmaf(pdp, x[i], t[r][i]);
                    e[r][i] = fmaf(p, x[i], e[r][i]);
                }
                if (c8 == 0 && key < w.k1) pd[(key - w.k0) * R + r] = make_float2(p, dp);
            }
        }
    }
#pragma unroll
    for (int x = LPR; x < 32; x <<= 1) count += __shfl_xor_sync(0xffffffffu, count, x);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int x = LPR; x < 32; x <<= 1) {
            delta[r] += __shfl_xor_sync(0xffffffffu, delta[r], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[r][i] += __shfl_xor_sync(0xffffffffu, t[r][i], x);
                e[r][i] += __shfl_xor_sync(0xffffffffu, e[r][i], x);
            }
        }
        if (lane < LPR) {
            float *dst = w_s + (warp * R + r) * S;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dst[c8 * 8 + i] = t[r][i];
                dst[D + c8 * 8 + i] = e[r][i];
            }
            if (c8 == 0) {
                dst[2 * D] = delta[r];
                dst[2 * D + 1] = count;
            }
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < R * S; x += kFewThreads) {
        float s = 0.f;
        for (int i = 0; i < kFewWarps; ++i) s += w_s[i * R * S + x];
        c_s[x] = s;
    }
    cluster.sync();
    // of a single key p is 1 whatever its score: no gradient reaches q and k, not even the roundings of dp - D
    float keys = 0.f;
    for (int x = 0; x < ranks; ++x) keys += cluster.map_shared_rank(c_s, x)[2 * D + 1];
    const float scale = keys == 1.f ? 0.f : a.scale;
    if (threadIdx.x < R) {
        float s = 0.f;
        for (int x = 0; x < ranks; ++x) s += cluster.map_shared_rank(c_s, x)[threadIdx.x * S + 2 * D];
        s_D[threadIdx.x] = s;
    }
    __syncthreads();
    if (rank == 0)
        for (int x = threadIdx.x; x < rows * D; x += kFewThreads) {
            const int r = x / D, d = x % D;
            float st = 0.f, se = 0.f;
            for (int i = 0; i < ranks; ++i) {
                const float *c = cluster.map_shared_rank(c_s, i) + r * S;
                st += c[d];
                se += c[D + d];
            }
            const FewRow z = few_row(a, w.bk, w.hk, r);
            T *dst = static_cast<T *>(a.dq) + z.b * a.dqB + z.h * a.dqH + z.n * a.dqN + d;
            *reinterpret_cast<uint16_t *>(dst) = (uint16_t)pack2(T(), fmaf(-s_D[r], se, st) * scale, 0.f);
        }
    // dk, dv of the range, zeros where no row reads the key
    T *dk = static_cast<T *>(a.dk) + w.bk * a.dkB + w.hk * a.dkH + c8 * 8;
    T *dv = static_cast<T *>(a.dv) + w.bk * a.dvB + w.hk * a.dvH + c8 * 8;
    float D_r[R];
#pragma unroll
    for (int r = 0; r < R; ++r) D_r[r] = s_D[r];
    for (int key = w.k0 + g; key < w.k1; key += NG) {
        float sk[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 x = pd[(key - w.k0) * R + r];
            if (x.x == 0.f) continue;  // (NaN is not)
            const float ds = x.x * (x.y - D_r[r]) * scale;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sk[i] = fmaf(ds, q[r][i], sk[i]);
                sv[i] = fmaf(x.x, y[r][i], sv[i]);
            }
        }
        store8(dk + key * a.dkN, sk);
        store8(dv + key * a.dvN, sv);
    }
    cluster.sync();  // nobody leaves while its sums are read
}

// CTAs of a key set's cluster, or 0 where the tensor-core kernels serve better:
// more rows, more keys than a CTA's (those kernels split them further), and
// forward, where the products of a second row cost more than those kernels' fixed
// time (24 heads of 512 keys: 1 row 5.5 us for 10, 4 rows 8.3 for 10; 512 heads of
// 2048 keys: 4 rows 313 us for 118) or long keys of few heads leave SMs idle
// (8 heads of 16000 keys: 34 us for 25).  The ranks double while a CTA has more than 128
// keys (so 65 are the fewest) and the sets fewer than eight CTAs a SM (so sixteen are the
// most).  Not all of those are resident: the bf16 kernel of one row takes 106 registers,
// two CTAs a SM, so 192 sets of 512 keys on four ranks come in 2.6 rounds.
int cross_few_ranks(int64_t sets, int64_t rows, int64_t M, bool backward, int sms)
{
    if (rows < 1 || rows > kFewRows || M < 1) return 0;
    int ranks = 1;
    while (ranks < 8 && M > 128 * ranks && (sets * ranks < 8 * (int64_t)sms || M > (int64_t)kFewKeys * ranks)) ranks *= 2;
    if (M > (int64_t)kFewKeys * ranks) return 0;
    if (!backward && (sets * M * (rows - 1) > 1024 * (int64_t)sms || (sets * ranks < sms && M > 1200 * ranks))) return 0;
    return ranks;
}

template <typename... Args>
static void launch_cluster(void (*kernel)(Args...), unsigned blocks, unsigned ranks, size_t smem, cudaStream_t st,
                           Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, args...);
    count_launches(1);
}

template <typename T, int D, int R>
static void few(const CrossArgs &a, bool backward, cudaStream_t st)
{
    const unsigned blocks = (unsigned)(a.sets * a.few_ranks);
    if (!backward) {
        launch_cluster(cross_few_kernel<T, D, R>, blocks, (unsigned)a.few_ranks, 0, st, a);
    } else {
        const int cap = (a.M + a.few_ranks - 1) / a.few_ranks;
        launch_cluster(cross_few_bwd_kernel<T, D, R>, blocks, (unsigned)a.few_ranks, few_bwd_smem<D, R>(cap), st, a, cap);
    }
}

template <typename T, int D>
static void few_rows(const CrossArgs &a, bool backward, cudaStream_t st)
{
    const int rows = a.heads * a.N;
    if (rows == 1) few<T, D, 1>(a, backward, st);
    else if (rows == 2) few<T, D, 2>(a, backward, st);
    else few<T, D, 4>(a, backward, st);
}

void launch_cross_few(const CrossArgs &a, int D, bool f16, bool backward, cudaStream_t st)
{
    if (f16) {
        if (D == 128) few_rows<__half, 128>(a, backward, st);
        else few_rows<__half, 64>(a, backward, st);
    } else {
        if (D == 128) few_rows<__nv_bfloat16, 128>(a, backward, st);
        else few_rows<__nv_bfloat16, 64>(a, backward, st);
    }
}

template <typename T, int D, int R>
static cudaError_t few_attr()
{
    return cudaFuncSetAttribute(cross_few_bwd_kernel<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)few_bwd_smem<D, R>(kFewKeys));
}

template <typename T, int D>
static cudaError_t few_attrs()
{
    const cudaError_t e[3] = {few_attr<T, D, 1>(), few_attr<T, D, 2>(), few_attr<T, D, 4>()};
    for (cudaError_t x : e)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}

cudaError_t cross_few_configure()
{
    const cudaError_t e[4] = {few_attrs<__nv_bfloat16, 128>(), few_attrs<__nv_bfloat16, 64>(), few_attrs<__half, 128>(),
                              few_attrs<__half, 64>()};
    for (cudaError_t x : e)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}

}  // namespace op
}  // namespace scope
