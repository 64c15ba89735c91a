// Cross attention, backward.  With p_ij = e^(s_ij - lse_i) recomputed from q, k
// and lse, D_i = do_i . o_i:
//
//   dv_j = sum_i p_ij do_i      dp_ij = do_i . v_j     ds_ij = p_ij (dp_ij - D_i)
//   dq_i = scale sum_j ds_ij k_j            dk_j = scale sum_i ds_ij q_i
//
// dk and dv sum over every query row that reads the key: the N queries, the
// query heads of the group and, for keys shared by the batch, its entries.
//
// Two tensor-core kernels, one per direction of the sum: cross_dq_kernel owns
// 128 rows and walks the keys (3 products a tile: S, dP, dQ), cross_dkv_kernel
// owns 128 keys and walks the rows (4 products: S^T, dP^T, dV, dK).  S and dP
// are computed twice, 14 D flops a pair instead of 10 D, and in exchange every
// accumulator stays in TMEM and no result is added up by atomics, so equal
// calls give equal bits.  (One kernel for both would send a fp32 dQ or dK/dV
// tile to memory per tile step.)  Bound: the tensor cores, 512 clocks a
// product of 128 x 128 x 128, against one exponential a pair in each kernel.
//
// Rows split over CTAs (few keys, many rows) or keys split (few rows, many
// keys) leave fp32 partial sums that a join adds in a fixed order.
//
// p and ds are rounded to the inputs' 16-bit type as operands of dV, dK, dQ;
// S, dP, D, lse and all sums are fp32.  Barriers, rings, bounded waits as in
// cross_attn.cu.
#include "cross_common.cuh"

namespace scope {
namespace op {

using namespace tc;

static __device__ int32_t g_cross_bwd_err[4];

constexpr int kBwdThreads = 384;
constexpr int kT = 128;      // rows or keys of a tile
constexpr int kQRing = 3;    // dq kernel: Q, dO tiles in flight
constexpr int kKvRing = 4;   // dq kernel: K, V tiles in flight
constexpr int kRowRing = 5;  // dk/dv kernel: Q, dO tiles in flight

constexpr size_t dq_smem(int D) { return (size_t)(kQRing + kKvRing) * kT * D * 2 + 1024; }
// tiles, three row tiles of nlse and two of ndelta, barriers.  At D = 128 that
// leaves no room to align the base by hand (227 KB a block), so the kernel has
// no static shared memory and checks that its base is aligned.
constexpr size_t dkv_smem(int D) { return (size_t)(2 + kRowRing) * kT * D * 2 + 5 * kT * 4 + 256; }

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// A-operand column of 16-element step k: each half of the warpgroups' 64
// packed values sits at the start of its own half of the fp32 columns.
__device__ __forceinline__ uint32_t half_col(int k) { return (uint32_t)((k >> 2) * 64 + (k & 3) * 8); }

__device__ __forceinline__ void bwd_prologue(int warp, uint32_t *tmem_base)
{
    if (warp == 11) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_base)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

__device__ __forceinline__ void bwd_epilogue(int warp, uint32_t tmem)
{
    tc_fence_before();
    __syncthreads();
    if (warp == 11) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// nlse and ndelta of every row of every key set, in the sets' row order.
template <typename T>
__global__ void __launch_bounds__(256) cross_rows_kernel(const __grid_constant__ CrossArgs a, int D)
{
    const int lpr = D / 8;
    const int64_t at = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / lpr;
    const int c8 = threadIdx.x % lpr;
    if (at >= (int64_t)a.sets * a.rows_pad) return;  // whole row groups of lanes
    const int set = (int)(at / a.rows_pad), r = (int)(at % a.rows_pad);
    const unsigned lanes = (lpr == 16 ? 0xffffu : 0xffu) << ((threadIdx.x & 31) & ~(lpr - 1));
    float sum = 0.f, nl = -INFINITY;
    if (r < a.rows) {
        int b, h, n;
        row_of(a, set / a.Hk, set % a.Hk, r, b, h, n);
        float o[8], d[8];
        load8(static_cast<const T *>(a.o) + b * a.oB + h * a.oH + n * a.oN + c8 * 8, o);
        load8(static_cast<const T *>(a.dout) + b * a.dB + h * a.dH + n * a.dN + c8 * 8, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(o[i], d[i], sum);
        const float lse = a.lse[((int64_t)b * a.H + h) * a.N + n];
        if (lse != -INFINITY) nl = -lse * 1.4426950408889634f;
    }
    for (int o = lpr >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(lanes, sum, o);
    if (c8 == 0) {
        a.nlse[at] = nl;
        a.ndelta[at] = -sum;
    }
}

// ---------------------------------------------------------------- dq
struct DqItem {
    int bk, hk, set, r0, nq, t0, t1, nk, split;
};

__device__ __forceinline__ DqItem dq_item(const CrossArgs &a, int item)
{
    DqItem w;
    const int tiles = a.rows_pad / kT;
    const int rt = item % tiles, rest = item / tiles;
    w.split = rest % a.dq_splits;
    w.set = rest / a.dq_splits;
    w.bk = w.set / a.Hk;
    w.hk = w.set % a.Hk;
    w.r0 = rt * kT;
    w.nq = min(kT, a.rows - w.r0);
    w.nk = keys_of(a, w.bk);
    const int kt = (w.nk + kT - 1) / kT;
    w.t0 = (int)((int64_t)kt * w.split / a.dq_splits);
    w.t1 = (int)((int64_t)kt * (w.split + 1) / a.dq_splits);
    return w;
}

// One persistent CTA per SM; item = 128 rows of a key set.  TMEM: S in two
// buffers [0,128) [128,256), so S(j+1) is computed under the softmax of j; dP
// [256,384); dQ [384,384+D).  Warps 0-3 take the keys 0-63 of a tile, warps
// 4-7 the keys 64-127, one thread per row and half; ds (16 bit) overwrites the
// half's own part of S.  S and dP of step j+1 are out before ds of j is awaited,
// so the warps may arrive for both steps before the issuer looks: one ds_full
// barrier per S buffer (a single one would have passed the awaited phase twice).
template <typename T, int D>
__global__ void __launch_bounds__(kBwdThreads, 1) cross_dq_kernel(const __grid_constant__ CrossArgs a, int items)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    constexpr int TB = kT * D * 2;
    unsigned char *sR = sm, *sKV = sm + kQRing * TB;
    __shared__ uint64_t r_full[kQRing], r_empty[kQRing], kv_full[kKvRing], kv_empty[kKvRing], s_full[2], dp_full, dp_read,
        ds_full[2], dq_full, dq_empty;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kQRing; ++i) {
            mbar_init(&r_full[i], 1);
            mbar_init(&r_empty[i], 1);
        }
        for (int i = 0; i < kKvRing; ++i) {
            mbar_init(&kv_full[i], 2);
            mbar_init(&kv_empty[i], 1);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(&dp_full, 1);
        mbar_init(&dp_read, 8);
        mbar_init(&ds_full[0], 8);
        mbar_init(&ds_full[1], 8);
        mbar_init(&dq_full, 1);
        mbar_init(&dq_empty, 8);
        abort_sh = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    bwd_prologue(warp, &tmem_base_sh);
    const uint32_t tmem = tmem_base_sh;
    const Waiter wait{&abort_sh, g_cross_bwd_err};

    if (warp == 8) {
        // ------------------------------------------------------------ Q, dO rows
        RingFill<kQRing> ring(r_full, r_empty);
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const DqItem w = dq_item(a, item);
            if (w.t0 == w.t1) continue;
            if (!ring.acquire(wait, 0x50)) break;
            copy_rows<T, D>(a, w.bk, w.hk, w.r0, w.nq, kT, static_cast<const T *>(a.q), a.qB, a.qH, a.qN,
                            smem_u32(sR + ring.slot * TB), lane, 32);
            ring.issued();
            if (!ring.acquire(wait, 0x50)) break;
            copy_rows<T, D>(a, w.bk, w.hk, w.r0, w.nq, kT, static_cast<const T *>(a.dout), a.dB, a.dH, a.dN,
                            smem_u32(sR + ring.slot * TB), lane, 32);
            ring.issued();
        }
        ring.flush();
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------------------ K, V rows
        const int tid = threadIdx.x - 9 * 32;
        RingFill<kKvRing> ring(kv_full, kv_empty);
        KeyTile<T, D, 64> tile;
        bool ok = true;
        for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
            const DqItem w = dq_item(a, item);
            const T *k = static_cast<const T *>(a.k) + w.bk * a.kB + w.hk * a.kH;
            const T *v = static_cast<const T *>(a.v) + w.bk * a.vB + w.hk * a.vH;
            const int32_t *list = a.idx ? a.idx + (int64_t)w.bk * a.M : nullptr;
            for (int j = w.t0; j < w.t1; ++j) {
                tile.load(list, w.nk, j, tid);
                if (!(ok = ring.acquire(wait, 0x51))) break;
                tile.copy(k, a.kN, smem_u32(sKV + ring.slot * TB), tid);
                ring.issued();
                if (!(ok = ring.acquire(wait, 0x51))) break;
                tile.copy(v, a.vN, smem_u32(sKV + ring.slot * TB), tid);
                ring.issued();
            }
        }
        ring.flush();
    } else if (warp == 11) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t id_s = idesc16<T>(kT, false), id_q = idesc16<T>(D, true);
            const uint64_t dr = sw128_desc(smem_u32(sR), 16, 1024);
            const uint64_t dkv = sw128_desc(smem_u32(sKV), 16, 1024);
            const uint64_t dmn = sw128_desc(smem_u32(sKV), kT * 128, 1024);
            RingRead<kQRing> rr;
            RingRead<kKvRing> kv;
            int ns = 0, nd = 0, no = 0;  // steps issued in all (S buffer), dP reads awaited, dQ tiles done
            auto product = [&](uint32_t d, int rslot, int kvslot) {  // d = rows x keys
                const uint64_t ar = dr + (uint64_t)((rslot * TB) >> 4), bk = dkv + (uint64_t)((kvslot * TB) >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t o = (uint64_t)(((k >> 2) * (kT * 128) + (k & 3) * 32) >> 4);
                    mma_ss(d, ar + o, bk + o, id_s, k > 0);
                }
            };
            bool ok = true;
            for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
                const DqItem w = dq_item(a, item);
                if (w.t0 == w.t1) continue;
                const int qs = rr.slot;
                if (!(ok = wait(&r_full[qs], rr.use & 1, 0x52))) break;
                rr.next();
                const int os = rr.slot, o_use = rr.use;
                rr.next();
                int ks = kv.slot;  // K of the current step
                if (!(ok = wait(&kv_full[ks], kv.use & 1, 0x53))) break;
                kv.next();
                tc_fence_after();
                product(tmem + (ns & 1) * 128, qs, ks);
                mma_commit(&s_full[ns & 1]);
                if (w.t0 + 1 == w.t1) mma_commit(&r_empty[qs]);
                if (!(ok = wait(&r_full[os], o_use & 1, 0x54) && wait(&kv_full[kv.slot], kv.use & 1, 0x55))) break;
                // the softmax has read the dP before this one
                if (nd > 0 && !(ok = wait(&dp_read, (nd - 1) & 1, 0x56))) break;
                tc_fence_after();
                product(tmem + 256, os, kv.slot);
                mma_commit(&dp_full);
                mma_commit(&kv_empty[kv.slot]);
                if (w.t0 + 1 == w.t1) mma_commit(&r_empty[os]);
                kv.next();
                ++nd;
                for (int j = w.t0; j < w.t1; ++j) {
                    const bool more = j + 1 < w.t1, last = j + 2 == w.t1;
                    const int cur = ns & 1;
                    int kn = 0;
                    if (more) {
                        kn = kv.slot;
                        if (!(ok = wait(&kv_full[kn], kv.use & 1, 0x57))) break;
                        kv.next();
                        tc_fence_after();
                        product(tmem + (cur ^ 1) * 128, qs, kn);
                        mma_commit(&s_full[cur ^ 1]);
                        if (last) mma_commit(&r_empty[qs]);
                        if (!(ok = wait(&kv_full[kv.slot], kv.use & 1, 0x58) && wait(&dp_read, (nd - 1) & 1, 0x59))) break;
                        tc_fence_after();
                        product(tmem + 256, os, kv.slot);
                        mma_commit(&dp_full);
                        mma_commit(&kv_empty[kv.slot]);
                        if (last) mma_commit(&r_empty[os]);
                        kv.next();
                        ++nd;
                    }
                    if (!(ok = wait(&ds_full[cur], (ns >> 1) & 1, 0x5a))) break;
                    // the previous item's dQ has been read
                    if (j == w.t0 && no > 0 && !(ok = wait(&dq_empty, (no - 1) & 1, 0x5b))) break;
                    tc_fence_after();
                    const uint64_t bk = dmn + (uint64_t)((ks * TB) >> 4);
#pragma unroll
                    for (int k = 0; k < kT / 16; ++k)
                        mma_ts(tmem + 384, tmem + cur * 128 + half_col(k), bk + (uint64_t)((k * 2048) >> 4), id_q,
                               j > w.t0 || k > 0);
                    mma_commit(&kv_empty[ks]);
                    if (!more) mma_commit(&dq_full);
                    ks = kn;
                    ++ns;
                }
                ++no;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        const int half = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        int ns = 0, no = 0;
        bool ok = true;
        const uint64_t scp = f2pack(a.scale * 1.4426950408889634f, a.scale * 1.4426950408889634f);
        for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
            const DqItem w = dq_item(a, item);
            const int64_t at = (int64_t)w.set * a.rows_pad + w.r0 + row;
            const float nl = a.nlse[at], nd = a.ndelta[at];
            const uint64_t nlp = f2pack(nl, nl), ndp = f2pack(nd, nd);
            for (int j = w.t0; j < w.t1; ++j) {
                const uint32_t tS = tmem + lane_off + (ns & 1) * 128 + half * 64;
                const uint32_t tP = tmem + lane_off + 256 + half * 64;
                if (!(ok = wait.warp(&s_full[ns & 1], (ns >> 1) & 1, 0x5c))) break;
                tc_fence_after();
                uint32_t r[64];
                tmem_ld32(tS, r);
                tmem_ld32(tS + 32, r + 32);
                tmem_wait_ld();
                const int valid = w.nk - j * kT - half * 64;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float x0, x1;
                    f2unpack(ffma2(f2pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), scp, nlp), x0, x1);
                    r[2 * i] = __float_as_uint(ex2(x0));
                    r[2 * i + 1] = __float_as_uint(ex2(x1));
                }
                if (valid < 64) {  // keys past the end: their K rows are zeros, but p must not overflow
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (i >= valid) r[i] = 0u;
                }
                if (!(ok = wait.warp(&dp_full, ns & 1, 0x5d))) break;
                tc_fence_after();
                uint32_t d[64];
                tmem_ld32(tP, d);
                tmem_ld32(tP + 32, d + 32);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&dp_read);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int e = c * 32 + 2 * i;
                        float x0, x1;
                        f2unpack(fmul2(f2pack(__uint_as_float(r[e]), __uint_as_float(r[e + 1])),
                                       fadd2(f2pack(__uint_as_float(d[e]), __uint_as_float(d[e + 1])), ndp)),
                                 x0, x1);
                        pk[i] = pack2(T(), x0, x1);
                    }
                    tmem_st16(tS + c * 16, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_full[ns & 1]);
                ++ns;
            }
            if (!ok) break;
            const bool some = w.t0 < w.t1;
            if (some) {
                if (!(ok = wait.warp(&dq_full, no & 1, 0x5e))) break;
                ++no;
                tc_fence_after();
            }
            const bool store = row < w.nq;
            int b, h, n;
            row_of(a, w.bk, w.hk, w.r0 + (store ? row : 0), b, h, n);
            const int64_t total = (int64_t)a.B * a.H * a.N, flat = ((int64_t)b * a.H + h) * a.N + n;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int col = half * (D / 2) + c * 32;
                uint32_t o[32];
                if (some) {
                    tmem_ld32(tmem + lane_off + 384 + col, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                if (some && c == D / 64 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&dq_empty);
                }
                if (store) {
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * a.scale;
                    if (a.dq_splits > 1) {
                        float *dst = a.part_dq + (w.split * total + flat) * D + col;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) store8(dst + i, f + i);
                    } else {
                        T *dst = static_cast<T *>(a.dq) + b * a.dqB + h * a.dqH + n * a.dqN + col;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) store8(dst + i, f + i);
                    }
                }
            }
        }
    }
    bwd_epilogue(warp, tmem);
}

// dq = sum of the key ranges' parts.
template <typename T>
__global__ void __launch_bounds__(256) cross_dq_join_kernel(const __grid_constant__ CrossArgs a, int D)
{
    const int lpr = D / 8;
    const int64_t total = (int64_t)a.B * a.H * a.N;
    const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / lpr;
    const int c8 = threadIdx.x % lpr;
    if (row >= total) return;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.dq_splits; ++s) {
        float x[8];
        load8(a.part_dq + (s * total + row) * D + c8 * 8, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += x[i];
    }
    const int64_t bh = row / a.N, n = row % a.N;
    store8(static_cast<T *>(a.dq) + (bh / a.H) * a.dqB + (bh % a.H) * a.dqH + n * a.dqN + c8 * 8, acc);
}

// ---------------------------------------------------------------- dk, dv
// One CTA per (key set, 128 keys, row range).  TMEM: S^T [0,128), dP^T
// [128,256), dV [256,256+D), dK [384,384+D).  P^T and dS^T (16 bit) overwrite
// S^T and dP^T.  Two phases alternate: dV(i) and S^T(i+1) run under the ds of
// row tile i, dK(i) and dP^T(i+1) under the exponentials of i+1.  Warps 0-3
// take the rows 0-63 of a row tile, warps 4-7 the rows 64-127, one thread per
// key and half.
template <typename T, int D>
__global__ void __launch_bounds__(kBwdThreads, 1) cross_dkv_kernel(const __grid_constant__ CrossArgs a, int key_tiles)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw;
    constexpr int TB = kT * D * 2;
    unsigned char *sK = sm, *sV = sm + TB, *sR = sm + 2 * TB;
    float *s_nl = reinterpret_cast<float *>(sm + (2 + kRowRing) * TB);  // [3][kT]
    float *s_nd = s_nl + 3 * kT;                                        // [2][kT]
    struct Barriers {
        uint64_t k_full, r_full[kRowRing], r_empty[kRowRing], s_full, dp_full, p_full, ds_full, acc_full;
        uint32_t tmem_base;
        int abort;
    };
    static_assert(sizeof(Barriers) <= 256, "room kept in dkv_smem");
    Barriers &bar = *reinterpret_cast<Barriers *>(s_nd + 2 * kT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int kt = blockIdx.x % key_tiles, rest = blockIdx.x / key_tiles;
    const int split = rest % a.dkv_splits, set = rest / a.dkv_splits;
    const int bk = set / a.Hk, hk = set % a.Hk;
    const int nk = keys_of(a, bk);
    const int row_tiles = a.rows_pad / kT;
    const int i0 = (int)((int64_t)row_tiles * split / a.dkv_splits);
    const int i1 = (int)((int64_t)row_tiles * (split + 1) / a.dkv_splits);
    // uniform for the CTA: no keys here, or a base that is not aligned
    if (kt * kT >= nk) return;
    if (smem_u32(sm) & 1023u) {
        if (threadIdx.x == 0) set_error(g_cross_bwd_err, kErrRange, 0x70);
        return;
    }
    if (threadIdx.x == 0) {
        mbar_init(&bar.k_full, 2);
        for (int i = 0; i < kRowRing; ++i) {
            mbar_init(&bar.r_full[i], 2);
            mbar_init(&bar.r_empty[i], 1);
        }
        mbar_init(&bar.s_full, 1);
        mbar_init(&bar.dp_full, 1);
        mbar_init(&bar.p_full, 8);
        mbar_init(&bar.ds_full, 8);
        mbar_init(&bar.acc_full, 1);
        bar.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    bwd_prologue(warp, &bar.tmem_base);
    const uint32_t tmem = bar.tmem_base;
    const Waiter wait{&bar.abort, g_cross_bwd_err};

    if (warp == 9 || warp == 10) {
        // ------------------------------------------------------------ producers: K, V once, then Q, dO row tiles
        const int tid = threadIdx.x - 9 * 32;
        {
            KeyTile<T, D, 64> tile;
            tile.load(a.idx ? a.idx + (int64_t)bk * a.M : nullptr, nk, kt, tid);
            tile.copy(static_cast<const T *>(a.k) + bk * a.kB + hk * a.kH, a.kN, smem_u32(sK), tid);
            tile.copy(static_cast<const T *>(a.v) + bk * a.vB + hk * a.vH, a.vN, smem_u32(sV), tid);
            cp_async_commit();
        }
        RingFill<kRowRing> ring(bar.r_full, bar.r_empty);
        const float *nl = a.nlse + (int64_t)set * a.rows_pad, *nd = a.ndelta + (int64_t)set * a.rows_pad;
        for (int i = i0; i < i1; ++i) {
            const int r0 = i * kT, nq = min(kT, a.rows - r0), u = i - i0;
            if (!ring.acquire(wait, 0x60)) break;
            copy_rows<T, D>(a, bk, hk, r0, nq, kT, static_cast<const T *>(a.q), a.qB, a.qH, a.qN,
                            smem_u32(sR + ring.slot * TB), tid, 64);
            if (tid < kT / 4) cp_async16(smem_u32(s_nl + (u % 3) * kT + tid * 4), nl + r0 + tid * 4, true);
            if (i == i0) {
                // K and V travel with the first Q tile: announce them together
                cp_async_commit();
                cp_async_wait_all();
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.k_full);
            }
            ring.issued();
            if (!ring.acquire(wait, 0x60)) break;
            copy_rows<T, D>(a, bk, hk, r0, nq, kT, static_cast<const T *>(a.dout), a.dB, a.dH, a.dN,
                            smem_u32(sR + ring.slot * TB), tid, 64);
            if (tid < kT / 4) cp_async16(smem_u32(s_nd + (u & 1) * kT + tid * 4), nd + r0 + tid * 4, true);
            ring.issued();
        }
        ring.flush();
    } else if (warp == 11) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t id_s = idesc16<T>(kT, false), id_acc = idesc16<T>(D, true);
            const uint64_t dK = sw128_desc(smem_u32(sK), 16, 1024), dV = sw128_desc(smem_u32(sV), 16, 1024);
            const uint64_t dr = sw128_desc(smem_u32(sR), 16, 1024);
            const uint64_t dmn = sw128_desc(smem_u32(sR), kT * 128, 1024);
            RingRead<kRowRing> rr;
            auto product = [&](uint32_t d, uint64_t keys, int slot) {  // d = keys x rows
                const uint64_t br = dr + (uint64_t)((slot * TB) >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t o = (uint64_t)(((k >> 2) * (kT * 128) + (k & 3) * 32) >> 4);
                    mma_ss(d, keys + o, br + o, id_s, k > 0);
                }
            };
            auto accumulate = [&](uint32_t d, uint32_t p, int slot, bool first) {  // d += p x rows
                const uint64_t b = dmn + (uint64_t)((slot * TB) >> 4);
#pragma unroll
                for (int k = 0; k < kT / 16; ++k)
                    mma_ts(d, p + half_col(k), b + (uint64_t)((k * 2048) >> 4), id_acc, !first || k > 0);
            };
            int qs = rr.slot;
            bool ok = wait(&bar.k_full, 0, 0x61) && wait(&bar.r_full[qs], rr.use & 1, 0x62);
            int os = 0;
            if (ok) {
                tc_fence_after();
                product(tmem, dK, qs);
                mma_commit(&bar.s_full);
                rr.next();
                os = rr.slot;
                ok = wait(&bar.r_full[os], rr.use & 1, 0x63);
            }
            if (ok) {
                tc_fence_after();
                product(tmem + 128, dV, os);
                mma_commit(&bar.dp_full);
                rr.next();
            }
            for (int i = i0; ok && i < i1; ++i) {
                const int u = i - i0;
                const bool more = i + 1 < i1;
                int qn = 0, on = 0;
                if (!(ok = wait(&bar.p_full, u & 1, 0x64))) break;
                tc_fence_after();
                accumulate(tmem + 256, tmem, os, u == 0);
                mma_commit(&bar.r_empty[os]);
                if (more) {
                    qn = rr.slot;
                    if (!(ok = wait(&bar.r_full[qn], rr.use & 1, 0x65))) break;
                    rr.next();
                    tc_fence_after();
                    product(tmem, dK, qn);
                    mma_commit(&bar.s_full);
                }
                if (!(ok = wait(&bar.ds_full, u & 1, 0x66))) break;
                tc_fence_after();
                accumulate(tmem + 384, tmem + 128, qs, u == 0);
                mma_commit(&bar.r_empty[qs]);
                if (more) {
                    on = rr.slot;
                    if (!(ok = wait(&bar.r_full[on], rr.use & 1, 0x67))) break;
                    rr.next();
                    tc_fence_after();
                    product(tmem + 128, dV, on);
                    mma_commit(&bar.dp_full);
                } else {
                    mma_commit(&bar.acc_full);
                }
                qs = qn;
                os = on;
            }
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------ softmax and epilogue
        const int half = warp >> 2, wq = warp & 3, key = wq * 32 + lane;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t tS = tmem + lane_off + half * 64, tP = tmem + lane_off + 128 + half * 64;
        const uint64_t scp = f2pack(a.scale * 1.4426950408889634f, a.scale * 1.4426950408889634f);
        bool ok = true;
        RingRead<kRowRing> rr;  // nlse, ndelta land with the Q, dO tiles
        for (int i = i0; i < i1; ++i) {
            const int u = i - i0;
            const ulonglong2 *nl = reinterpret_cast<const ulonglong2 *>(s_nl + (u % 3) * kT + half * 64);
            const ulonglong2 *nd = reinterpret_cast<const ulonglong2 *>(s_nd + (u & 1) * kT + half * 64);
            if (!(ok = wait.warp(&bar.r_full[rr.slot], rr.use & 1, 0x6b))) break;
            rr.next();
            if (!(ok = wait.warp(&bar.s_full, u & 1, 0x68))) break;
            tc_fence_after();
            uint32_t r[64];
            tmem_ld32(tS, r);
            tmem_ld32(tS + 32, r + 32);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const ulonglong2 n2 = nl[c];
                float x0, x1;
                f2unpack(ffma2(f2pack(__uint_as_float(r[4 * c]), __uint_as_float(r[4 * c + 1])), scp, n2.x), x0, x1);
                r[4 * c] = __float_as_uint(ex2(x0));
                r[4 * c + 1] = __float_as_uint(ex2(x1));
                f2unpack(ffma2(f2pack(__uint_as_float(r[4 * c + 2]), __uint_as_float(r[4 * c + 3])), scp, n2.y), x0, x1);
                r[4 * c + 2] = __float_as_uint(ex2(x0));
                r[4 * c + 3] = __float_as_uint(ex2(x1));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    pk[e] = pack2(T(), __uint_as_float(r[c * 32 + 2 * e]), __uint_as_float(r[c * 32 + 2 * e + 1]));
                tmem_st16(tS + c * 16, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full);
            if (!(ok = wait.warp(&bar.r_full[rr.slot], rr.use & 1, 0x6c))) break;
            rr.next();
            if (!(ok = wait.warp(&bar.dp_full, u & 1, 0x69))) break;
            tc_fence_after();
            uint32_t d[64];
            tmem_ld32(tP, d);
            tmem_ld32(tP + 32, d + 32);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const ulonglong2 n2 = nd[c * 8 + e];
                    const int q = c * 32 + 4 * e;
                    float x0, x1;
                    f2unpack(fmul2(f2pack(__uint_as_float(r[q]), __uint_as_float(r[q + 1])),
                                   fadd2(f2pack(__uint_as_float(d[q]), __uint_as_float(d[q + 1])), n2.x)),
                             x0, x1);
                    pk[2 * e] = pack2(T(), x0, x1);
                    f2unpack(fmul2(f2pack(__uint_as_float(r[q + 2]), __uint_as_float(r[q + 3])),
                                   fadd2(f2pack(__uint_as_float(d[q + 2]), __uint_as_float(d[q + 3])), n2.y)),
                             x0, x1);
                    pk[2 * e + 1] = pack2(T(), x0, x1);
                }
                tmem_st16(tP + c * 16, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.ds_full);
        }
        if (ok && wait.warp(&bar.acc_full, 0, 0x6a)) {
            tc_fence_after();
            const int m = kt * kT + key;
            const int64_t at = ((int64_t)split * a.sets + set) * a.M + m;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int col = half * (D / 2) + c * 32;
                uint32_t o[32];
                float f[32];
                tmem_ld32(tmem + lane_off + 256 + col, o);
                tmem_wait_ld();
                if (m < nk) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]);
#pragma unroll
                    for (int i = 0; i < 32; i += 8) store8(a.part_dv + at * D + col + i, f + i);
                }
                tmem_ld32(tmem + lane_off + 384 + col, o);
                tmem_wait_ld();
                if (m < nk) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * a.scale;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) store8(a.part_dk + at * D + col + i, f + i);
                }
            }
        }
    }
    bwd_epilogue(warp, tmem);
}

// dk, dv of every key: the row ranges' parts added in order; keys that no row
// may read get zeros.
struct DkvOut {
    void *dk, *dv;
    int64_t ks[3], vs[3];  // element strides of batch, head, key
    const int32_t *inv;    // place of a key in its list or -1, or null
};

template <typename T>
__global__ void __launch_bounds__(256) cross_dkv_join_kernel(const __grid_constant__ CrossArgs a,
                                                             const __grid_constant__ DkvOut out, int D)
{
    const int lpr = D / 8;
    const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / lpr;  // set * M + m
    const int c8 = threadIdx.x % lpr;
    if (row >= (int64_t)a.sets * a.M) return;
    const int set = (int)(row / a.M), m = (int)(row % a.M), bk = set / a.Hk, hk = set % a.Hk;
    const int place = out.inv ? out.inv[(int64_t)bk * a.M + m] : (m < keys_of(a, bk) ? m : -1);
    float sk[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (place >= 0) {
#pragma unroll 2
        for (int s = 0; s < a.dkv_splits; ++s) {
            const int64_t at = (((int64_t)s * a.sets + set) * a.M + place) * D + c8 * 8;
            float x[8], y[8];
            load8(a.part_dk + at, x);
            load8(a.part_dv + at, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sk[i] += x[i];
                sv[i] += y[i];
            }
        }
    }
    store8(static_cast<T *>(out.dk) + bk * out.ks[0] + hk * out.ks[1] + m * out.ks[2] + c8 * 8, sk);
    store8(static_cast<T *>(out.dv) + bk * out.vs[0] + hk * out.vs[1] + m * out.vs[2] + c8 * 8, sv);
}

template <typename T, int D>
static cudaError_t bwd_attr()
{
    const cudaError_t e = cudaFuncSetAttribute(cross_dq_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)dq_smem(D));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(cross_dkv_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dkv_smem(D));
}

cudaError_t cross_bwd_configure()
{
    const cudaError_t e[4] = {bwd_attr<__nv_bfloat16, 128>(), bwd_attr<__nv_bfloat16, 64>(), bwd_attr<__half, 128>(),
                              bwd_attr<__half, 64>()};
    for (cudaError_t x : e)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}

cudaError_t cross_bwd_error(int32_t *err, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(err, g_cross_bwd_err, sizeof g_cross_bwd_err);
    const int32_t zero[4] = {0, 0, 0, 0};
    if (e == cudaSuccess && clear && err[0]) e = cudaMemcpyToSymbol(g_cross_bwd_err, zero, sizeof zero);
    return e;
}

// Ranges of `len` tiles for `items` pieces of work: the count with the least
// modelled time in tile steps (some 1.3 us), a piece costing its tiles and
// `fixed` more, a range's partial sums `part` steps of join traffic.
static int best_split(int64_t items, int64_t len, int sms, double fixed, double part, double join)
{
    int best = 1;
    double least = 0.0;
    for (int64_t s = 1; s <= len && s <= 128 && (s == 1 || items * (s - 1) < 8 * (int64_t)sms); ++s) {
        const double waves = (double)((items * s + sms - 1) / sms);
        const double t = waves * ((double)((len + s - 1) / s) + fixed) + part * (double)s + (s > 1 ? join : 0.0);
        if (s == 1 || t < least) {
            least = t;
            best = (int)s;
        }
    }
    return best;
}

int cross_dq_splits(int64_t sets, int64_t rows, int64_t M, int64_t rows_total, int D, int sms)
{
    const int64_t items = sets * ((rows + kT - 1) / kT), len = (M + kT - 1) / kT;
    if (items >= sms) return 1;  // persistent: items even out by themselves
    return best_split(items, len, sms, 2.0, (double)rows_total * D * 8.0 / 6e6, 3.0);
}

int cross_dkv_splits(int64_t sets, int64_t rows, int64_t M, int D, int sms)
{
    const int64_t items = sets * ((M + kT - 1) / kT), len = (rows + kT - 1) / kT;
    return best_split(items, len, sms, 4.0, (double)(sets * M) * D * 16.0 / 6e6, 0.0);
}

template <typename T, int D>
static void launch_bwd_t(const CrossArgs &a, int sms, const DkvOut &out, cudaStream_t st)
{
    const int64_t key_threads = (int64_t)a.sets * a.M * (D / 8);
    const unsigned join_blocks = (unsigned)((key_threads + 255) / 256);
    if (a.N == 0) {  // no row: dk = dv = 0
        CrossArgs none = a;
        none.dkv_splits = 0;
        cross_dkv_join_kernel<T><<<join_blocks, 256, 0, st>>>(none, out, D);
        count_launches(1);
        return;
    }
    const int64_t row_threads = (int64_t)a.sets * a.rows_pad * (D / 8);
    cross_rows_kernel<T><<<(unsigned)((row_threads + 255) / 256), 256, 0, st>>>(a, D);
    const int dq_items = a.sets * a.dq_splits * (a.rows_pad / kT);
    cross_dq_kernel<T, D><<<dq_items < sms ? dq_items : sms, kBwdThreads, dq_smem(D), st>>>(a, dq_items);
    count_launches(2);
    if (a.dq_splits > 1) {
        const int64_t threads = (int64_t)a.B * a.H * a.N * (D / 8);
        cross_dq_join_kernel<T><<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(a, D);
        count_launches(1);
    }
    if (a.M == 0) return;
    const int key_tiles = (a.M + kT - 1) / kT;
    cross_dkv_kernel<T, D><<<(unsigned)(a.sets * a.dkv_splits * key_tiles), kBwdThreads, dkv_smem(D), st>>>(a, key_tiles);
    cross_dkv_join_kernel<T><<<join_blocks, 256, 0, st>>>(a, out, D);
    count_launches(2);
}

void launch_cross_bwd(const CrossArgs &a, int D, bool f16, int sms, const int32_t *inv, void *dk, const int64_t *dks,
                      void *dv, const int64_t *dvs, cudaStream_t st)
{
    DkvOut out{dk, dv, {dks[0], dks[1], dks[2]}, {dvs[0], dvs[1], dvs[2]}, inv};
    if (f16) {
        if (D == 128) launch_bwd_t<__half, 128>(a, sms, out, st);
        else launch_bwd_t<__half, 64>(a, sms, out, st);
    } else {
        if (D == 128) launch_bwd_t<__nv_bfloat16, 128>(a, sms, out, st);
        else launch_bwd_t<__nv_bfloat16, 64>(a, sms, out, st);
    }
}

}  // namespace op
}  // namespace scope
