// Cross attention, forward: each of N queries attends over M keys of another
// sequence (an encoder's states), M and N any lengths.
//
//   s_ij = scale q_i . k_j over the allowed keys j,  lse_i = log sum_j e^s_ij,
//   o_i = sum_j e^(s_ij - lse_i) v_j;  a row without keys gets o = 0, lse = -inf.
//
// Bound: 4 D flops a (row, key) pair on the tensor cores against one
// exponential a pair (16 a clock and SM), both 1024 clocks a 128 x 128 tile at
// D = 128; but S with operands in shared memory reads that at its full rate, so
// with the copies into it shared memory is the first limit (1280 clocks).  Below
// some 300 keys the rows' own bytes (q in, o out) take longer and HBM is the bound.
//
// One persistent CTA per SM walks work items = (key set, key range, 256
// rows).  The two 128-row tiles of an item share every K/V tile, which halves
// the L2 traffic.  The keys go in tiles of 64 with two S buffers a row tile, so
// the products of the tile after next are out while the softmax works on this
// one: neither waits for the other's latency (one buffer of 128 keys took 4200
// clocks a row tile and 128 keys, of which the products are 1024; but then one warp
// issued for both row tiles and was a limit too, see below).  The steps run on
// over item borders: the next item's first S tiles are there before this one's
// epilogue.  Q rows have two buffers for the same reason.
//
// Warp roles (416 threads):
//   warps 0-3, 4-7  softmax and epilogue of row tile 0, 1 (one thread per row); O
//                   leaves by TMA through the item's Q buffer
//   warps 8, 9, 10  Q, K, V rows by TMA, or cp.async where a tile's rows are not
//                   in order (cross_common.cuh)
//   warps 11, 12    tcgen05.mma issuers of row tile 0, 1; warp 11 owns the TMEM
//                   allocation.  (One issuer for both was the limit: its waits,
//                   commits and issues came to 3200 clocks for 1280 of products.)
// TMEM, of each row tile's 256 columns: S0 [0,64) S1 [64,128) O [128,128+D);
// P (16 bit) overwrites its S.  The softmax runs in base 2 with a lazy
// rescale: O and l move to a new maximum only when it grew by more than 2^8,
// so P stays below 2^8.  P is rounded to the inputs' type for the product
// (the tensor cores take 16-bit operands); its sum l is taken before that
// rounding, in fp32, as are S, O and lse.  f16 holds P 2^7 (up to 2^15), of which l and O
// are made alike, so that weights down to 2^-21 of the largest are normal numbers: of a
// long tail of small ones, as a whole no small share of o, each is else off by more than
// a rounding (3% at 2^-20).
//
// Few rows (a single token, a short prompt reading a long video) leave most
// SMs without an item: the keys are then split into ranges whose normalised
// outputs and lse meet in cross_join_kernel, in a fixed order.
//
// Measured: 40 heads of 32760 rows x 512 keys 410 us (838 TFLOP/s; 17300 clocks an
// item of 8 steps, 1700 a step, at the 1.5 to 1.7 GHz that the power cap leaves),
// 24 heads of 118800 x 256 538 us, 24 heads of 77 x 118800 332 us (4.4 TB/s); on a card
// that held its clock 353, 497 and 271.
//
// Every mbarrier wait is bounded (about two seconds); on timeout the thread
// records it in the operators' error word, the CTA drops its items and all
// threads still meet at the end so the TMEM is released.
#include "cross_common.cuh"

namespace scope {
namespace op {

using namespace tc;

static __device__ int32_t g_cross_err[4];

constexpr int kFwdThreads = 416;
constexpr int kTile = 128;  // rows of a Q tile

constexpr int fwd_stages(int D) { return D == 128 ? 3 : 6; }  // of K and of V
constexpr size_t fwd_smem(int D) { return (size_t)(4 * kTile + 2 * fwd_stages(D) * kFwdKeys) * D * 2 + 1024; }

// P and its sums are held by 2^kFwdUp.
template <typename T> constexpr float kFwdUp = 0.f;
template <> constexpr float kFwdUp<__half> = 7.f;

struct FwdItem {
    int bk, hk, t0, t1, nk, split;
    RowTile r;
};

__device__ __forceinline__ FwdItem fwd_item(const CrossArgs &a, int item)
{
    FwdItem w;
    int rt, set;
    item = min(item, a.items - 1);  // behind the last one any
    set = a.by_splits(a.by_tiles(item, rt), w.split);
    w.bk = a.by_Hk(set, w.hk);
    w.r = row_tile<2 * kTile>(a, w.bk, w.hk, rt);
    w.nk = keys_of(a, w.bk);
    split_range((w.nk + kFwdKeys - 1) / kFwdKeys, w.split, a.by_splits, w.t0, w.t1);
    return w;
}

// A CTA's key tiles in order, over its items; by a whole warp.
struct FwdSteps {
    int item, j, t1, nt;  // nt: row tiles of the item
    int seq = -1;         // items begun before this one
    bool first;           // of its item
    __device__ __forceinline__ bool seek(const CrossArgs &a, int from)
    {
#pragma unroll 1
        for (item = from; item < a.items; item += gridDim.x) {
            const FwdItem w = fwd_item(a, item);
            j = uniform(w.t0);
            t1 = uniform(w.t1);
            if (j == t1) continue;
            nt = uniform(w.r.nq) > kTile ? 2 : 1;
            first = true;
            ++seq;
            return true;
        }
        return false;
    }
    __device__ __forceinline__ bool next(const CrossArgs &a)
    {
        first = false;
        return ++j < t1 || seek(a, item + gridDim.x);
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kFwdThreads, 1) cross_fwd_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ CrossMaps m)
{
    wait_for_previous();
    let_next_start();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    constexpr int TB = kTile * D * 2, KB = kFwdKeys * D * 2;  // bytes of a row tile, of a key tile
    constexpr int NS = fwd_stages(D);
    const uint32_t sQ = smem_u32(sm);  // 2 buffers of 2 tiles
    const uint32_t sK = sQ + 4 * TB, sV = sK + NS * KB;

    __shared__ uint64_t q_full[2], q_empty[2], k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
    // Of each row tile.  Steps alternate between two barriers each: with one, S being two steps ahead, a waiter
    // could find the phase after next, which looks like the phase before.
    __shared__ uint64_t s_full[2][2], p_full[2][2], o_full[2][2], o_empty[2];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 8);  // the softmax warps, or for those without rows their issuer
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s_full[i][b], 1);
                mbar_init(&p_full[i][b], 4);
                mbar_init(&o_full[i][b], 1);
            }
            mbar_init(&o_empty[i], 4);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 2);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 2);
        }
        abort_sh = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 11) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base_sh)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(tmem_base_sh);
    const Waiter wait{&abort_sh, g_cross_err};

    if (warp == 8) {
        // ------------------------------------------------------------ Q rows
        int qi = 0;
        bool ok = true;
#pragma unroll 1
        for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
            const FwdItem w = fwd_item(a, item);
            if (w.t0 == w.t1) continue;
            const int buf = qi & 1;
            if (qi >= 2 && !(ok = wait.warp(&q_empty[buf], ((qi >> 1) - 1) & 1, 0x40))) break;
            fence_async_smem();  // O has gone through the buffer
            load_rows<T, D>(a, w.r, w.hk, w.r.nq > kTile ? 2 : 1, &m.q, a.q, a.qB, a.qH, a.qN, sQ + buf * 2 * TB,
                            &q_full[buf]);
            ++qi;
        }
        if (!ok)
            for (int i = max(0, qi - 2); i < qi; ++i) drain(&q_full[i & 1], (i >> 1) & 1);
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------------------ K rows, V rows
        auto decode = [&](int item) { return fwd_item(a, item); };
        auto any_time = [](int) { return true; };
        if (warp == 9)
            fill_keys<T, D, kFwdKeys>(a, RingFill<NS>(k_full, k_empty), &m.k, a.k, a.kB, a.kH, a.kN, sK, a.items, wait,
                                      0x41, decode, any_time);
        else
            fill_keys<T, D, kFwdKeys>(a, RingFill<NS>(v_full, v_empty), &m.v, a.v, a.vB, a.vH, a.vN, sV, a.items, wait,
                                      0x42, decode, any_time);
    } else if (warp >= 11) {
        // ------------------------------------------------------------ MMA issuer of row tile t
        // The whole warp runs the steps, so their values are uniform, and one lane issues (where a single lane ran
        // them, each operand of an instruction cost a search for the lanes that share it: 1.3 times the call's time)
        const int t = warp - 11;
        const uint32_t id_qk = idesc16<T>(kFwdKeys, false), id_pv = idesc16<T>(D, true);
        const uint64_t dq = sw128_desc(sQ + t * TB, 16, 1024), dk = sw128_desc(sK, 16, 1024);
        const uint64_t dv = sw128_desc(sV, kFwdKeys * 128, 1024);
        const uint32_t tS = tmem + t * 256, tO = tS + 128;
        FwdSteps front;  // the step whose S is next, two ahead of the one whose PV is
        constexpr uint32_t kStep = 1, kFirst = 2, kLast = 4, kHas = 8;  // of an item; kHas: has this row tile
        uint32_t back = 0, mid = 0;                                     // the steps behind the front one; 0: none
        RingRead<NS> kr, vr;
        int ns = 0, np = 0, no = 0;  // of this row tile: S, PV issued, items done
        bool ok, more = front.seek(a, blockIdx.x);
#pragma unroll 1
        while (more | (back | mid) != 0) {
            if (back) {  // O (+)= P V
                uint64_t *v = &v_full[vr.slot];
                if (back & kHas) {
                    const int b = np & 1;
                    if (!(ok = wait.all(&p_full[t][b], (np >> 1) & 1, 0x45, v, vr.use & 1, 0x47))) break;
                    // the previous item's epilogue has read O
                    if ((back & kFirst) && no > 0 && !(ok = wait.warp(&o_empty[t], (no - 1) & 1, 0x46))) break;
                    tc_fence_after();
                    const uint64_t bv = dv + (uint64_t)((vr.slot * KB) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kFwdKeys / 16; ++k)
                            mma_ts(tO, tS + b * 64 + k * 8, bv + (uint64_t)((k * 2048) >> 4), id_pv, !(back & kFirst) || k > 0);
                        mma_commit(&o_full[t][b]);
                        mma_commit(&v_empty[vr.slot]);
                    }
                    __syncwarp();
                    ++np;
                    if (back & kLast) ++no;
                } else {
                    if (!(ok = wait.warp(v, vr.use & 1, 0x4f))) break;
                    if (lane == 0) mbar_arrive(&v_empty[vr.slot]);
                }
                vr.next();
            }
            back = mid;
            mid = 0;
            if (more) {  // S = Q K^T
                const int buf = front.seq & 1;
                // Q once an item (K again else), and by both issuers: nothing frees the item's buffer before this one has
                // looked at it, so its barrier is never two phases ahead, nor one behind of an item that was passed over
                uint64_t *k = &k_full[kr.slot], *q = front.first ? &q_full[buf] : k;
                if (!(ok = wait.all(k, kr.use & 1, 0x44, q, (front.first ? front.seq >> 1 : kr.use) & 1, 0x43))) break;
                mid = kStep | (front.first ? kFirst : 0) | (front.j + 1 == front.t1 ? kLast : 0);
                if (t < front.nt) {
                    mid |= kHas;
                    tc_fence_after();
                    const uint64_t aq = dq + (uint64_t)((buf * 2 * TB) >> 4), bk = dk + (uint64_t)((kr.slot * KB) >> 4);
                    const int b = ns & 1;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_ss(tS + b * 64, aq + (uint64_t)(((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4),
                                   bk + (uint64_t)(((k >> 2) * (kFwdKeys * 128) + (k & 3) * 32) >> 4), id_qk, k > 0);
                        mma_commit(&s_full[t][b]);
                        mma_commit(&k_empty[kr.slot]);
                    }
                    __syncwarp();
                    ++ns;
                } else if (lane == 0) {
                    if (front.first) mbar_arrive(&q_empty[buf], 4);  // for the row tile's softmax warps, which have no rows
                    mbar_arrive(&k_empty[kr.slot]);
                }
                kr.next();
                more = front.next(a);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        const int t = warp >> 2, wq = warp & 3;
        const uint32_t tT = tmem + ((uint32_t)(wq * 32) << 16) + t * 256, tO = tT + 128;
        const uint64_t scp = f2pack(a.scale_log2, a.scale_log2);
        int ns = 0, qi = 0;
        bool ok = true, leaving = false;  // leaving: the last item's O may still be on its way out of the Q buffer
        auto q_free = [&]() {             // of the item before qi's
            if (lane == 0) {
                stored();
                mbar_arrive(&q_empty[(qi & 1) ^ 1]);
            }
            leaving = false;
        };
        FwdItem w = fwd_item(a, blockIdx.x);
#pragma unroll 1
        for (int item = blockIdx.x; ok && item < a.items; item += gridDim.x) {
            const bool some = w.t0 < w.t1;  // uniform for the CTA
            const int buf = qi & 1;
            if (w.r.nq <= t * kTile) {  // no rows here: the row tile's issuer frees the item's Q
                if (some) {
                    if (leaving) q_free();
                    ++qi;
                }
                w = fwd_item(a, item + gridDim.x);
                continue;
            }
            float m_run = -INFINITY;
            uint64_t lA = 0ull, lB = 0ull;
#pragma unroll 1
            for (int j = w.t0; j < w.t1; ++j, ++ns) {
                const uint32_t tS = tT + (ns & 1) * 64;
                if (!(ok = wait.warp(&s_full[t][ns & 1], (ns >> 1) & 1, 0x48 + t))) break;
                tc_fence_after();
                uint32_t r[kFwdKeys];
                tmem_ld32(tS, r);
                tmem_ld32(tS + 32, r + 32);
                tmem_wait_ld();
                const int valid = w.nk - j * kFwdKeys;
                if (valid < kFwdKeys) {
#pragma unroll
                    for (int i = 0; i < kFwdKeys; ++i)
                        if (i >= valid) r[i] = __float_as_uint(-INFINITY);
                }
                float m4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m4[i] = __uint_as_float(r[i]);
#pragma unroll
                for (int i = 4; i < kFwdKeys; i += 2)
                    m4[(i >> 1) & 3] = fmax3(m4[(i >> 1) & 3], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                const float mt = fmax3(fmax3(m4[0], m4[1], m4[2]), m4[3], m4[3]) * a.scale_log2;
                if (j == w.t0) {
                    m_run = mt;
                } else if (__any_sync(0xffffffffu, mt > m_run + 8.f)) {
                    const float mn = fmaxf(m_run, mt);
                    // every logit so far -inf: l = 0 and O = 0, nothing to scale
                    const float alpha = m_run == -INFINITY ? 0.f : ex2(m_run - mn);
                    m_run = mn;
                    const uint64_t al = f2pack(alpha, alpha);
                    lA = fmul2(lA, al);
                    lB = fmul2(lB, al);
                    // O holds the sum up to the step before once its PV is done (this step's waits for this warp)
                    if (!(ok = wait.warp(&o_full[t][(ns - 1) & 1], ((ns - 1) >> 1) & 1, 0x4e))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16(tO + c * 16, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st16(tO + c * 16, o);
                    }
                }
                float shift = m_run == -INFINITY ? 0.f : -m_run;
                if constexpr (kFwdUp<T> != 0.f) shift += kFwdUp<T>;
                const uint64_t nmp = f2pack(shift, shift);
#pragma unroll
                for (int c = 0; c < kFwdKeys / 32; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int e = c * 32 + 2 * i;
                        float x0, x1;
                        f2unpack(ffma2(f2pack(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), scp, nmp), x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        if (i & 1) lB = fadd2(lB, f2pack(x0, x1));
                        else lA = fadd2(lA, f2pack(x0, x1));
                        pk[i] = pack2(T(), x0, x1);
                    }
                    tmem_st16(tS + c * 16, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t][ns & 1]);
                if (leaving) q_free();
            }
            if (!ok) break;
            float la, lb, lc, ld;
            f2unpack(lA, la, lb);
            f2unpack(lB, lc, ld);
            const float l = (la + lc) + (lb + ld);
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a NaN sum stays one
            const int row = t * kTile + wq * 32 + lane;
            const bool store = row < w.r.nq;
            int b, h, n;  // of this thread's row; behind the last one, of the tile's first
            tile_row(a, w.r, w.hk, store ? row : 0, b, h, n);
            const int64_t flat = ((int64_t)b * a.H + h) * a.N + n, part = w.split * (int64_t)a.B * a.H * a.N + flat;
            T *o = static_cast<T *>(a.o) + b * a.oB + h * a.oH + n * a.oN;
            float *po = a.part_o + part * D;
            if (store) {
                const float lse2 = l == 0.f ? -INFINITY : m_run + (log2f(l) - kFwdUp<T>);
                if (a.splits > 1) a.part_lse[part] = lse2;
                else if (a.lse) a.lse[flat] = lse2 * 0.6931471805599453f;
            }
            const bool boxes = a.tma_o && a.splits == 1;
            const int first = t * kTile + wq * 32, bh = w.r.h, bb = w.r.b, bn = w.r.n + first;
            const bool rows = first < w.r.nq;            // uniform for the warp
            w = fwd_item(a, item + gridDim.x);           // while the last products run
            if (some) {
                if (!(ok = wait.warp(&o_full[t][(ns - 1) & 1], ((ns - 1) >> 1) & 1, 0x4a + t))) break;
                tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
                uint32_t r[64];
#pragma unroll
                for (int i = 0; i < 64; ++i) r[i] = 0u;
                if (some) {
                    tmem_ld32(tO + c * 64, r);
                    tmem_ld32(tO + c * 64 + 32, r + 32);
                    tmem_wait_ld();
                    if (c == D / 64 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&o_empty[t]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 64; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * inv);
                const float *f = reinterpret_cast<const float *>(r);
                if (boxes && some) {
                    uint4 u[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = pack8<T>(f + 8 * i);
                    if (rows) store_box(sQ + (buf * 2 + t) * TB + c * (kTile * 128) + wq * (32 * 128), u, &m.o, c * 64, bn, bh, bb);
                } else if (store) {
                    if (a.splits > 1) store_row<64>(po + c * 64, r);
                    else store_row<T, 64>(o + c * 64, f, a.wide);
                }
            }
            if (some) {
                ++qi;
                leaving = true;
            }
        }
        if (leaving && lane == 0) stored();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 11) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// Joins the key ranges of each row: o = sum_s w_s o_s / sum_s w_s with
// w_s = 2^(lse_s - max), D/8 lanes a row.
template <typename T>
__global__ void __launch_bounds__(256) cross_join_kernel(const __grid_constant__ CrossArgs a, int D)
{
    wait_for_previous();
    const int lpr = D / 8;
    const int64_t total = (int64_t)a.B * a.H * a.N;
    const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / lpr;
    const int c8 = threadIdx.x % lpr;
    if (row >= total) return;
    float m = -INFINITY;
    for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_lse[s * total + row]);
    const float ref = m == -INFINITY ? 0.f : m;
    float sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float w = exp2f(a.part_lse[s * total + row] - ref);
        float o[8];
        load8(a.part_o + (s * total + row) * D + c8 * 8, o);
        sum += w;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, o[i], acc[i]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= inv;
    const int64_t bh = row / a.N, n = row % a.N;
    store8(static_cast<T *>(a.o) + (bh / a.H) * a.oB + (bh % a.H) * a.oH + n * a.oN + c8 * 8, acc);
    if (a.lse && c8 == 0) a.lse[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}

// Kept keys of a byte mask, one block per batch entry: ascending list, count
// and (for the backward pass) each key's place in the list or -1.  16 keys a
// thread and step, block-wide scan of the counts.
__global__ void __launch_bounds__(1024) key_lists_kernel(const uint8_t *mask, int64_t stride, int M, int32_t *idx,
                                                         int32_t *cnt, int32_t *inv)
{
    let_next_start();
    __shared__ int tmp[33];
    const uint8_t *mk = mask + blockIdx.x * stride;
    int32_t *list = idx + (int64_t)blockIdx.x * M;
    int32_t *place = inv ? inv + (int64_t)blockIdx.x * M : nullptr;
    int carry = 0;
    for (int64_t m0 = 0; m0 < M; m0 += 16 * 1024) {
        const int64_t first = m0 + threadIdx.x * 16;
        uint32_t bits = 0;
        for (int i = 0; i < 16; ++i)
            if (first + i < M && mk[first + i]) bits |= 1u << i;
        int total;
        int at = carry + block_excl_scan(__popc(bits), tmp, total);
        for (int i = 0; i < 16 && first + i < M; ++i) {
            const bool kept = (bits >> i) & 1u;
            if (place) place[first + i] = kept ? at : -1;
            if (kept) list[at++] = (int32_t)(first + i);
        }
        carry += total;
    }
    if (threadIdx.x == 0) cnt[blockIdx.x] = carry;
}

void launch_key_lists(const uint8_t *mask, int64_t stride, int Bk, int M, int32_t *idx, int32_t *cnt, int32_t *inv,
                      cudaStream_t st)
{
    key_lists_kernel<<<Bk, 1024, 0, st>>>(mask, stride, M, idx, cnt, inv);
    count_launches(1);
}

template <typename T, int D>
static cudaError_t fwd_attr()
{
    return cudaFuncSetAttribute(cross_fwd_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fwd_smem(D));
}

cudaError_t cross_fwd_configure()
{
    const cudaError_t e[4] = {fwd_attr<__nv_bfloat16, 128>(), fwd_attr<__nv_bfloat16, 64>(), fwd_attr<__half, 128>(),
                              fwd_attr<__half, 64>()};
    for (cudaError_t x : e)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}

cudaError_t cross_fwd_error(int32_t *err, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(err, g_cross_err, sizeof g_cross_err);
    const int32_t zero[4] = {0, 0, 0, 0};
    if (e == cudaSuccess && clear && err[0]) e = cudaMemcpyToSymbol(g_cross_err, zero, sizeof zero);
    return e;
}

int32_t *cross_fwd_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_cross_err) == cudaSuccess ? static_cast<int32_t *>(p) : nullptr;
}

// Key ranges per row tile: the count with the least modelled time, in steps of
// one 64-key tile (some 0.7 us a CTA).  An item costs its tiles and about four
// more for its Q rows and epilogue; a split adds a launch (about 5 steps) and
// the partial outputs' traffic.
int cross_fwd_splits(int64_t sets, int64_t pairs, int64_t M, int64_t rows_total, int D, int sms)
{
    const int64_t tiles = (M + kFwdKeys - 1) / kFwdKeys, items = sets * pairs;
    int best = 1;
    double least = 0.0;
    for (int64_t s = 1; s <= tiles && s <= 128 && (s == 1 || items * (s - 1) < sms); ++s) {
        const double waves = (double)((items * s + sms - 1) / sms);
        double t = waves * (double)((tiles + s - 1) / s + 4);
        if (s > 1) t += 5.0 + (double)(s * rows_total) * D * 8.0 / 4e6;
        if (s == 1 || t < least) {
            least = t;
            best = (int)s;
        }
    }
    return best;
}

// The first kernel of a call is launched as any other: it follows whatever the stream holds.
template <typename T, int D>
static void launch_fwd_t(const CrossArgs &a, const CrossMaps &m, int grid, cudaStream_t st)
{
    if (a.idx) {
        launch_next(cross_fwd_kernel<T, D>, grid, kFwdThreads, fwd_smem(D), st, a, m);
    } else {
        cross_fwd_kernel<T, D><<<grid, kFwdThreads, fwd_smem(D), st>>>(a, m);
        count_launches(1);
    }
    if (a.splits > 1) {
        const int64_t threads = (int64_t)a.B * a.H * a.N * (D / 8);
        launch_next(cross_join_kernel<T>, (threads + 255) / 256, 256, 0, st, a, D);
    }
}

void launch_cross_fwd(const CrossArgs &a, const CrossMaps &m, int D, bool f16, int sms, cudaStream_t st)
{
    const int grid = a.items < sms ? a.items : sms;
    if (f16) {
        if (D == 128) launch_fwd_t<__half, 128>(a, m, grid, st);
        else launch_fwd_t<__half, 64>(a, m, grid, st);
    } else {
        if (D == 128) launch_fwd_t<__nv_bfloat16, 128>(a, m, grid, st);
        else launch_fwd_t<__nv_bfloat16, 64>(a, m, grid, st);
    }
}

}  // namespace op
}  // namespace scope
