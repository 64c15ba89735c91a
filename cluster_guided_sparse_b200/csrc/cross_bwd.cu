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
// 128 rows and walks the keys, cross_dkv_kernel owns 128 keys and walks the rows,
// four products a tile each.  S and dP are computed twice, and in exchange every
// accumulator stays in TMEM and no result is added up by atomics, so equal
// calls give equal bits.  (One kernel for both would send a fp32 dQ or dK/dV
// tile to memory per tile step.)
//
// The given o is rounded to 16 bits, and D' = do . o with it: its error is a
// share of |do| |o|, which all of a row's ds would carry (more than their own
// rounding, and many times more where the values have a common offset).  The dq
// kernel therefore sums t_ij = p_ij (dp_ij - D'_i), which sum to D_i - D'_i over
// a row (held in fp32), next to E_i = sum_j p_ij k_j, and takes
//   dq_i = scale (sum_j t_ij k_j - (D_i - D'_i) E_i),
// and the dk/dv kernel after it reads the corrected D_i.  Where a row reads a
// single key, p is 1 whatever its score, and dq, dk are set to 0 instead of to
// what the roundings of t leave.
//
// Both run the same pipeline over two TMEM buffers X0, X1 of 128 columns: S of
// step i goes to X[i%2], dP to the other; p and ds (16 bit, 64 columns each)
// overwrite S.  S of the next step is out as soon as dP has been read, under
// the ds of this one, and the exponentials of the next step run under the
// accumulations and dP.  Bound: 2048 clocks of products a step at D = 128, half of
// them (S, dP) with shared memory at its full rate too, which the next tiles'
// copies share.  Measured by clock: 2700 a step of the dk/dv kernel, 3400 of the
// dq kernel, whose items add about 3500 each for their ends (a wait that is ready
// takes some 60, so the issuers look at operands before they wait for the
// softmax).  40 heads of 32760 rows x 512 keys: dq 774 us, dk/dv 573 us, the join 19.
//
// Rows split over CTAs (few keys, many rows) or keys split (few rows, many
// keys) leave fp32 partial sums that a join adds in a fixed order.
//
// p and ds are rounded to the inputs' 16-bit type as operands of the products
// (the tensor cores take 16-bit operands); S, dP, D, lse and all sums are fp32.
// f16's smallest normal number is 2^-14, which the p of a flat row passes at 16000
// keys (at 60000 its rounding was 4 times that of a normal number, and from 2^25 on
// p vanished), so f16 holds p 2^14; the power is added to -lse and taken off dP and
// D' (whose sum and product with p then give ds as it is), dv and E.
// Barriers, rings, bounded waits as in cross_attn.cu.
#include "cross_common.cuh"

namespace scope {
namespace op {

using namespace tc;

static __device__ int32_t g_cross_bwd_err[4];

constexpr int kBwdThreads = 384;
constexpr int kT = 128;      // rows or keys of a tile
constexpr int kTiles = 7;    // tiles in shared memory, both kernels

// Tiles, 5 x 128 floats, barriers.  At D = 128 that leaves no room to align the
// base by hand (227 KB a block), so the kernels have no static shared memory and
// check that their base is aligned.
constexpr int kFloats = 5 * kT;
constexpr size_t bwd_smem(int D) { return (size_t)kTiles * kT * D * 2 + kFloats * 4 + 256; }

// Column of 16-element step k of p (ds: 32 further on) as an A operand: the 64
// values of each half of the warps sit, packed, in the half's own columns of S.
__device__ __forceinline__ uint32_t half_col(int k) { return (uint32_t)((k >> 2) * 64 + (k & 3) * 8); }

// Softmax weights are held as p 2^kUp: p is 1 at most, up to the error of lse, so a
// factor of 4 is left in f16.  kDown = 2^-kUp.
template <typename T> constexpr float kUp = 0.f;
template <> constexpr float kUp<__half> = 14.f;
template <typename T> constexpr float kDown = 1.f;
template <> constexpr float kDown<__half> = 1.f / 16384.f;

// dP - D' of two values, by 2^-kUp (nd is).
template <typename T>
__device__ __forceinline__ uint64_t dp_less_d(uint32_t dp0, uint32_t dp1, uint64_t nd)
{
    const uint64_t dp = f2pack(__uint_as_float(dp0), __uint_as_float(dp1));
    if constexpr (kUp<T> == 0.f) return fadd2(dp, nd);
    else return ffma2(dp, f2pack(kDown<T>, kDown<T>), nd);
}

// rows x cols = A B^T of two [128][D] tiles.
template <typename T, int D>
__device__ __forceinline__ void tile_product(uint32_t d, uint32_t a_smem, uint32_t b_smem)
{
    const uint32_t id = idesc16<T>(kT, false);
    const uint64_t da = sw128_desc(a_smem, 16, 1024), db = sw128_desc(b_smem, 16, 1024);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const uint64_t o = (uint64_t)(((k >> 2) * (kT * 128) + (k & 3) * 32) >> 4);
        mma_ss(d, da + o, db + o, id, k > 0);
    }
}

// d (+)= P B, P [128][128] packed at TMEM column p, B a [128][D] tile.
template <typename T, int D>
__device__ __forceinline__ void tile_accumulate(uint32_t d, uint32_t p, uint32_t b_smem, bool first)
{
    const uint32_t id = idesc16<T>(D, true);
    const uint64_t db = sw128_desc(b_smem, kT * 128, 1024);
#pragma unroll
    for (int k = 0; k < kT / 16; ++k)
        mma_ts(d, p + half_col(k), db + (uint64_t)((k * 2048) >> 4), id, !first || k > 0);
}

// 64 values as 32 packed columns.
template <typename T>
__device__ __forceinline__ void store_half(uint32_t col, const uint32_t *r)
{
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            pk[i] = pack2(T(), __uint_as_float(r[c * 32 + 2 * i]), __uint_as_float(r[c * 32 + 2 * i + 1]));
        tmem_st16(col + c * 16, pk);
    }
}

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

// ---------------------------------------------------------------- dq
struct DqItem {
    int bk, hk, t0, t1, nk, split;
    int64_t at;  // padded row of its first row
    RowTile r;
};

__device__ __forceinline__ DqItem dq_item(const CrossArgs &a, int item)
{
    DqItem w;
    int rt;
    item = min(item, a.sets * a.dq_splits * a.tiles - 1);  // behind the last one any
    const int set = a.by_splits(a.by_tiles(item, rt), w.split);
    w.bk = a.by_Hk(set, w.hk);
    w.r = row_tile<kT>(a, w.bk, w.hk, rt);
    w.at = ((int64_t)set * a.tiles + rt) * kT;
    w.nk = keys_of(a, w.bk);
    split_range((w.nk + kT - 1) / kT, w.split, a.by_splits, w.t0, w.t1);
    return w;
}

// -D' (do . o, of the rounded o) 2^-kUp of 16 rows of a tile by each of eight warps,
// and kUp - lse in base 2 of this thread's own row: -inf, so that p is 0, where the
// row reads nothing or does not exist.
template <typename T, int D>
__device__ __forceinline__ float row_values(const CrossArgs &a, RowTile w, int hk, float *s_nd)
{
    constexpr int LPR = D / 8, RPP = 32 / LPR, U = 16 / RPP;  // lanes a row, rows a pass, passes
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c8 = lane % LPR, row = (warp & 3) * 32 + lane;
    Raw8<T> o[U], y[U];
    int b, h, n;
    // each lane's row address, handed round: 64-bit products for each row would take longer than the loads
    const int mine = warp * 16 + (lane & 15);
    tile_row(a, w, hk, min(mine, w.nq - 1), b, h, n);
    const T *po = static_cast<const T *>(a.o) + b * a.oB + h * a.oH + n * a.oN;
    const T *py = static_cast<const T *>(a.dout) + b * a.dB + h * a.dH + n * a.dN;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int from = u * RPP + lane / LPR;
        const T *to = reinterpret_cast<const T *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(po), from));
        const T *ty = reinterpret_cast<const T *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(py), from));
        o[u].u = y[u].u = make_uint4(0u, 0u, 0u, 0u);
        if (warp * 16 + from < w.nq) {
            o[u].load(to + c8 * 8);
            y[u].load(ty + c8 * 8);
        }
    }
    float nl = -INFINITY;
    if (row < w.nq) {
        tile_row(a, w, hk, row, b, h, n);
        const float lse = a.lse[((int64_t)b * a.H + h) * a.N + n];
        if (lse != -INFINITY) nl = fmaf(-lse, 1.4426950408889634f, kUp<T>);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float x[8], z[8], sum = 0.f;
        o[u].values(x);
        y[u].values(z);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(x[e], z[e], sum);
#pragma unroll
        for (int e = LPR >> 1; e > 0; e >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, e);
        if (c8 == 0) s_nd[warp * 16 + u * RPP + lane / LPR] = -sum * kDown<T>;
    }
    return nl;
}

// A CTA's key tiles in order, over its items; by a whole warp.
struct DqStep {
    int item, j, t0, t1;
    __device__ __forceinline__ bool seek(const CrossArgs &a, int from, int items)
    {
#pragma unroll 1
        for (item = from; item < items; item += gridDim.x) {
            const DqItem w = dq_item(a, item);
            j = t0 = uniform(w.t0);
            t1 = uniform(w.t1);
            if (t0 < t1) return true;
        }
        return false;
    }
    __device__ __forceinline__ bool next(const CrossArgs &a, int items)
    {
        return ++j < t1 || seek(a, item + gridDim.x, items);
    }
};

// One persistent CTA per SM; item = 128 rows of a key set and a key range.  TMEM:
// X0 [0,128), X1 [128,256), sum t k [256,256+D), sum p k [384,384+D).  Shared
// memory: 2 Q tiles (the next item's comes early; dq leaves through it), 1 dO
// tile, rings of 3 K and 1 V tiles.  Warps 0-3 take the keys 0-63 of a tile,
// warps 4-7 the keys 64-127, one thread per row and half; warps 8, 9, 10 load
// Q and dO, K, V; warp 11 issues.  The softmax warps compute the next item's D'
// while this one waits for its sums, which saves a launch: with gradients 16 heads of
// 2048 rows x 77 keys took 84 us with it and 74 without; 40 heads of 32760 rows x 512
// keys, where it hid under the others, 1890 with and 1927 without.  One form serves
// both.  One loader warp for all rows of an item was three times too slow.
template <typename T, int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    cross_dq_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ CrossMaps m, int items)
{
    wait_for_previous();
    let_next_start();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    constexpr int TB = kT * D * 2;
    const uint32_t sQ = smem_u32(smem_raw), sO = sQ + 2 * TB, sK = sQ + 3 * TB, sV = sQ + 6 * TB;
    // [2 halves][kT] and, of items in turn, [2][kT].  Every warp announces the next item's D' after it has read this
    // one's sums, and waits for all before it uses them, so neither is written before it has been read.
    float *s_delta = reinterpret_cast<float *>(smem_raw + kTiles * TB), *s_nd = s_delta + 2 * kT;
    struct Barriers {
        uint64_t q_full[2], q_empty[2], o_full, o_empty, k_full[3], k_empty[3], v_full, v_empty;
        uint64_t s_full, dp_full, dp_read, ds_full, dq_full, delta_full[4], rows_full[2];
        uint32_t tmem_base;
        int abort;
    };
    static_assert(sizeof(Barriers) <= 256, "room kept in bwd_smem");
    Barriers &bar = *reinterpret_cast<Barriers *>(smem_raw + kTiles * TB + kFloats * 4);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (sQ & 1023u) {  // uniform
        if (threadIdx.x == 0) set_error(g_cross_bwd_err, kErrRange, 0x70);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 8);
            mbar_init(&bar.rows_full[i], 8);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bar.k_full[i], 1);
            mbar_init(&bar.k_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bar.delta_full[i], 2);
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_empty, 1);
        mbar_init(&bar.v_full, 1);
        mbar_init(&bar.v_empty, 1);
        mbar_init(&bar.s_full, 1);
        mbar_init(&bar.dp_full, 1);
        mbar_init(&bar.dp_read, 8);
        mbar_init(&bar.ds_full, 8);
        mbar_init(&bar.dq_full, 1);
        bar.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    bwd_prologue(warp, &bar.tmem_base);
    const uint32_t tmem = uniform(bar.tmem_base);
    const Waiter wait{&bar.abort, g_cross_bwd_err};

    if (warp == 8) {
        // ------------------------------------------------------------ Q, dO rows
        int qi = 0;
        bool ok = true;
#pragma unroll 1
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const DqItem w = dq_item(a, item);
            if (w.t0 == w.t1) continue;
            const int buf = qi & 1;
            if (qi >= 2 && !(ok = wait.warp(&bar.q_empty[buf], ((qi >> 1) - 1) & 1, 0x50))) break;
            fence_async_smem();  // dq has gone through the buffer
            load_rows<T, D>(a, w.r, w.hk, 1, &m.q, a.q, a.qB, a.qH, a.qN, sQ + buf * TB, &bar.q_full[buf]);
#pragma unroll 1
            for (int i = lane; i < w.r.nq; i += 32) {  // o and do will be read soon
                int b, h, n;
                tile_row(a, w.r, w.hk, i, b, h, n);
                const T *o = static_cast<const T *>(a.o) + b * a.oB + h * a.oH + n * a.oN;
                const T *y = static_cast<const T *>(a.dout) + b * a.dB + h * a.dH + n * a.dN;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(o));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(y));
                if (D == 128) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(o + 64));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(y + 64));
                }
            }
            ++qi;
            if (qi >= 2 && !(ok = wait.warp(&bar.o_empty, (qi - 2) & 1, 0x50))) break;
            load_rows<T, D>(a, w.r, w.hk, 1, &m.d, a.dout, a.dB, a.dH, a.dN, sO, &bar.o_full);
        }
        if (!ok) {  // the last dO has been waited for (it is free) or belongs to the item before
            for (int i = max(0, qi - 2); i < qi; ++i) drain(&bar.q_full[i & 1], (i >> 1) & 1);
            if (qi >= 2) drain(&bar.o_full, (qi - 2) & 1);
        }
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------------------ K rows, V rows
        auto decode = [&](int item) { return dq_item(a, item); };
        if (warp == 9)
            fill_keys<T, D, kT>(a, RingFill<3>(bar.k_full, bar.k_empty), &m.k, a.k, a.kB, a.kH, a.kN, sK, items, wait, 0x51,
                                decode, [](int) { return true; });
        else
            fill_keys<T, D, kT>(a, RingFill<1>(&bar.v_full, &bar.v_empty), &m.v, a.v, a.vB, a.vH, a.vN, sV, items, wait,
                                0x5c, decode,
                                // not while S(n) is computed, which takes shared memory's full rate
                                [&](int n) { return n == 0 || wait.warp(&bar.s_full, n & 1, 0x5d); });
    } else if (warp == 11) {
        // ------------------------------------------------------------ MMA issuer
        // (by the whole warp, one lane issuing, as in cross_attn.cu)
        RingRead<3> kr;
        DqStep cur, nxt;
        int ns = 0, qi = 0;  // steps, items begun
        // S of a step has its operands (looked at early: each ready wait takes as long as an instruction's product)
        auto s_ready = [&](const DqStep &st) {
            if (st.j == st.t0) {
                ++qi;
                if (!wait.warp(&bar.q_full[(qi - 1) & 1], ((qi - 1) >> 1) & 1, 0x52)) return false;
            }
            return wait.warp(&bar.k_full[kr.slot], kr.use & 1, 0x53);
        };
        auto issue_s = [&](int step, int &slot) {
            slot = kr.slot;
            kr.next();
            tc_fence_after();
            if (elect_one()) {
                tile_product<T, D>(tmem + (step & 1) * 128, sQ + ((qi - 1) & 1) * TB, sK + slot * TB);
                mma_commit(&bar.s_full);
            }
            __syncwarp();
        };
        auto issue_dp = [&](const DqStep &st, int step) {
            if (!wait.all(&bar.o_full, (qi - 1) & 1, 0x54, &bar.v_full, step & 1, 0x55)) return false;
            tc_fence_after();
            const bool last = st.j + 1 == st.t1;
            if (elect_one()) {
                tile_product<T, D>(tmem + ((step & 1) ^ 1) * 128, sO, sV);
                mma_commit(&bar.dp_full);
                mma_commit(&bar.v_empty);
                if (last) mma_commit(&bar.o_empty);
            }
            __syncwarp();
            return true;
        };
        int ks = 0, kn = 0;
        bool more = cur.seek(a, blockIdx.x, items), ok = more && s_ready(cur);
        if (ok) {
            issue_s(0, ks);
            ok = issue_dp(cur, 0);
        }
#pragma unroll 1
        while (ok && more) {
            nxt = cur;
            more = nxt.next(a, items);
            const bool first = cur.j == cur.t0, last = cur.j + 1 == cur.t1;
            // The next S is out before this step's ds is awaited; at an item's end, where the epilogue waits for the
            // sums, after them.  dP of this step has been read: its buffer is free for that S.
            if (more && !last) {
                if (!(ok = s_ready(nxt) && wait.warp(&bar.dp_read, ns & 1, 0x56))) break;
                issue_s(ns + 1, kn);
            }
            if (!(ok = wait.warp(&bar.ds_full, ns & 1, 0x57))) break;
            tc_fence_after();
            const uint32_t p = tmem + (ns & 1) * 128;
            if (elect_one()) {
                tile_accumulate<T, D>(tmem + 256, p + 32, sK + ks * TB, first);
                tile_accumulate<T, D>(tmem + 384, p, sK + ks * TB, first);
                mma_commit(&bar.k_empty[ks]);
                if (last) mma_commit(&bar.dq_full);
            }
            __syncwarp();
            if (more && last) {
                if (!(ok = s_ready(nxt) && wait.warp(&bar.dp_read, ns & 1, 0x56))) break;
                issue_s(ns + 1, kn);
            }
            if (more && !(ok = issue_dp(nxt, ns + 1))) break;
            cur = nxt;
            ks = kn;
            ++ns;
        }
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        const int half = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        int ns = 0, qi = 0;
        bool ok = true, leaving = false;  // leaving: the last item's dq may still be on its way out of the Q buffer
        auto q_free = [&]() {             // of the item before qi's
            if (lane == 0) {
                stored();
                mbar_arrive(&bar.q_empty[(qi & 1) ^ 1]);
            }
            leaving = false;
        };
        const uint64_t scp = f2pack(a.scale_log2, a.scale_log2);
        DqItem w{};
        float nl = 0.f;
        bool begun = false;  // w is an item, the one before `next`
#pragma unroll 1
        for (int next = blockIdx.x;; next += gridDim.x) {
            const bool keys = begun && w.t0 < w.t1;
            float nd = 0.f, delta = 0.f;
            if (keys) {
                if (!(ok = wait.warp(&bar.rows_full[qi & 1], (qi >> 1) & 1, 0x5e))) break;
                nd = s_nd[(qi & 1) * kT + row];
            }
            const uint64_t nlp = f2pack(nl, nl), ndp = f2pack(nd, nd);
            uint64_t dA = 0ull, dB = 0ull;
#pragma unroll 1
            for (int j = w.t0; keys && j < w.t1; ++j, ++ns) {
                const uint32_t tS = tmem + lane_off + (ns & 1) * 128 + half * 64;
                const uint32_t tP = tmem + lane_off + ((ns & 1) ^ 1) * 128 + half * 64;
                if (!(ok = wait.warp(&bar.s_full, ns & 1, 0x58))) break;
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
                store_half<T>(tS, r);
                if (!(ok = wait.warp(&bar.dp_full, ns & 1, 0x59))) break;
                tc_fence_after();
                uint32_t d[64];
                tmem_ld32(tP, d);
                tmem_ld32(tP + 32, d + 32);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.dp_read);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint64_t t2 = fmul2(f2pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                                              dp_less_d<T>(d[2 * i], d[2 * i + 1], ndp));
                    if (i & 1) dB = fadd2(dB, t2);
                    else dA = fadd2(dA, t2);
                    float x0, x1;
                    f2unpack(t2, x0, x1);
                    d[2 * i] = __float_as_uint(x0);
                    d[2 * i + 1] = __float_as_uint(x1);
                }
                store_half<T>(tS + 32, d);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.ds_full);
                if (leaving) q_free();
            }
            if (!ok) break;
            // D - D' of the row: both halves' sums
            float *pair = s_delta + row;
            if (keys) {
                float d0, d1, d2, d3;
                f2unpack(dA, d0, d1);
                f2unpack(dB, d2, d3);
                pair[half * kT] = (d0 + d2) + (d1 + d3);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.delta_full[wq]);
            }
            const bool store = begun && row < w.r.nq;
            int b, h, n;
            tile_row(a, w.r, w.hk, store ? row : 0, b, h, n);
            const int64_t part = w.split * (int64_t)a.B * a.H * a.N + ((int64_t)b * a.H + h) * a.N + n;
            T *dq = static_cast<T *>(a.dq) + b * a.dqB + h * a.dqH + n * a.dqN + half * (D / 2);
            float *pt = a.part_t + part * D + half * (D / 2), *pe = a.part_e + part * D + half * (D / 2);
            if (keys) {
                if (!(ok = wait.warp(&bar.delta_full[wq], qi & 1, 0x5a))) break;
                delta = pair[0] + pair[kT];
                // for the dk/dv kernel; of split keys the join takes the sum of the ranges' deltas off
                if (half == 0) {
                    if (a.dq_splits > 1 && store) a.part_delta[part] = delta;
                    if (w.split == 0 || a.dq_splits == 1) {
                        a.nlse[w.at + row] = nl;
                        a.ndelta[w.at + row] = a.dq_splits > 1 ? nd : fmaf(-delta, kDown<T>, nd);
                    }
                }
            } else if (store) {
                const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int i = 0; i < D / 2; i += 8) {
                    if (a.dq_splits > 1) {
                        store8(pt + i, zero);
                        store8(pe + i, zero);
                    } else {
                        store8(dq + i, zero);
                    }
                }
                if (a.dq_splits > 1 && half == 0) a.part_delta[part] = 0.f;
            }
            const float scale = w.nk == 1 ? 0.f : a.scale;
            const int bh = w.r.h, bb = w.r.b, bn = w.r.n + wq * 32;
            const bool rows = begun && wq * 32 < w.r.nq;  // uniform for the warp
            // the next item's values while this one's last products run
            const bool more = next < items;
            begun = true;
            if (more) {
                w = dq_item(a, next);
                if (w.t0 < w.t1) {
                    const int to = (qi + (keys ? 1 : 0)) & 1;
                    nl = row_values<T, D>(a, w.r, w.hk, s_nd + to * kT);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.rows_full[to]);
                }
            }
            if (!keys) {
                if (more) continue;
                break;
            }
            if (!(ok = wait.warp(&bar.dq_full, qi & 1, 0x5b))) break;
            tc_fence_after();
            if (a.dq_splits > 1) {
#pragma unroll 1
                for (int x = 0; x < 2 * (D / 64); ++x) {
                    const int e = x & 1, c = x >> 1;
                    uint32_t r[32];
                    tmem_ld32(tmem + lane_off + 256 + e * 128 + half * (D / 2) + c * 32, r);
                    tmem_wait_ld();
                    if (store) store_row<32>((e ? pe : pt) + c * 32, r);
                }
            } else {
                uint4 u[D / 16];
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t r[32], e[32];
                    tmem_ld32(tmem + lane_off + 256 + half * (D / 2) + c * 32, r);
                    tmem_ld32(tmem + lane_off + 384 + half * (D / 2) + c * 32, e);
                    tmem_wait_ld();
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        f[i] = fmaf(-delta * kDown<T>, __uint_as_float(e[i]), __uint_as_float(r[i])) * scale;
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[c * 4 + i] = pack8<T>(f + 8 * i);
                    // a half row is one box's 64 columns at D = 128
                    if ((D == 64 || !a.tma_o) && store) store_row<T, 32>(dq + c * 32, f, a.wide);
                }
                if constexpr (D == 128) {
                    if (a.tma_o && rows)
                        store_box(sQ + (qi & 1) * TB + half * (TB / 2) + wq * (32 * 128), u, &m.o, half * 64, bn, bh, bb);
                }
            }
            tc_fence_before();
            ++qi;
            leaving = true;
            if (!more) break;
        }
        if (leaving && lane == 0) stored();
        __syncwarp();
    }
    bwd_epilogue(warp, tmem);
}

// dq from the key ranges' parts, and the corrected ndelta.
template <typename T>
__global__ void __launch_bounds__(256) cross_dq_join_kernel(const __grid_constant__ CrossArgs a, int D)
{
    wait_for_previous();
    let_next_start();
    const int lpr = D / 8;
    const int64_t total = (int64_t)a.B * a.H * a.N;
    const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / lpr;
    const int c8 = threadIdx.x % lpr;
    if (row >= total) return;
    float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, e[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, delta = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.dq_splits; ++s) {
        float x[8], y[8];
        load8(a.part_t + (s * total + row) * D + c8 * 8, x);
        load8(a.part_e + (s * total + row) * D + c8 * 8, y);
        delta += a.part_delta[s * total + row];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i] += x[i];
            e[i] += y[i];
        }
    }
    const int64_t bh = row / a.N, n = row % a.N;
    const float scale = keys_of(a, a.Bk == a.B ? (int)(bh / a.H) : 0) == 1 ? 0.f : a.scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = fmaf(-delta * kDown<T>, e[i], t[i]) * scale;
    store8(static_cast<T *>(a.dq) + (bh / a.H) * a.dqB + (bh % a.H) * a.dqH + n * a.dqN + c8 * 8, t);
    if (c8 == 0) a.ndelta[padded_row(a, (int)(bh / a.H), (int)(bh % a.H), (int)n)] -= delta * kDown<T>;
}

// ---------------------------------------------------------------- dk, dv
// One CTA per (key set, 128 keys, row range); keys are the rows of its products:
// S^T = K Q^T and dP^T = V dO^T in X0, X1, dV [256,256+D), dK [384,384+D).
// Shared memory: K, V, rings of 3 Q and 2 dO tiles with the rows' nlse, ndelta.
// Warps 0-3 take the rows 0-63 of a row tile, warps 4-7 the rows 64-127, one
// thread per key and half; warps 8, 9, 10 load K and V, Q, dO; warp 11 issues.
template <typename T, int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
    cross_dkv_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ CrossMaps m, int key_tiles)
{
    wait_for_previous();
    let_next_start();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    constexpr int TB = kT * D * 2;
    const uint32_t sK = smem_u32(smem_raw), sV = sK + TB, sQ = sK + 2 * TB, sO = sK + 5 * TB;
    float *s_nl = reinterpret_cast<float *>(smem_raw + kTiles * TB);  // [3][kT]
    float *s_nd = s_nl + 3 * kT;                                      // [2][kT]
    struct Barriers {
        uint64_t kv_full, q_full[3], q_empty[3], o_full[2], o_empty[2], s_full, dp_full, dp_read, ds_full, acc_full;
        uint32_t tmem_base;
        int abort;
    };
    static_assert(sizeof(Barriers) <= 256, "room kept in bwd_smem");
    Barriers &bar = *reinterpret_cast<Barriers *>(smem_raw + kTiles * TB + kFloats * 4);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

    const int kt = blockIdx.x % key_tiles, rest = blockIdx.x / key_tiles;
    const int split = rest % a.dkv_splits, set = rest / a.dkv_splits;
    const int bk = set / a.Hk, hk = set % a.Hk;
    const int nk = keys_of(a, bk);
    int i0, i1;
    split_range(a.tiles, split, a.by_dkv_splits, i0, i1);
    // uniform for the CTA: no keys here, or a base that is not aligned
    if (kt * kT >= nk) return;
    if (sK & 1023u) {
        if (threadIdx.x == 0) set_error(g_cross_bwd_err, kErrRange, 0x71);
        return;
    }
    if (threadIdx.x == 0) {
        mbar_init(&bar.kv_full, 1);
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.o_full[i], 1);
            mbar_init(&bar.o_empty[i], 1);
        }
        mbar_init(&bar.s_full, 1);
        mbar_init(&bar.dp_full, 1);
        mbar_init(&bar.dp_read, 8);
        mbar_init(&bar.ds_full, 8);
        mbar_init(&bar.acc_full, 1);
        bar.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // keys of a list, or a last tile that ends inside its set, are copied by all threads
    const bool whole = tma_keys<kT>(a, nk, kt);
    if (!whole) {
        const int32_t *list = a.idx ? a.idx + (int64_t)bk * a.M : nullptr;
        copy_keys<T, D, kT, kBwdThreads>(list, nk, kt, static_cast<const T *>(a.k) + bk * a.kB + hk * a.kH, a.kN, sK);
        copy_keys<T, D, kT, kBwdThreads>(list, nk, kt, static_cast<const T *>(a.v) + bk * a.vB + hk * a.vH, a.vN, sV);
        cp_async_commit();
        cp_async_wait_all();
        fence_async_smem();
    }
    bwd_prologue(warp, &bar.tmem_base);
    const uint32_t tmem = uniform(bar.tmem_base);
    const Waiter wait{&bar.abort, g_cross_bwd_err};

    if (warp == 8) {
        // ------------------------------------------------------------ K, V
        if (lane == 0) {
            if (whole) {
                mbar_expect_tx(&bar.kv_full, 2 * TB);
                tma_tile<D>(sK, &m.k, kt * kT, hk, bk, &bar.kv_full);
                tma_tile<D>(sV, &m.v, kt * kT, hk, bk, &bar.kv_full);
            } else {
                mbar_arrive(&bar.kv_full);
            }
        }
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------------------ Q rows, dO rows
        const bool q = warp == 9;
        const int ns = q ? 3 : 2;
        uint64_t *full = q ? bar.q_full : bar.o_full, *empty = q ? bar.q_empty : bar.o_empty;
        float *s_vec = q ? s_nl : s_nd;
        const float *vec = (q ? a.nlse : a.ndelta) + (int64_t)set * a.tiles * kT;
        const CUtensorMap *map = q ? &m.q : &m.d;
        const void *src = q ? a.q : a.dout;
        const int64_t sB = q ? a.qB : a.dB, sH = q ? a.qH : a.dH, sN = q ? a.qN : a.dN;
        const uint32_t smem = q ? sQ : sO;
        bool ok = true;
        int u = 0;
#pragma unroll 1
        for (int i = i0; i < i1; ++i, ++u) {
            const int slot = u % ns, use = u / ns;
            if (use > 0 && !(ok = wait.warp(&empty[slot], (use - 1) & 1, 0x60))) break;
            // the rows' 128 values first: they are announced together with the tile
            reinterpret_cast<float4 *>(s_vec + slot * kT)[lane] = reinterpret_cast<const float4 *>(vec + (int64_t)i * kT)[lane];
            __syncwarp();
            load_rows<T, D>(a, row_tile<kT>(a, bk, hk, i), hk, 1, map, src, sB, sH, sN, smem + slot * TB, &full[slot]);
        }
        if (!ok)
            for (int i = max(0, u - ns); i < u; ++i) drain(&full[i % ns], (i / ns) & 1);
    } else if (warp == 11) {
        // ------------------------------------------------------------ MMA issuer
        RingRead<3> qr;
        RingRead<2> dr;
        const int n = uniform(i1 - i0);
        auto s_ready = [&]() { return wait.warp(&bar.q_full[qr.slot], qr.use & 1, 0x61); };
        auto issue_s = [&](int u, int &slot) {
            slot = qr.slot;
            qr.next();
            tc_fence_after();
            if (elect_one()) {
                tile_product<T, D>(tmem + (u & 1) * 128, sK, sQ + slot * TB);
                mma_commit(&bar.s_full);
            }
            __syncwarp();
        };
        auto issue_dp = [&](int u, int &slot) {
            slot = dr.slot;
            if (!wait.warp(&bar.o_full[slot], dr.use & 1, 0x62)) return false;
            dr.next();
            tc_fence_after();
            if (elect_one()) {
                tile_product<T, D>(tmem + ((u & 1) ^ 1) * 128, sV, sO + slot * TB);
                mma_commit(&bar.dp_full);
            }
            __syncwarp();
            return true;
        };
        int qs = 0, qn = 0, os = 0;
        bool ok = wait.warp(&bar.kv_full, 0, 0x63) && s_ready();
        if (ok) {
            issue_s(0, qs);
            ok = issue_dp(0, os);
        }
#pragma unroll 1
        for (int u = 0; ok && u < n; ++u) {
            const bool more = u + 1 < n;
            if (more) {
                if (!(ok = s_ready() && wait.warp(&bar.dp_read, u & 1, 0x64))) break;
                issue_s(u + 1, qn);
            }
            if (!(ok = wait.warp(&bar.ds_full, u & 1, 0x65))) break;
            tc_fence_after();
            const uint32_t p = tmem + (u & 1) * 128;
            if (elect_one()) {
                tile_accumulate<T, D>(tmem + 256, p, sO + os * TB, u == 0);
                mma_commit(&bar.o_empty[os]);
                tile_accumulate<T, D>(tmem + 384, p + 32, sQ + qs * TB, u == 0);
                mma_commit(&bar.q_empty[qs]);
                if (!more) mma_commit(&bar.acc_full);
            }
            __syncwarp();
            if (more && !(ok = issue_dp(u + 1, os))) break;
            qs = qn;
        }
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        const int half = warp >> 2, wq = warp & 3, key = wq * 32 + lane;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint64_t scp = f2pack(a.scale_log2, a.scale_log2);
        bool ok = true;
        RingRead<3> qr;  // nlse, ndelta come with the Q, dO tiles
        RingRead<2> dr;
#pragma unroll 1
        for (int u = 0; u < i1 - i0; ++u) {
            const ulonglong2 *nl = reinterpret_cast<const ulonglong2 *>(s_nl + qr.slot * kT + half * 64);
            const ulonglong2 *nd = reinterpret_cast<const ulonglong2 *>(s_nd + dr.slot * kT + half * 64);
            const uint32_t tS = tmem + lane_off + (u & 1) * 128 + half * 64;
            const uint32_t tP = tmem + lane_off + ((u & 1) ^ 1) * 128 + half * 64;
            if (!(ok = wait.all(&bar.q_full[qr.slot], qr.use & 1, 0x66, &bar.s_full, u & 1, 0x67))) break;
            qr.next();
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
            store_half<T>(tS, r);
            if (!(ok = wait.all(&bar.o_full[dr.slot], dr.use & 1, 0x68, &bar.dp_full, u & 1, 0x69))) break;
            dr.next();
            tc_fence_after();
            uint32_t d[64];
            tmem_ld32(tP, d);
            tmem_ld32(tP + 32, d + 32);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.dp_read);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const ulonglong2 n2 = nd[c];
                float x0, x1;
                f2unpack(fmul2(f2pack(__uint_as_float(r[4 * c]), __uint_as_float(r[4 * c + 1])),
                               dp_less_d<T>(d[4 * c], d[4 * c + 1], n2.x)),
                         x0, x1);
                d[4 * c] = __float_as_uint(x0);
                d[4 * c + 1] = __float_as_uint(x1);
                f2unpack(fmul2(f2pack(__uint_as_float(r[4 * c + 2]), __uint_as_float(r[4 * c + 3])),
                               dp_less_d<T>(d[4 * c + 2], d[4 * c + 3], n2.y)),
                         x0, x1);
                d[4 * c + 2] = __float_as_uint(x0);
                d[4 * c + 3] = __float_as_uint(x1);
            }
            store_half<T>(tS + 32, d);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.ds_full);
        }
        if (ok && wait.warp(&bar.acc_full, 0, 0x6a)) {
            tc_fence_after();
            const int key_at = kt * kT + key;
            const float scale = nk == 1 ? 0.f : a.scale;
            const int64_t at = ((int64_t)split * a.sets + set) * a.M + key_at;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int col = half * (D / 2) + c * 32;
                uint32_t o[32];
                float f[32];
                tmem_ld32(tmem + lane_off + 256 + col, o);
                tmem_wait_ld();
                if (key_at < nk) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * kDown<T>;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) store8(a.part_dv + at * D + col + i, f + i);
                }
                tmem_ld32(tmem + lane_off + 384 + col, o);
                tmem_wait_ld();
                if (key_at < nk) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * scale;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) store8(a.part_dk + at * D + col + i, f + i);
                }
            }
        }
    }
    bwd_epilogue(warp, tmem);
}

// dk, dv of every key: the row ranges' parts added in order; keys that no row
// may read get zeros.  inv: a key's place in its list or -1, or null.
template <typename T>
__global__ void __launch_bounds__(256) cross_dkv_join_kernel(const __grid_constant__ CrossArgs a,
                                                             const int32_t *inv, int D)
{
    wait_for_previous();
    const int lpr = D / 8;
    const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / lpr;  // set * M + m
    const int c8 = threadIdx.x % lpr;
    if (row >= (int64_t)a.sets * a.M) return;
    const int set = (int)(row / a.M), m = (int)(row % a.M), bk = set / a.Hk, hk = set % a.Hk;
    const int place = inv ? inv[(int64_t)bk * a.M + m] : (m < keys_of(a, bk) ? m : -1);
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
    store8(static_cast<T *>(a.dk) + bk * a.dkB + hk * a.dkH + m * a.dkN + c8 * 8, sk);
    store8(static_cast<T *>(a.dv) + bk * a.dvB + hk * a.dvH + m * a.dvN + c8 * 8, sv);
}

template <typename T, int D>
static cudaError_t bwd_attr()
{
    const cudaError_t e = cudaFuncSetAttribute(cross_dq_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)bwd_smem(D));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(cross_dkv_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bwd_smem(D));
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

int32_t *cross_bwd_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_cross_bwd_err) == cudaSuccess ? static_cast<int32_t *>(p) : nullptr;
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

int cross_dq_splits(int64_t sets, int64_t tiles, int64_t M, int64_t rows_total, int D, int sms)
{
    const int64_t items = sets * tiles, len = (M + kT - 1) / kT;
    if (items >= sms) return 1;  // persistent: items even out by themselves
    return best_split(items, len, sms, 2.0, (double)rows_total * D * 16.0 / 6e6, 3.0);
}

int cross_dkv_splits(int64_t sets, int64_t tiles, int64_t M, int D, int sms)
{
    const int64_t items = sets * ((M + kT - 1) / kT), len = tiles;
    return best_split(items, len, sms, 4.0, (double)(sets * M) * D * 16.0 / 6e6, 0.0);
}

template <typename T, int D>
static void launch_bwd_t(const CrossArgs &a, const CrossMaps &m, int sms, const int32_t *inv, cudaStream_t st)
{
    const int64_t join_blocks = ((int64_t)a.sets * a.M * (D / 8) + 255) / 256;
    if (a.N == 0) {  // no row: dk = dv = 0
        CrossArgs none = a;
        none.dkv_splits = 0;
        cross_dkv_join_kernel<T><<<(unsigned)join_blocks, 256, 0, st>>>(none, inv, D);
        count_launches(1);
        return;
    }
    const int dq_items = a.sets * a.dq_splits * a.tiles, dq_grid = dq_items < sms ? dq_items : sms;
    if (a.idx) {  // after the key lists
        launch_next(cross_dq_kernel<T, D>, dq_grid, kBwdThreads, bwd_smem(D), st, a, m, dq_items);
    } else {
        cross_dq_kernel<T, D><<<dq_grid, kBwdThreads, bwd_smem(D), st>>>(a, m, dq_items);
        count_launches(1);
    }
    if (a.dq_splits > 1) {
        const int64_t threads = (int64_t)a.B * a.H * a.N * (D / 8);
        launch_next(cross_dq_join_kernel<T>, (threads + 255) / 256, 256, 0, st, a, D);
    }
    if (a.M == 0) return;
    const int key_tiles = (a.M + kT - 1) / kT;
    launch_next(cross_dkv_kernel<T, D>, (int64_t)a.sets * a.dkv_splits * key_tiles, kBwdThreads, bwd_smem(D), st, a, m, key_tiles);
    launch_next(cross_dkv_join_kernel<T>, join_blocks, 256, 0, st, a, inv, D);
}

void launch_cross_bwd(const CrossArgs &a, const CrossMaps &m, int D, bool f16, int sms, const int32_t *inv,
                      cudaStream_t st)
{
    if (f16) {
        if (D == 128) launch_bwd_t<__half, 128>(a, m, sms, inv, st);
        else launch_bwd_t<__half, 64>(a, m, sms, inv, st);
    } else {
        if (D == 128) launch_bwd_t<__nv_bfloat16, 128>(a, m, sms, inv, st);
        else launch_bwd_t<__nv_bfloat16, 64>(a, m, sms, inv, st);
    }
}

}  // namespace op
}  // namespace scope
