// Shared by the cross-attention kernels (cross_attn.cu, cross_bwd.cu).
//
// A "key set" is one (key batch entry, key head): the rows that read it are the
// N queries of its G query heads, of one batch entry or (keys of batch 1) of all.
// They are cut into tiles in one of two ways:
//   by head  tiles start at each head's first query; their rows are loaded by
//            TMA, which fills rows past the head's end with zeros
//   folded   tiles run on over the borders of heads and batch entries, so short
//            query lengths of many heads still fill tiles; rows are copied by
//            cp.async (as by head, where a stride is too large for TMA)
// K and V tiles come by TMA where every row of the tile is a key in order (or
// past the end of the tensor); with a key list, or a length that ends inside
// the tile, by cp.async, which writes zeros for the rows past the end and never
// reads them.
#pragma once

#include "op_common.cuh"
#include "tcgen05.cuh"

namespace scope {
namespace op {

struct CrossMaps {
    // [B][H][N][D] boxes of 128 (forward k, v: kFwdKeys; o, in the backward pass dq: 32) rows x 64 columns, 128B
    // swizzle
    CUtensorMap q, k, v, d, o;
};

constexpr int kFwdKeys = 64;  // keys of a tile of the forward kernel

// n / d for 0 <= n < 2^31 without a division, by a multiplication's high half, an addition
// and a shift (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994): a decoded work item costs some
// hundred clocks with these and 1500 with the divide instructions' sequences.
struct Div {
    uint32_t mul;
    int shift, d;
    Div() = default;
    explicit Div(int by) : mul(0), shift(0), d(by < 1 ? 1 : by)
    {
        while (((int64_t)1 << shift) < d) ++shift;
        mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ int operator()(int n) const
    {
        return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
    }
    __device__ __forceinline__ int operator()(int n, int &rest) const
    {
        const int q = (*this)(n);
        rest = n - q * d;
        return q;
    }
};

struct CrossArgs {
    const void *q, *k, *v;
    void *o;
    float *lse;                // [B][H][N] or null
    int64_t qB, qH, qN, kB, kH, kN, vB, vH, vN, oB, oH, oN;  // element strides
    const int32_t *kv_len;     // [Bk] or null: all M keys
    const int32_t *idx, *cnt;  // kept keys of a mask: [Bk][M] ascending, [Bk]; or null
    const uint8_t *mask;       // the mask itself, [Bk][M] with mask_stride between rows (few rows), or null
    int64_t mask_stride;
    int few_ranks;             // CTAs of a key set where it has few rows (cross_few.cu), or 0
    int B, Bk, H, Hk, G, N, M;
    int heads;                 // heads whose rows read one key set: G, or B * G
    int fold;                  // how rows are cut into tiles
    int wide;                  // rows of o (backward: dq) start on 32 bytes
    int tma_kv, tma_rows, tma_o;  // whether the k, v maps are valid, and the q, d and o ones (by head only)
    int sets;                  // Bk * Hk
    int pairs, splits;         // 256-row tiles per set, key ranges (forward)
    // per: row tiles of a head; tiles, splits: of the forward's, of the dq kernel's items
    Div by_N, by_G, by_Hk, by_per, by_tiles, by_splits, by_dkv_splits;
    int items;                 // sets * splits * pairs
    float scale, scale_log2;   // scale, scale * log2(e)
    float *part_o;             // [splits][B*H*N][D], normalised per split (splits > 1)
    float *part_lse;           // [splits][B*H*N], base 2
    // backward
    const void *dout;
    int64_t dB, dH, dN;
    int tiles;                 // 128-row tiles per set
    // per set, tile and row: -lse in base 2 (-inf where the row reads nothing or
    // does not exist: its p is then 0) and -D (f16: with p's power of two, and less it)
    float *nlse, *ndelta;
    void *dq;
    int64_t dqB, dqH, dqN;
    int dq_splits;             // key ranges of the dq kernel
    float *part_t, *part_e;    // [dq_splits][B*H*N][D] (dq_splits > 1)
    float *part_delta;         // [dq_splits][B*H*N]
    int dkv_splits;            // row ranges of the dk/dv kernel
    float *part_dk, *part_dv;  // [dkv_splits][sets][M][D], kept keys in list order
    void *dk, *dv;
    int64_t dkB, dkH, dkN, dvB, dvH, dvN;
};

// Row tile: its first row (batch entry, head, query) and its row count.
struct RowTile {
    int b, h, n, nq;
};

template <int T>
__device__ __forceinline__ RowTile row_tile(const CrossArgs &a, int bk, int hk, int rt)
{
    RowTile w;
    int hh;
    if (a.fold) {
        const int r0 = rt * T;
        hh = a.by_N(r0, w.n);
        w.nq = min(T, a.heads * a.N - r0);
    } else {
        hh = a.by_per(rt, w.n);
        w.n *= T;
        w.nq = min(T, a.N - w.n);
    }
    w.b = bk;
    if (a.Bk != a.B) w.b = a.by_G(hh, hh);
    w.h = hk * a.G + hh;
    return w;
}

// Row i of a tile of key head hk.
__device__ __forceinline__ void tile_row(const CrossArgs &a, const RowTile &w, int hk, int i, int &b, int &h, int &n)
{
    b = w.b;
    h = w.h;
    n = w.n + i;
    if (n >= a.N) {  // folded: a later head
        h += a.by_N(n, n);
        const int over = a.by_G(h - hk * a.G);
        b += over;
        h -= over * a.G;
    }
}

// Where (batch entry b, head h, query n) sits among its set's padded rows.
__device__ __forceinline__ int64_t padded_row(const CrossArgs &a, int b, int h, int n)
{
    const int hk = a.by_G(h), shared = a.Bk != a.B;
    const int hh = (shared ? b * a.G : 0) + h - hk * a.G, set = (shared ? 0 : b) * a.Hk + hk;
    const int64_t at = a.fold ? (int64_t)hh * a.N + n : (int64_t)hh * ((a.N + 127) / 128 * 128) + n;
    return (int64_t)set * a.tiles * 128 + at;
}

// Keys the set may read: the mask's count, or the length kept inside [0, M].
__device__ __forceinline__ int keys_of(const CrossArgs &a, int bk)
{
    if (a.idx) return a.cnt[bk];
    return a.kv_len ? min(max(a.kv_len[bk], 0), a.M) : a.M;
}

// A value that is the same in all lanes, as one that the compiler knows to be.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Tiles [t0, t1) of range `split` of `by.d` even ranges of n tiles.
__device__ __forceinline__ void split_range(int n, int split, const Div &by, int &t0, int &t1)
{
    int rest;
    const int base = by(n, rest);
    t0 = base * split + min(split, rest);
    t1 = t0 + base + (split < rest ? 1 : 0);
}

// Byte offset of 16-byte chunk `c` of row `r` in a [rows][D] tile of 16-bit
// elements stored as D/64 column blocks of rows x 128 B, 128B-swizzled.
__device__ __forceinline__ uint32_t tile_off(int r, int c, int rows)
{
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// kind::f16 instruction descriptor for 16-bit type T (A and B alike), fp32
// accumulators, M = 128.
template <typename T>
__device__ __forceinline__ uint32_t idesc16(int n, bool b_mn_major);
template <>
__device__ __forceinline__ uint32_t idesc16<__nv_bfloat16>(int n, bool b_mn_major)
{
    return tc::idesc_bf16(n, b_mn_major);
}
template <>
__device__ __forceinline__ uint32_t idesc16<__half>(int n, bool b_mn_major)
{
    return tc::idesc_bf16(n, b_mn_major) & ~((7u << 7) | (7u << 10));
}

// Bounded mbarrier wait of these kernels: by one lane, or by a whole warp, all
// of whose lanes get the same answer (so a warp never splits around its
// warp-wide instructions when a wait gives up).  A look at a barrier takes some
// 60 clocks, so a warp that needs several looks at all of them first (`all`).
// The loop is a call: inlined at each wait it made the kernels' code several
// times as long, and the roles, which run in turn, ran out of the instruction
// caches (a ready wait of the issuer took 160 clocks instead of 45).
static __device__ __noinline__ bool wait_longer(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int32_t *err, int where)
{
    return tc::mbar_wait(bar, parity, abort_flag, err, where);
}

struct Waiter {
    volatile int *abort_flag;
    int32_t *err;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity, int where) const
    {
        return tc::mbar_try_wait(bar, parity) || wait_longer(bar, parity, abort_flag, err, where);
    }
    __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity, int where) const
    {
        return __all_sync(0xffffffffu, (*this)(bar, parity, where));
    }
    __device__ __forceinline__ bool all(uint64_t *b0, uint32_t p0, int w0, uint64_t *b1, uint32_t p1, int w1) const
    {
        const bool r0 = tc::mbar_try_wait(b0, p0), r1 = tc::mbar_try_wait(b1, p1);
        if (__all_sync(0xffffffffu, r0 && r1)) return true;
        return warp(b0, p0, w0) && warp(b1, p1, w1);
    }
};

// TMA load of rows [n, n + ROWS) of head (b, h) into a swizzled tile.
template <int D, int ROWS = 128>
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap *m, int n, int h, int b, uint64_t *bar)
{
#pragma unroll
    for (int x = 0; x < D / 64; ++x)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst + x * (ROWS * 128)),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(x * 64), "r"(n), "r"(h), "r"(b), "r"(tc::smem_u32(bar))
            : "memory");
}

// After a wait gave up: lets a copy that was issued earlier land (its barrier
// completes by itself), so that nothing writes shared memory after the block
// has gone.  Bounded as well.
__device__ __forceinline__ void drain(uint64_t *full, uint32_t parity)
{
    for (int i = 0; i < 20000 && !tc::mbar_try_wait(full, parity); ++i) {
    }
}

// Ring of shared-memory stages filled by one warp.  A stage filled by cp.async is
// announced once its copies landed, which is checked after the next stage's copies were issued, so two are in
// flight; a stage filled by TMA announces itself.
template <int NS>
struct RingFill {
    uint64_t *full, *empty;
    int slot, use, pending;
    __device__ __forceinline__ RingFill(uint64_t *f, uint64_t *e) : full(f), empty(e), slot(0), use(0), pending(-1) {}
    __device__ __forceinline__ void announce()
    {
        tc::fence_async_smem();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&full[pending]);
        pending = -1;
    }
    __device__ __forceinline__ void advance()
    {
        if (++slot == NS) {
            slot = 0;
            ++use;
        }
    }
    // Waits until the stage `slot` is free; false: a wait gave up.
    __device__ __forceinline__ bool acquire(const Waiter &wait, int where)
    {
        if (use == 0 || __all_sync(0xffffffffu, tc::mbar_try_wait(&empty[slot], (use - 1) & 1))) return true;
        flush();  // the consumers may be waiting for what is in flight
        return wait.warp(&empty[slot], (use - 1) & 1, where);
    }
    __device__ __forceinline__ void issued()
    {
        tc::cp_async_commit();
        if (pending >= 0) {
            tc::cp_async_wait1();
            announce();
        }
        pending = slot;
        advance();
    }
    // Fills the stage by TMA.
    template <int D, int ROWS>
    __device__ __forceinline__ void tma(uint32_t dst, const CUtensorMap *m, int n, int h, int b)
    {
        if (pending >= 0) flush();
        if ((threadIdx.x & 31) == 0) {
            tc::mbar_expect_tx(&full[slot], ROWS * D * 2);
            tma_tile<D, ROWS>(dst, m, n, h, b, &full[slot]);
        }
        __syncwarp();
        advance();
    }
    __device__ __forceinline__ void flush()
    {
        tc::cp_async_wait_all();
        if (pending >= 0) announce();
    }
    // The end of a producer: everything that it issued has landed.
    __device__ __forceinline__ void finish(bool aborted)
    {
        flush();
        if (!aborted) return;
        const int total = use * NS + slot;
        for (int i = max(0, total - NS); i < total; ++i) drain(&full[i % NS], (i / NS) & 1);
    }
};

// The consumer's place in such a ring.
template <int NS>
struct RingRead {
    int slot = 0, use = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == NS) {
            slot = 0;
            ++use;
        }
    }
};

// Copies the first `fill` rows of a row tile (element strides sB, sH, sN) into
// swizzled tiles of 128 rows, rows from w.nq on as zeros, by one warp.
template <typename T, int D>
__device__ __noinline__ void copy_rows(const CrossArgs &a, const RowTile &w, int hk, int fill, const T *src, int64_t sB,
                                          int64_t sH, int64_t sN, uint32_t dst)
{
    constexpr int CH = D / 8, RPI = 32 / CH;
    const int lane = threadIdx.x & 31, ch = lane % CH;
    src += ch * 8;
#pragma unroll 4
    for (int i = lane / CH; i < fill; i += RPI) {
        const bool ok = i < w.nq;
        int b, h, n;
        tile_row(a, w, hk, ok ? i : 0, b, h, n);
        tc::cp_async16(dst + (i / 128) * (128 * D * 2) + tile_off(i % 128, ch, 128), src + b * sB + h * sH + n * sN, ok);
    }
}

// One warp fills `tiles` 128-row tiles with a row tile's rows and announces
// them on `full` (one arrival).
template <typename T, int D>
__device__ __forceinline__ void load_rows(const CrossArgs &a, const RowTile &w, int hk, int tiles, const CUtensorMap *map,
                                          const void *src, int64_t sB, int64_t sH, int64_t sN, uint32_t dst, uint64_t *full)
{
    constexpr int TB = 128 * D * 2;
    if (!a.tma_rows) {
        copy_rows<T, D>(a, w, hk, tiles * 128, static_cast<const T *>(src), sB, sH, sN, dst);
        tc::cp_async_commit();
        tc::cp_async_wait_all();
        tc::fence_async_smem();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(full);
    } else if ((threadIdx.x & 31) == 0) {
        tc::mbar_expect_tx(full, tiles * TB);
        for (int t = 0; t < tiles; ++t) tma_tile<D>(dst + t * TB, map, w.n + t * 128, w.h, w.b, full);
    }
    __syncwarp();
}

// Whether the keys of tile j (of ROWS keys) can come by TMA.
template <int ROWS>
__device__ __forceinline__ bool tma_keys(const CrossArgs &a, int nk, int j)
{
    return a.tma_kv && !a.idx && (nk == a.M || nk - j * ROWS >= ROWS);
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack2(T(), x[0], x[1]), pack2(T(), x[2], x[3]), pack2(T(), x[4], x[5]), pack2(T(), x[6], x[7]));
}

// One warp's 32 rows x 64 columns of 16-bit values, this lane's row as 8 chunks,
// into its part of a swizzled tile and from there to rows [n, n + 32) of head
// (b, h) by TMA, which drops rows past the head's end.  The tile may be written
// again after stored().  (Rows of 256 bytes straight from registers, 32 bytes a
// thread and store, keep the load/store unit at one line a clock: 3000 clocks for
// an item's 64 KB.)
__device__ __forceinline__ void store_box(uint32_t smem, const uint4 *u, const CUtensorMap *m, int x, int n, int h, int b)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(smem + lane * 128 + ((c ^ (lane & 7)) << 4)),
                     "r"(u[c].x), "r"(u[c].y), "r"(u[c].z), "r"(u[c].w)
                     : "memory");
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0)
        asm volatile(
            "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n\t"
            "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(m)),
            "r"(smem), "r"(x), "r"(n), "r"(h), "r"(b)
            : "memory");
}

// This thread's store_box copies have left shared memory.
__device__ __forceinline__ void stored() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// 16 values to 32 bytes of 16-bit elements, 8 to 32 bytes of fp32: whole sectors
// of a row from one thread.
__device__ __forceinline__ void store32(void *p, const uint32_t *u)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                 "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}

// N values as 16-bit elements of a row; wide: every row starts on 32 bytes (else on 16).
template <typename T, int N>
__device__ __forceinline__ void store_row(T *p, const float *x, bool wide)
{
#pragma unroll
    for (int i = 0; i < N; i += 16) {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = pack2(T(), x[i + 2 * e], x[i + 2 * e + 1]);
        if (wide) {
            store32(p + i, u);
        } else {
            reinterpret_cast<uint4 *>(p + i)[0] = make_uint4(u[0], u[1], u[2], u[3]);
            reinterpret_cast<uint4 *>(p + i)[1] = make_uint4(u[4], u[5], u[6], u[7]);
        }
    }
}

template <int N>
__device__ __forceinline__ void store_row(float *p, const uint32_t *x)
{
#pragma unroll
    for (int i = 0; i < N; i += 8) store32(p + i, x + i);
}

// THREADS threads (one warp, or a block) copy the keys of tile j (rows of a key list, if any) into a tile,
// rows past the set's nk keys as zeros: their memory is never read.
template <typename T, int D, int ROWS, int THREADS = 32>
__device__ __noinline__ void copy_keys(const int32_t *list, int nk, int j, const T *base, int64_t sn, uint32_t dst)
{
    constexpr int CH = D / 8, RPI = THREADS / CH;
    const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x, ch = tid % CH;
#pragma unroll 8
    for (int i = tid / CH; i < ROWS; i += RPI) {
        const int kj = j * ROWS + i;
        const bool ok = kj < nk;
        const int key = ok ? (list ? list[kj] : kj) : 0;
        tc::cp_async16(dst + tile_off(i, ch, ROWS), base + key * sn + ch * 8, ok);
    }
}

// One warp fills a ring with the key tiles (of k or of v) of its CTA's items;
// `before(n)` waits for what the n-th copy is to come after.
template <typename T, int D, int ROWS, int NS, typename Decode, typename Before>
__device__ __forceinline__ void fill_keys(const CrossArgs &a, RingFill<NS> ring, const CUtensorMap *map, const void *src,
                                          int64_t sB, int64_t sH, int64_t sN, uint32_t smem, int items, const Waiter &wait,
                                          int where, const Decode &decode, const Before &before)
{
    bool ok = true;
    int n = 0;
#pragma unroll 1
    for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
        const auto w = decode(item);
        const T *base = static_cast<const T *>(src) + w.bk * sB + w.hk * sH;
        const int32_t *list = a.idx ? a.idx + (int64_t)w.bk * a.M : nullptr;
#pragma unroll 1
        for (int j = w.t0; j < w.t1; ++j) {
            if (!(ok = ring.acquire(wait, where) && before(n++))) break;
            const uint32_t dst = smem + ring.slot * (ROWS * D * 2);
            if (tma_keys<ROWS>(a, w.nk, j)) {
                ring.template tma<D, ROWS>(dst, map, j * ROWS, w.hk, w.bk);
            } else {
                copy_keys<T, D, ROWS>(list, w.nk, j, base, sN, dst);
                ring.issued();
            }
        }
    }
    ring.finish(!ok);
}

int cross_few_ranks(int64_t sets, int64_t rows, int64_t M, bool backward, int sms);
void launch_cross_few(const CrossArgs &a, int D, bool f16, bool backward, cudaStream_t st);
cudaError_t cross_few_configure();
cudaError_t cross_fwd_configure();
cudaError_t cross_bwd_configure();
int cross_fwd_splits(int64_t sets, int64_t pairs, int64_t M, int64_t rows_total, int D, int sms);
int cross_dq_splits(int64_t sets, int64_t tiles, int64_t M, int64_t rows_total, int D, int sms);
int cross_dkv_splits(int64_t sets, int64_t tiles, int64_t M, int D, int sms);
void launch_key_lists(const uint8_t *mask, int64_t stride, int Bk, int M, int32_t *idx, int32_t *cnt, int32_t *inv,
                      cudaStream_t st);
void launch_cross_fwd(const CrossArgs &a, const CrossMaps &m, int D, bool f16, int sms, cudaStream_t st);
void launch_cross_bwd(const CrossArgs &a, const CrossMaps &m, int D, bool f16, int sms, const int32_t *inv,
                      cudaStream_t st);
cudaError_t cross_fwd_error(int32_t *err, bool clear);
cudaError_t cross_bwd_error(int32_t *err, bool clear);
int32_t *cross_fwd_error_word();  // its device address, or null
int32_t *cross_bwd_error_word();

}  // namespace op
}  // namespace scope
