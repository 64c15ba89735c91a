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
    CUtensorMap q, k, v, d;  // [B][H][N][D] boxes of 128 rows x 64 columns, 128B swizzle
};

struct CrossArgs {
    const void *q, *k, *v;
    void *o;
    float *lse;                // [B][H][N] or null
    int64_t qB, qH, qN, kB, kH, kN, vB, vH, vN, oB, oH, oN;  // element strides
    const int32_t *kv_len;     // [Bk] or null: all M keys
    const int32_t *idx, *cnt;  // kept keys of a mask: [Bk][M] ascending, [Bk]; or null
    int B, Bk, H, Hk, G, N, M;
    int heads;                 // heads whose rows read one key set: G, or B * G
    int fold;                  // how rows are cut into tiles
    int tma_kv, tma_rows;      // whether the k, v maps are valid, and the q, d ones (by head only)
    int sets;                  // Bk * Hk
    int pairs, splits;         // 256-row tiles per set, key ranges (forward)
    int items;                 // sets * splits * pairs
    float scale, scale_log2;   // scale, scale * log2(e)
    float *part_o;             // [splits][B*H*N][D], normalised per split (splits > 1)
    float *part_lse;           // [splits][B*H*N], base 2
    // backward
    const void *dout;
    int64_t dB, dH, dN;
    int tiles;                 // 128-row tiles per set
    // per set, tile and row: -lse in base 2 (-inf where the row reads nothing or
    // does not exist: its p is then 0) and -D
    float *nlse, *ndelta;
    void *dq;
    int64_t dqB, dqH, dqN;
    int dq_splits;             // key ranges of the dq kernel
    float *part_t, *part_e;    // [dq_splits][B*H*N][D] (dq_splits > 1)
    float *part_delta;         // [dq_splits][B*H*N]
    int dkv_splits;            // row ranges of the dk/dv kernel
    float *part_dk, *part_dv;  // [dkv_splits][sets][M][D], kept keys in list order (dkv_splits > 1 or a list)
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
        hh = r0 / a.N;
        w.n = r0 - hh * a.N;
        w.nq = min(T, a.heads * a.N - r0);
    } else {
        const int per = (a.N + T - 1) / T;
        hh = rt / per;
        w.n = (rt - hh * per) * T;
        w.nq = min(T, a.N - w.n);
    }
    w.b = bk;
    if (a.Bk != a.B) {
        w.b = hh / a.G;
        hh -= w.b * a.G;
    }
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
        const int step = n / a.N;
        n -= step * a.N;
        h += step;
        const int over = (h - hk * a.G) / a.G;
        b += over;
        h -= over * a.G;
    }
}

// Where (batch entry b, head h, query n) sits among its set's padded rows.
__device__ __forceinline__ int64_t padded_row(const CrossArgs &a, int b, int h, int n)
{
    const int hk = h / a.G, shared = a.Bk != a.B;
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
// warp-wide instructions when a wait gives up).
struct Waiter {
    volatile int *abort_flag;
    int32_t *err;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity, int where) const
    {
        return tc::mbar_wait(bar, parity, abort_flag, err, where);
    }
    __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity, int where) const
    {
        return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, err, where));
    }
};

// TMA load of rows [n, n + 128) of head (b, h) into a swizzled tile.
template <int D>
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap *m, int n, int h, int b, uint64_t *bar)
{
#pragma unroll
    for (int x = 0; x < D / 64; ++x)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst + x * (128 * 128)),
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

// Ring of shared-memory stages filled by one or more whole warps.  A stage
// filled by cp.async is announced (one arrival per warp) once its copies landed,
// which is checked after the next stage's copies were issued, so two are in
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
    // Fills the stage by TMA; of several warps one is the lead.
    template <int D>
    __device__ __forceinline__ void tma(bool lead, uint32_t dst, const CUtensorMap *m, int n, int h, int b)
    {
        if (pending >= 0) flush();
        if ((threadIdx.x & 31) == 0) {
            if (lead) {
                tc::mbar_expect_tx(&full[slot], 128 * D * 2);
                tma_tile<D>(dst, m, n, h, b, &full[slot]);
            } else {
                tc::mbar_arrive(&full[slot]);
            }
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
__device__ __forceinline__ void copy_rows(const CrossArgs &a, const RowTile &w, int hk, int fill, const T *src, int64_t sB,
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

// Whether the 128 keys of tile j can come by TMA.
__device__ __forceinline__ bool tma_keys(const CrossArgs &a, int nk, int j)
{
    return a.tma_kv && !a.idx && (nk == a.M || nk - j * 128 >= 128);
}

// One warp's rows through shared memory to global memory: each lane holds CH
// 16-byte chunks of its own row; they leave as whole row segments.  `dst(i)`
// is the address of row i's segment; rows from n_rows on are dropped.
template <int CH, typename Dst>
__device__ __forceinline__ void store_staged(uint32_t stage, const uint4 *v, int n_rows, Dst dst)
{
    const int lane = threadIdx.x & 31;
    auto at = [&](int row, int c) {
        return stage + row * (CH * 16) + ((CH == 8 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4);
    };
    __syncwarp();
#pragma unroll
    for (int c = 0; c < CH; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(lane, c)), "r"(v[c].x), "r"(v[c].y), "r"(v[c].z),
                     "r"(v[c].w)
                     : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int row = i * (32 / CH) + lane / CH, c = lane % CH;
        uint4 u;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "r"(at(row, c))
                     : "memory");
        if (row < n_rows) reinterpret_cast<uint4 *>(dst(row))[c] = u;
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack2(T(), x[0], x[1]), pack2(T(), x[2], x[3]), pack2(T(), x[4], x[5]), pack2(T(), x[6], x[7]));
}

__device__ __forceinline__ uint4 bits4(const float *x)
{
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// Copies the 128 keys of tile j (rows of a key list, if any) into a tile, rows
// past the set's nk keys as zeros: their memory is never read.
template <typename T, int D, int THREADS>
__device__ __forceinline__ void copy_keys(const int32_t *list, int nk, int j, const T *base, int64_t sn, uint32_t dst,
                                          int tid)
{
    constexpr int CH = D / 8, RPI = THREADS / CH;
    const int ch = tid % CH;
#pragma unroll 8
    for (int i = tid / CH; i < 128; i += RPI) {
        const int kj = j * 128 + i;
        const bool ok = kj < nk;
        const int key = ok ? (list ? list[kj] : kj) : 0;
        tc::cp_async16(dst + tile_off(i, ch, 128), base + key * sn + ch * 8, ok);
    }
}

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

}  // namespace op
}  // namespace scope
