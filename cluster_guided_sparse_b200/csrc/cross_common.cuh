// Shared by the cross-attention kernels (cross_attn.cu, cross_bwd.cu).
//
// A "key set" is one (key batch entry, key head): its rows are the query rows
// that read it, numbered r = (b' * G + g) * N + n over the batch entries b'
// that share the keys (one, or all of B when the keys have batch 1), the G
// query heads of the key head and the N queries.  Row tiles cross head and
// batch borders, so short query lengths of many heads still fill tiles.
#pragma once

#include "op_common.cuh"
#include "tcgen05.cuh"

namespace scope {
namespace op {

struct CrossArgs {
    const void *q, *k, *v;
    void *o;
    float *lse;                // [B][H][N] or null
    int64_t qB, qH, qN, kB, kH, kN, vB, vH, vN, oB, oH, oN;  // element strides
    const int32_t *kv_len;     // [Bk] or null: all M keys
    const int32_t *idx, *cnt;  // kept keys of a mask: [Bk][M] ascending, [Bk]; or null
    int B, Bk, H, Hk, G, N, M, GN;
    int rows;                  // per key set
    int sets;                  // Bk * Hk
    int row_tiles, splits;
    int items;                 // sets * splits * row_tiles
    float scale_log2;          // scale * log2(e)
    float *part_o;             // [splits][B*H*N][D], normalised per split (splits > 1)
    float *part_lse;           // [splits][B*H*N], base 2
    // backward
    const void *dout;
    int64_t dB, dH, dN;
    // per key set, rows padded to rows_pad (a multiple of 128): -lse in base 2
    // (-inf where the row reads nothing: its p is then 0) and -sum_d do * o
    float *nlse, *ndelta;
    int rows_pad;
    void *dq;
    int64_t dqB, dqH, dqN;
    int dq_splits;             // key ranges of the dq kernel
    float *part_dq;            // [dq_splits][B*H*N][D] (dq_splits > 1)
    int dkv_splits;            // row ranges of the dk/dv kernel
    float *part_dk, *part_dv;  // [dkv_splits][sets][M][D], kept keys in list order
    float scale;
};

// Queries of row r of key set (bk, hk).
__device__ __forceinline__ void row_of(const CrossArgs &a, int bk, int hk, int r, int &b, int &h, int &n)
{
    b = bk;
    if (a.Bk != a.B) {
        b = r / a.GN;
        r -= b * a.GN;
    }
    const int g = r / a.N;
    n = r - g * a.N;
    h = hk * a.G + g;
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

// Ring of shared-memory stages filled by cp.async from W whole warps: a stage
// is announced (one arrival per warp) once its copies landed, which is checked
// after the next stage's copies were issued, so two are in flight.
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
        if (++slot == NS) {
            slot = 0;
            ++use;
        }
    }
    __device__ __forceinline__ void flush()
    {
        tc::cp_async_wait_all();
        if (pending >= 0) announce();
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

// Copies rows [r0, r0 + fill) of a key set's query rows (element strides
// sB, sH, sN) into swizzled tiles of 128 rows, rows from `n_rows` on as zeros.
// `threads` threads (whole warps), `tid` this one's number.
template <typename T, int D>
__device__ __forceinline__ void copy_rows(const CrossArgs &a, int bk, int hk, int r0, int n_rows, int fill, const T *src,
                                          int64_t sB, int64_t sH, int64_t sN, uint32_t dst, int tid, int threads)
{
    constexpr int CH = D / 8;
    const int ch = tid % CH, rl = tid / CH, step = threads / CH;
    int b, h, n;
    row_of(a, bk, hk, r0, b, h, n);
    const bool one_head = n + n_rows <= a.N;
    src += ch * 8;
    const T *p0 = src + b * sB + h * sH + n * sN;
#pragma unroll 8
    for (int i = rl; i < fill; i += step) {
        const bool ok = i < n_rows;
        const T *p = p0;
        if (one_head) {
            if (ok) p = p0 + i * sN;
        } else if (ok) {
            row_of(a, bk, hk, r0 + i, b, h, n);
            p = src + b * sB + h * sH + n * sN;
        }
        tc::cp_async16(dst + (i / 128) * (128 * D * 2) + tile_off(i % 128, ch, 128), p, ok);
    }
}

// Copies the 128 keys of tile j (rows of a key list, if any) into a tile, rows
// past the set's nk keys as zeros: their memory is never read.
template <typename T, int D, int THREADS>
struct KeyTile {
    static constexpr int CH = D / 8, RPI = THREADS / CH, NR = 128 / RPI;
    int keys[NR];
    __device__ __forceinline__ void load(const int32_t *list, int nk, int j, int tid)
    {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int kj = j * 128 + i * RPI + tid / CH;
            keys[i] = kj < nk ? (list ? list[kj] : kj) : -1;
        }
    }
    __device__ __forceinline__ void copy(const T *base, int64_t sn, uint32_t dst, int tid) const
    {
        const int ch = tid % CH, rl = tid / CH;
#pragma unroll
        for (int i = 0; i < NR; ++i)
            tc::cp_async16(dst + tile_off(i * RPI + rl, ch, 128), base + max(keys[i], 0) * sn + ch * 8, keys[i] >= 0);
    }
};

cudaError_t cross_fwd_configure();
cudaError_t cross_bwd_configure();
int cross_fwd_splits(int64_t sets, int64_t row_tiles, int64_t M, int64_t rows_total, int D, int sms);
int cross_dq_splits(int64_t sets, int64_t rows, int64_t M, int64_t rows_total, int D, int sms);
int cross_dkv_splits(int64_t sets, int64_t rows, int64_t M, int D, int sms);
void launch_key_lists(const uint8_t *mask, int64_t stride, int Bk, int M, int32_t *idx, int32_t *cnt, int32_t *inv,
                      cudaStream_t st);
void launch_cross_fwd(const CrossArgs &a, int D, bool f16, int sms, cudaStream_t st);
void launch_cross_bwd(const CrossArgs &a, int D, bool f16, int sms, const int32_t *inv, void *dk, const int64_t *dks,
                      void *dv, const int64_t *dvs, cudaStream_t st);
cudaError_t cross_fwd_error(int32_t *err, bool clear);
cudaError_t cross_bwd_error(int32_t *err, bool clear);

}  // namespace op
}  // namespace scope
