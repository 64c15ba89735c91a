// Cross attention, forward: each of N queries attends over M keys of another
// sequence (an encoder's states), M and N any lengths.
//
//   s_ij = scale q_i . k_j over the allowed keys j,  lse_i = log sum_j e^s_ij,
//   o_i = sum_j e^(s_ij - lse_i) v_j;  a row without keys gets o = 0, lse = -inf.
//
// Bound: 4 D flops a (row, key) pair on the tensor cores against one
// exponential a pair (16 a clock and SM): at D = 128 both take 1024 clocks a
// 128 x 128 tile, so the two must overlap; below some 300 keys the rows' own
// bytes (q in, o out) take longer than either and HBM is the bound.
//
// One persistent CTA per SM walks work items = (key set, key range, 256
// rows).  The two 128-row tiles of an item share every K/V tile, which halves
// the L2 traffic, and are in opposite phases: one's softmax runs under the
// other's products.  K and V tiles of 128 keys go through one ring of
// shared-memory stages; the next item's Q rows land in a second buffer while
// this item runs, and an item's epilogue overlaps the next item's first
// products.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax and epilogue of tile 0, 1 (one thread per row); O
//                   leaves through the item's Q buffer as whole row segments
//   warp 8          Q rows     } by TMA, or cp.async where a tile's rows are not
//   warps 9-10      K, V rows  } in order (cross_common.cuh)
//   warp 11         tcgen05.mma issuer (one lane), owns the TMEM allocation
// TMEM (512 columns): S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D);
// P (16 bit) overwrites its S.  The softmax runs in base 2 with a lazy
// rescale: O and l move to a new maximum only when it grew by more than 2^8,
// so P stays below 2^8.  P is rounded to the inputs' type for the product
// (the tensor cores take 16-bit operands); its sum l is taken before that
// rounding, in fp32, as are S, O and lse.
//
// Few rows (a single token, a short prompt reading a long video) leave most
// SMs without an item: the keys are then split into ranges whose normalised
// outputs and lse meet in cross_join_kernel, in a fixed order.
//
// Every mbarrier wait is bounded (about two seconds); on timeout the thread
// records it in the operators' error word, the CTA drops its items and all
// threads still meet at the end so the TMEM is released.
#include "cross_common.cuh"

namespace scope {
namespace op {

using namespace tc;

static __device__ int32_t g_cross_err[4];

constexpr int kFwdThreads = 384;
constexpr int kTile = 128;  // rows of a Q tile, keys of a K/V tile

constexpr int fwd_stages(int D) { return D == 128 ? 3 : 4; }
constexpr size_t fwd_smem(int D) { return (size_t)(4 + fwd_stages(D)) * kTile * D * 2 + 1024; }

struct FwdItem {
    int bk, hk, t0, t1, nk, split;
    RowTile r;
};

__device__ __forceinline__ FwdItem fwd_item(const CrossArgs &a, int item)
{
    FwdItem w;
    const int rt = item % a.pairs, rest = item / a.pairs;
    w.split = rest % a.splits;
    const int set = rest / a.splits;
    w.bk = set / a.Hk;
    w.hk = set % a.Hk;
    w.r = row_tile<2 * kTile>(a, w.bk, w.hk, rt);
    w.nk = keys_of(a, w.bk);
    const int tiles = (w.nk + kTile - 1) / kTile;
    w.t0 = (int)((int64_t)tiles * w.split / a.splits);
    w.t1 = (int)((int64_t)tiles * (w.split + 1) / a.splits);
    return w;
}

template <typename T, int D>
__global__ void __launch_bounds__(kFwdThreads, 1) cross_fwd_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ CrossMaps m)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    constexpr int TB = kTile * D * 2;  // bytes of a tile
    constexpr int NS = fwd_stages(D);
    unsigned char *sQ = sm;            // 2 buffers of 2 tiles
    unsigned char *sKV = sm + 4 * TB;  // NS stages

    __shared__ uint64_t q_full[2], q_empty[2], kv_full[NS], kv_empty[NS], s_full[2], p_full[2], o_full[2], o_empty[2];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 8);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], 4);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&kv_full[i], 2);
            mbar_init(&kv_empty[i], 1);
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
    const uint32_t tmem = tmem_base_sh;
    const Waiter wait{&abort_sh, g_cross_err};

    if (warp == 8) {
        // ------------------------------------------------------------ Q rows
        int qi = 0;
        bool ok = true;
        for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
            const FwdItem w = fwd_item(a, item);
            if (w.t0 == w.t1) continue;
            const int buf = qi & 1;
            if (qi >= 2 && !(ok = wait.warp(&q_empty[buf], ((qi >> 1) - 1) & 1, 0x40))) break;
            load_rows<T, D>(a, w.r, w.hk, w.r.nq > kTile ? 2 : 1, &m.q, a.q, a.qB, a.qH, a.qN,
                            smem_u32(sQ + buf * 2 * TB), &q_full[buf]);
            ++qi;
        }
        if (!ok)
            for (int i = qi - 2; i < qi; ++i) drain(&q_full[i & 1], (i >> 1) & 1);
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------------------ K, V rows
        const int tid = threadIdx.x - 9 * 32;
        RingFill<NS> ring(kv_full, kv_empty);
        bool ok = true;
        for (int item = blockIdx.x; ok && item < a.items; item += gridDim.x) {
            const FwdItem w = fwd_item(a, item);
            const T *k = static_cast<const T *>(a.k) + w.bk * a.kB + w.hk * a.kH;
            const T *v = static_cast<const T *>(a.v) + w.bk * a.vB + w.hk * a.vH;
            const int32_t *list = a.idx ? a.idx + (int64_t)w.bk * a.M : nullptr;
            for (int j = w.t0; ok && j < w.t1; ++j) {
                const bool whole = tma_keys(a, w.nk, j);
#pragma unroll 1
                for (int x = 0; x < 2; ++x) {
                    if (!(ok = ring.acquire(wait, 0x41))) break;
                    const uint32_t dst = smem_u32(sKV + ring.slot * TB);
                    if (whole) {
                        ring.template tma<D>(warp == 9, dst, x ? &m.v : &m.k, j * kTile, w.hk, w.bk);
                    } else {
                        copy_keys<T, D, 64>(list, w.nk, j, x ? v : k, x ? a.vN : a.kN, dst, tid);
                        ring.issued();
                    }
                }
            }
        }
        ring.finish(!ok);
    } else if (warp == 11) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t id_qk = idesc16<T>(kTile, false), id_pv = idesc16<T>(D, true);
            const uint64_t dq = sw128_desc(smem_u32(sQ), 16, 1024);
            const uint64_t dk = sw128_desc(smem_u32(sKV), 16, 1024);
            const uint64_t dv = sw128_desc(smem_u32(sKV), kTile * 128, 1024);
            int qi = 0, np[2] = {0, 0}, no[2] = {0, 0};
            RingRead<NS> kv;
            bool ok = true;
            for (int item = blockIdx.x; ok && item < a.items; item += gridDim.x) {
                const FwdItem w = fwd_item(a, item);
                if (w.t0 == w.t1) continue;
                const int nt = w.r.nq > kTile ? 2 : 1, buf = qi & 1;
                // S_t = Q_t K^T
                auto issue_qk = [&](int t, int ks) {
                    const uint64_t aq = dq + (uint64_t)(((buf * 2 + t) * TB) >> 4);
                    const uint64_t bk = dk + (uint64_t)((ks * TB) >> 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t o = (uint64_t)(((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4);
                        mma_ss(tmem + t * 128, aq + o, bk + o, id_qk, k > 0);
                    }
                    mma_commit(&s_full[t]);
                    if (t == nt - 1) mma_commit(&kv_empty[ks]);
                };
                ok = wait(&q_full[buf], (qi >> 1) & 1, 0x42) && wait(&kv_full[kv.slot], kv.use & 1, 0x43);
                if (!ok) break;
                tc_fence_after();
                for (int t = 0; t < nt; ++t) issue_qk(t, kv.slot);
                kv.next();
                for (int j = w.t0; ok && j < w.t1; ++j) {
                    const int vs = kv.slot;
                    if (!(ok = wait(&kv_full[vs], kv.use & 1, 0x44))) break;
                    kv.next();
                    const bool more = j + 1 < w.t1;
                    for (int t = 0; t < nt; ++t) {
                        if (!(ok = wait(&p_full[t], np[t] & 1, 0x45))) break;
                        ++np[t];
                        // the previous item's epilogue has read O_t
                        if (j == w.t0 && no[t] > 0 && !(ok = wait(&o_empty[t], (no[t] - 1) & 1, 0x46))) break;
                        tc_fence_after();
                        const uint64_t bv = dv + (uint64_t)((vs * TB) >> 4);
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            mma_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, bv + (uint64_t)((k * 2048) >> 4), id_pv,
                                   j > w.t0 || k > 0);
                        if (t == nt - 1) mma_commit(&kv_empty[vs]);
                        if (more) {
                            if (t == 0 && !(ok = wait(&kv_full[kv.slot], kv.use & 1, 0x47))) break;
                            tc_fence_after();
                            issue_qk(t, kv.slot);
                        } else {
                            mma_commit(&o_full[t]);
                            ++no[t];
                        }
                    }
                    if (more) kv.next();
                }
                ++qi;
            }
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------------------ softmax and epilogue
        const int t = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * 128, tO = tmem + lane_off + 256 + t * 128;
        int ns = 0, no = 0, qi = 0;
        bool ok = true;
        for (int item = blockIdx.x; ok && item < a.items; item += gridDim.x) {
            const FwdItem w = fwd_item(a, item);
            const bool some = w.t0 < w.t1;  // uniform for the CTA
            const int buf = qi & 1;
            if (some) ++qi;
            if (w.r.nq <= t * kTile) {
                // no rows here: the item's Q is free as far as this tile goes (but not before it has come)
                if (some) {
                    if (!(ok = wait.warp(&q_full[buf], ((qi - 1) >> 1) & 1, 0x4c))) break;
                    if (lane == 0) mbar_arrive(&q_empty[buf]);
                }
                continue;
            }
            float m_run = -INFINITY, l = 0.f;
            for (int j = w.t0; j < w.t1; ++j) {
                if (!(ok = wait.warp(&s_full[t], ns & 1, 0x48 + t))) break;
                ++ns;
                tc_fence_after();
                uint32_t r[kTile];
#pragma unroll
                for (int c4 = 0; c4 < kTile / 32; ++c4) tmem_ld32(tS + c4 * 32, r + c4 * 32);
                tmem_wait_ld();
                const int valid = w.nk - j * kTile;
                if (valid < kTile) {
#pragma unroll
                    for (int i = 0; i < kTile; ++i)
                        if (i >= valid) r[i] = __float_as_uint(-INFINITY);
                }
                float m4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m4[i] = __uint_as_float(r[i]);
#pragma unroll
                for (int i = 4; i < kTile; i += 2)
                    m4[(i >> 1) & 3] = fmax3(m4[(i >> 1) & 3], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                const float mt = fmax3(fmax3(m4[0], m4[1], m4[2]), m4[3], m4[3]) * a.scale_log2;
                bool rescale = false;
                float alpha = 1.f;
                if (j == w.t0) {
                    m_run = mt;
                } else if (__any_sync(0xffffffffu, mt > m_run + 8.f)) {
                    const float mn = fmaxf(m_run, mt);
                    // every logit so far -inf: l = 0 and O = 0, nothing to scale
                    alpha = m_run == -INFINITY ? 0.f : ex2(m_run - mn);
                    m_run = mn;
                    l *= alpha;
                    rescale = true;
                }
                const float m_ref = m_run == -INFINITY ? 0.f : m_run;
                const uint64_t scp = f2pack(a.scale_log2, a.scale_log2), nmp = f2pack(-m_ref, -m_ref);
                uint64_t sA = 0ull, sB = 0ull;
#pragma unroll
                for (int c4 = 0; c4 < kTile / 32; ++c4) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t x2 = ffma2(
                            f2pack(__uint_as_float(r[c4 * 32 + 2 * i]), __uint_as_float(r[c4 * 32 + 2 * i + 1])), scp, nmp);
                        float x0, x1;
                        f2unpack(x2, x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        if (i & 1) sB = fadd2(sB, f2pack(p0, p1));
                        else sA = fadd2(sA, f2pack(p0, p1));
                        pk[i] = pack2(T(), p0, p1);
                    }
                    tmem_st16(tS + c4 * 16, pk);
                }
                float la, lb, lc, ld;
                f2unpack(sA, la, lb);
                f2unpack(sB, lc, ld);
                l += (la + lc) + (lb + ld);
                if (rescale) {
#pragma unroll
                    for (int c4 = 0; c4 < D / 32; ++c4) {
                        uint32_t o[32];
                        tmem_ld32(tO + c4 * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(tO + c4 * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t]);
            }
            if (!ok) break;
            if (some) {
                if (!(ok = wait.warp(&o_full[t], no & 1, 0x4a + t))) break;
                ++no;
                tc_fence_after();
            }
            // all products of the item are done: the O rows leave through this tile's part of the Q buffer
            const uint32_t stage = smem_u32(sQ + (buf * 2 + t) * TB) + wq * (TB / 4);
            const int first = t * kTile + wq * 32, n_rows = w.r.nq - first;
            const bool store = lane < n_rows;
            int b, h, n;
            tile_row(a, w.r, w.hk, store ? first + lane : 0, b, h, n);
            const int64_t total = (int64_t)a.B * a.H * a.N, flat = ((int64_t)b * a.H + h) * a.N + n;
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a NaN sum stays one
            const float lse2 = l == 0.f ? -INFINITY : m_run + log2f(l);
            T *o = static_cast<T *>(a.o);
            auto o_row = [&](int i) {
                int rb, rh, rn;
                tile_row(a, w.r, w.hk, first + i, rb, rh, rn);
                return o + rb * a.oB + rh * a.oH + rn * a.oN;
            };
            auto part_row = [&](int i) {
                int rb, rh, rn;
                tile_row(a, w.r, w.hk, first + i, rb, rh, rn);
                return a.part_o + (w.split * total + ((int64_t)rb * a.H + rh) * a.N + rn) * D;
            };
            if (some) {
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t r[64];
                    tmem_ld32(tO + c * 64, r);
                    tmem_ld32(tO + c * 64 + 32, r + 32);
                    tmem_wait_ld();
                    if (c == D / 64 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&o_empty[t]);
                    }
                    float f[64];
#pragma unroll
                    for (int i = 0; i < 64; ++i) f[i] = __uint_as_float(r[i]) * inv;
                    uint4 u[8];
                    if (a.splits > 1) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) u[i] = bits4(f + x * 32 + 4 * i);
                            store_staged<8>(stage, u, n_rows, [&](int i) { return part_row(i) + c * 64 + x * 32; });
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = pack8<T>(f + 8 * i);
                        store_staged<8>(stage, u, n_rows, [&](int i) { return o_row(i) + c * 64; });
                    }
                }
                fence_async_smem();  // before a TMA load writes the buffer again
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_empty[buf]);
            } else if (store) {
                const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                for (int i = 0; i < D; i += 8) {
                    if (a.splits > 1) store8(part_row(lane) + i, zero);
                    else store8(o_row(lane) + i, zero);
                }
            }
            if (store) {
                if (a.splits > 1) a.part_lse[w.split * total + flat] = lse2;
                else if (a.lse) a.lse[flat] = lse2 * 0.6931471805599453f;
            }
        }
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

// Key ranges per row tile: the count with the least modelled time, in steps of
// one 128-key tile (some 1.2 us a CTA).  An item costs its tiles and about two
// more for its Q rows and epilogue; a split adds a launch (about 3 steps) and
// the partial outputs' traffic.
int cross_fwd_splits(int64_t sets, int64_t pairs, int64_t M, int64_t rows_total, int D, int sms)
{
    const int64_t tiles = (M + kTile - 1) / kTile, items = sets * pairs;
    int best = 1;
    double least = 0.0;
    for (int64_t s = 1; s <= tiles && s <= 128 && (s == 1 || items * (s - 1) < sms); ++s) {
        const double waves = (double)((items * s + sms - 1) / sms);
        double t = waves * (double)((tiles + s - 1) / s + 2);
        if (s > 1) t += 3.0 + (double)(s * rows_total) * D * 8.0 / 6e6;
        if (s == 1 || t < least) {
            least = t;
            best = (int)s;
        }
    }
    return best;
}

template <typename T>
static void launch_fwd_t(const CrossArgs &a, const CrossMaps &m, int D, int grid, cudaStream_t st)
{
    if (D == 128) cross_fwd_kernel<T, 128><<<grid, kFwdThreads, fwd_smem(128), st>>>(a, m);
    else cross_fwd_kernel<T, 64><<<grid, kFwdThreads, fwd_smem(64), st>>>(a, m);
    count_launches(1);
    if (a.splits > 1) {
        const int64_t threads = (int64_t)a.B * a.H * a.N * (D / 8);
        cross_join_kernel<T><<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(a, D);
        count_launches(1);
    }
}

void launch_cross_fwd(const CrossArgs &a, const CrossMaps &m, int D, bool f16, int sms, cudaStream_t st)
{
    const int grid = a.items < sms ? a.items : sms;
    if (f16) launch_fwd_t<__half>(a, m, D, grid, st);
    else launch_fwd_t<__nv_bfloat16>(a, m, D, grid, st);
}

}  // namespace op
}  // namespace scope
