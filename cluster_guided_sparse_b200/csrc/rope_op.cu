// Rotary positions with three axes as an operator of its own, optionally
// behind a per-head RMS norm, and the gradient of both.
//
//   r = (mean_d x_d^2 + eps)^-1/2,  z = x r w          (norm; else z = x)
//   y_2i   = z_2i cos a_i - z_2i+1 sin a_i
//   y_2i+1 = z_2i sin a_i + z_2i+1 cos a_i             a_i = p_axis theta^(-2i'/d_axis)
// Without the norm the gradient is the rotation by -a of dy.  With it, for
// dz = R(-a) dy and g = dz w:
//   dx = r (g - x r^2 mean_d(g x)),   dw = sum over rows of dz x r.
//
// Bound by HBM: each tensor is read or written once in 16-byte chunks (32 for
// fp32).  One thread owns 8 dims (4 pairs) of one token and walks that token's
// heads, which share the 4 angles, so the sines cost one evaluation per token
// and pair, not per element, and no table or second launch is needed.  The
// D/8 lanes of a row sit in one warp, so the norm's sum is a few shuffles and
// x may be overwritten in place.  Four heads' chunks are under way at any
// time, the first ones before the angles are evaluated.
//
// With the norm the instructions come close to the bytes' time, so the
// arithmetic runs on pairs of fp32 values in one register pair: the first halves
// of two rotations, and their second halves.
//
// The angle in turns is reduced in fp64 (positions are 32-bit integers: in
// fp32 a position of 1e5 would lose 1e-2 rad); sine, cosine, norm and
// rotation run in fp32 and each output is rounded once.
#include "../../include/scope.h"
#include "op_common.cuh"

namespace scope {
namespace op {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // heads in flight per thread

// Batch entry and place of a token.
__device__ __forceinline__ void token_at(const RopeArgs &a, int64_t tok, int &b, int &n)
{
    if (a.tokens <= 0x7fffffff) {
        b = (int)((uint32_t)tok / (uint32_t)a.N);
        n = (int)tok - b * a.N;
    } else {
        b = (int)(tok / a.N);
        n = (int)(tok % a.N);
    }
}

__device__ __forceinline__ void rope_angles(const RopeArgs &a, const RopeTurns &t, int b, int n, int c8, float *cs,
                                            float *sn)
{
    int pos[3];
    if (a.positions) {
        const int32_t *p = a.positions + b * a.posB + (int64_t)n * 3;
        pos[0] = p[0]; pos[1] = p[1]; pos[2] = p[2];
    } else {
        pos[0] = n / (a.Hh * a.W); pos[1] = (n / a.W) % a.Hh; pos[2] = n % a.W;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int pair = c8 * 4 + i;
        const int axis = pair < t.pt ? 0 : (pair < t.pt + t.ph ? 1 : 2);
        double f = (double)(axis == 0 ? pos[0] : axis == 1 ? pos[1] : pos[2]) * t.turns[pair];
        f -= rint(f);
        sincospif(2.f * (float)f, &sn[i], &cs[i]);
        sn[i] *= a.sign;
    }
}

__device__ __forceinline__ void load_weight(const RopeArgs &a, int c8, float *w)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = c8 * 8 + i;
        w[i] = a.w_dtype == SCOPE_F32    ? static_cast<const float *>(a.weight)[d]
               : a.w_dtype == SCOPE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.weight)[d])
                                         : __half2float(static_cast<const __half *>(a.weight)[d]);
    }
}

// Sum over the LPR lanes that share a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Two fp32 values, worked on by one instruction.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ void get(float &x, float &y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
    __device__ __forceinline__ float sum() const
    {
        float x, y;
        get(x, y);
        return x + y;
    }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

// 8 dims of a row: first halves e and second halves o of rotations 0, 1 and 2, 3.
struct Row8 {
    F2 e[2], o[2];
    __device__ __forceinline__ explicit Row8(const float *x)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            e[i] = F2(x[4 * i], x[4 * i + 2]);
            o[i] = F2(x[4 * i + 1], x[4 * i + 3]);
        }
    }
    __device__ __forceinline__ void get(float *x) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            e[i].get(x[4 * i], x[4 * i + 2]);
            o[i].get(x[4 * i + 1], x[4 * i + 3]);
        }
    }
};

__device__ __forceinline__ float dot(const Row8 &a, const Row8 &b)
{
    F2 s = a.e[0] * b.e[0];
    s = fma2(a.o[0], b.o[0], s);
    s = fma2(a.e[1], b.e[1], s);
    return fma2(a.o[1], b.o[1], s).sum();
}

template <typename T, bool NORM, int LPR>
__global__ void __launch_bounds__(kRopeThreads)
    rope_op_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTurns t)
{
    const int c8 = threadIdx.x % LPR;
    const int64_t tok = (int64_t)blockIdx.x * (kRopeThreads / LPR) + threadIdx.x / LPR;
    const bool valid = tok < a.tokens;
    // idle lanes of the last block follow the last token (shuffles) and store nothing
    int b, n;
    token_at(a, valid ? tok : a.tokens - 1, b, n);
    const T *x = static_cast<const T *>(a.x) + b * a.xB + n * a.xN + c8 * 8;
    T *y = static_cast<T *>(a.y) + b * a.yB + n * a.yN + c8 * 8;
    const int h0 = blockIdx.y * a.heads_per_block, h1 = min(a.H, h0 + a.heads_per_block);
    Raw8<T> next[kRopeBatch];
#pragma unroll
    for (int j = 0; j < kRopeBatch; ++j) next[j].load(x + min(h0 + j, h1 - 1) * a.xH);
    float cs[4], sn[4], w[8];
    rope_angles(a, t, b, n, c8, cs, sn);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if constexpr (NORM) load_weight(a, c8, w);
    // y_e = x_e (w_e cos) - x_o (w_o sin), y_o = x_e (w_e sin) + x_o (w_o cos)
    F2 ec[2], es[2], oc[2], os[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        ec[i] = F2(w[4 * i] * cs[2 * i], w[4 * i + 2] * cs[2 * i + 1]);
        es[i] = F2(w[4 * i] * sn[2 * i], w[4 * i + 2] * sn[2 * i + 1]);
        oc[i] = F2(w[4 * i + 1] * cs[2 * i], w[4 * i + 3] * cs[2 * i + 1]);
        os[i] = F2(-w[4 * i + 1] * sn[2 * i], -w[4 * i + 3] * sn[2 * i + 1]);
    }
    for (int h = h0; h < h1; h += kRopeBatch) {
#pragma unroll
        for (int j = 0; j < kRopeBatch; ++j) {
            float v[8];
            next[j].values(v);
            if (h + j + kRopeBatch < h1) next[j].load(x + (h + j + kRopeBatch) * a.xH);
            Row8 q(v);
            if constexpr (NORM) {
                const float r = rsqrtf(row_sum<LPR>(dot(q, q)) * (1.f / (LPR * 8)) + a.eps);
                const F2 r2(r, r);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    q.e[i] = q.e[i] * r2;
                    q.o[i] = q.o[i] * r2;
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const F2 e = fma2(q.e[i], ec[i], q.o[i] * os[i]);
                q.o[i] = fma2(q.e[i], es[i], q.o[i] * oc[i]);
                q.e[i] = e;
            }
            float o[8];
            q.get(o);
            if (valid && h + j < h1) store8(y + (h + j) * a.yH, o);
        }
    }
}

// Gradient behind the norm.  Blocks walk the tokens with a fixed stride, so
// each thread keeps its 8 columns of dw in registers; the block's rows meet
// in shared memory and its partial sums in rope_dw_kernel, always in the same
// order.
template <typename T, int LPR>
__global__ void __launch_bounds__(kRopeThreads, 2)
    rope_op_bwd_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTurns t)
{
    constexpr int D = LPR * 8, TPB = kRopeThreads / LPR, kB = sizeof(T) == 4 ? 2 : 4;
    let_next_start();
    __shared__ float part[TPB][D];
    const int c8 = threadIdx.x % LPR;
    const int h0 = blockIdx.y * a.heads_per_block, h1 = min(a.H, h0 + a.heads_per_block);
    float w[8], dw[8];
    load_weight(a, c8, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0.f;
    const Row8 wr(w);
    Row8 dwr(dw);
    for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < a.tokens; t0 += (int64_t)gridDim.x * TPB) {
        const int64_t tok = t0 + threadIdx.x / LPR;
        const bool valid = tok < a.tokens;
        int b, n;
        token_at(a, valid ? tok : a.tokens - 1, b, n);
        const T *x = static_cast<const T *>(a.x) + b * a.xB + n * a.xN + c8 * 8;
        const T *dy = static_cast<const T *>(a.dy) + b * a.dB + n * a.dN + c8 * 8;
        T *dx = static_cast<T *>(a.y) + b * a.yB + n * a.yN + c8 * 8;
        Raw8<T> xn[kB], gn[kB];
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            const int hj = min(h0 + j, h1 - 1);
            xn[j].load(x + hj * a.xH);
            gn[j].load(dy + hj * a.dH);
        }
        float cs[4], sn[4];
        rope_angles(a, t, b, n, c8, cs, sn);
        F2 c2[2], s2[2], m2[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c2[i] = F2(cs[2 * i], cs[2 * i + 1]);
            s2[i] = F2(sn[2 * i], sn[2 * i + 1]);
            m2[i] = F2(-sn[2 * i], -sn[2 * i + 1]);
        }
        for (int h = h0; h < h1; h += kB) {
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                float xv[8], gv[8];
                xn[j].values(xv);
                gn[j].values(gv);
                if (h + j + kB < h1) {
                    xn[j].load(x + (h + j + kB) * a.xH);
                    gn[j].load(dy + (h + j + kB) * a.dH);
                }
                const bool store = valid && h + j < h1;
                const Row8 xr(xv);
                Row8 dz(gv), g = dz;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const F2 e = fma2(dz.e[i], c2[i], dz.o[i] * s2[i]);
                    dz.o[i] = fma2(dz.o[i], c2[i], dz.e[i] * m2[i]);
                    dz.e[i] = e;
                    g.e[i] = dz.e[i] * wr.e[i];
                    g.o[i] = dz.o[i] * wr.o[i];
                }
                const float r = rsqrtf(row_sum<LPR>(dot(xr, xr)) * (1.f / D) + a.eps);
                const float m = -row_sum<LPR>(dot(g, xr)) * (1.f / D) * r * r;
                const F2 r2(r, r), mm(m, m);
                // Rows that are not this thread's are left out, not multiplied by zero: an idle lane may hold an
                // infinity, in place even one that the row's own lanes have just written.
                if (store) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        dwr.e[i] = fma2(dz.e[i], xr.e[i] * r2, dwr.e[i]);
                        dwr.o[i] = fma2(dz.o[i], xr.o[i] * r2, dwr.o[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    g.e[i] = fma2(xr.e[i], mm, g.e[i]) * r2;
                    g.o[i] = fma2(xr.o[i], mm, g.o[i]) * r2;
                }
                float o[8];
                g.get(o);
                if (store) store8(dx + (h + j) * a.yH, o);
            }
        }
    }
    dwr.get(dw);
#pragma unroll
    for (int i = 0; i < 8; ++i) part[threadIdx.x / LPR][c8 * 8 + i] = dw[i];
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
        for (int g = 0; g < TPB; ++g) s += part[g][threadIdx.x];
        a.dw_part[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
    }
}

// dw[d] = sum of the blocks' partial sums, in fp64; one block per 8 columns.
__global__ void __launch_bounds__(512) rope_dw_kernel(const float *part, int parts, int D, void *dw, int w_dtype)
{
    wait_for_previous();
    __shared__ double acc[64][8];
    const int c = threadIdx.x & 7, g = threadIdx.x >> 3, d = blockIdx.x * 8 + c;
    double s = 0.0;
#pragma unroll 4
    for (int p = g; p < parts; p += 64) s += part[(int64_t)p * D + d];
    acc[g][c] = s;
    __syncthreads();
    if (g == 0) {
        for (int i = 1; i < 64; ++i) s += acc[i][c];
        if (w_dtype == SCOPE_F32) static_cast<float *>(dw)[d] = (float)s;
        else if (w_dtype == SCOPE_BF16) static_cast<__nv_bfloat16 *>(dw)[d] = __double2bfloat16(s);
        else static_cast<__half *>(dw)[d] = __double2half(s);
    }
}

// Heads per block: all of them (the angles are then evaluated once per token)
// unless that leaves fewer blocks than some six per place on the GPU, whose
// last ones would run alone (480p, 40 heads: 3.5 blocks a place took 130 us,
// 7 a place, with the arithmetic below, 115 us); at least eight heads, or a batch where that is
// needed to fill the GPU at all, as for one token of many heads.  Forward, a place is a
// quarter of an SM, as the 16-bit kernels fit (52 to 64 registers); of the fp32 ones
// (80 and 86) an SM holds three or two.
static int heads_per_block(int64_t token_blocks, int H, int batch, int places)
{
    int hpb = H;
    while (hpb > 8 && token_blocks * ((H + hpb - 1) / hpb) < 6 * places) hpb = (hpb + 1) / 2;
    while (hpb > batch && token_blocks * ((H + hpb - 1) / hpb) < places) hpb = (hpb + 1) / 2;
    return hpb;
}

template <typename T, bool NORM>
static void launch_fwd(const RopeArgs &a, const RopeTurns &t, dim3 grid, cudaStream_t st)
{
    if (a.D == 128) rope_op_kernel<T, NORM, 16><<<grid, kRopeThreads, 0, st>>>(a, t);
    else rope_op_kernel<T, NORM, 8><<<grid, kRopeThreads, 0, st>>>(a, t);
}

template <typename T>
static void launch_fwd_t(const RopeArgs &a, const RopeTurns &t, dim3 grid, cudaStream_t st)
{
    if (a.weight) launch_fwd<T, true>(a, t, grid, st);
    else launch_fwd<T, false>(a, t, grid, st);
}

void launch_rope_op(const RopeArgs &args, const RopeTurns &t, int dtype, cudaStream_t st)
{
    RopeArgs a = args;
    const int tpb = kRopeThreads / (a.D / 8);
    const int64_t blocks = (a.tokens + tpb - 1) / tpb;
    a.heads_per_block = heads_per_block(blocks, a.H, kRopeBatch, 148 * 4);
    const dim3 grid((unsigned)blocks, (unsigned)((a.H + a.heads_per_block - 1) / a.heads_per_block));
    if (dtype == SCOPE_F32) launch_fwd_t<float>(a, t, grid, st);
    else if (dtype == SCOPE_BF16) launch_fwd_t<__nv_bfloat16>(a, t, grid, st);
    else launch_fwd_t<__half>(a, t, grid, st);
    count_launches(1);
}

// Blocks of the backward kernel: two per SM (its registers allow no more) walk the tokens.
static dim3 bwd_grid(int64_t tokens, int H, int D, int *hpb)
{
    const int tpb = kRopeThreads / (D / 8);
    int64_t bx = (tokens + tpb - 1) / tpb;
    *hpb = heads_per_block(bx, H, 2, 148 * 2);
    const int64_t by = (H + *hpb - 1) / *hpb;
    const int64_t most = (148 * 2) / by > 0 ? (148 * 2) / by : 1;
    if (bx > most) bx = most;
    return dim3((unsigned)bx, (unsigned)by);
}

int rope_bwd_blocks(int64_t tokens, int H, int D, int *hpb)
{
    const dim3 g = bwd_grid(tokens, H, D, hpb);
    return (int)(g.x * g.y);
}

template <typename T>
static void launch_bwd_t(const RopeArgs &a, const RopeTurns &t, dim3 grid, cudaStream_t st)
{
    if (a.D == 128) rope_op_bwd_kernel<T, 16><<<grid, kRopeThreads, 0, st>>>(a, t);
    else rope_op_bwd_kernel<T, 8><<<grid, kRopeThreads, 0, st>>>(a, t);
}

void launch_rope_op_bwd(RopeArgs a, const RopeTurns &t, int dtype, void *dw, cudaStream_t st)
{
    const dim3 grid = bwd_grid(a.tokens, a.H, a.D, &a.heads_per_block);
    if (dtype == SCOPE_F32) launch_bwd_t<float>(a, t, grid, st);
    else if (dtype == SCOPE_BF16) launch_bwd_t<__nv_bfloat16>(a, t, grid, st);
    else launch_bwd_t<__half>(a, t, grid, st);
    count_launches(1);
    launch_next(rope_dw_kernel, a.D / 8, 512, 0, st, a.dw_part, (int)(grid.x * grid.y), a.D, dw, a.w_dtype);
}

}  // namespace op
}  // namespace scope
