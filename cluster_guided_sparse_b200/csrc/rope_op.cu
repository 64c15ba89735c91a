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
// x may be overwritten in place.  Four heads' chunks are loaded before the
// first is used.
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

template <typename T, bool NORM, int LPR>
__global__ void __launch_bounds__(kRopeThreads)
    rope_op_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTurns t)
{
    const int c8 = threadIdx.x % LPR;
    const int64_t tok = (int64_t)blockIdx.x * (kRopeThreads / LPR) + threadIdx.x / LPR;
    const bool valid = tok < a.tokens;
    // idle lanes of the last block follow the last token (shuffles) and store nothing
    const int64_t tk = valid ? tok : a.tokens - 1;
    const int b = (int)(tk / a.N), n = (int)(tk % a.N);
    float cs[4], sn[4], w[8];
    rope_angles(a, t, b, n, c8, cs, sn);
    if constexpr (NORM) load_weight(a, c8, w);
    const T *x = static_cast<const T *>(a.x) + b * a.xB + n * a.xN + c8 * 8;
    T *y = static_cast<T *>(a.y) + b * a.yB + n * a.yN + c8 * 8;
    const int h0 = blockIdx.y * a.heads_per_block, h1 = min(a.H, h0 + a.heads_per_block);
    for (int h = h0; h < h1; h += kRopeBatch) {
        float v[kRopeBatch][8];
#pragma unroll
        for (int j = 0; j < kRopeBatch; ++j) load8(x + min(h + j, h1 - 1) * a.xH, v[j]);
#pragma unroll
        for (int j = 0; j < kRopeBatch; ++j) {
            if constexpr (NORM) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
                const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / (LPR * 8)) + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] *= r * w[i];
            }
            float o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x0 = v[j][2 * i], x1 = v[j][2 * i + 1];
                o[2 * i] = fmaf(x0, cs[i], -x1 * sn[i]);
                o[2 * i + 1] = fmaf(x0, sn[i], x1 * cs[i]);
            }
            if (valid && h + j < h1) store8(y + (h + j) * a.yH, o);
        }
    }
}

// Gradient behind the norm.  Blocks walk the tokens with a fixed stride, so
// each thread keeps its 8 columns of dw in registers; the block's rows meet
// in shared memory and its partial sums in rope_dw_kernel, always in the same
// order.
template <typename T, int LPR>
__global__ void __launch_bounds__(kRopeThreads)
    rope_op_bwd_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTurns t)
{
    constexpr int D = LPR * 8, TPB = kRopeThreads / LPR, kB = 2;
    __shared__ float part[TPB][D];
    const int c8 = threadIdx.x % LPR;
    const int h0 = blockIdx.y * a.heads_per_block, h1 = min(a.H, h0 + a.heads_per_block);
    float w[8], dw[8];
    load_weight(a, c8, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0.f;
    for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < a.tokens; t0 += (int64_t)gridDim.x * TPB) {
        const int64_t tok = t0 + threadIdx.x / LPR;
        const bool valid = tok < a.tokens;
        const int64_t tk = valid ? tok : a.tokens - 1;
        const int b = (int)(tk / a.N), n = (int)(tk % a.N);
        float cs[4], sn[4];
        rope_angles(a, t, b, n, c8, cs, sn);
        const T *x = static_cast<const T *>(a.x) + b * a.xB + n * a.xN + c8 * 8;
        const T *dy = static_cast<const T *>(a.dy) + b * a.dB + n * a.dN + c8 * 8;
        T *dx = static_cast<T *>(a.y) + b * a.yB + n * a.yN + c8 * 8;
        for (int h = h0; h < h1; h += kB) {
            float xv[kB][8], gv[kB][8];
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                const int hj = min(h + j, h1 - 1);
                load8(x + hj * a.xH, xv[j]);
                load8(dy + hj * a.dH, gv[j]);
            }
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                const bool store = valid && h + j < h1;
                float dz[8], ss = 0.f, gx = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y0 = gv[j][2 * i], y1 = gv[j][2 * i + 1];
                    dz[2 * i] = fmaf(y0, cs[i], y1 * sn[i]);
                    dz[2 * i + 1] = fmaf(y1, cs[i], -y0 * sn[i]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ss = fmaf(xv[j][i], xv[j][i], ss);
                    gx = fmaf(dz[i] * w[i], xv[j][i], gx);
                }
                const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
                const float m = row_sum<LPR>(gx) * (1.f / D) * r * r;
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[i] = r * fmaf(-xv[j][i], m, dz[i] * w[i]);
                    if (store) dw[i] = fmaf(dz[i], xv[j][i] * r, dw[i]);
                }
                if (store) store8(dx + (h + j) * a.yH, o);
            }
        }
    }
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
// unless that leaves fewer than `want` blocks, as for one token of many heads.
static int heads_per_block(int64_t token_blocks, int H, int batch, int want)
{
    int hpb = H;
    while (hpb > batch && token_blocks * ((H + hpb - 1) / hpb) < want) hpb = (hpb + 1) / 2;
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

// Blocks of the backward kernel: four per SM walk the tokens.
static dim3 bwd_grid(int64_t tokens, int H, int D, int *hpb)
{
    const int tpb = kRopeThreads / (D / 8);
    int64_t bx = (tokens + tpb - 1) / tpb;
    *hpb = heads_per_block(bx, H, 2, 148 * 4);
    const int64_t by = (H + *hpb - 1) / *hpb;
    const int64_t most = (148 * 4 + by - 1) / by;
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
    rope_dw_kernel<<<a.D / 8, 512, 0, st>>>(a.dw_part, (int)(grid.x * grid.y), a.D, dw, a.w_dtype);
    count_launches(2);
}

}  // namespace op
}  // namespace scope
