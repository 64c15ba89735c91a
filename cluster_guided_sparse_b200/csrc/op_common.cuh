// Shared by the operators around the sparse attention (rope_op.cu, cross_*.cu,
// ops_api.cu): 8-element row chunks of the three float types, and the host
// launchers.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace scope {
namespace op {

// ---------------------------------------------------------------- 8 consecutive elements as fp32
__device__ __forceinline__ void load8(const float *p, float *x)
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *x)
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void load8(const __half *p, float *x)
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const __half2 *h = reinterpret_cast<const __half2 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The same in two steps: the bits, and later their values (half the registers of
// a load in flight for 16-bit types).
template <typename T>
struct Raw8 {
    uint4 u;
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void values(float *x) const { load8(reinterpret_cast<const T *>(&u), x); }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void values(float *x) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

__device__ __forceinline__ void store8(float *p, const float *x)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack2(__half, float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float *x)
{
    uint4 u;
    u.x = pack2(T(), x[0], x[1]);
    u.y = pack2(T(), x[2], x[3]);
    u.z = pack2(T(), x[4], x[5]);
    u.w = pack2(T(), x[6], x[7]);
    *reinterpret_cast<uint4 *>(p) = u;
}

// ---------------------------------------------------------------- launches
// The kernels of a call follow each other by programmatic launch: the next one's
// blocks come to the SMs as this one's leave them, and wait before they read
// anything until it has ended.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Args, typename... Given>
void launch_next(void (*kernel)(Args...), int64_t blocks, int threads, size_t smem, cudaStream_t st, const Given &...given)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, Args(given)...);
    count_launches(1);
}

// ---------------------------------------------------------------- rotary positions (rope_op.cu)
// Turns (1 = a full rotation) per unit of position of each pair of the head
// dim; pairs [0, pt) belong to the t axis, [pt, pt + ph) to h, the rest to w.
struct RopeTurns {
    double turns[64];
    int pt, ph;
};

struct RopeArgs {
    const void *x, *dy;       // backward reads both
    void *y;                  // forward: y, backward: dx
    int64_t xB, xH, xN, dB, dH, dN, yB, yH, yN;  // element strides of x, dy, y
    const int32_t *positions; // [pos_B][N][3], or null: raster order of the grid
    int64_t posB;             // elements between batch entries (0: shared by the batch)
    int Hh, W;
    const void *weight;       // [D] or null
    int w_dtype;              // scope_dtype of weight and dw
    float eps;
    float sign;               // +1 forward, -1 the inverse rotation
    int H, N, D;
    int64_t tokens;           // B * N
    int heads_per_block;
    float *dw_part;           // backward: [blocks][D]
};

void launch_rope_op(const RopeArgs &a, const RopeTurns &t, int dtype, cudaStream_t st);
int rope_bwd_blocks(int64_t tokens, int H, int D, int *heads_per_block);
void launch_rope_op_bwd(RopeArgs a, const RopeTurns &t, int dtype, void *dw, cudaStream_t st);

}  // namespace op
}  // namespace scope
