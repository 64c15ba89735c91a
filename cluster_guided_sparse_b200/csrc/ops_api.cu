// Host side of the operators around the sparse attention: argument checks,
// workspace layout and launches.  Every argument check runs before any CUDA
// call.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/scope.h"
#include "cross_common.cuh"

scope_status scope_set_error(scope_status s, const char *msg);

namespace scope {
void launch_wait_timeout(int32_t *err, long long limit, cudaStream_t st);
namespace op {
bool check_tensor(const scope_tensor *t, const char *name, int64_t min_n, scope_status *st);
RowStrides strides_of(const scope_tensor *t);
}  // namespace op
}  // namespace scope

using namespace scope;

namespace {

scope_status fail(scope_status s, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return scope_set_error(s, buf);
}

bool same_shape(const scope_tensor *a, const scope_tensor *b)
{
    return a->B == b->B && a->H == b->H && a->N == b->N && a->D == b->D;
}

// Written in place: the very same rows.
bool same_rows(const scope_tensor *a, const scope_tensor *b)
{
    const RowStrides x = op::strides_of(a), y = op::strides_of(b);
    return (a->B == 1 || x.sB == y.sB) && (a->H == 1 || x.sH == y.sH) && (a->N == 1 || x.sN == y.sN);
}

scope_status check_over(const scope_tensor *out, const scope_tensor *in, const char *names)
{
    if (out->ptr == in->ptr && out->N > 0 && !same_rows(out, in))
        return fail(SCOPE_EINVAL, "%s: same memory with other strides", names);
    return SCOPE_OK;
}

bool float_type(int t) { return t == SCOPE_F32 || t == SCOPE_BF16 || t == SCOPE_F16; }

size_t take(size_t &cur, size_t bytes)
{
    const size_t at = cur;
    cur += (bytes + 255) & ~(size_t)255;
    return at;
}

scope_status check_workspace(const void *ws, size_t have, size_t need)
{
    if (!ws) return fail(SCOPE_EWORKSPACE, "workspace: null");
    if (((uintptr_t)ws) & 255) return fail(SCOPE_EALIGN, "workspace must be 256-byte aligned");
    if (have < need) return fail(SCOPE_EWORKSPACE, "workspace too small: %zu < %zu bytes", have, need);
    return SCOPE_OK;
}

// The current device is an sm_100 one.  (A stream of another device makes the
// launch itself fail; asking for a stream's device would end a capture.)
scope_status check_device()
{
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(SCOPE_EDEVICE, "no CUDA device");
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (major != 10)
        return fail(SCOPE_EDEVICE, "libscope.so is built for sm_100a; device has compute capability %d.x", major);
    return SCOPE_OK;
}

scope_status launch_status(const char *what)
{
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(SCOPE_ECUDA, "%s: %s", what, cudaGetErrorString(e));
    return SCOPE_OK;
}

// ---------------------------------------------------------------- rotary positions
scope_status check_rope(const scope_tensor *x, const scope_grid *g, const scope_params *p, const scope_positions *pos)
{
    if (!p) return fail(SCOPE_EINVAL, "params: null");
    const int ds[3] = {p->d_t, p->d_h, p->d_w};
    for (int s = 0; s < 3; ++s)
        if (ds[s] < 0 || (ds[s] & 1)) return fail(SCOPE_ESHAPE, "params: d_t/d_h/d_w must be even and >= 0");
    if ((int64_t)ds[0] + ds[1] + ds[2] != x->D) return fail(SCOPE_ESHAPE, "params: d_t + d_h + d_w must equal D");
    if (!(p->theta > 0.0) || !std::isfinite(p->theta)) return fail(SCOPE_EINVAL, "params: theta must be finite and > 0");
    const bool has_grid = g && (g->T || g->Hh || g->W);
    if (pos) {
        if (has_grid) return fail(SCOPE_EINVAL, "give a grid or positions, not both");
        if (!pos->ptr && x->N) return fail(SCOPE_EINVAL, "positions: null data pointer");
        if (((uintptr_t)pos->ptr) & 3) return fail(SCOPE_EALIGN, "positions: pointer not 4-byte aligned");
        if (pos->B != 1 && pos->B != x->B) return fail(SCOPE_ESHAPE, "positions: B must be 1 or that of x");
        return SCOPE_OK;
    }
    if (!has_grid) return fail(SCOPE_EINVAL, "give a grid or positions");
    if (g->T < 1 || g->Hh < 1 || g->W < 1 || (int64_t)g->Hh * g->W > x->N || (int64_t)g->T * g->Hh * g->W != x->N)
        return fail(SCOPE_ESHAPE, "grid: T*Hh*W must equal N");
    return SCOPE_OK;
}

scope_status check_weight(const scope_vector *w, const char *name, float eps)
{
    if (!w->ptr) return fail(SCOPE_EINVAL, "%s: null data pointer", name);
    if (!float_type(w->dtype)) return fail(SCOPE_EDTYPE, "%s: dtype must be f32, bf16 or f16", name);
    if (((uintptr_t)w->ptr) & (w->dtype == SCOPE_F32 ? 3 : 1)) return fail(SCOPE_EALIGN, "%s: pointer not aligned", name);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(SCOPE_EINVAL, "eps must be finite and >= 0");
    return SCOPE_OK;
}

// The last call's angles of this thread serve again where their parameters are the same: 64 powers take longer
// than a small call's kernel.
const op::RopeTurns &rope_turns(const scope_params *p)
{
    static thread_local op::RopeTurns t;
    static thread_local int32_t ds[3];
    static thread_local double theta = 0.0;  // never valid
    if (theta == p->theta && ds[0] == p->d_t && ds[1] == p->d_h && ds[2] == p->d_w) return t;
    theta = p->theta;
    ds[0] = p->d_t;
    ds[1] = p->d_h;
    ds[2] = p->d_w;
    t = op::RopeTurns{};
    t.pt = p->d_t / 2;
    t.ph = p->d_h / 2;
    int at = 0;
    for (int s = 0; s < 3; ++s)
        for (int i = 0; i < ds[s] / 2; ++i)
            t.turns[at++] = std::pow(p->theta, -2.0 * i / ds[s]) / (2.0 * M_PI);
    return t;
}

op::RopeArgs rope_args(const scope_tensor *x, const scope_grid *g, const scope_positions *pos, const scope_vector *w,
                       float eps, const scope_tensor *y)
{
    op::RopeArgs a{};
    const RowStrides xs = op::strides_of(x), ys = op::strides_of(y);
    a.x = x->ptr;
    a.y = y->ptr;
    a.xB = xs.sB; a.xH = xs.sH; a.xN = xs.sN;
    a.yB = ys.sB; a.yH = ys.sH; a.yN = ys.sN;
    a.Hh = 1;
    a.W = 1;
    if (pos) {
        a.positions = pos->ptr;
        a.posB = pos->B > 1 ? x->N * 3 : 0;
    } else {
        a.Hh = g->Hh;
        a.W = g->W;
    }
    if (w) {
        a.weight = w->ptr;
        a.w_dtype = w->dtype;
        a.eps = eps;
    }
    a.sign = 1.f;
    a.H = (int)x->H;
    a.N = (int)x->N;
    a.D = (int)x->D;
    a.tokens = x->B * x->N;
    return a;
}

size_t rope_bwd_bytes(const scope_tensor *x)
{
    int hpb;
    return 256 + (size_t)op::rope_bwd_blocks(x->B * x->N, (int)x->H, (int)x->D, &hpb) * x->D * 4;
}

}  // namespace

extern "C" scope_status scope_rope(const scope_tensor *x, const scope_grid *grid, const scope_params *p,
                                   const scope_positions *pos, const scope_vector *weight, float eps, int inverse,
                                   scope_tensor *y, void *stream)
{
    scope_status st;
    if (!op::check_tensor(x, "x", 0, &st) || !op::check_tensor(y, "y", 0, &st)) return st;
    if (!same_shape(x, y)) return fail(SCOPE_ESHAPE, "x and y shapes differ");
    if (x->dtype != y->dtype) return fail(SCOPE_EDTYPE, "x and y dtypes differ");
    if ((st = check_over(y, x, "y, x")) != SCOPE_OK) return st;
    if ((st = check_rope(x, grid, p, pos)) != SCOPE_OK) return st;
    if (inverse != 0 && inverse != 1) return fail(SCOPE_EINVAL, "inverse must be 0 or 1");
    if (weight) {
        if ((st = check_weight(weight, "weight", eps)) != SCOPE_OK) return st;
        if (inverse) return fail(SCOPE_EINVAL, "inverse does not go with a weight (see scope_rope_backward)");
    }
    if (x->N == 0) return SCOPE_OK;
    if ((st = check_device()) != SCOPE_OK) return st;
    op::RopeArgs a = rope_args(x, grid, pos, weight, eps, y);
    if (inverse) a.sign = -1.f;
    op::launch_rope_op(a, rope_turns(p), x->dtype, (cudaStream_t)stream);
    return launch_status("scope_rope");
}

extern "C" size_t scope_rope_backward_workspace_bytes(const scope_tensor *x)
{
    scope_status st;
    if (!op::check_tensor(x, "x", 0, &st)) return 0;
    return rope_bwd_bytes(x);
}

extern "C" scope_status scope_rope_backward(const scope_tensor *dy, const scope_tensor *x, const scope_grid *grid,
                                            const scope_params *p, const scope_positions *pos,
                                            const scope_vector *weight, float eps, scope_tensor *dx, scope_vector *dw,
                                            void *workspace, size_t ws_bytes, void *stream)
{
    scope_status st;
    if (!op::check_tensor(dy, "dy", 0, &st) || !op::check_tensor(x, "x", 0, &st) || !op::check_tensor(dx, "dx", 0, &st))
        return st;
    if (!same_shape(x, dy) || !same_shape(x, dx)) return fail(SCOPE_ESHAPE, "x, dy and dx shapes differ");
    if (x->dtype != dy->dtype || x->dtype != dx->dtype) return fail(SCOPE_EDTYPE, "x, dy and dx dtypes differ");
    if ((st = check_over(dx, x, "dx, x")) != SCOPE_OK || (st = check_over(dx, dy, "dx, dy")) != SCOPE_OK) return st;
    if ((st = check_rope(x, grid, p, pos)) != SCOPE_OK) return st;
    if (!weight || !dw) return fail(SCOPE_EINVAL, "weight, dw: null (without a norm the gradient is scope_rope, inverse = 1)");
    if ((st = check_weight(weight, "weight", eps)) != SCOPE_OK) return st;
    if ((st = check_weight(dw, "dw", eps)) != SCOPE_OK) return st;
    if (dw->dtype != weight->dtype) return fail(SCOPE_EDTYPE, "weight and dw dtypes differ");
    if (dw->ptr == weight->ptr) return fail(SCOPE_EINVAL, "dw may not overlap weight");
    if ((st = check_workspace(workspace, ws_bytes, rope_bwd_bytes(x))) != SCOPE_OK) return st;
    if ((st = check_device()) != SCOPE_OK) return st;
    if (x->N == 0) {
        cudaMemsetAsync(dw->ptr, 0, (size_t)x->D * (dw->dtype == SCOPE_F32 ? 4 : 2), (cudaStream_t)stream);
        return launch_status("scope_rope_backward");
    }
    op::RopeArgs a = rope_args(x, grid, pos, weight, eps, dx);
    const RowStrides ds = op::strides_of(dy);
    a.dy = dy->ptr;
    a.dB = ds.sB; a.dH = ds.sH; a.dN = ds.sN;
    a.dw_part = (float *)workspace;
    op::launch_rope_op_bwd(a, rope_turns(p), x->dtype, dw->ptr, (cudaStream_t)stream);
    return launch_status("scope_rope_backward");
}

// ---------------------------------------------------------------- cross attention
namespace {

constexpr int kSms = 148;  // of a B200; work is split for this many whatever part of one is visible

scope_status check_keys(const scope_tensor *k, const scope_keys *keys)
{
    if (!keys) return SCOPE_OK;
    if (keys->len && keys->mask) return fail(SCOPE_EINVAL, "keys: give a length or a mask, not both");
    if (((uintptr_t)keys->len) & 3) return fail(SCOPE_EALIGN, "keys: len not 4-byte aligned");
    if (keys->mask && keys->mask_stride < 0)
        return fail(SCOPE_ESHAPE, "keys: mask_stride must be >= 0");
    return SCOPE_OK;
}

scope_status check_qk(const scope_tensor *q, const scope_tensor *k)
{
    scope_status st;
    if (!op::check_tensor(q, "q", 0, &st) || !op::check_tensor(k, "k", 0, &st)) return st;
    if (q->dtype == SCOPE_F32) return fail(SCOPE_EDTYPE, "q: dtype must be bf16 or f16");
    if (q->dtype != k->dtype) return fail(SCOPE_EDTYPE, "q and k dtypes differ");
    if (q->D != k->D) return fail(SCOPE_ESHAPE, "q and k head dims differ");
    if (k->B != q->B && k->B != 1) return fail(SCOPE_ESHAPE, "k: B must be 1 or that of q");
    if (q->H % k->H) return fail(SCOPE_ESHAPE, "the key heads must divide the query heads");
    if (q->B * q->H * q->N > ((int64_t)1 << 30)) return fail(SCOPE_ESHAPE, "q: B*H*N must be <= 2^30");
    return SCOPE_OK;
}

scope_status check_cross(const scope_tensor *q, const scope_tensor *k, const scope_tensor *v, const scope_keys *keys,
                         float scale)
{
    scope_status st;
    if ((st = check_qk(q, k)) != SCOPE_OK) return st;
    if (!op::check_tensor(v, "v", 0, &st)) return st;
    if (!same_shape(k, v)) return fail(SCOPE_ESHAPE, "k and v shapes differ");
    if (v->dtype != k->dtype) return fail(SCOPE_EDTYPE, "k and v dtypes differ");
    if ((st = check_keys(k, keys)) != SCOPE_OK) return st;
    if (scale != 0.f && !(scale >= 1e-30f && scale <= 1e30f))
        return fail(SCOPE_EINVAL, "scale must be 0 (1/sqrt(D)) or in [1e-30, 1e30]");
    return SCOPE_OK;
}

// `t` has the shape and dtype of `like`.
scope_status check_as(const scope_tensor *t, const char *name, const scope_tensor *like, const char *like_name)
{
    scope_status st;
    if (!op::check_tensor(t, name, 0, &st)) return st;
    if (!same_shape(t, like)) return fail(SCOPE_ESHAPE, "%s and %s shapes differ", name, like_name);
    if (t->dtype != like->dtype) return fail(SCOPE_EDTYPE, "%s and %s dtypes differ", name, like_name);
    return SCOPE_OK;
}

// No two of an output and any other tensor start at one address.
scope_status check_apart(const scope_tensor *const *t, int n, int outputs)
{
    for (int i = 0; i < outputs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (t[i]->ptr && t[i]->ptr == t[j]->ptr)
                return fail(SCOPE_EINVAL, "an output may not overlap another tensor");
    return SCOPE_OK;
}

scope_status cross_ready()
{
    const scope_status st = check_device();
    if (st != SCOPE_OK) return st;
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && configured[dev]) return SCOPE_OK;
    if (op::cross_fwd_configure() != cudaSuccess || op::cross_bwd_configure() != cudaSuccess ||
        op::cross_few_configure() != cudaSuccess)
        return fail(SCOPE_ECUDA, "kernel attribute setup failed");
    if (dev < 64) configured[dev] = true;
    return SCOPE_OK;
}

// Offsets into the workspace.
struct CrossLayout {
    size_t idx, cnt, part_o, part_lse, total;
};

op::CrossArgs cross_sizes(const scope_tensor *q, const scope_tensor *k)
{
    op::CrossArgs a{};
    a.B = (int)q->B; a.Bk = (int)k->B; a.H = (int)q->H; a.Hk = (int)k->H; a.N = (int)q->N; a.M = (int)k->N;
    a.G = a.H / a.Hk;
    a.heads = a.Bk == a.B ? a.G : a.B * a.G;
    a.sets = a.Bk * a.Hk;
    // Tiles by head waste up to 127 rows a head, folded ones cost copies by
    // threads instead of TMA.
    const int padded = (a.N + 127) / 128 * 128;
    a.fold = a.heads > 1 && padded > 1.25 * a.N;
    const int rows = a.heads * a.N;
    a.pairs = a.fold ? (rows + 255) / 256 : a.heads * ((a.N + 255) / 256);
    a.tiles = a.fold ? (rows + 127) / 128 : a.heads * (padded / 128);
    a.by_N = op::Div(a.N);
    a.by_G = op::Div(a.G);
    a.by_Hk = op::Div(a.Hk);
    return a;
}

CrossLayout cross_layout(op::CrossArgs &a, int D, bool masked)
{
    CrossLayout L{};
    L.total = 256;
    a.few_ranks = op::cross_few_ranks(a.sets, (int64_t)a.heads * a.N, a.M, false, kSms);
    if (a.few_ranks) return L;
    const int64_t total = (int64_t)a.B * a.H * a.N;
    a.splits = op::cross_fwd_splits(a.sets, a.pairs, a.M, total, D, kSms);
    a.items = a.sets * a.splits * a.pairs;
    a.by_per = op::Div((a.N + 255) / 256);
    a.by_tiles = op::Div(a.pairs);
    a.by_splits = op::Div(a.splits);
    size_t cur = 256;
    L.idx = take(cur, masked ? (size_t)a.Bk * a.M * 4 : 0);
    L.cnt = take(cur, masked ? (size_t)a.Bk * 4 : 0);
    L.part_o = take(cur, a.splits > 1 ? (size_t)a.splits * total * D * 4 : 0);
    L.part_lse = take(cur, a.splits > 1 ? (size_t)a.splits * total * 4 : 0);
    L.total = cur;
    return L;
}

struct CrossBwdLayout {
    size_t idx, cnt, inv, nlse, ndelta, part_t, part_e, part_delta, part_dk, part_dv, total;
};

CrossBwdLayout cross_bwd_layout(op::CrossArgs &a, int D, bool masked)
{
    CrossBwdLayout L{};
    L.total = 256;
    a.few_ranks = op::cross_few_ranks(a.sets, (int64_t)a.heads * a.N, a.M, true, kSms);
    if (a.few_ranks) return L;
    const int64_t total = (int64_t)a.B * a.H * a.N;
    a.dq_splits = op::cross_dq_splits(a.sets, a.tiles, a.M, total, D, kSms);
    a.dkv_splits = op::cross_dkv_splits(a.sets, a.tiles, a.M, D, kSms);
    a.by_per = op::Div((a.N + 127) / 128);
    a.by_tiles = op::Div(a.tiles);
    a.by_splits = op::Div(a.dq_splits);
    a.by_dkv_splits = op::Div(a.dkv_splits);
    size_t cur = 256;
    const size_t keys = masked ? (size_t)a.Bk * a.M * 4 : 0, rows = (size_t)a.sets * a.tiles * 128 * 4;
    L.idx = take(cur, keys);
    L.inv = take(cur, keys);
    L.cnt = take(cur, masked ? (size_t)a.Bk * 4 : 0);
    L.nlse = take(cur, rows);
    L.ndelta = take(cur, rows);
    const size_t rows_split = a.dq_splits > 1 ? (size_t)a.dq_splits * total * 4 : 0;
    L.part_t = take(cur, rows_split * D);
    L.part_e = take(cur, rows_split * D);
    L.part_delta = take(cur, rows_split);
    const size_t parts = (size_t)a.dkv_splits * a.sets * a.M * D * 4;
    L.part_dk = take(cur, parts);
    L.part_dv = take(cur, parts);
    L.total = cur;
    return L;
}

// Every row of a tensor of 16-bit elements starts on 32 bytes.
bool rows_on_32(const scope_tensor *t, const RowStrides &s)
{
    return !(((uintptr_t)t->ptr | (uintptr_t)(2 * ((t->B > 1 ? s.sB : 0) | (t->H > 1 ? s.sH : 0) | (t->N > 1 ? s.sN : 0)))) & 31);
}

void cross_tensors(op::CrossArgs &a, const scope_tensor *q, const scope_tensor *k, const scope_tensor *v,
                   const scope_tensor *o, const scope_keys *keys, float scale)
{
    const RowStrides qs = op::strides_of(q), ks = op::strides_of(k), vs = op::strides_of(v), os = op::strides_of(o);
    a.q = q->ptr; a.k = k->ptr; a.v = v->ptr; a.o = o->ptr;
    a.qB = qs.sB; a.qH = qs.sH; a.qN = qs.sN;
    a.kB = ks.sB; a.kH = ks.sH; a.kN = ks.sN;
    a.vB = vs.sB; a.vH = vs.sH; a.vN = vs.sN;
    a.oB = os.sB; a.oH = os.sH; a.oN = os.sN;
    a.kv_len = keys ? keys->len : nullptr;
    a.mask = keys ? keys->mask : nullptr;
    a.mask_stride = keys ? keys->mask_stride : 0;
    a.scale = scale != 0.f ? scale : 1.f / std::sqrt((float)q->D);
    a.scale_log2 = a.scale * 1.4426950408889634f;
    a.wide = rows_on_32(o, os);
}

// Tensor map of boxes of `rows` rows x 64 columns; false where TMA cannot address the
// layout (a stride of 2^40 bytes or more).
bool tile_map(CUtensorMap *m, const scope_tensor *t, int rows)
{
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<Encode> found{nullptr};
    Encode encode = found;
    if (!encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess || !fn)
            return false;
        found = encode = (Encode)fn;
    }
    const RowStrides s = op::strides_of(t);
    // a dimension of one entry may have any stride
    const int64_t ext[3] = {t->N, t->H, t->B}, str[3] = {s.sN, s.sH, s.sB};
    cuuint64_t dims[4] = {(cuuint64_t)t->D}, strides[3];
    for (int i = 0; i < 3; ++i) {
        dims[i + 1] = (cuuint64_t)ext[i];
        strides[i] = (cuuint64_t)(ext[i] > 1 ? str[i] : t->D) * 2;
        if (strides[i] >= (cuuint64_t)1 << 40) return false;
    }
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
    return encode(m, t->dtype == SCOPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t->ptr,
                  dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps that a call's kernels use; what has none is copied by threads.
// d: do, in the backward pass; o: what the rows' kernel writes, o or dq.
void cross_maps(op::CrossArgs &a, op::CrossMaps &m, const scope_tensor *q, const scope_tensor *k, const scope_tensor *v,
                const scope_tensor *d, const scope_tensor *o)
{
    const int keys = d ? 128 : op::kFwdKeys;
    a.tma_kv = a.M > 0 && !a.idx && tile_map(&m.k, k, keys) && tile_map(&m.v, v, keys);
    a.tma_rows = !a.fold && a.N > 0 && tile_map(&m.q, q, 128) && (!d || tile_map(&m.d, d, 128));
    a.tma_o = !a.fold && a.N > 0 && tile_map(&m.o, o, 32);
}

}  // namespace

extern "C" size_t scope_cross_attn_workspace_bytes(const scope_tensor *q, const scope_tensor *k, int masked)
{
    if (check_qk(q, k) != SCOPE_OK) return 0;
    op::CrossArgs a = cross_sizes(q, k);
    return cross_layout(a, (int)q->D, masked != 0).total;
}

extern "C" scope_status scope_cross_attn(const scope_tensor *q, const scope_tensor *k, const scope_tensor *v,
                                         const scope_keys *keys, float scale, scope_tensor *o, float *lse,
                                         void *workspace, size_t ws_bytes, void *stream)
{
    scope_status st;
    if ((st = check_cross(q, k, v, keys, scale)) != SCOPE_OK) return st;
    if ((st = check_as(o, "o", q, "q")) != SCOPE_OK) return st;
    const scope_tensor *all[4] = {o, q, k, v};
    if ((st = check_apart(all, 4, 1)) != SCOPE_OK) return st;
    if (((uintptr_t)lse) & 3) return fail(SCOPE_EALIGN, "lse: pointer not 4-byte aligned");
    op::CrossArgs a = cross_sizes(q, k);
    const bool masked = keys && keys->mask;
    const CrossLayout L = cross_layout(a, (int)q->D, masked);
    if ((st = check_workspace(workspace, ws_bytes, L.total)) != SCOPE_OK) return st;
    if (q->N == 0) return SCOPE_OK;
    if ((st = cross_ready()) != SCOPE_OK) return st;
    cross_tensors(a, q, k, v, o, keys, scale);
    a.lse = lse;
    char *ws = (char *)workspace;
    a.part_o = (float *)(ws + L.part_o);
    a.part_lse = (float *)(ws + L.part_lse);
    cudaStream_t s = (cudaStream_t)stream;
    if (a.few_ranks) {
        op::launch_cross_few(a, (int)q->D, q->dtype == SCOPE_F16, false, s);
        return launch_status("scope_cross_attn");
    }
    if (masked) {
        int32_t *idx = (int32_t *)(ws + L.idx), *cnt = (int32_t *)(ws + L.cnt);
        op::launch_key_lists(keys->mask, keys->mask_stride, a.Bk, a.M, idx, cnt, nullptr, s);
        a.idx = idx;
        a.cnt = cnt;
    }
    op::CrossMaps m;
    cross_maps(a, m, q, k, v, nullptr, o);
    op::launch_cross_fwd(a, m, (int)q->D, q->dtype == SCOPE_F16, kSms, s);
    return launch_status("scope_cross_attn");
}

extern "C" size_t scope_cross_attn_backward_workspace_bytes(const scope_tensor *q, const scope_tensor *k, int masked)
{
    if (check_qk(q, k) != SCOPE_OK) return 0;
    op::CrossArgs a = cross_sizes(q, k);
    return cross_bwd_layout(a, (int)q->D, masked != 0).total;
}

extern "C" scope_status scope_cross_attn_backward(const scope_tensor *d_o, const scope_tensor *q, const scope_tensor *k,
                                                  const scope_tensor *v, const scope_tensor *o, const float *lse,
                                                  const scope_keys *keys, float scale, scope_tensor *dq,
                                                  scope_tensor *dk, scope_tensor *dv, void *workspace, size_t ws_bytes,
                                                  void *stream)
{
    scope_status st;
    if ((st = check_cross(q, k, v, keys, scale)) != SCOPE_OK) return st;
    if ((st = check_as(d_o, "d_o", q, "q")) != SCOPE_OK || (st = check_as(o, "o", q, "q")) != SCOPE_OK ||
        (st = check_as(dq, "dq", q, "q")) != SCOPE_OK || (st = check_as(dk, "dk", k, "k")) != SCOPE_OK ||
        (st = check_as(dv, "dv", k, "k")) != SCOPE_OK)
        return st;
    const scope_tensor *all[8] = {dq, dk, dv, d_o, q, k, v, o};
    if ((st = check_apart(all, 8, 3)) != SCOPE_OK) return st;
    if (!lse && q->N) return fail(SCOPE_EINVAL, "lse: null data pointer");
    if (((uintptr_t)lse) & 3) return fail(SCOPE_EALIGN, "lse: pointer not 4-byte aligned");
    op::CrossArgs a = cross_sizes(q, k);
    const bool masked = keys && keys->mask;
    const CrossBwdLayout L = cross_bwd_layout(a, (int)q->D, masked);
    if ((st = check_workspace(workspace, ws_bytes, L.total)) != SCOPE_OK) return st;
    if (q->N == 0 && k->N == 0) return SCOPE_OK;
    if ((st = cross_ready()) != SCOPE_OK) return st;
    cross_tensors(a, q, k, v, o, keys, scale);
    const RowStrides ds = op::strides_of(d_o), qs = op::strides_of(dq), ks = op::strides_of(dk), vs = op::strides_of(dv);
    a.dout = d_o->ptr;
    a.dB = ds.sB; a.dH = ds.sH; a.dN = ds.sN;
    a.dq = dq->ptr;
    a.dqB = qs.sB; a.dqH = qs.sH; a.dqN = qs.sN;
    a.wide = rows_on_32(dq, qs);
    a.lse = const_cast<float *>(lse);  // read only here
    char *ws = (char *)workspace;
    a.nlse = (float *)(ws + L.nlse);
    a.ndelta = (float *)(ws + L.ndelta);
    a.part_t = (float *)(ws + L.part_t);
    a.part_e = (float *)(ws + L.part_e);
    a.part_delta = (float *)(ws + L.part_delta);
    a.part_dk = (float *)(ws + L.part_dk);
    a.part_dv = (float *)(ws + L.part_dv);
    a.dk = dk->ptr;
    a.dkB = ks.sB; a.dkH = ks.sH; a.dkN = ks.sN;
    a.dv = dv->ptr;
    a.dvB = vs.sB; a.dvH = vs.sH; a.dvN = vs.sN;
    cudaStream_t s = (cudaStream_t)stream;
    if (a.few_ranks) {
        op::launch_cross_few(a, (int)q->D, q->dtype == SCOPE_F16, true, s);
        return launch_status("scope_cross_attn_backward");
    }
    int32_t *inv = nullptr;
    if (masked) {
        int32_t *idx = (int32_t *)(ws + L.idx), *cnt = (int32_t *)(ws + L.cnt);
        inv = (int32_t *)(ws + L.inv);
        op::launch_key_lists(keys->mask, keys->mask_stride, a.Bk, a.M, idx, cnt, inv, s);
        a.idx = idx;
        a.cnt = cnt;
    }
    op::CrossMaps m;
    cross_maps(a, m, q, k, v, d_o, dq);
    op::launch_cross_bwd(a, m, (int)q->D, q->dtype == SCOPE_F16, kSms, inv, s);
    return launch_status("scope_cross_attn_backward");
}

extern "C" scope_status scope_ops_sync_status(void *stream)
{
    const scope_status st = check_device();
    if (st != SCOPE_OK) return st;
    cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return fail(SCOPE_ECUDA, "stream: %s", cudaGetErrorString(e));
    int32_t err[4] = {0, 0, 0, 0};
    e = op::cross_fwd_error(err, true);
    int32_t bwd[4] = {0, 0, 0, 0};
    if (e == cudaSuccess) e = op::cross_bwd_error(bwd, true);
    if (!err[1]) err[1] = bwd[1];
    err[0] |= bwd[0];
    if (e != cudaSuccess) return fail(SCOPE_ECUDA, "reading the error word: %s", cudaGetErrorString(e));
    if (err[0] & kErrTimeout) return fail(SCOPE_ETIMEOUT, "a bounded device wait gave up (detail 0x%x)", err[1]);
    if (err[0]) return fail(SCOPE_EDEVICE, "device range check fired (flags 0x%x, detail 0x%x)", err[0], err[1]);
    return SCOPE_OK;
}

extern "C" scope_status scope_ops_selftest_wait_timeout(int backward, int64_t wait_cycles, void *stream)
{
    if (backward != 0 && backward != 1) return fail(SCOPE_EINVAL, "backward must be 0 or 1");
    if (wait_cycles < 1000 || wait_cycles > 4000000000ll)
        return fail(SCOPE_EINVAL, "wait_cycles must be in [1e3, 4e9]");
    const scope_status st = check_device();
    if (st != SCOPE_OK) return st;
    int32_t *err = backward ? op::cross_bwd_error_word() : op::cross_fwd_error_word();
    if (!err) return fail(SCOPE_ECUDA, "no address of the error word");
    launch_wait_timeout(err, (long long)wait_cycles, (cudaStream_t)stream);
    return launch_status("scope_ops_selftest_wait_timeout");
}
