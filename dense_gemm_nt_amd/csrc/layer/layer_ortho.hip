// layer_ortho.hip -- the orthogonalized update of a weight: Newton-Schulz products.
//
//   X = G / (||G|| + eps), r x k with r <= k (a tall G's transpose), then `steps` times
//   A = X X^T,  X = a X + (b A + c A^2) X
// which takes every singular value s of X to a s + b s^3 + c s^5.
//
// Numbers.  The products run on FP16 operands with FP32 sums; X itself is kept in FP32, and
// its FP16 copy (in units of 1 / s, s the power of two near sqrt(k), so that entries of
// 1 / sqrt(r k) are not below fp16's steps) only enters the products, so an X of steep spectrum, whose
// small singular values the first steps multiply by a alone, keeps them: with X in FP16
// a spectrum falling as 1 / i ended 2.9e-3 off, so 0.5e-3.  From the third step on, when the singular
// values are near 1, the squares are held as what they differ from the identity by:
//   A = I + A':  b A + c A^2 = (b + c) I + (b + 2 c) A' + c A'^2
// whose diagonal does not fill FP16's bits with what is known already; the multiple of I goes
// into X's factor, exactly (a random 512 x 512: 1.5e-3 off without, 0.9e-3 with).  A BF16
// result's rounding is 1.7e-3 by itself; iterates in BF16 would be 1e-2 off.
#include "layer_host.hpp"
#include "ortho_common.hpp"

namespace gnt {

hipError_t launch_ortho(const OrthoArgs &a, int tile, bool mn_major, unsigned grid, hipStream_t s);

constexpr int kOrthoParts = 1024;          // partial sums of squares of a stack, at most

__device__ __forceinline__ float read_any(const void *x, int64_t i, int dtype)
{
    return dtype == OUT_FP32 ? static_cast<const float *>(x)[i]
                             : from_bits16(dtype, static_cast<const uint16_t *>(x)[i]);
}

__device__ __forceinline__ double block_sum(double v, double *part)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    if (threadIdx.x % 64 == 0)
        part[threadIdx.x / 64] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

// Partial sums of squares, in FP64 (an FP32 gradient's squares leave FP32's range on both
// sides): block (i, b) takes every gridDim.x-th row of matrix b.
__global__ __launch_bounds__(256) void ortho_squares(const void *G, int m, int n, int64_t ld, int64_t step, int dtype,
                                                     double *parts)
{
    __shared__ double part[4];
    double s = 0.0;
    for (int r = blockIdx.x; r < m; r += gridDim.x) {
        const int64_t row = blockIdx.y * step + (int64_t)r * ld;
        for (int c = threadIdx.x; c < n; c += 256) {
            const double v = read_any(G, row + c, dtype);
            s += v * v;
        }
    }
    s = block_sum(s, part);
    if (threadIdx.x == 0)
        parts[blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// X = G / (||G|| + eps) in FP32 and, times s, in FP16, [rows8][cols8] with zeros past the
// matrix; a tall G (flip) is transposed on the way.  A block has 64 x 64 values.
__global__ __launch_bounds__(256) void ortho_begin(const void *G, int m, int n, int64_t ld, int64_t step, int dtype,
                                                   int flip, const double *parts, int num_parts, double eps, float s,
                                                   float *x, uint16_t *xh, int rows8, int cols8)
{
    __shared__ double part[4];
    __shared__ float tile[64][65];
    double sum = 0.0;
    for (int i = threadIdx.x; i < num_parts; i += 256)
        sum += parts[blockIdx.z * num_parts + i];
    const double inv = 1.0 / (__builtin_sqrt(block_sum(sum, part)) + eps);
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;         // of X
    const int g_r0 = flip ? c0 : r0, g_c0 = flip ? r0 : c0;       // of G
    const int64_t from = blockIdx.z * step;
    for (int i = threadIdx.x; i < 4096; i += 256) {
        const int r = g_r0 + (i >> 6), c = g_c0 + (i & 63);
        tile[i >> 6][i & 63] = r < m && c < n ? (float)(read_any(G, from + (int64_t)r * ld + c, dtype) * inv) : 0.0f;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 512; i += 256) {
        const int r = i >> 3, c = (i & 7) * 8;
        if (r0 + r >= rows8 || c0 + c >= cols8)
            continue;
        const int64_t at = (int64_t)blockIdx.z * rows8 * cols8 + (int64_t)(r0 + r) * cols8 + c0 + c;
        float y[8], h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] = flip ? tile[c + e][r] : tile[r][c + e];
            h[e] = s * y[e];
        }
        store_run<OUT_FP32, 8>(x, at, y, true, 8);
        store_run<OUT_FP16, 8>(xh, at, h, true, 8);
    }
}

// The update of no steps at all: X as it begins.
__global__ __launch_bounds__(256) void ortho_copy(const float *x, int rows8, int cols8, OrthoArgs p)
{
    const int m = p.flip ? p.update_cols : p.update_rows, n = p.flip ? p.update_rows : p.update_cols;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= (int64_t)m * n)
        return;
    const int r = (int)(t / n), c = (int)(t - (int64_t)r * n);
    const float v = x[(int64_t)blockIdx.y * rows8 * cols8 + (p.flip ? (int64_t)c * cols8 + r : (int64_t)r * cols8 + c)];
    const int64_t at = blockIdx.y * p.update_step + (int64_t)r * p.ldu + c;
    if (p.update_dtype == OUT_FP32)
        static_cast<float *>(p.update)[at] = v;
    else
        static_cast<uint16_t *>(p.update)[at] =
            (uint16_t)(p.update_dtype == OUT_BF16 ? to_bits16<OUT_BF16>(v) : to_bits16<OUT_FP16>(v));
}

namespace {

struct OrthoPlan {
    int tile, splits;
    Plan plan;               // of one of the stack's matrices
    int64_t blocks;          // of the stack
};

// Tile and K splits of a stack's product.  A pass of the machine takes about 10 + 1.5 us a
// 64-deep slab on the ping-pong tile and 5 + 0.62 on the 128 x 128 one; splits are summed in
// the kernel (two on the ping-pong tile), in about 6 and 3 + s / 2 us, and keep 4 slabs.
OrthoPlan plan_ortho(int64_t batch, int64_t M, int64_t N, int64_t K)
{
    OrthoPlan best{};
    double least = 0.0;
    const int64_t slabs = cdiv(K, 64);
    for (int tile : {256, 128}) {
        const int64_t tm = cdiv(M, tile), tn = cdiv(N, tile), tiles = tm * tn * batch;
        for (int64_t s = 1; s <= (tile == 256 ? 2 : 16) && (s == 1 || slabs / s >= 4); ++s) {
            const int64_t per = cdiv(slabs, s), splits = slabs ? cdiv(slabs, per) : 1;
            if (splits != s || (s > 1 && (tiles * s * tile * tile * 4 > kPartialBytes * 4 || tiles * s > 4 * kNumCUs)))
                continue;
            const double passes = (double)cdiv(tiles * s, kNumCUs);
            const double cost = tile == 256 ? passes * (10 + 1.5 * per) + (s > 1 ? 6 : 0)
                                            : passes * (5 + 0.62 * per) + (s > 1 ? 3 + 0.5 * s : 0);
            if (best.tile == 0 || cost < least) {
                least = cost;
                best.tile = tile;
                best.splits = (int)s;
                Plan &p = best.plan;
                p = Plan{};
                p.tiles_m = (int)tm, p.tiles_n = (int)tn;
                p.k_tiles = (int)slabs;
                p.splits = (int)s;
                p.kt_per_split = (int)per;
                p.group_m = std::min<int>(4, p.tiles_m);
                p.inreduce = s > 1;
                p.ws_bytes = s > 1 ? tiles * s * tile * tile * 4 : 0;
                p.grid = tiles * s;
            }
        }
    }
    best.blocks = best.plan.grid;
    return best;
}

struct OrthoWs {
    int64_t r, k, r8, k8;
    int parts;               // partial sums a matrix
    OrthoPlan plan[3];
    double *sums;
    float *x, *partials;
    uint16_t *xh, *a, *b;
    unsigned *counters;
    int num_counters[3];
    int64_t bytes;
};

OrthoWs carve_ortho(int64_t batch, int64_t m, int64_t n, void *base)
{
    OrthoWs w{};
    Carver c{static_cast<uint8_t *>(base)};
    w.r = std::min(m, n), w.k = std::max(m, n);
    w.r8 = cdiv(w.r, 8) * 8, w.k8 = cdiv(w.k, 8) * 8;
    w.parts = (int)std::max<int64_t>(1, std::min<int64_t>(m, kOrthoParts / std::max<int64_t>(1, batch)));
    w.plan[ORTHO_SQUARE] = plan_ortho(batch, w.r8, w.r8, w.k8);
    w.plan[ORTHO_POLY] = plan_ortho(batch, w.r8, w.r8, w.r8);
    w.plan[ORTHO_STEP] = plan_ortho(batch, w.r8, w.k8, w.r8);
    w.sums = c.take<double>(batch * w.parts);
    w.x = c.take<float>(batch * w.r8 * w.k8);
    w.xh = c.take<uint16_t>(2 * batch * w.r8 * w.k8);      // two, in turn: a step reads one and writes the other
    w.a = c.take<uint16_t>(batch * w.r8 * w.r8);
    w.b = c.take<uint16_t>(batch * w.r8 * w.r8);
    int64_t partial = 0, counters = 0;
    for (int i = 0; i < 3; ++i) {
        const Plan &p = w.plan[i].plan;
        partial = std::max(partial, p.ws_bytes / 4);
        w.num_counters[i] = p.inreduce ? (int)(batch * p.tiles_m * p.tiles_n) : 0;
        counters = std::max<int64_t>(counters, w.num_counters[i]);
    }
    w.partials = c.take<float>(partial);
    w.counters = c.take<unsigned>(counters);               // (each call of a tile leaves them zero)
    w.num_counters[0] = (int)counters;
    w.bytes = c.used;
    return w;
}

gemm_status_t check_sizes(int64_t batch, int64_t m, int64_t n, int in_dtype, int out_dtype)
{
    if (batch < 0 || m < 0 || n < 0)
        return GEMM_ERR_INVALID_ARG;
    if (!is_out(in_dtype) || !is_out(out_dtype))
        return GEMM_ERR_UNSUPPORTED;
    // (a stack's tiles, blocks and counters stay far inside 32 bits)
    if (batch > 65535 || m > (1 << 20) || n > (1 << 20))
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

}  // namespace
}  // namespace gnt

using namespace gnt;

extern "C" {

gemm_status_t gemm_orthogonalize_workspace(int64_t batch, int64_t m, int64_t n, int64_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = check_sizes(batch, m, n, GEMM_FP32, GEMM_FP32);
    if (st != GEMM_OK)
        return st;
    *bytes = batch && m && n ? carve_ortho(batch, m, n, nullptr).bytes : 0;
    return GEMM_OK;
}

gemm_status_t gemm_run_orthogonalize(const void *G, void *U, int64_t batch, int64_t m, int64_t n, int64_t ldg,
                                     int64_t ldu, int64_t g_step, int64_t u_step, int in_dtype, int out_dtype,
                                     int64_t steps, const float *coefficients, double eps, void *workspace,
                                     int64_t workspace_bytes, hipStream_t stream)
{
    gemm_status_t st = check_sizes(batch, m, n, in_dtype, out_dtype);
    if (st != GEMM_OK)
        return st;
    if (steps < 0 || (steps > 0 && !coefficients) || g_step < 0 || u_step < 0 || !(eps >= 0.0))
        return GEMM_ERR_INVALID_ARG;
    if (batch == 0 || m == 0 || n == 0)
        return GEMM_OK;
    for (int64_t i = 0; i < 3 * steps; ++i)
        if (!std::isfinite(coefficients[i]))
            return GEMM_ERR_UNSUPPORTED;
    if (!G || ldg < n)
        return GEMM_ERR_INVALID_ARG;
    if ((uintptr_t)G % size_of(in_dtype))
        return GEMM_ERR_MISALIGNED;
    if ((st = check_output(U, n, ldu, out_dtype)) != GEMM_OK)
        return st;
    const OrthoWs w = carve_ortho(batch, m, n, workspace);
    if ((st = check_workspace(workspace, workspace_bytes, w.bytes)) != GEMM_OK)
        return st;
    const bool flip = m > n;
    for (const OrthoPlan &p : w.plan)
        if (p.blocks <= 0 || p.blocks >= kMaxBlocks)
            return GEMM_ERR_UNSUPPORTED;

    hipLaunchKernelGGL(ortho_squares, dim3(w.parts, (unsigned)batch), dim3(256), 0, stream, G, (int)m, (int)n, ldg,
                       g_step, in_dtype, w.sums);
    hipError_t e = hipGetLastError();
    const SplitWs counters{w.partials, w.counters, w.num_counters[0]};
    if (e == hipSuccess)
        e = clear_counters(&counters, 1, stream);
    const float s = std::exp2(std::round(0.5f * std::log2((float)w.k))), t = 64.0f;
    if (e == hipSuccess) {
        hipLaunchKernelGGL(ortho_begin, dim3((unsigned)cdiv(w.k8, 64), (unsigned)cdiv(w.r8, 64), (unsigned)batch), dim3(256),
                           0, stream, G, (int)m, (int)n, ldg, g_step, in_dtype, (int)flip, w.sums, w.parts, eps, s, w.x,
                           w.xh, (int)w.r8, (int)w.k8);
        e = hipGetLastError();
    }
    OrthoArgs last{};
    last.update = U;
    last.update_step = u_step;
    last.update_dtype = out_dtype;
    last.ldu = (int)ldu;
    last.update_rows = (int)w.r, last.update_cols = (int)w.k;
    last.flip = flip;
    const int64_t size = size_of(out_dtype);
    last.update16 = (ldu * size) % 16 == 0 && (uintptr_t)U % 16 == 0 && (batch == 1 || (u_step * size) % 16 == 0);
    if (e == hipSuccess && steps == 0) {
        hipLaunchKernelGGL(ortho_copy, dim3((unsigned)cdiv(m * n, 256), (unsigned)batch), dim3(256), 0, stream, w.x,
                           (int)w.r8, (int)w.k8, last);
        e = hipGetLastError();
    }
    const int64_t x_step = w.r8 * w.k8, sq_step = w.r8 * w.r8;
    for (int64_t i = 0; i < steps && e == hipSuccess; ++i) {
        const float ca = coefficients[3 * i], cb = coefficients[3 * i + 1], cc = coefficients[3 * i + 2];
        const float sigma = i >= 2 ? 1.0f : 0.0f;
        uint16_t *xh = w.xh + (i & 1) * batch * x_step, *next = w.xh + ((i + 1) & 1) * batch * x_step;
        const SplitWs split{w.partials, w.counters, 0};
        for (int mode = ORTHO_SQUARE; mode <= ORTHO_STEP && e == hipSuccess; ++mode) {
            const OrthoPlan &plan = w.plan[mode];
            OrthoArgs a = mode == ORTHO_STEP && i + 1 == steps ? last : OrthoArgs{};
            a.mode = mode;
            a.all_splits = plan.splits;
            const bool step = mode == ORTHO_STEP;
            fill_args(a, plan.plan, split, mode == ORTHO_SQUARE ? w.a : mode == ORTHO_POLY ? w.b : next, w.r8,
                      step ? w.k8 : w.r8, mode == ORTHO_SQUARE ? w.k8 : w.r8, step ? w.k8 : w.r8, GEMM_FP16);
            a.A = mode == ORTHO_SQUARE ? xh : mode == ORTHO_POLY ? w.a : w.b;
            a.B = mode == ORTHO_SQUARE ? xh : mode == ORTHO_POLY ? w.a : xh;
            a.lda = (int)(mode == ORTHO_SQUARE ? w.k8 : w.r8);
            a.ldb = (int)(mode == ORTHO_POLY ? w.r8 : w.k8);
            a.a_step = mode == ORTHO_SQUARE ? x_step : sq_step;
            a.b_step = mode == ORTHO_POLY ? sq_step : x_step;
            a.c_step = step ? x_step : sq_step;
            a.old = w.a;
            a.x = w.x;
            if (mode == ORTHO_SQUARE) {
                a.alpha = t / (s * s);
                a.shift = t * sigma;
            } else if (mode == ORTHO_POLY) {
                a.alpha = cc / t;
                a.beta = cb + 2.0f * cc * sigma;
            } else {
                a.alpha = 1.0f / (t * s);
                a.beta = (float)((double)ca + (double)sigma * ((double)cb + (double)cc));
                a.scale = s;
            }
            e = launch_ortho(a, plan.tile, step, (unsigned)plan.blocks, stream);
        }
    }
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
