// layer_ortho.hip -- the orthogonalized update of a weight: Newton-Schulz products.
//
//   X = G / (||G|| + eps), r x k with r <= k (a tall G's transpose), then `steps` times
//   A = X X^T,  X = a X + (b A + c A^2) X
// which takes every singular value s of X to a s + b s^3 + c s^5.
//
// Numbers.  The products run on FP16 operands with FP32 sums.  X is the sum of two FP16 values (in
// units of 1 / s, s the power of two near 16 sqrt(k), so that entries of 1 / sqrt(r k) have 22 bits in
// them), of which only the first enters the products; so an X of steep spectrum, whose small
// singular values the first steps multiply by a alone, keeps them: with X in one FP16 value
// a spectrum falling as 1 / i ended 2.9e-3 off, so 0.5e-3.  (In FP32 beside the copy for the
// products it was as exact, for 12 bytes a value and step to move where this has 8: 12 of 2048 x
// 768 564 us against 504, 4096 x 8192 2543 against 2445.)  From the third step on, when the
// singular values are near 1, the squares are held as what they differ from the identity by:
//   A = I + A':  b A + c A^2 = (b + c) I + (b + 2 c) A' + c A'^2
// whose diagonal does not fill FP16's bits with what is known already; the multiple of I goes
// into X's factor, exactly (a random 512 x 512: 1.5e-3 off without, 0.9e-3 with).  A BF16
// result's rounding is 1.7e-3 by itself; iterates in BF16 would be 1e-2 off.
#include "layer_host.hpp"
#include "ortho_common.hpp"

namespace gnt {

hipError_t launch_ortho(const OrthoArgs &a, OrthoTile tile, unsigned grid, hipStream_t s);

constexpr int kOrthoParts = 1024;          // partial sums of squares of a stack, at most

__device__ __forceinline__ float read_any(const void *x, int64_t i, int dtype)
{
    return dtype == OUT_FP32 ? static_cast<const float *>(x)[i]
                             : from_bits16(dtype, static_cast<const uint16_t *>(x)[i]);
}

// Eight values from element i on, of which the first `left` are there; zeros behind them.
__device__ __forceinline__ void read_eight(const void *x, int64_t i, int dtype, int left, float (&v)[8])
{
    if (left >= 8 && dtype == OUT_FP32) {
        const run32_t *s = reinterpret_cast<const run32_t *>(static_cast<const float *>(x) + i);
        const f32x4 a = s[0], b = s[1];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = a[e], v[4 + e] = b[e];
    } else if (left >= 8) {
        const u32x4 w = *reinterpret_cast<const run16_t *>(static_cast<const uint16_t *>(x) + i);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = from_bits16(dtype, (w[e >> 1] >> (16 * (e & 1))) & 0xffffu);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = e < left ? read_any(x, i + e, dtype) : 0.0f;
    }
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
// sides): the threads of matrix b's blocks (x, b) take eight values of a row each in turn, four
// loads of them at a time (one at a time 2 TB/s, of a long row 5.6).  The arrival counters of
// the products to come are cleared on the way.
__global__ __launch_bounds__(256) void ortho_squares(const void *G, int m, int n, int64_t ld, int64_t step, int dtype,
                                                     double *parts, unsigned *counters, int num_counters)
{
    __shared__ double part[4];
    const int id = blockIdx.x * 256 + threadIdx.x, threads = gridDim.x * 256;
    if (blockIdx.y == 0)
        for (int i = id; i < num_counters; i += threads)
            counters[i] = 0u;
    const int runs = (n + 7) / 8;
    const int64_t all = (int64_t)m * runs, from = blockIdx.y * step;
    double s = 0.0;
    for (int64_t i = id; i < all; i += 4 * (int64_t)threads) {
        float v[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = i + j * (int64_t)threads;
            const int64_t r = at / runs;
            const int c = (int)(at - r * runs) * 8;
            read_eight(G, from + r * ld + c, dtype, at < all ? n - c : 0, v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += (double)v[j][e] * (double)v[j][e];
    }
    s = block_sum(s, part);
    if (threadIdx.x == 0)
        parts[blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// s X = s G / (||G|| + eps) as two FP16 values, [rows8][cols8] with zeros past the matrix, and
// with xt the first also transposed, [cols8][rows8]; a tall G (flip) is transposed on the way.
// A block has 64 x 64 values.
__global__ __launch_bounds__(256) void ortho_begin(const void *G, int m, int n, int64_t ld, int64_t step, int dtype,
                                                   int flip, const double *parts, int num_parts, double eps,
                                                   float s, uint16_t *hi, uint16_t *lo, uint16_t *xt, int rows8, int cols8)
{
    __shared__ double part[4];
    __shared__ float tile[64][65];
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;         // of X
    const int g_r0 = flip ? c0 : r0, g_c0 = flip ? r0 : c0;       // of G
    const int64_t from = blockIdx.z * step;
    float v[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = threadIdx.x + 256 * i, r = g_r0 + (t >> 3), c = g_c0 + 8 * (t & 7);
        read_eight(G, from + (int64_t)r * ld + c, dtype, r < m ? n - c : 0, v[i]);
    }
    double sum = 0.0;
    for (int i = threadIdx.x; i < num_parts; i += 256)
        sum += parts[blockIdx.z * num_parts + i];
    // (an infinity alone would leave the other values 0: what is not finite takes the whole matrix)
    const double squares = block_sum(sum, part);
    const double inv = __builtin_isfinite(squares) ? (double)s / (__builtin_sqrt(squares) + eps) : __builtin_nan("");
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = threadIdx.x + 256 * i;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            tile[t >> 3][8 * (t & 7) + e] = (float)((double)v[i][e] * inv);
    }
    __syncthreads();
    const int64_t at = (int64_t)blockIdx.z * rows8 * cols8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = threadIdx.x + 256 * i, r = t >> 3, c = (t & 7) * 8;
        float y[8], z[8];
        if (r0 + r < rows8 && c0 + c < cols8) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] = flip ? tile[c + e][r] : tile[r][c + e];
            two_halves(y, z);
            store_run<OUT_FP16, 8, false>(hi, at + (int64_t)(r0 + r) * cols8 + c0 + c, y, 8);
            store_run<OUT_FP16, 8, false>(lo, at + (int64_t)(r0 + r) * cols8 + c0 + c, z, 8);
        }
        if (xt && c0 + r < cols8 && r0 + c < rows8) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] = flip ? tile[r][c + e] : tile[c + e][r];
            store_run<OUT_FP16, 8, false>(xt, at + (int64_t)(c0 + r) * rows8 + r0 + c, y, 8);
        }
    }
}

// The update of no steps at all: X as it begins.  (A launch has fewer than 2^32 threads:
// kCopyBlocks a matrix at most, which take its values in turn.)
constexpr int64_t kCopyBlocks = (int64_t)1 << 20;

__global__ __launch_bounds__(256) void ortho_copy(const uint16_t *hi, const uint16_t *lo, float unit, int rows8, int cols8,
                                                  OrthoArgs p)
{
    const int m = p.flip ? p.update_cols : p.update_rows, n = p.flip ? p.update_rows : p.update_cols;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < (int64_t)m * n; t += (int64_t)gridDim.x * 256) {
        const int r = (int)(t / n), c = (int)(t - (int64_t)r * n);
        const int64_t i = (int64_t)blockIdx.y * rows8 * cols8 + (p.flip ? (int64_t)c * cols8 + r : (int64_t)r * cols8 + c);
        const float v = unit * (from_bits16(IN_FP16, hi[i]) + from_bits16(IN_FP16, lo[i]));
        const int64_t at = blockIdx.y * p.update_step + (int64_t)r * p.ldu + c;
        if (p.update_dtype == OUT_FP32)
            static_cast<float *>(p.update)[at] = v;
        else
            static_cast<uint16_t *>(p.update)[at] =
                (uint16_t)(p.update_dtype == OUT_BF16 ? to_bits16<OUT_BF16>(v) : to_bits16<OUT_FP16>(v));
    }
}

namespace {

// One launch of a product: its tile and K splits, and which of the stack's tiles.
struct OrthoLaunch {
    OrthoTile tile;
    int size;                // of a tile
    int first, quarters;     // OrthoArgs'
    int splits, kt_per_split;
    int64_t blocks;
};

struct OrthoPlan {
    int half;                // a square's lower half only: the size of its tiles
    int tiles;               // of a matrix
    int tiles_m, tiles_n, k_tiles;
    int count;
    OrthoLaunch part[2];
    int64_t partials;        // values
    int64_t counters;
};

// What a pass of the machine takes, in us: begin + slab a 64-deep slab (alone: with one block a
// compute unit where two fit); the most splits (summed in the kernel), and us a split
// (a step's K is the smaller side, too short to split: 1000 x 2047 210 us in two, 183 whole).  From
// the kernels' times: steps of 12 matrices of 768 x 2048 and of one of 4096 x 8192 (12 and 64 slabs)
// on 256_MN 32 and 117 a pass, 128_MN 19 and 83, 128_S2 21 and 86, 128 16 and 45; squares of 4096 on
// 256 88 (64 slabs) and 155 (128), of 12 x 768 on 128 16 (12) and 26 (32), of 1000 on 64 9 (16), 11 (32) and
// 28 (125); steps of 1000 on 64_MN 8.  Over twenty-two shapes swept during development the choices
// were within 4% of the best tile and split of each product.
struct OrthoKind {
    OrthoTile tile;
    int size, at_once, splits;
    bool mn;
    double begin, slab, alone, split;
};
constexpr OrthoKind kOrthoKinds[] = {
    {ORTHO_256, 256, 1, 2, false, 18.0, 1.3, 1.3, 16.0},  {ORTHO_256_MN, 256, 1, 1, true, 11.0, 1.62, 1.62, 0.0},
    {ORTHO_128, 128, 1, 16, false, 11.5, 0.52, 0.52, 5.0}, {ORTHO_128_S2, 128, 2, 1, false, 15.0, 1.1, 0.6, 0.0},
    {ORTHO_128_MN, 128, 2, 1, true, 7.0, 1.05, 1.0, 0.0}, {ORTHO_64, 64, 2, 16, false, 5.5, 0.55, 0.28, 0.8},
    {ORTHO_64_MN, 64, 2, 1, true, 3.0, 0.55, 0.28, 0.0},
};

double cost_of(const OrthoKind &k, int64_t blocks, int64_t slabs, int64_t splits)
{
    const double slab = blocks <= kNumCUs ? k.alone : k.slab;
    return (double)cdiv(blocks, kNumCUs * k.at_once) * (k.begin + slab * (double)slabs) +
           (splits > 1 ? 2.0 + k.split * (double)splits : 0.0);
}

// Splits of `slabs` that keep four slabs each and fill `s` whole; 0: not that many.
int64_t slabs_per(int64_t slabs, int64_t s)
{
    const int64_t per = cdiv(slabs, s);
    return s == 1 ? per : slabs / s >= 4 && cdiv(slabs, per) == s ? per : 0;
}

// The launches of a stack's product [M][N] over K, the least by what they are expected to take:
// `square` (M = N, symmetric, both operands K-major: the lower half of its tiles) or the step.
OrthoPlan plan_ortho(int64_t batch, int64_t M, int64_t N, int64_t K, bool square)
{
    OrthoPlan best{};
    double least = -1.0;
    const int64_t slabs = cdiv(K, 64);
    auto fits = [&](int64_t blocks, int64_t s, int size) {
        return s == 1 || (blocks * size * size * 4 <= 2 * kPartialBytes && blocks <= 4 * kNumCUs);
    };
    auto begin = [&](const OrthoKind &k) {
        OrthoPlan p{};
        p.tiles_m = (int)cdiv(M, k.size), p.tiles_n = (int)cdiv(N, k.size);
        p.k_tiles = (int)slabs;
        p.half = square ? k.size : 0;
        p.tiles = square ? p.tiles_m * (p.tiles_m + 1) / 2 : p.tiles_m * p.tiles_n;
        return p;
    };
    auto add = [&](OrthoPlan &p, const OrthoKind &k, int64_t first, bool quarters, int64_t tiles, int64_t s) {
        const int64_t blocks = tiles * s;
        p.part[p.count++] = {k.tile, k.size, (int)first, quarters, (int)s, (int)slabs_per(slabs, s), blocks};
        if (s > 1) {
            p.partials = std::max<int64_t>(p.partials, blocks * k.size * k.size);
            p.counters = std::max<int64_t>(p.counters, tiles);
        }
    };
    for (const OrthoKind &k : kOrthoKinds) {
        // (a step's 64 x 64 tiles read X as it is: 1000 x 2047 189 us, with X transposed 203)
        if (square ? k.mn : k.tile == ORTHO_256 || k.tile == ORTHO_64)
            continue;
        for (int64_t s = 1; s <= k.splits; ++s) {
            const int64_t per = slabs_per(slabs, s);
            OrthoPlan p = begin(k);
            const int64_t all = batch * p.tiles;
            if ((slabs && !per) || !fits(all * s, s, k.size))
                continue;
            add(p, k, 0, false, all, s);
            const double cost = cost_of(k, all * s, per, s);
            if (least < 0.0 || cost < least)
                least = cost, best = p;
        }
    }
    // A square's 256 x 256 tiles that fill whole passes of the machine, and the quarters of the
    // rest on the 128 x 128 tile, with splits: two matrices of 4096 rows (272 tiles) 3.29 ms for
    // the update, on the one tile 3.53.  (Whole passes of tiles split in two did not pay: one
    // matrix of 4096 x 8192, 128 tiles twice and 8 over, 3.18 against 3.14; nor did 192 x 192 tiles, four
    // waves of 96 x 96: there 253 of them fill the machine and took 1.1 us a slab, 2.52 against 2.56.)
    if (square) {
        const OrthoKind &k = kOrthoKinds[0], &q = kOrthoKinds[2];
        OrthoPlan p = begin(k);
        const int64_t all = batch * p.tiles, whole = all / kNumCUs * kNumCUs, rest = 4 * (all - whole);
        if (whole > 0 && rest > 0) {
            int64_t rs = 1;
            double rest_cost = cost_of(q, rest, slabs, 1);
            for (int64_t t = 2; t <= q.splits; ++t)
                if (slabs_per(slabs, t) && fits(rest * t, t, q.size) && cost_of(q, rest * t, slabs_per(slabs, t), t) < rest_cost)
                    rest_cost = cost_of(q, rest * t, slabs_per(slabs, t), t), rs = t;
            if (cost_of(k, whole, slabs, 1) + rest_cost < least) {
                add(p, k, 0, false, whole, 1);
                add(p, q, whole, true, rest, rs);
                best = p;
            }
        }
    }
    return best;
}

struct OrthoWs {
    int64_t r, k, r8, k8;
    int parts;               // partial sums a matrix
    bool turned;             // the step reads X transposed
    OrthoPlan plan[3];
    double *sums;
    float *partials;
    uint16_t *hi, *lo, *xt, *a, *b;
    unsigned *counters;
    int num_counters;
    int64_t bytes;
};

OrthoWs carve_ortho(int64_t batch, int64_t m, int64_t n, void *base)
{
    OrthoWs w{};
    Carver c{static_cast<uint8_t *>(base)};
    w.r = std::min(m, n), w.k = std::max(m, n);
    // whole 128-byte lines a row: 1000 x 2047 with rows of 1000 and 2048 took 19.8 us a step,
    // 1024 x 2048 14.9
    w.r8 = cdiv(w.r, 64) * 64, w.k8 = cdiv(w.k, 64) * 64;
    w.parts = (int)std::max<int64_t>(1, std::min<int64_t>(cdiv(m * cdiv(n, 8), 1024), kOrthoParts / std::max<int64_t>(1, batch)));
    w.plan[ORTHO_SQUARE] = plan_ortho(batch, w.r8, w.r8, w.k8, true);
    w.plan[ORTHO_POLY] = plan_ortho(batch, w.r8, w.r8, w.r8, true);
    w.plan[ORTHO_STEP] = plan_ortho(batch, w.r8, w.k8, w.r8, false);
    const int64_t size = batch * w.r8 * w.k8;
    w.sums = c.take<double>(batch * w.parts);
    w.hi = c.take<uint16_t>(2 * size);       // two, in turn: a step reads one and writes the other
    w.lo = c.take<uint16_t>(size);
    const OrthoTile step = w.plan[ORTHO_STEP].part[0].tile;
    // (every tile but those reads B by rows of K)
    w.turned = step != ORTHO_256_MN && step != ORTHO_128_MN && step != ORTHO_64_MN;
    w.xt = c.take<uint16_t>(w.turned ? 2 * size : 0);
    w.a = c.take<uint16_t>(batch * w.r8 * w.r8);
    w.b = c.take<uint16_t>(batch * w.r8 * w.r8);
    int64_t partial = 0, counters = 0;
    for (const OrthoPlan &p : w.plan) {
        partial = std::max(partial, p.partials);
        counters = std::max(counters, p.counters);
    }
    w.partials = c.take<float>(partial);
    w.counters = c.take<unsigned>(counters);               // (each call of a tile leaves them zero)
    w.num_counters = (int)counters;
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
        for (int i = 0; i < p.count; ++i)
            if (p.part[i].blocks <= 0 || p.part[i].blocks >= kMaxBlocks)
                return GEMM_ERR_UNSUPPORTED;

    hipLaunchKernelGGL(ortho_squares, dim3(w.parts, (unsigned)batch), dim3(256), 0, stream, G, (int)m, (int)n, ldg,
                       g_step, in_dtype, w.sums, w.counters, w.num_counters);
    hipError_t e = hipGetLastError();
    const float s = 16.0f * std::exp2(std::round(0.5f * std::log2((float)w.k))), t = 64.0f;
    if (e == hipSuccess) {
        hipLaunchKernelGGL(ortho_begin, dim3((unsigned)cdiv(w.k8, 64), (unsigned)cdiv(w.r8, 64), (unsigned)batch), dim3(256),
                           0, stream, G, (int)m, (int)n, ldg, g_step, in_dtype, (int)flip, w.sums, w.parts, eps,
                           s, w.hi, w.lo, w.turned ? w.xt : nullptr, (int)w.r8, (int)w.k8);
        e = hipGetLastError();
    }
    OrthoArgs last{};
    last.update = U;
    last.update_step = u_step;
    last.update_dtype = out_dtype;
    last.ldu = (int)ldu;
    last.update_rows = (int)w.r, last.update_cols = (int)w.k;
    last.flip = flip;
    if (e == hipSuccess && steps == 0) {
        hipLaunchKernelGGL(ortho_copy, dim3((unsigned)std::min(cdiv(m * n, 256), kCopyBlocks), (unsigned)batch), dim3(256), 0,
                           stream, w.hi, w.lo, 1.0f / s, (int)w.r8, (int)w.k8, last);
        e = hipGetLastError();
    }
    const int64_t x_step = w.r8 * w.k8, sq_step = w.r8 * w.r8;
    for (int64_t i = 0; i < steps && e == hipSuccess; ++i) {
        const float ca = coefficients[3 * i], cb = coefficients[3 * i + 1], cc = coefficients[3 * i + 2];
        const float sigma = i >= 2 ? 1.0f : 0.0f;
        uint16_t *xh = w.hi + (i & 1) * batch * x_step, *next = w.hi + ((i + 1) & 1) * batch * x_step;
        const uint16_t *xt = w.turned ? w.xt + (i & 1) * batch * x_step : nullptr;
        for (int mode = ORTHO_SQUARE; mode <= ORTHO_STEP && e == hipSuccess; ++mode) {
            const OrthoPlan &plan = w.plan[mode];
            OrthoArgs a = mode == ORTHO_STEP && i + 1 == steps ? last : OrthoArgs{};
            a.mode = mode;
            a.tiles = plan.tiles;
            a.half = plan.half;
            const bool step = mode == ORTHO_STEP;
            a.C = mode == ORTHO_SQUARE ? w.a : mode == ORTHO_POLY ? w.b : next;
            a.M = (int)w.r8, a.N = (int)(step ? w.k8 : w.r8), a.K = (int)(mode == ORTHO_SQUARE ? w.k8 : w.r8);
            a.ldc = a.N;
            a.tiles_m = plan.tiles_m, a.tiles_n = plan.tiles_n, a.k_tiles = plan.k_tiles;
            a.group_m = std::min(4, plan.tiles_m);
            a.partials = w.partials;
            a.counters = w.counters;
            a.A = mode == ORTHO_SQUARE ? xh : mode == ORTHO_POLY ? w.a : w.b;
            a.B = mode == ORTHO_SQUARE ? xh : mode == ORTHO_POLY ? w.a : w.turned ? xt : xh;
            a.lda = (int)(mode == ORTHO_SQUARE ? w.k8 : w.r8);
            a.ldb = (int)(mode == ORTHO_POLY || (step && w.turned) ? w.r8 : w.k8);
            a.a_step = mode == ORTHO_SQUARE ? x_step : sq_step;
            a.b_step = mode == ORTHO_POLY ? sq_step : x_step;
            a.c_step = step ? x_step : sq_step;
            a.old = w.a;
            a.hi = xh;
            a.lo = w.lo;
            a.xt = step && w.turned ? w.xt + ((i + 1) & 1) * batch * x_step : nullptr;
            a.ldt = (int)w.r8;
            if (mode == ORTHO_SQUARE) {
                a.alpha = t / (s * s);
                a.shift = t * sigma;
            } else if (mode == ORTHO_POLY) {
                a.alpha = cc / t;
                a.beta = cb + 2.0f * cc * sigma;
            } else {
                // (of s X; the last step's X itself)
                const float unit = a.update ? 1.0f / s : 1.0f;
                a.alpha = unit / t;
                a.beta = unit * (float)((double)ca + (double)sigma * ((double)cb + (double)cc));
            }
            for (int j = 0; j < plan.count && e == hipSuccess; ++j) {
                const OrthoLaunch &l = plan.part[j];
                a.first = l.first;
                a.quarters = l.quarters;
                a.splits = a.all_splits = l.splits;
                a.kt_per_split = l.kt_per_split;
                a.inreduce = l.splits > 1;
                e = launch_ortho(a, l.tile, (unsigned)l.blocks, stream);
            }
        }
    }
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
