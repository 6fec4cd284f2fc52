// layer_gated.hip -- the gated block and its gradients: argument checks, plans, launches, and
// the small kernels beside the tiles.
//
//   h  = act(g) * u,  g = x Wg^T,  u = x Wu^T
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// The two weights are one B whose rows alternate in groups of eight between them
// (GNT_EXT_PAIRED), so one product of 2 F columns makes both sums, and a gate and its up value
// are in one lane's registers: the activation and the product need nothing from another
// lane, and neither sum goes through memory.  The backward call makes the sums again rather
// than read them (its caller keeps x alone; 12 M F K operations against 8, and 4 M F
// values less to keep and read), turns them into dg and du where they are, and stores those
// once, in the sums' column order: the contraction of dx then runs over both weights'
// rows in the same turns, and the rows of dW fall to the two arrays in the same turns, so that
// each is one launch.
//
// dg and du are rounded to the operands' type once, to nearest: the matrix cores take 16 bits,
// and what the rounding leaves (2^-9 of each BF16 value, 2^-12 FP16, independent) is no more than
// the rounding of dx and dW themselves.  FP16's would end at 2^-24: dh is multiplied by the
// power of two that brings its largest magnitude to 1 .. 2, and the sums are divided by it.
#include "layer_host.hpp"
#include "layer_launch.hpp"

namespace gnt {

// The partial maxima of |dh| (16-bit patterns without the sign, which order as the values do), of
// its finite values: what is not finite has its own row and column only, and no say in the rest's
// scale.
__global__ __launch_bounds__(256) void most_of(const uint16_t *x, int64_t M, int F, int ld, uint32_t *most)
{
    __shared__ uint32_t part[4];
    uint32_t b = 0;
    auto take1 = [&](uint32_t v) { b = max(b, v < 0x7c00u ? v : 0u); };
    auto take = [&](uint32_t w) { take1(w & 0x7fffu), take1((w >> 16) & 0x7fffu); };
    const int64_t step = gridDim.x;
    for (int64_t m = blockIdx.x; m < M; m += step) {
        const uint16_t *row = x + m * ld;
        int n = threadIdx.x * 8;
        for (; n + 8 <= F; n += 2048) {
            const u32x4 w = *reinterpret_cast<const run16_t *>(row + n);
            take(w[0]), take(w[1]), take(w[2]), take(w[3]);
        }
        for (; n < F; n += 2048)
            for (int i = 0; i < 8; ++i)
                if (n + i < F)
                    take(row[n + i]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        b = max(b, (uint32_t)__shfl_xor((int)b, o));
    if (threadIdx.x % 64 == 0)
        part[threadIdx.x / 64] = b;
    __syncthreads();
    if (threadIdx.x == 0)
        most[blockIdx.x] = max(max(part[0], part[1]), max(part[2], part[3]));
}

__global__ __launch_bounds__(256) void clear_words(ClearList l)
{
    clear_list(l, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

ClearList clear_of(const SplitWs *w, int count)
{
    ClearList l{};
    for (int i = 0; i < count; ++i) {
        l.at[i] = w[i].counters;
        l.count[i] = w[i].num_counters;
    }
    return l;
}

hipError_t clear_counters(const SplitWs *w, int count, hipStream_t stream)
{
    const ClearList l = clear_of(w, count);
    int most = 0;
    for (int n : l.count)
        most = std::max(most, n);
    if (most == 0)
        return hipSuccess;
    hipLaunchKernelGGL(clear_words, dim3((unsigned)std::min<int64_t>(32, cdiv(most, 256))), dim3(256), 0, stream, l);
    return hipGetLastError();
}

// The second pass of a product split along K (tiles whose splits are not summed in the
// kernel): the partials in split order, then what the tile's store does.  A thread has
// four of a group's columns, or with ROWS four columns of one of a group's rows.
enum : int { SUM_GATED = 0, SUM_GRAD = 1, SUM_ROWS = 2 };

template <int MODE, int IN, int OUT>
__global__ __launch_bounds__(256) void paired_sum(PairedArgs p)
{
    float scale = 1.0f;                     // (by whole waves, before any lane leaves)
    if constexpr (MODE == SUM_GRAD && IN == IN_FP16)
        scale = __builtin_ldexpf(1.0f, most_shift(p.most, threadIdx.x & 63));
    const int per = MODE == SUM_ROWS ? p.N / 4 : p.N / 8;        // threads per row
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= (int64_t)p.M * per)
        return;
    const int m = (int)(t / per), i = (int)(t - (int64_t)m * per);
    const int64_t plane = (int64_t)p.M * p.N;
    auto sum = [&](int n) {
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < p.splits; ++k)
            s += *reinterpret_cast<const f32x4 *>(p.partials + k * plane + (int64_t)m * p.N + n);
        return s;
    };
    if constexpr (MODE == SUM_ROWS) {
        const int f = (m >> 4) * 8 + (m & 7);
        if (f < p.cols)
            store4<OUT>((m >> 3) & 1 ? p.C2 : p.C, (int64_t)f * p.ldc + 4 * i, sum(4 * i), p.vec_store != 0, 4);
    } else {
        const int f = 4 * i, n = (f >> 3) * 16 + (f & 7);
        const f32x4 g = sum(n), u = sum(n + 8);
        float slope;
        if constexpr (MODE == SUM_GATED) {
            f32x4 y;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = gate_value<false>(p.act, g[e], slope) * u[e];
            if (f < p.cols)
                store4<OUT>(p.C, (int64_t)m * p.ldc + f, y, p.vec_store != 0, p.cols - f);
        } else {
            f32x4 dg, du;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = f + e < p.cols;
                const float d = in ? scale * from_bits16(IN, p.dh[(int64_t)m * p.lddh + f + e]) : 0.0f;
                const float a = gate_value<true>(p.act, g[e], slope);
                dg[e] = in ? d * u[e] * slope : 0.0f;
                du[e] = in ? d * a : 0.0f;
            }
            store4<OUT>(p.C, (int64_t)m * p.ldc + n, dg, true, 4);
            store4<OUT>(p.C, (int64_t)m * p.ldc + n + 8, du, true, 4);
        }
    }
}

namespace {

int64_t both(int64_t F) { return cdiv(F, 8) * 16; }        // columns of the paired product

gemm_status_t check_sizes(int64_t M, int64_t F, int64_t K, int in_dtype, int out_dtype, int activation)
{
    if (M < 0 || F < 0 || K < 0)
        return GEMM_ERR_INVALID_ARG;
    if (activation != GEMM_GATE_RELU && activation != GEMM_GATE_GELU && activation != GEMM_GATE_SILU)
        return GEMM_ERR_INVALID_ARG;
    if (!is_16bit(in_dtype) || !is_out(out_dtype))
        return GEMM_ERR_UNSUPPORTED;
    if (M >= kMaxRows || F >= kMaxLeadingDim / 2 || K >= kMaxSize || K % 8)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// The input gradient's plan: the library's for an MN-major B, or (`small`) the 64 x 64 tile where its
// tiles all run at once, two a compute unit, split along K to be as many, with at most 64
// slabs each.  In us, the sums' part with it (the 128 x 128 tile's first): 64 rows, F 1408, K 2048
// 31 and 24; 777 rows 52 and 50; 1024 x 2048 x 1024 54 and 44; 64 x 14336 x 4096 (8 splits of 56 slabs)
// 120 and 104; but 512 x 5632 x 2048 (2 of 88) 88 and 86, 777 x 5461 x 2048 (171 slabs) 137 and 163.
struct DxPlan : GradPlan {
    bool small;
};
DxPlan plan_dx(int64_t M, int64_t F, int64_t K)
{
    DxPlan g{plan_mn_major(M, K, both(F), kPartialBytes), false};
    Plan p{};
    p.tiles_m = (int)cdiv(M, 64);
    p.tiles_n = (int)cdiv(K, 64);
    p.k_tiles = (int)cdiv(both(F), 64);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, most = 2 * kNumCUs;
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(most / tiles, p.k_tiles / 8));
    p.kt_per_split = (int)cdiv(p.k_tiles, splits);
    if (tiles > most || p.kt_per_split > 64)
        return g;
    p.splits = p.k_tiles ? (int)cdiv(p.k_tiles, p.kt_per_split) : 1;
    p.group_m = std::min(4, p.tiles_m);
    p.grid = tiles * p.splits;
    if (p.splits > 1) {
        p.inreduce = 1;
        p.ws_bytes = p.grid * 64 * 64 * 4;
    }
    g.plan = p, g.small = true;
    return g;
}
// (the contraction runs over rows, which the MN-major operands take in any number)
Plan plan_dw(int64_t M, int64_t F, int64_t K)
{
    return make_plan(both(F), K, cdiv(M, 8) * 8, kPartialBytes, CFG_PP2_256x256, -1, 0);
}

// The workspaces of the two sums' pieces.
struct SumsWs {
    Pieces pieces;
    SplitWs split[2];
};

SumsWs carve_sums(Carver &c, int64_t M, int64_t F, int64_t K)
{
    SumsWs w;
    w.pieces = plan_pieces(M, both(F), K);
    for (int i = 0; i < w.pieces.count; ++i)
        w.split[i] = carve_splits(c, w.pieces.at[i].plan);
    return w;
}

bool launchable(const Pieces &p)
{
    return launchable(p.at[0].plan) && (p.count == 1 || launchable(p.at[1].plan));
}

struct BackwardWs {
    SumsWs sums;
    DxPlan dx;
    Plan plan[2];                       // dx, dW
    SplitWs split[2];
    uint16_t *d;                        // [M][both(F)]
    uint32_t *most;
    int64_t bytes;
};

BackwardWs carve_backward(int64_t M, int64_t F, int64_t K, void *base)
{
    BackwardWs w{};
    Carver c{static_cast<uint8_t *>(base)};
    w.d = c.take<uint16_t>(M * both(F));
    w.most = c.take<uint32_t>(kMostParts);
    // (a product of no rows or columns has no plan)
    if (M > 0 && F > 0)
        w.sums = carve_sums(c, M, F, K);
    if (M > 0 && K > 0) {
        w.dx = plan_dx(M, F, K);
        w.plan[0] = w.dx.plan;
        w.split[0] = carve_splits(c, w.plan[0]);
    }
    if (F > 0 && K > 0) {
        w.plan[1] = plan_dw(M, F, K);
        w.split[1] = carve_splits(c, w.plan[1]);
    }
    w.bytes = c.used;
    return w;
}

// The arguments of the sums' rows from `row` on and `cols` of the block's columns (F counts
// the last ones) from `col` on.
PairedArgs piece(PairedArgs a, int64_t row, int64_t col, int64_t cols)
{
    a.A += row * a.lda;
    a.B += col * a.ldb;
    a.B2 += col * a.ldb2;
    a.cols = (int)std::min<int64_t>(a.cols - col, cols);
    if (a.dh)
        a.dh += row * a.lddh + col;
    return a;
}

template <int MODE, int IN, int OUT>
hipError_t run_sum(const PairedArgs &a, hipStream_t stream)
{
    const int64_t per = MODE == SUM_ROWS ? a.N / 4 : a.N / 8;
    hipLaunchKernelGGL((paired_sum<MODE, IN, OUT>), dim3((unsigned)cdiv(a.M * per, 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <int MODE>
hipError_t run_sum_out(const PairedArgs &a, int out_dtype, hipStream_t stream)
{
    if (out_dtype == GEMM_BF16)
        return run_sum<MODE, 0, OUT_BF16>(a, stream);
    return out_dtype == GEMM_FP16 ? run_sum<MODE, 0, OUT_FP16>(a, stream) : run_sum<MODE, 0, OUT_FP32>(a, stream);
}

}  // namespace
}  // namespace gnt

using namespace gnt;

extern "C" {

gemm_status_t gemm_gated_workspace(int64_t M, int64_t F, int64_t K, int64_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = check_sizes(M, F, K, GEMM_BF16, GEMM_BF16, GEMM_GATE_SILU);
    if (st != GEMM_OK)
        return st;
    Carver c{nullptr};
    if (M > 0 && F > 0)
        carve_sums(c, M, F, K);
    *bytes = c.used;
    return GEMM_OK;
}

gemm_status_t gemm_run_gated(const void *X, const void *Wg, const void *Wu, void *H, int64_t M, int64_t F,
                             int64_t K, int64_t ldx, int64_t ldwg, int64_t ldwu, int64_t ldh, int in_dtype,
                             int out_dtype, int activation, void *workspace, int64_t workspace_bytes,
                             hipStream_t stream)
{
    gemm_status_t st = check_sizes(M, F, K, in_dtype, out_dtype, activation);
    if (st != GEMM_OK)
        return st;
    if (M == 0 || F == 0)
        return GEMM_OK;
    if ((st = check_output(H, F, ldh, out_dtype)) != GEMM_OK)
        return st;
    if (K > 0 && ((st = check_operand(X, K, ldx)) != GEMM_OK || (st = check_operand(Wg, K, ldwg)) != GEMM_OK ||
                  (st = check_operand(Wu, K, ldwu)) != GEMM_OK))
        return st;
    Carver c{static_cast<uint8_t *>(workspace)};
    const SumsWs w = carve_sums(c, M, F, K);
    if ((st = check_workspace(workspace, workspace_bytes, c.used)) != GEMM_OK)
        return st;
    if (!launchable(w.pieces))
        return GEMM_ERR_UNSUPPORTED;
    if (clear_counters(w.split, w.pieces.count, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    PairedArgs a{};
    a.A = static_cast<const uint16_t *>(X);
    a.B = static_cast<const uint16_t *>(Wg);
    a.B2 = static_cast<const uint16_t *>(Wu);
    a.lda = (int)ldx, a.ldb = (int)ldwg, a.ldb2 = (int)ldwu;
    a.cols = (int)F;
    a.act = activation;
    const int64_t size = size_of(out_dtype);
    hipError_t e = hipSuccess;
    for (int i = 0; i < w.pieces.count && e == hipSuccess; ++i) {
        const auto &q = w.pieces.at[i];
        const Plan &p = q.plan;
        PairedArgs b = piece(a, q.row, q.col / 2, q.cols / 2);
        fill_args(b, p, w.split[i], static_cast<uint8_t *>(H) + (q.row * ldh + q.col / 2) * size, q.rows, q.cols, K, ldh,
                  out_dtype);
        const bool rot = rotate_slabs(1, q.rows);
        paired_fn fn;
        switch (p.cfg) {
        case CFG_T128x128: fn = (rot ? kGated_128_s4_rot : kGated_128_s4)[in_dtype][out_dtype]; break;
        case CFG_T128x128_S2: fn = (rot ? kGated_128_s2_rot : kGated_128_s2)[in_dtype][out_dtype]; break;
        case CFG_T32x128: fn = kGated_32_rot[in_dtype][out_dtype]; break;
        case CFG_W4_256x128: fn = kGated_w4[in_dtype][out_dtype]; break;
        default: fn = kGated_pp2[in_dtype][out_dtype];
        }
        e = fn(b, (unsigned)p.grid, stream);
        if (e == hipSuccess && p.splits > 1 && !p.inreduce)
            e = run_sum_out<SUM_GATED>(b, out_dtype, stream);
    }
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

gemm_status_t gemm_gated_backward_workspace(int64_t M, int64_t F, int64_t K, int64_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = check_sizes(M, F, K, GEMM_BF16, GEMM_BF16, GEMM_GATE_SILU);
    if (st != GEMM_OK)
        return st;
    *bytes = carve_backward(M, F, K, nullptr).bytes;
    return GEMM_OK;
}

gemm_status_t gemm_run_gated_backward(const void *dH, const void *X, const void *Wg, const void *Wu, void *dX,
                                      void *dWg, void *dWu, int64_t M, int64_t F, int64_t K, int64_t lddh,
                                      int64_t ldx, int64_t ldwg, int64_t ldwu, int64_t lddx, int in_dtype,
                                      int dx_dtype, int grad_dtype, int activation, void *workspace,
                                      int64_t workspace_bytes, hipStream_t stream)
{
    gemm_status_t st = check_sizes(M, F, K, in_dtype, dx_dtype, activation);
    if (st != GEMM_OK)
        return st;
    if (!is_out(grad_dtype))
        return GEMM_ERR_UNSUPPORTED;
    const bool want_dx = dX && M > 0 && K > 0;
    const bool want_dw = (dWg || dWu) && F > 0 && K > 0;
    if (!dWg != !dWu && F > 0 && K > 0)
        return GEMM_ERR_INVALID_ARG;
    if (!want_dx && !want_dw)
        return GEMM_OK;
    if (M > 0 && F > 0) {
        if (lddh < F || !dH)
            return GEMM_ERR_INVALID_ARG;
        if (lddh >= kMaxSize)
            return GEMM_ERR_UNSUPPORTED;
        if ((uintptr_t)dH % 2)
            return GEMM_ERR_MISALIGNED;
        if ((st = check_operand(X, K, ldx)) != GEMM_OK || (st = check_operand(Wg, K, ldwg)) != GEMM_OK ||
            (st = check_operand(Wu, K, ldwu)) != GEMM_OK)
            return st;
    }
    if (want_dx && (st = check_output(dX, K, lddx, dx_dtype)) != GEMM_OK)
        return st;
    if (want_dw && ((st = check_output(dWg, K, K, grad_dtype)) != GEMM_OK ||
                    (st = check_output(dWu, K, K, grad_dtype)) != GEMM_OK))
        return st;
    const BackwardWs w = carve_backward(M, F, K, workspace);
    if ((st = check_workspace(workspace, workspace_bytes, w.bytes)) != GEMM_OK)
        return st;
    const bool inner = M > 0 && F > 0;
    if ((inner && !launchable(w.sums.pieces)) || (want_dx && !launchable(w.plan[0])) || (want_dw && !launchable(w.plan[1])))
        return GEMM_ERR_UNSUPPORTED;
    SplitWs split[4] = {w.split[0], w.split[1], w.sums.split[0], w.sums.split[1]};
    const int splits = inner ? 2 + w.sums.pieces.count : 2;
    // what the later products count on is cleared by the first's blocks, each of which stores a
    // tile, or where those are split themselves by a launch
    const bool clear_first = inner && w.sums.pieces.at[0].plan.splits == 1;
    hipError_t e = clear_first ? hipSuccess : clear_counters(split, splits, stream);
    const int64_t both_cols = both(F);
    PairedArgs a{};
    a.B = static_cast<const uint16_t *>(Wg);
    a.B2 = static_cast<const uint16_t *>(Wu);
    a.ldb = (int)ldwg, a.ldb2 = (int)ldwu;
    a.cols = (int)F;
    a.act = activation;
    a.dh = static_cast<const uint16_t *>(dH);
    a.lddh = (int)lddh;
    a.most = w.most;
    if (e == hipSuccess && in_dtype == GEMM_FP16) {
        hipLaunchKernelGGL(most_of, dim3(kMostParts), dim3(256), 0, stream, a.dh, F > 0 ? M : 0, (int)F, a.lddh,
                           w.most);
        e = hipGetLastError();
    }
    for (int i = 0; inner && i < w.sums.pieces.count && e == hipSuccess; ++i) {
        const auto &q = w.sums.pieces.at[i];
        const Plan &p = q.plan;
        PairedArgs b = a;
        b.A = static_cast<const uint16_t *>(X);
        b.lda = (int)ldx;
        b = piece(b, q.row, q.col / 2, q.cols / 2);
        if (clear_first && i == 0)
            b.clear = clear_of(split, splits);
        fill_args(b, p, w.sums.split[i], w.d + q.row * both_cols + q.col, q.rows, q.cols, K, both_cols, in_dtype);
        const bool rot = rotate_slabs(1, q.rows);
        paired_fn fn;
        switch (p.cfg) {
        case CFG_T128x128: fn = (rot ? kGateGrad_128_s4_rot : kGateGrad_128_s4)[in_dtype]; break;
        case CFG_T128x128_S2: fn = kGateGrad_128_s2[in_dtype]; break;
        case CFG_T32x128: fn = kGateGrad_32_rot[in_dtype]; break;
        case CFG_W4_256x128: fn = kGateGrad_w4[in_dtype]; break;
        default: fn = kGateGrad_pp2[in_dtype];
        }
        e = fn(b, (unsigned)p.grid, stream);
        if (e == hipSuccess && p.splits > 1 && !p.inreduce)
            e = in_dtype == GEMM_BF16 ? run_sum<SUM_GRAD, IN_BF16, OUT_BF16>(b, stream)
                                      : run_sum<SUM_GRAD, IN_FP16, OUT_FP16>(b, stream);
    }
    if (e == hipSuccess && want_dx) {
        const Plan &p = w.plan[0];
        PairedArgs b = a;
        fill_args(b, p, w.split[0], dX, M, K, both_cols, lddx, dx_dtype);
        b.A = w.d;
        b.lda = (int)both_cols;
        e = (w.dx.small ? kGatedDx_64 : w.dx.tile ? kGatedDx_tile : kGatedDx_pp2)[in_dtype][dx_dtype](b, (unsigned)p.grid, stream);
        if (e == hipSuccess && p.splits > 1 && !p.inreduce) {
            const KernelArgs &k = b;
            const unsigned grid = (unsigned)cdiv(M * (K / 4), 256);
            if (dx_dtype == GEMM_BF16)
                hipLaunchKernelGGL(splitk_sum<OUT_BF16>, dim3(grid), dim3(256), 0, stream, k);
            else if (dx_dtype == GEMM_FP16)
                hipLaunchKernelGGL(splitk_sum<OUT_FP16>, dim3(grid), dim3(256), 0, stream, k);
            else
                hipLaunchKernelGGL(splitk_sum<OUT_FP32>, dim3(grid), dim3(256), 0, stream, k);
            e = hipGetLastError();
        }
    }
    if (e == hipSuccess && want_dw) {
        const Plan &p = w.plan[1];
        PairedArgs b = a;
        fill_args(b, p, w.split[1], dWg, both_cols, K, M, K, grad_dtype);
        b.vec_store = b.vec_store && (uintptr_t)dWu % (4 * size_of(grad_dtype)) == 0;
        b.C2 = dWu;
        b.A = w.d;
        b.lda = (int)both_cols;
        b.B = static_cast<const uint16_t *>(X);
        b.ldb = (int)ldx;
        e = kGatedDw_pp2[in_dtype][grad_dtype](b, (unsigned)p.grid, stream);
        if (e == hipSuccess && p.splits > 1 && !p.inreduce)
            e = run_sum_out<SUM_ROWS>(b, grad_dtype, stream);
    }
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
