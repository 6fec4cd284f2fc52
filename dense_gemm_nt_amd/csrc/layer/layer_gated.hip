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
// lane, and neither sum goes through memory but for K splits' partials (few rows or columns, which
// the last of a tile's splits or a second pass adds up).  The backward call makes the sums again rather
// than read them (its caller keeps x alone; 12 M F K operations against 8, and 4 M F
// values less to keep and read), turns them into dg and du where they are, and stores those
// once, in the sums' column order: the contraction of dx then runs over both weights'
// rows in the same turns, and the rows of dW fall to the two arrays in the same turns, so that
// each is one launch.
//
// dg and du are rounded to the operands' type once, to nearest: the matrix cores take 16 bits,
// and what the rounding leaves (2^-9 of each BF16 value, 2^-12 FP16, independent) is no more than
// the rounding of dx and dW themselves.  FP16's would end at 2^-24 and 2^16: they are stored in units
// of powers of two, once of their row for dx and once of their column for the weights'
// gradients, and the sums divided by them (bound_exponent).  The units take a launch that reads
// every operand (gate_units) and a second copy of dg and du; one scale for all of dh, which needs
// neither, lost the bits of every row beside a large one, and all where a sum was large.
#include "layer_host.hpp"
#include "layer_launch.hpp"

namespace gnt {

// What the units of FP16 gradients are made of (PairedArgs): the largest finite |dh| of each row,
// and of the columns of each chunk of rows (16-bit patterns, which order as the values do); and
// partial maxima of the squared norms of X's rows and of the weights' rows, of those that are
// finite.  (A value that is not finite makes its own row's and column's gradients what they are,
// and has no say in the others'.)  The first kNormParts blocks take rows in turn, a wave each or a block
// those of more than 8192 values; `strips * chunks` after them 64 columns of dh's rows of a
// chunk each.  Bound by its reads, dh's twice: 470 MB of 8192 x 8192 x 4096 80 us, 5.9 TB/s (with the
// columns' blocks first and four rows a wave 114); 777 x 1408 x 2048 7.7 us, of which a launch's
// beginning and end are 4.
struct UnitArgs {
    const uint16_t *dh, *x, *wg, *wu;
    int64_t M, F;
    int K, lddh, ldx, ldg, ldu;
    int strips, chunks, chunk_rows;
    uint16_t *row_most, *col_most;
    float *norms;
};

constexpr int kRowsAtOnce = 2;

typedef short s16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float squares8(u32x4 w)
{
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = from_bits16(IN_FP16, (w[e >> 1] >> (16 * (e & 1))) & 0xffffu);
        s += v * v;
    }
    return s;
}

__global__ __launch_bounds__(256) void gate_units(UnitArgs a)
{
    __shared__ uint32_t part[4][32];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // the running maxima of pairs of values: 0x400 is added to a pattern without its sign, so that
    // what is not finite is negative
    const s16x2 kZero = {0x400, 0x400};
    auto take = [&](s16x2 &most, uint32_t w) {
        most = __builtin_elementwise_max(most, __builtin_bit_cast(s16x2, w & 0x7fff7fffu) + kZero);
    };
    auto read = [&](const uint16_t *at, int64_t left) -> u32x4 {      // eight values, or `left` and zeros
        u32x4 w = {0u, 0u, 0u, 0u};
        if (left >= 8) {
            w = *reinterpret_cast<const run16_t *>(at);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    w[i >> 1] |= (uint32_t)at[i] << (16 * (i & 1));
        }
        return w;
    };
    if (blockIdx.x >= kNormParts) {
        const int tile = blockIdx.x - kNormParts;
        const int chunk = tile / a.strips, strip = tile - chunk * a.strips;
        const int64_t f = (int64_t)strip * 64 + 8 * (lane & 7);
        const int64_t end = min(a.M, (int64_t)(chunk + 1) * a.chunk_rows);
        s16x2 most[4] = {kZero, kZero, kZero, kZero};
        if (f < a.F) {
#pragma unroll 8
            for (int64_t m = (int64_t)chunk * a.chunk_rows + (threadIdx.x >> 3); m < end; m += 32) {
                const u32x4 w = read(a.dh + m * a.lddh + f, a.F - f);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    take(most[i], w[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 8; o < 64; o <<= 1)
                most[i] = __builtin_elementwise_max(
                    most[i], __builtin_bit_cast(s16x2, __shfl_xor(__builtin_bit_cast(int, most[i]), o)));
            if (lane < 8)
                part[wave][4 * lane + i] = __builtin_bit_cast(uint32_t, most[i] - kZero);
        }
        __syncthreads();
        const int64_t c = (int64_t)strip * 64 + threadIdx.x;
        if (threadIdx.x < 64 && c < a.F) {
            uint32_t b = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                b = max(b, (part[w][threadIdx.x >> 1] >> (16 * (threadIdx.x & 1))) & 0xffffu);
            a.col_most[(int64_t)chunk * a.F + c] = (uint16_t)b;
        }
        return;
    }
    // (what every wave of the block joins of its waves' values)
    auto across = [&](uint32_t v, auto join) {
        __syncthreads();
        if (lane == 0)
            part[wave][0] = v;
        __syncthreads();
        return join(join(part[0][0], part[1][0]), join(part[2][0], part[3][0]));
    };
    // Rows of `len` values from at(r) on, kRowsAtOnce of them read at once: one(i, eight values), then
    // done(r, i, wide) by every lane.  The `last` first: so that the waves that have the fewest of one
    // kind of rows begin with the other.
    auto rows = [&](int64_t count, int64_t len, bool last, auto at, auto one, auto done) {
        const bool wide = len > 8192;
        const int threads = wide ? 256 : 64, t = wide ? (int)threadIdx.x : lane;
        const int64_t units = wide ? kNormParts : 4 * kNormParts;
        const int64_t id = wide ? blockIdx.x : 4 * blockIdx.x + wave;
        for (int64_t r = last ? units - 1 - id : id; r < count; r += kRowsAtOnce * units) {
            const uint16_t *row[kRowsAtOnce];
#pragma unroll
            for (int i = 0; i < kRowsAtOnce; ++i)
                row[i] = at(min(r + i * units, count - 1));      // (past the last, that one again)
#pragma unroll 4
            for (int64_t n = 8 * t; n < len; n += 8 * threads)
#pragma unroll
                for (int i = 0; i < kRowsAtOnce; ++i)
                    one(i, read(row[i] + n, len - n));
#pragma unroll
            for (int i = 0; i < kRowsAtOnce; ++i)
                done(min(r + i * units, count - 1), i, wide);
        }
    };
    float sum[kRowsAtOnce] = {}, norm_x = 0.0f, norm_w = 0.0f;
    rows(2 * a.F + a.M, a.K, false,
         [&](int64_t r) {
             return r < a.F ? a.wg + r * a.ldg : r < 2 * a.F ? a.wu + (r - a.F) * a.ldu : a.x + (r - 2 * a.F) * a.ldx;
         },
         [&](int i, u32x4 w) { sum[i] += squares8(w); },
         [&](int64_t r, int i, bool wide) {
#pragma unroll
             for (int o = 32; o > 0; o >>= 1)
                 sum[i] += __shfl_xor(sum[i], o);
             if (wide)
                 sum[i] = __builtin_bit_cast(float, across(__builtin_bit_cast(uint32_t, sum[i]), [](uint32_t p, uint32_t q) {
                     return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, p) + __builtin_bit_cast(float, q));
                 }));
             if (__builtin_isfinite(sum[i])) {
                 if (r < 2 * a.F)
                     norm_w = fmaxf(norm_w, sum[i]);
                 else
                     norm_x = fmaxf(norm_x, sum[i]);
             }
             sum[i] = 0.0f;
         });
    s16x2 most[kRowsAtOnce];
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i)
        most[i] = kZero;
    rows(a.M, a.F, true, [&](int64_t r) { return a.dh + r * a.lddh; },
         [&](int i, u32x4 w) { take(most[i], w[0]), take(most[i], w[1]), take(most[i], w[2]), take(most[i], w[3]); },
         [&](int64_t r, int i, bool wide) {
#pragma unroll
             for (int o = 32; o > 0; o >>= 1)
                 most[i] = __builtin_elementwise_max(most[i], __builtin_bit_cast(s16x2, __shfl_xor(__builtin_bit_cast(int, most[i]), o)));
             const s16x2 m = most[i] - kZero;
             uint32_t b = max((uint32_t)(uint16_t)m[0], (uint32_t)(uint16_t)m[1]);
             if (wide)
                 b = across(b, [](uint32_t p, uint32_t q) { return max(p, q); });
             if (wide ? threadIdx.x == 0 : lane == 0)
                 a.row_most[r] = (uint16_t)b;
             most[i] = kZero;
         });
    auto top = [](uint32_t p, uint32_t q) { return max(p, q); };     // (of values that are not negative)
    const uint32_t x = across(__builtin_bit_cast(uint32_t, norm_x), top), w = across(__builtin_bit_cast(uint32_t, norm_w), top);
    if (threadIdx.x == 0) {
        a.norms[blockIdx.x] = __builtin_bit_cast(float, x);
        a.norms[kNormParts + blockIdx.x] = __builtin_bit_cast(float, w);
    }
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
    constexpr bool UNITS = MODE == SUM_GRAD && IN == IN_FP16;
    int bound = 0;                          // (by whole waves, before any lane leaves)
    if constexpr (UNITS)
        bound = bound_exponent(p.norms, threadIdx.x & 63);
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
                const float d = in ? from_bits16(IN, p.dh[(int64_t)m * p.lddh + f + e]) : 0.0f;
                const float a = gate_value<true>(p.act, g[e], slope);
                dg[e] = in ? d * u[e] * slope : 0.0f;
                du[e] = in ? d * a : 0.0f;
            }
            auto put = [&](void *to, f32x4 unit) {
                store4<OUT>(to, (int64_t)m * p.ldc + n, unit * dg, true, 4);
                store4<OUT>(to, (int64_t)m * p.ldc + n + 8, unit * du, true, 4);
            };
            if constexpr (UNITS) {
                if (p.C) {
                    const int row = unit_exponent(p.row_most[m], bound);
                    const float unit = __builtin_ldexpf(1.0f, row);
                    put(p.C, (f32x4){unit, unit, unit, unit});
                    if (i == 0)
                        p.row_back[m] = __builtin_ldexpf(1.0f, -row);
                }
                if (p.C2) {
                    f32x4 unit;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int column = unit_exponent(column_most(p, min(f + e, p.cols - 1)), bound);
                        unit[e] = __builtin_ldexpf(1.0f, column);
                        if (m == 0 && f + e < p.cols)
                            p.col_back[f + e] = __builtin_ldexpf(1.0f, -column);
                    }
                    put(p.C2, unit);
                }
            } else {
                put(p.C, (f32x4){1.0f, 1.0f, 1.0f, 1.0f});
            }
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
    uint16_t *d, *dc;                   // dg and du [M][both(F)], FP16's in units of rows and of columns
    int strips, chunks, chunk_rows;     // gate_units'
    uint16_t *row_most, *col_most;
    float *norms, *row_back, *col_back;
    int64_t bytes;
};

BackwardWs carve_backward(int64_t M, int64_t F, int64_t K, int in_dtype, void *base)
{
    BackwardWs w{};
    Carver c{static_cast<uint8_t *>(base)};
    w.d = c.take<uint16_t>(M * both(F));
    w.dc = w.d;
    if (in_dtype == GEMM_FP16 && M > 0 && F > 0) {
        w.dc = c.take<uint16_t>(M * both(F));
        // chunks of 256 rows or more, up to 32 of them, that make about four blocks a compute unit
        w.strips = (int)cdiv(F, 64);
        const int64_t most = std::min<int64_t>(32, std::max<int64_t>(1, 4 * kNumCUs / w.strips));
        w.chunk_rows = (int)std::max<int64_t>(256, cdiv(M, most));
        w.chunks = (int)cdiv(M, w.chunk_rows);
        w.row_most = c.take<uint16_t>(M);
        w.col_most = c.take<uint16_t>(w.chunks * F);
        w.norms = c.take<float>(2 * kNormParts);
        w.row_back = c.take<float>(M);
        w.col_back = c.take<float>(F);
    }
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
    if (a.norms) {
        a.row_most += row;
        a.col_most += col;
        a.row_back += row;
        a.col_back += col;
    }
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
    // (FP16's, the larger one)
    return gemm_gated_backward_workspace_of(M, F, K, GEMM_FP16, bytes);
}

gemm_status_t gemm_gated_backward_workspace_of(int64_t M, int64_t F, int64_t K, int in_dtype, int64_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = check_sizes(M, F, K, in_dtype, GEMM_BF16, GEMM_GATE_SILU);
    if (st != GEMM_OK)
        return st;
    *bytes = carve_backward(M, F, K, in_dtype, nullptr).bytes;
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
    const BackwardWs w = carve_backward(M, F, K, in_dtype, workspace);
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
    a.row_most = w.row_most;
    a.col_most = w.col_most;
    a.col_chunks = w.chunks;
    a.col_step = (int)F;
    a.norms = w.norms;
    a.row_back = w.row_back;
    a.col_back = w.col_back;
    if (e == hipSuccess && w.norms) {
        UnitArgs u{a.dh, static_cast<const uint16_t *>(X), a.B, a.B2, M, F, (int)K, a.lddh, (int)ldx, a.ldb, a.ldb2,
                   w.strips, w.chunks, w.chunk_rows, w.row_most, w.col_most, w.norms};
        hipLaunchKernelGGL(gate_units, dim3((unsigned)(w.strips * w.chunks + kNormParts)), dim3(256), 0, stream, u);
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
        const int64_t at = q.row * both_cols + q.col;
        fill_args(b, p, w.sums.split[i], w.d + at, q.rows, q.cols, K, both_cols, in_dtype);
        if (w.norms) {
            // (a copy that nothing reads is not made)
            b.C = want_dx ? w.d + at : nullptr;
            b.C2 = want_dw ? w.dc + at : nullptr;
        }
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
        b.A = w.dc;
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
