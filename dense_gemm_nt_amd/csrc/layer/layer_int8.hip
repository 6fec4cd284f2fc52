// layer_int8.hip -- the product in 8-bit integers and its activations' quantization.
//
// y[m][n] = s_m t_n sum_k q[m][k] w[n][k].  v_mfma_i32_32x32x32_i8 takes 16 bytes of a row per
// lane, as the 16-bit MFMA does, and sums exactly in 32 bits, so the tiles run as they are on
// K / 2 elements of 16 bits; the scales come in when the sum is whole, K splits and all
// (int8_scale, int8_sum).
#include "layer_host.hpp"
#include "layer_launch.hpp"

namespace gnt {

template <int IN>
__device__ __forceinline__ float read_value(const void *x, int64_t i)
{
    if constexpr (IN == OUT_FP32)
        return static_cast<const float *>(x)[i];
    else
        return from_bits16(IN, static_cast<const uint16_t *>(x)[i]);
}

// Eight values from element i on; those at or past K are zero.
template <int IN>
__device__ __forceinline__ void read8(const void *x, int64_t i, int left, float (&v)[8])
{
    if (left >= 8) {
        if constexpr (IN == OUT_FP32) {
            const run32_t *s = reinterpret_cast<const run32_t *>(static_cast<const float *>(x) + i);
            const f32x4 a = s[0], b = s[1];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = a[e], v[4 + e] = b[e];
        } else {
            const u32x4 w = *reinterpret_cast<const run16_t *>(static_cast<const uint16_t *>(x) + i);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = from_bits16(IN, (w[e >> 1] >> (16 * (e & 1))) & 0xffffu);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = e < left ? read_value<IN>(x, i + e) : 0.0f;
    }
}

typedef uint32_t codes8_t __attribute__((ext_vector_type(2), aligned(1)));    // of rows of any length

// Codes and scale of a row: s = max |x| / 127, q = the nearest integer (even at a tie) to x / s,
// both quotients rounded to FP32 as IEEE division does.  A row of zeros: scale 0, codes 0; a row
// with an infinity or NaN: scale NaN, codes 0, so that its products are NaN.  TPR threads a
// row hold its first 32 TPR values in registers between the two passes; what is
// longer is read again (from L2).  A launch has fewer than 2^32 threads along an axis of its grid, so
// the blocks past 2^20 are on its second axis.  (With blocks that take rows in turn instead, 8111 x
// 8192 FP16 took 45.5 us, and 37.5 so.)
constexpr int64_t kQuantizeBlocks = (int64_t)1 << 20;

template <int IN, int TPR>
__global__ __launch_bounds__(256) void quantize_rows(const void *x, int8_t *codes, float *scale, int64_t M, int K,
                                                     int64_t ldx, int64_t ldq)
{
    constexpr int ROWS = 256 / TPR, HELD = 4;
    __shared__ uint32_t part[4];
    const int t = threadIdx.x % TPR;
    const int64_t m = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * ROWS + threadIdx.x / TPR;
    const bool live = m < M;
    const int64_t row = (live ? m : 0) * ldx;
    float v[HELD][8];
    uint32_t top = 0;
    auto most = [&](const float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max(top, __builtin_bit_cast(uint32_t, y[e]) & 0x7fffffffu);
    };
    if (live) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int k = (i * TPR + t) * 8;
            if (k < K) {
                read8<IN>(x, row + k, K - k, v[i]);
                most(v[i]);
            }
        }
        for (int k = (HELD * TPR + t) * 8; k < K; k += TPR * 8) {
            float y[8];
            read8<IN>(x, row + k, K - k, y);
            most(y);
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if constexpr (TPR > 64) {
        if (threadIdx.x % 64 == 0)
            part[threadIdx.x / 64] = top;
        __syncthreads();
        top = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    if (!live)
        return;
    const bool finite = top < 0x7f800000u;
    const float s = finite ? __builtin_bit_cast(float, top) / 127.0f : __builtin_nanf("");
    if (t == 0)
        scale[m] = s;
    const bool some = finite && s > 0.0f;
    // x times the reciprocal is within 127 * 2^-22 = 3.1e-5 of the quotient (s and its reciprocal
    // normal numbers, two roundings and the quotient's own), so further than that from a half it
    // rounds to the same integer; the eight values that hold a nearer one are divided.  Adding
    // 1.5 * 2^23 rounds to the integer, even at a tie, which is then in the low byte.
    // 8111 x 8192 FP16 40 us (4.9 TB/s), with eight divisions 53.
    constexpr float kRound = 12582912.0f;
    const bool quick = some && s > 1e-35f && s < 1e35f;
    const float inv = quick ? 1.0f / s : 0.0f;
    auto put = [&](int k, const float (&y)[8]) {
        uint32_t q[8];
        float far = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float t = y[e] * inv, r = t + kRound;
            far = fmaxf(far, fabsf(t - (r - kRound)));
            q[e] = __builtin_bit_cast(uint32_t, r);
        }
        if (!quick || far > 0.4999f) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                q[e] = some ? (uint32_t)(int)fminf(fmaxf(__builtin_rintf(y[e] / s), -127.0f), 127.0f) : 0u;
        }
        int8_t *dst = codes + m * ldq + k;
        if (k + 8 <= K) {
            codes8_t w;
#pragma unroll
            for (int d = 0; d < 2; ++d)
                w[d] = (q[4 * d] & 0xffu) | (q[4 * d + 1] & 0xffu) << 8 | (q[4 * d + 2] & 0xffu) << 16 | q[4 * d + 3] << 24;
            *reinterpret_cast<codes8_t *>(dst) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < K)
                    dst[e] = (int8_t)q[e];
        }
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int k = (i * TPR + t) * 8;
        if (k < K)
            put(k, v[i]);
    }
    for (int k = (HELD * TPR + t) * 8; k < K; k += TPR * 8) {
        float y[8];
        read8<IN>(x, row + k, K - k, y);
        put(k, y);
    }
}

// A few tokens' product without the tiles: all of it is the stream of B, which the lanes take 16
// bytes each straight into registers and multiply with v_dot4.  A block has four rows of B, its
// waves every fourth KB of them, two KB of each row in flight; exact sums, so their order does
// not matter.  No K splits, hence no counters and no second launch.  One and two rows, in us,
// against the tiles: 8192 x 8192 14.2 and 14.9 / 19.6, 28672 x 8192 36.0 and 37.0 / 38.8, 1024 x 4096 11.3 / 16.7,
// 8192 x 1024 11.5 / 11.4 (so from 2048 on); with four rows the loads of A, as many as B's, take over:
// 28672 x 8192 44.4 / 38.8.
constexpr int kFewRows = 2;

template <int OUT, int MR>
__global__ __launch_bounds__(256) void int8_few(Int8Args p, int K, int lda, int ldb)
{
    constexpr int R = 4;
    __shared__ int part[4][R][MR];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n0 = blockIdx.x * R;
    const int8_t *A = reinterpret_cast<const int8_t *>(p.A);
    const int8_t *B = reinterpret_cast<const int8_t *>(p.B);
    int acc[R][MR];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MR; ++m)
            acc[r][m] = 0;
#pragma unroll 2
    for (int k = wave * 1024 + lane * 16; k < K; k += 4096) {
        i32x4 b[R], a[MR];
#pragma unroll
        for (int r = 0; r < R; ++r)
            b[r] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(B + (int64_t)min(n0 + r, p.N - 1) * ldb + k));
#pragma unroll
        for (int m = 0; m < MR; ++m)
            a[m] = *reinterpret_cast<const i32x4 *>(A + (int64_t)min(m, p.M - 1) * lda + k);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int m = 0; m < MR; ++m)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    acc[r][m] = __builtin_amdgcn_sdot4(a[m][d], b[r][d], acc[r][m], false);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MR; ++m) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1)
                acc[r][m] += __shfl_xor(acc[r][m], o);
            if (lane == 0)
                part[wave][r][m] = acc[r][m];
        }
    __syncthreads();
    const int m = threadIdx.x;
    if (m >= p.M)
        return;
    f32x4 y;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int sum = (part[0][r][m] + part[1][r][m]) + (part[2][r][m] + part[3][r][m]);
        y[r] = (static_cast<float>(sum) * p.sa[m * p.sa_step]) * p.sb[(int64_t)min(n0 + r, p.N - 1) * p.sb_step];
    }
    store_result<OUT>(p, 0, m, n0, y);
}

// The second pass of a product split along K (tiles whose splits are not summed in the
// kernel): the integer partials, the scales as int8_scale has them, the epilogue.
template <int OUT>
__global__ __launch_bounds__(256) void int8_sum(Int8Args p)
{
    const int nvec = (p.N + 3) >> 2;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= (int64_t)p.M * nvec)
        return;
    const int m = (int)(t / nvec);
    const int n = (int)(t - (int64_t)m * nvec) * 4;
    const int valid = min(p.N - n, 4);
    const int64_t plane = (int64_t)p.M * p.N;
    const int *src = reinterpret_cast<const int *>(p.partials) + (int64_t)m * p.N + n;
    i32x4 sum = {0, 0, 0, 0};
    if ((p.N & 3) == 0) {
        for (int s = 0; s < p.splits; ++s)
            sum += *reinterpret_cast<const i32x4 *>(src + s * plane);
    } else {
        for (int s = 0; s < p.splits; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < valid)
                    sum[i] += src[s * plane + i];
    }
    const float sa = p.sa[(int64_t)m * p.sa_step];
    f32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = (static_cast<float>(sum[i]) * sa) * p.sb[(int64_t)min(n + i, p.N - 1) * p.sb_step];
    if (p.epi)
        y = epilogue4<OUT>(p, m, n, y, valid);
    store4<OUT>(p.C, (int64_t)m * p.ldc + n, y, p.vec_store != 0, valid);
}

namespace {

gemm_status_t check_sizes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0)
        return GEMM_ERR_INVALID_ARG;
    // (2^17 products of two codes of -128 end INT32's range)
    return M >= kMaxRows || N >= kMaxSize || K >= (1 << 17) || K % 16 ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

// The workspaces of a product's pieces.
struct Int8Ws {
    Pieces pieces;
    SplitWs split[2];
};

Int8Ws carve_int8(Carver &c, int64_t M, int64_t N, int64_t K)
{
    Int8Ws w;
    w.pieces = plan_pieces(M, N, K / 2);
    for (int i = 0; i < w.pieces.count; ++i)
        w.split[i] = carve_splits(c, w.pieces.at[i].plan);
    return w;
}

template <int MR>
hipError_t run_few_of(const Int8Args &a, int K, int lda, int ldb, int out_dtype, hipStream_t stream)
{
    const dim3 grid((unsigned)cdiv(a.N, 4));
    if (out_dtype == GEMM_BF16)
        hipLaunchKernelGGL((int8_few<OUT_BF16, MR>), grid, dim3(256), 0, stream, a, K, lda, ldb);
    else if (out_dtype == GEMM_FP16)
        hipLaunchKernelGGL((int8_few<OUT_FP16, MR>), grid, dim3(256), 0, stream, a, K, lda, ldb);
    else
        hipLaunchKernelGGL((int8_few<OUT_FP32, MR>), grid, dim3(256), 0, stream, a, K, lda, ldb);
    return hipGetLastError();
}

hipError_t run_few(const Int8Args &a, int K, int lda, int ldb, int out_dtype, hipStream_t stream)
{
    return a.M == 1 ? run_few_of<1>(a, K, lda, ldb, out_dtype, stream)
                    : run_few_of<2>(a, K, lda, ldb, out_dtype, stream);
}

// (a launch has fewer than 2^32 threads)
bool few_rows(int64_t M, int64_t N, int64_t K) { return M <= kFewRows && K >= 2048 && N < (1 << 25); }

gemm_status_t check_codes(const void *p, int64_t row, int64_t ld)
{
    if (ld < row || !p)
        return GEMM_ERR_INVALID_ARG;
    if (ld / 2 >= kMaxLeadingDim)
        return GEMM_ERR_UNSUPPORTED;
    return (uintptr_t)p % 16 || ld % 16 ? GEMM_ERR_MISALIGNED : GEMM_OK;
}

}  // namespace
}  // namespace gnt

using namespace gnt;

extern "C" {

gemm_status_t gemm_run_quantize_int8(const void *X, void *codes, float *scale, int64_t M, int64_t K, int64_t ldx,
                                     int64_t ldq, int in_dtype, hipStream_t stream)
{
    if (M < 0 || K < 0)
        return GEMM_ERR_INVALID_ARG;
    if (!is_out(in_dtype) || M >= kMaxRows || K >= kMaxSize - 16384)
        return GEMM_ERR_UNSUPPORTED;
    if (M == 0)
        return GEMM_OK;
    if (!scale || (K > 0 && (!X || !codes || ldx < K || ldq < K)))
        return GEMM_ERR_INVALID_ARG;
    const int64_t size = size_of(in_dtype);
    if ((uintptr_t)scale % 4 || (uintptr_t)X % size)
        return GEMM_ERR_MISALIGNED;
    const bool wave = K <= 2048;
    const int64_t blocks = cdiv(M, wave ? 4 : 1);
    const dim3 grid((unsigned)std::min(blocks, kQuantizeBlocks), (unsigned)cdiv(blocks, kQuantizeBlocks));
    auto launch = [&](auto in) {
        if (wave)
            hipLaunchKernelGGL((quantize_rows<in.value, 64>), grid, dim3(256), 0, stream, X,
                               static_cast<int8_t *>(codes), scale, M, (int)K, ldx, ldq);
        else
            hipLaunchKernelGGL((quantize_rows<in.value, 256>), grid, dim3(256), 0, stream, X,
                               static_cast<int8_t *>(codes), scale, M, (int)K, ldx, ldq);
    };
    if (in_dtype == GEMM_BF16)
        launch(std::integral_constant<int, OUT_BF16>{});
    else if (in_dtype == GEMM_FP16)
        launch(std::integral_constant<int, OUT_FP16>{});
    else
        launch(std::integral_constant<int, OUT_FP32>{});
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

gemm_status_t gemm_int8_workspace(int64_t M, int64_t N, int64_t K, int64_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = check_sizes(M, N, K);
    if (st != GEMM_OK)
        return st;
    Carver c{nullptr};
    if (M > 0 && N > 0 && !few_rows(M, N, K))
        carve_int8(c, M, N, K);
    *bytes = c.used;
    return GEMM_OK;
}

gemm_status_t gemm_run_int8(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K, int64_t lda,
                            int64_t ldb, int64_t ldc, int out_dtype, const float *scale_a, int64_t scales_a,
                            const float *scale_b, int64_t scales_b, const gemm_epilogue_t *epi, void *workspace,
                            int64_t workspace_bytes, hipStream_t stream)
{
    gemm_status_t st = check_sizes(M, N, K);
    if (st != GEMM_OK)
        return st;
    if (!is_out(out_dtype))
        return GEMM_ERR_UNSUPPORTED;
    if ((st = check_epilogue(epi)) != GEMM_OK)
        return st;
    if (M == 0 || N == 0)
        return GEMM_OK;
    if (!scale_a || !scale_b || (scales_a != 1 && scales_a != M) || (scales_b != 1 && scales_b != N))
        return GEMM_ERR_INVALID_ARG;
    if ((st = check_output(C, N, ldc, out_dtype)) != GEMM_OK)
        return st;
    if ((uintptr_t)scale_a % 4 || (uintptr_t)scale_b % 4)
        return GEMM_ERR_MISALIGNED;
    if (K > 0 && ((st = check_codes(A, K, lda)) != GEMM_OK || (st = check_codes(B, K, ldb)) != GEMM_OK))
        return st;
    const bool few = few_rows(M, N, K);
    Carver c{static_cast<uint8_t *>(workspace)};
    Int8Ws w{};
    if (!few) {
        w = carve_int8(c, M, N, K);
        if ((st = check_workspace(workspace, workspace_bytes, c.used)) != GEMM_OK)
            return st;
    }
    for (int i = 0; i < w.pieces.count; ++i)
        if (!launchable(w.pieces.at[i].plan))
            return GEMM_ERR_UNSUPPORTED;
    Int8Args a{};
    a.A = static_cast<const uint16_t *>(A);
    a.B = static_cast<const uint16_t *>(B);
    a.lda = (int)(lda / 2), a.ldb = (int)(ldb / 2);
    a.sa = scale_a, a.sb = scale_b;
    a.sa_step = scales_a != 1, a.sb_step = scales_b != 1;
    auto epilogue = [&](int64_t row, int64_t col) {       // after fill_args
        if (!epi)
            return;
        a.alpha = epi->alpha;
        a.beta = epi->beta;
        a.bias = epi->bias_along == GEMM_BIAS_N ? epi->bias + col : epi->bias_along == GEMM_BIAS_M ? epi->bias + row : nullptr;
        a.bias_along = epi->bias_along;
        a.act = epi->activation;
        a.bias_vec = (uintptr_t)a.bias % 16 == 0;
        a.epi = !(a.alpha == 1.0f && a.beta == 0.0f && a.bias_along == GEMM_BIAS_NONE && a.act == GEMM_ACT_NONE);
    };
    if (few) {
        Plan none{};
        none.tiles_m = none.tiles_n = none.splits = 1;
        fill_args(a, none, SplitWs{}, C, M, N, K / 2, ldc, out_dtype);
        epilogue(0, 0);
        return run_few(a, (int)K, (int)lda, (int)ldb, out_dtype, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
    }
    if (clear_counters(w.split, w.pieces.count, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    hipError_t e = hipSuccess;
    const Int8Args whole = a;
    for (int i = 0; i < w.pieces.count && e == hipSuccess; ++i) {
        const auto &q = w.pieces.at[i];
        const Plan &p = q.plan;
        a = whole;
        a.A += q.row * a.lda;
        a.B += q.col * a.ldb;
        a.sa += q.row * a.sa_step;
        a.sb += q.col * a.sb_step;
        fill_args(a, p, w.split[i], static_cast<uint8_t *>(C) + (q.row * ldc + q.col) * size_of(out_dtype), q.rows,
                  q.cols, K / 2, ldc, out_dtype);
        epilogue(q.row, q.col);
        const bool rot = rotate_slabs(1, q.rows);
        int8_fn fn;
        switch (p.cfg) {
        case CFG_T128x128: fn = (rot ? kInt8_128_s4_rot : kInt8_128_s4)[out_dtype]; break;
        case CFG_T128x128_S2: fn = (rot ? kInt8_128_s2_rot : kInt8_128_s2)[out_dtype]; break;
        case CFG_T32x128: fn = kInt8_32_rot[out_dtype]; break;
        case CFG_W4_256x128: fn = kInt8_w4[out_dtype]; break;
        default: fn = kInt8_pp2[out_dtype];
        }
        e = fn(a, (unsigned)p.grid, stream);
        if (e == hipSuccess && p.splits > 1 && !p.inreduce) {
            const unsigned grid = (unsigned)cdiv(q.rows * ((q.cols + 3) / 4), 256);
            if (out_dtype == GEMM_BF16)
                hipLaunchKernelGGL(int8_sum<OUT_BF16>, dim3(grid), dim3(256), 0, stream, a);
            else if (out_dtype == GEMM_FP16)
                hipLaunchKernelGGL(int8_sum<OUT_FP16>, dim3(grid), dim3(256), 0, stream, a);
            else
                hipLaunchKernelGGL(int8_sum<OUT_FP32>, dim3(grid), dim3(256), 0, stream, a);
            e = hipGetLastError();
        }
    }
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
