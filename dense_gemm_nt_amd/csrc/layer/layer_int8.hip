// layer_int8.hip -- the product in 8-bit integers and its activations' quantization.
//
// y[m][n] = s_m t_n sum_k q[m][k] w[n][k].  v_mfma_i32_32x32x32_i8 takes 16 bytes of a row per
// lane, as the 16-bit MFMA does, and sums exactly in 32 bits, so the tiles run as they are on
// K / 2 elements of 16 bits; the scales come in when the sum is whole (int8_scale).
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
__device__ __forceinline__ void read8(const void *x, int64_t i, bool wide, int left, float (&v)[8])
{
    if (wide && left >= 8) {
        if constexpr (IN == OUT_FP32) {
            const f32x4 *s = reinterpret_cast<const f32x4 *>(static_cast<const float *>(x) + i);
            const f32x4 a = s[0], b = s[1];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = a[e], v[4 + e] = b[e];
        } else {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(x) + i);
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

// Codes and scale of a row: s = max |x| / 127, q = the nearest integer (even at a tie) to x / s,
// both quotients rounded to FP32 as IEEE division does.  A row of zeros: scale 0, codes 0; a row
// with an infinity or NaN: scale NaN, codes 0, so that its products are NaN.  TPR threads a
// row hold its first 32 TPR values in registers between the two passes; what is
// longer is read again (from L2).
template <int IN, int TPR>
__global__ __launch_bounds__(256) void quantize_rows(const void *x, int8_t *codes, float *scale, int64_t M, int K,
                                                     int64_t ldx, int64_t ldq, int wide, int wide_q)
{
    constexpr int ROWS = 256 / TPR, HELD = 4;
    __shared__ uint32_t part[4];
    const int t = threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
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
                read8<IN>(x, row + k, wide, K - k, v[i]);
                most(v[i]);
            }
        }
        for (int k = (HELD * TPR + t) * 8; k < K; k += TPR * 8) {
            float y[8];
            read8<IN>(x, row + k, wide, K - k, y);
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
    auto put = [&](int k, const float (&y)[8]) {
        int8_t q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            q[e] = some ? (int8_t)fminf(fmaxf(__builtin_rintf(y[e] / s), -127.0f), 127.0f) : (int8_t)0;
        int8_t *dst = codes + m * ldq + k;
        if (wide_q && k + 8 <= K) {
            u32x2 w = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e >> 2] |= (uint32_t)(uint8_t)q[e] << (8 * (e & 3));
            *reinterpret_cast<u32x2 *>(dst) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < K)
                    dst[e] = q[e];
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
        read8<IN>(x, row + k, wide, K - k, y);
        put(k, y);
    }
}

namespace {

gemm_status_t check_sizes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0)
        return GEMM_ERR_INVALID_ARG;
    // (2^17 products of two codes of -128 end INT32's range)
    return M >= kMaxRows || N >= kMaxSize || K >= (1 << 17) || K % 16 ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

Plan plan_int8(int64_t M, int64_t N, int64_t K) { return make_plan(M, N, K / 2, kPartialBytes, -1, -1, 0); }

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
    const int wide = (ldx * size) % 16 == 0 && (uintptr_t)X % 16 == 0;
    const int wide_q = ldq % 8 == 0 && (uintptr_t)codes % 8 == 0;
    const bool wave = K <= 2048;
    const unsigned grid = (unsigned)cdiv(M, wave ? 4 : 1);
    auto launch = [&](auto in) {
        if (wave)
            hipLaunchKernelGGL((quantize_rows<in.value, 64>), dim3(grid), dim3(256), 0, stream, X,
                               static_cast<int8_t *>(codes), scale, M, (int)K, ldx, ldq, wide, wide_q);
        else
            hipLaunchKernelGGL((quantize_rows<in.value, 256>), dim3(grid), dim3(256), 0, stream, X,
                               static_cast<int8_t *>(codes), scale, M, (int)K, ldx, ldq, wide, wide_q);
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
    if (M > 0 && N > 0)
        carve_splits(c, plan_int8(M, N, K));
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
    const Plan p = plan_int8(M, N, K);
    Carver c{static_cast<uint8_t *>(workspace)};
    const SplitWs w = carve_splits(c, p);
    if ((st = check_workspace(workspace, workspace_bytes, c.used)) != GEMM_OK)
        return st;
    if (!launchable(p))
        return GEMM_ERR_UNSUPPORTED;
    Int8Args a{};
    fill_args(a, p, w, C, M, N, K / 2, ldc, out_dtype);
    a.A = static_cast<const uint16_t *>(A);
    a.B = static_cast<const uint16_t *>(B);
    a.lda = (int)(lda / 2), a.ldb = (int)(ldb / 2);
    a.sa = scale_a, a.sb = scale_b;
    a.sa_step = scales_a != 1, a.sb_step = scales_b != 1;
    if (epi) {
        a.alpha = epi->alpha;
        a.beta = epi->beta;
        a.bias = epi->bias_along != GEMM_BIAS_NONE ? epi->bias : nullptr;
        a.bias_along = epi->bias_along;
        a.act = epi->activation;
        a.bias_vec = (uintptr_t)a.bias % 16 == 0;
        a.epi = !(a.alpha == 1.0f && a.beta == 0.0f && a.bias_along == GEMM_BIAS_NONE && a.act == GEMM_ACT_NONE);
    }
    if (clear_counters(&w, 1, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    const bool rot = rotate_slabs(1, M);
    int8_fn fn;
    switch (p.cfg) {
    case CFG_T128x128: fn = (rot ? kInt8_128_s4_rot : kInt8_128_s4)[out_dtype]; break;
    case CFG_T128x128_S2: fn = kInt8_128_s2[out_dtype]; break;
    case CFG_T32x128: fn = kInt8_32_rot[out_dtype]; break;
    case CFG_W4_256x128: fn = kInt8_w4[out_dtype]; break;
    default: fn = kInt8_pp2[out_dtype];
    }
    hipError_t e = fn(a, (unsigned)p.grid, stream);
    if (e == hipSuccess && p.splits > 1 && !p.inreduce) {
        const KernelArgs &k = a;
        const unsigned grid = (unsigned)cdiv(M * ((N + 3) / 4), 256);
        if (out_dtype == GEMM_BF16)
            hipLaunchKernelGGL(splitk_sum<OUT_BF16>, dim3(grid), dim3(256), 0, stream, k);
        else if (out_dtype == GEMM_FP16)
            hipLaunchKernelGGL(splitk_sum<OUT_FP16>, dim3(grid), dim3(256), 0, stream, k);
        else
            hipLaunchKernelGGL(splitk_sum<OUT_FP32>, dim3(grid), dim3(256), 0, stream, k);
        e = hipGetLastError();
    }
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
