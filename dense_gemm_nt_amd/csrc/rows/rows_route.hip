// rows_route.hip -- the top-k router: softmax, choices, per-expert counts and
// order, balance loss; and its gradient.
//
// A token's logits are spread over LPR lanes of 4 Q columns each (columns
// 4 LPR q + 4 li + i for lane li), so a row is read once, coalesced, and held
// in registers: maximum, sum and the k choices come from reductions over the
// LPR lanes.  A choice is one maximum over the lanes and a ballot for its
// first holder, so ties fall to the lowest column.
#include <type_traits>

#include "rows_group.hpp"
#include "rows_host.hpp"

namespace gnt {
namespace {

enum : int { L_BF16 = 0, L_FP16 = 1, L_FP32 = 2 };

struct RouteArgs {
    const void *logits;
    const uint8_t *mask;
    int64_t T, ld;
    int E, k, renorm, vec;
    int64_t per_block;        // tokens of a block
    int blocks;
    int32_t *ids;
    float *weights;
    int32_t *counts, *offsets, *order, *tokens;
    float *loss;
    int *hist;                // [blocks][E + 1]
    float *psum;              // [blocks][E]
    int *live;                // [blocks]
    // backward
    const float *grad_w, *grad_loss;
    void *dlogits;
    int64_t ldd;
    int vec_d;
};

template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    const int v = __builtin_bit_cast(int, x);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, false));
}

// x combined over the LPR lanes of a row, in every one of them.
template <int LPR, typename F>
__device__ __forceinline__ float over_row(float x, F op)
{
    if constexpr (LPR >= 2)
        x = op(x, dpp<0xB1>(x));       // lanes 1 apart
    if constexpr (LPR >= 4)
        x = op(x, dpp<0x4E>(x));       // 2 apart
    if constexpr (LPR >= 8)
        x = op(x, dpp<0x141>(x));      // the other quad of eight
    if constexpr (LPR >= 16)
        x = op(x, dpp<0x140>(x));      // the other eight of sixteen
    if constexpr (LPR >= 32) {
        const unsigned v = __builtin_bit_cast(unsigned, x);
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        const unsigned lo = r[0], hi = r[1];   // (values: a bit cast of an element takes the first)
        x = op(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
    }
    if constexpr (LPR >= 64) {
        const unsigned v = __builtin_bit_cast(unsigned, x);
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        const unsigned lo = r[0], hi = r[1];   // (values: a bit cast of an element takes the first)
        x = op(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
    }
    return x;
}

template <int LPR>
__device__ __forceinline__ float row_max(float x)
{
    return over_row<LPR>(x, [](float a, float b) { return fmaxf(a, b); });
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
    return over_row<LPR>(x, [](float a, float b) { return a + b; });
}

// Four consecutive values of a row from column c; past E: -inf.
template <int DT>
__device__ __forceinline__ f32x4 load_logits(const void *base, int64_t row, int c, int E, int vec)
{
    f32x4 x;
    if constexpr (DT == L_FP32) {
        const float *p = static_cast<const float *>(base) + row + c;
        if (vec && c + 4 <= E)
            return *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = c + i < E ? p[i] : -INFINITY;
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + row + c;
        uint16_t h[4];
        if (vec && c + 4 <= E) {
            const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
            h[0] = (uint16_t)w[0], h[1] = (uint16_t)(w[0] >> 16);
            h[2] = (uint16_t)w[1], h[3] = (uint16_t)(w[1] >> 16);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = from16<DT>(h[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = c + i < E ? from16<DT>(p[i]) : -INFINITY;
        }
    }
    return x;
}

template <int DT>
__device__ __forceinline__ void store_logits(void *base, int64_t row, int c, int E, int vec, f32x4 x)
{
    if constexpr (DT == L_FP32) {
        float *p = static_cast<float *>(base) + row + c;
        if (vec && c + 4 <= E) {
            *reinterpret_cast<f32x4 *>(p) = x;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < E)
                p[i] = x[i];
    } else {
        uint16_t *p = static_cast<uint16_t *>(base) + row + c;
        if (vec && c + 4 <= E) {
            u32x2 w;
            w[0] = (uint32_t)to16<DT>(x[0]) | ((uint32_t)to16<DT>(x[1]) << 16);
            w[1] = (uint32_t)to16<DT>(x[2]) | ((uint32_t)to16<DT>(x[3]) << 16);
            *reinterpret_cast<u32x2 *>(p) = w;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < E)
                p[i] = to16<DT>(x[i]);
    }
}

// A row's softmax from its logits: p in place of x; false for a row without an
// open expert.  key is the ranking value of each logit (NaN as the lowest
// finite one).
template <int LPR, int Q>
__device__ __forceinline__ bool softmax_row(f32x4 (&x)[Q], f32x4 (&key)[Q])
{
    float top = -INFINITY;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            key[q][i] = x[q][i] != x[q][i] ? -3.402823466e38f : x[q][i];
            top = fmaxf(top, key[q][i]);
        }
    top = row_max<LPR>(top);
    const bool open = top > -INFINITY;
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[q][i] = open ? __expf(x[q][i] - top) : 0.0f;
            sum += x[q][i];
        }
    sum = row_sum<LPR>(sum);
    const float inv = open ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[q][i] *= inv;
    return open;
}

// The balance loss from counts (a function of e) and the routed tokens' sums of p.
template <typename P, typename C>
__device__ __forceinline__ void balance_loss(const RouteArgs &a, int n, P psum, C count, float *red)
{
    float part = 0.0f;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        part += (float)count(e) * psum(e);
    part = row_sum<64>(part);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = part;
    __syncthreads();
    if (threadIdx.x == 0) {
        float s = 0.0f;
        for (int w = 0; w < (int)(blockDim.x >> 6); ++w)
            s += red[w];
        const float nf = (float)n;
        *a.loss = n > 0 ? (float)a.E * (s / nf) / (nf * (float)a.k) : 0.0f;
        *a.tokens = n;
    }
}

// One block of tokens: choices, weights, the block's counts and sums of p.
// ONE: the only block, which then also finishes (counts, order, loss).
template <int DT, int LPR, int Q, bool ONE>
__global__ __launch_bounds__(kGroupThreads) void route_forward(RouteArgs a)
{
    constexpr int NW = kGroupThreads / 64, GPW = 64 / LPR, COLS = LPR * 4 * Q;
    __shared__ int hist[kMaxGroups + 1];
    __shared__ float ps[NW][COLS];
    __shared__ int live[NW];
    __shared__ std::conditional_t<ONE, PlaceLds, int> place;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int li = lane % LPR, grp = lane / LPR;
    for (int e = tid; e <= a.E; e += kGroupThreads)
        hist[e] = 0;
    __syncthreads();

    const int64_t t0 = blockIdx.x * a.per_block;
    const int64_t t1 = t0 + a.per_block < a.T ? t0 + a.per_block : a.T;
    f32x4 sum[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        sum[q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    int routed = 0;
    for (int64_t base = t0 + wave * GPW; base < t1; base += NW * GPW) {
        const int64_t t = base + grp;
        const bool in = t < t1;
        const bool on = in && (!a.mask || a.mask[t]);
        f32x4 x[Q], key[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q)
            x[q] = on ? load_logits<DT>(a.logits, t * a.ld, q * LPR * 4 + li * 4, a.E, a.vec)
                      : (f32x4){-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const bool open = softmax_row<LPR, Q>(x, key);
        routed += open && li == 0;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            sum[q] += x[q];
        // the k largest, one at a time: the maximum over the row, its first holder
        uint8_t place_of[4 * Q];
#pragma unroll
        for (int i = 0; i < 4 * Q; ++i)
            place_of[i] = 0xff;
        float chosen = 0.0f;
        int found = 0;
        for (int j = 0; j < a.k; ++j) {
            float best = -INFINITY;
#pragma unroll
            for (int q = 0; q < Q; ++q)
                best = fmaxf(best, fmaxf(fmaxf(key[q][0], key[q][1]), fmaxf(key[q][2], key[q][3])));
            best = row_max<LPR>(best);
            if (__builtin_amdgcn_ballot_w64(best > -INFINITY) == 0)
                break;
            bool open_yet = best > -INFINITY;
            found += open_yet;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const bool mine = open_yet && (key[q][0] == best || key[q][1] == best || key[q][2] == best ||
                                               key[q][3] == best);
                const uint64_t all = __builtin_amdgcn_ballot_w64(mine);
                const uint64_t row = LPR == 64 ? all : (all >> (grp * LPR)) & ((1ull << (LPR & 63)) - 1);
                if (row && mine && __builtin_ctzll(row) == li) {
                    bool taken = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!taken && key[q][i] == best) {
                            taken = true;
                            key[q][i] = -INFINITY;
                            place_of[4 * q + i] = (uint8_t)j;
                            chosen += x[q][i];
                        }
                }
                open_yet = open_yet && row == 0;
            }
        }
        chosen = row_sum<LPR>(chosen);
        const float scale = a.renorm && found ? 1.0f / chosen : 1.0f;
        if (in) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (place_of[4 * q + i] != 0xff) {
                        const int e = q * LPR * 4 + li * 4 + i;
                        a.ids[t * a.k + place_of[4 * q + i]] = e;
                        a.weights[t * a.k + place_of[4 * q + i]] = x[q][i] * scale;
                        atomicAdd(&hist[e], 1);
                    }
            for (int j = found + li; j < a.k; j += LPR) {
                a.ids[t * a.k + j] = -1;
                a.weights[t * a.k + j] = 0.0f;
                atomicAdd(&hist[a.E], 1);
            }
        }
    }
    // the block's sums of p: over the rows of a wave, then over the waves
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = sum[q][i];
            for (int o = LPR; o < 64; o <<= 1)
                v += __shfl_xor(v, o);
            if (grp == 0)
                ps[wave][q * LPR * 4 + li * 4 + i] = v;
        }
    for (int o = 32; o; o >>= 1)
        routed += __shfl_xor(routed, o);
    if (lane == 0)
        live[wave] = routed;
    __syncthreads();
    auto psum = [&](int e) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            v += ps[w][e];
        return v;
    };
    int n = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        n += live[w];
    if constexpr (ONE) {
        store_hist(hist, a.hist, a.E);
        balance_loss(a, n, psum, [&](int e) { return hist[e]; }, reinterpret_cast<float *>(place.part));
        __syncthreads();
        place_block(place, a.ids, a.T * a.k, a.E, a.per_block * a.k, a.hist, 0, 1, a.counts, a.offsets,
                    a.order);
    } else {
        store_hist(hist, a.hist, a.E);
        for (int e = tid; e < a.E; e += kGroupThreads)
            a.psum[(int64_t)blockIdx.x * a.E + e] = psum(e);
        if (tid == 0)
            a.live[blockIdx.x] = n;
    }
}

// The second launch of a larger batch: counts, offsets, order; the loss.
__global__ __launch_bounds__(kGroupThreads) void route_finish(RouteArgs a)
{
    __shared__ PlaceLds place;
    if ((int)blockIdx.x == a.blocks) {
        // one block more than the entries': the loss, from the blocks' sums in order
        int n = 0;
        for (int i = 0; i < a.blocks; ++i)
            n += a.live[i];
        auto psum = [&](int e) {
            float v = 0.0f;
#pragma unroll 8
            for (int i = 0; i < a.blocks; ++i)
                v += a.psum[(int64_t)i * a.E + e];
            return v;
        };
        auto count = [&](int e) {
            int c = 0;
#pragma unroll 8
            for (int i = 0; i < a.blocks; ++i)
                c += a.hist[(int64_t)i * (a.E + 1) + e];
            return c;
        };
        balance_loss(a, n, psum, count, reinterpret_cast<float *>(place.part));
        return;
    }
    place_block(place, a.ids, a.T * a.k, a.E, a.per_block * a.k, a.hist, blockIdx.x, a.blocks, a.counts,
                a.offsets, a.order);
}

// dlogit = p (dp - sum p dp), dp_e = g_loss E f_e / n + (the gradient of e's
// weight, if chosen): p is recomputed from the logits, which are read once.
template <int DT, int LPR, int Q>
__global__ __launch_bounds__(256) void route_backward(RouteArgs a)
{
    constexpr int GPW = 64 / LPR;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane % LPR, grp = lane / LPR;
    const float n = (float)*a.tokens;
    const float gl = a.grad_loss && n > 0.0f ? *a.grad_loss * (float)a.E / (n * n * (float)a.k) : 0.0f;
    f32x4 from_loss[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = q * LPR * 4 + li * 4 + i;
            from_loss[q][i] = e < a.E ? gl * (float)a.counts[e] : 0.0f;
        }
    const int64_t step = (int64_t)gridDim.x * 4 * GPW;
    for (int64_t base = ((int64_t)blockIdx.x * 4 + wave) * GPW; base < a.T; base += step) {
        const int64_t t = base + grp;
        const bool in = t < a.T;
        const bool on = in && a.ids[t * a.k] >= 0;     // a routed token has a first choice
        f32x4 x[Q], key[Q], dp[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q)
            x[q] = on ? load_logits<DT>(a.logits, t * a.ld, q * LPR * 4 + li * 4, a.E, a.vec)
                      : (f32x4){-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        softmax_row<LPR, Q>(x, key);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            dp[q] = from_loss[q];
        if (a.grad_w) {
            // sums over the choices: of g w, and (renormalized) of p
            float gw = 0.0f, total = 1.0f;
            if (a.renorm) {
                float s = 0.0f;
                for (int j = 0; j < a.k; ++j) {
                    const int e = on ? a.ids[t * a.k + j] : -1;
                    if (e >= 0)
                        gw += a.grad_w[t * a.k + j] * a.weights[t * a.k + j];
#pragma unroll
                    for (int q = 0; q < Q; ++q)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (e == q * LPR * 4 + li * 4 + i)
                                s += x[q][i];
                }
                s = row_sum<LPR>(s);
                total = s != 0.0f ? s : 1.0f;
            }
            for (int j = 0; j < a.k; ++j) {
                const int e = on ? a.ids[t * a.k + j] : -1;
                const float h = e >= 0 ? (a.grad_w[t * a.k + j] - gw) / total : 0.0f;
#pragma unroll
                for (int q = 0; q < Q; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dp[q][i] += e == q * LPR * 4 + li * 4 + i ? h : 0.0f;
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dot += x[q][i] * dp[q][i];
        dot = row_sum<LPR>(dot);
        if (in)
#pragma unroll
            for (int q = 0; q < Q; ++q)
                store_logits<DT>(a.dlogits, t * a.ldd, q * LPR * 4 + li * 4, a.E, a.vec_d, x[q] * (dp[q] - dot));
    }
}

// The number of blocks of the forward launch, at most 128: each later block
// reads every block's counts.
int64_t tokens_per_block(int64_t T)
{
    return std::max<int64_t>(cdiv(cdiv(T, 128), 64) * 64, 64);
}

template <typename F>
gemm_status_t by_width(int E, F launch)
{
    if (E <= 16)
        launch(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
    else if (E <= 64)
        launch(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    else if (E <= 256)
        launch(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (E <= 512)
        launch(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    else
        launch(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

template <typename F>
gemm_status_t by_type(int dtype, int E, F launch)
{
    if (dtype == GEMM_BF16)
        return by_width(E, [&](auto l, auto q) { launch(std::integral_constant<int, L_BF16>{}, l, q); });
    if (dtype == GEMM_FP16)
        return by_width(E, [&](auto l, auto q) { launch(std::integral_constant<int, L_FP16>{}, l, q); });
    return by_width(E, [&](auto l, auto q) { launch(std::integral_constant<int, L_FP32>{}, l, q); });
}

gemm_status_t check_route(int64_t T, int64_t E, int64_t k)
{
    if (T < 0 || E < 0 || k < 0)
        return GEMM_ERR_INVALID_ARG;
    if (E < 1 || E > kMaxGroups || k < 1 || k > E || k > 64 || T >= kMaxSize || T * k >= kMaxSize)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// four values of a row as one load: every row starts aligned to it
bool rows_vectorize(const void *p, int64_t ld, int dtype)
{
    return (uintptr_t)p % (4 * size_of(dtype)) == 0 && ld % 4 == 0;
}

void carve_route(Carver &c, RouteArgs &a)
{
    a.hist = c.take<int>((int64_t)a.blocks * (a.E + 1));
    a.psum = c.take<float>((int64_t)a.blocks * a.E);
    a.live = c.take<int>(a.blocks);
}

}  // namespace
}  // namespace gnt

using namespace gnt;

extern "C" {

gemm_status_t gemm_route_workspace(int64_t T, int64_t E, int64_t top_k, int64_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_INVALID_ARG;
    *bytes = 0;
    const gemm_status_t st = check_route(T, E, top_k);
    if (st != GEMM_OK)
        return st;
    RouteArgs a{};
    a.E = (int)E;
    a.blocks = (int)std::max<int64_t>(1, cdiv(T, tokens_per_block(T)));
    Carver c{nullptr};
    carve_route(c, a);
    *bytes = c.used;
    return GEMM_OK;
}

gemm_status_t gemm_run_route(const void *logits, const uint8_t *mask, int64_t T, int64_t E,
                             int64_t ld, int64_t top_k, int renormalize, int dtype,
                             const gemm_routing_t *out, void *workspace, int64_t workspace_bytes,
                             hipStream_t stream)
{
    gemm_status_t st = check_route(T, E, top_k);
    if (st != GEMM_OK)
        return st;
    if (!is_out(dtype) || ld >= kMaxSize)
        return GEMM_ERR_UNSUPPORTED;
    if (ld < E || !out || !out->counts || !out->offsets || !out->tokens || !out->loss ||
        (T > 0 && (!logits || !out->ids || !out->weights || !out->order)))
        return GEMM_ERR_INVALID_ARG;
    for (const void *p : {(const void *)out->ids, (const void *)out->weights, (const void *)out->counts,
                          (const void *)out->offsets, (const void *)out->order, (const void *)out->tokens,
                          (const void *)out->loss})
        if ((uintptr_t)p % 4)
            return GEMM_ERR_MISALIGNED;
    if ((uintptr_t)logits % size_of(dtype))
        return GEMM_ERR_MISALIGNED;
    RouteArgs a{};
    a.logits = logits;
    a.mask = mask;
    a.T = T;
    a.ld = ld;
    a.E = (int)E;
    a.k = (int)top_k;
    a.renorm = renormalize != 0;
    a.vec = rows_vectorize(logits, ld, dtype);
    a.per_block = tokens_per_block(T);
    a.blocks = (int)std::max<int64_t>(1, cdiv(T, a.per_block));
    a.ids = out->ids;
    a.weights = out->weights;
    a.counts = out->counts;
    a.offsets = out->offsets;
    a.order = out->order;
    a.tokens = out->tokens;
    a.loss = out->loss;
    Carver c{static_cast<uint8_t *>(workspace)};
    carve_route(c, a);
    if ((st = check_workspace(workspace, workspace_bytes, c.used)) != GEMM_OK)
        return st;
    const bool one = a.blocks == 1;
    st = by_type(dtype, a.E, [&](auto dt, auto lpr, auto q) {
        if (one)
            hipLaunchKernelGGL((route_forward<dt.value, lpr.value, q.value, true>), dim3(1), dim3(kGroupThreads),
                               0, stream, a);
        else
            hipLaunchKernelGGL((route_forward<dt.value, lpr.value, q.value, false>), dim3(a.blocks),
                               dim3(kGroupThreads), 0, stream, a);
    });
    if (st != GEMM_OK || one)
        return st;
    hipLaunchKernelGGL(route_finish, dim3(a.blocks + 1), dim3(kGroupThreads), 0, stream, a);
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

gemm_status_t gemm_run_route_backward(const void *logits, const gemm_routing_t *in,
                                      const float *grad_weights, const float *grad_loss,
                                      void *dlogits, int64_t T, int64_t E, int64_t ld, int64_t ldd,
                                      int64_t top_k, int renormalize, int dtype,
                                      hipStream_t stream)
{
    const gemm_status_t st = check_route(T, E, top_k);
    if (st != GEMM_OK)
        return st;
    if (!is_out(dtype) || ld >= kMaxSize || ldd >= kMaxSize)
        return GEMM_ERR_UNSUPPORTED;
    if (ld < E || ldd < E || !in)
        return GEMM_ERR_INVALID_ARG;
    if (T == 0)
        return GEMM_OK;
    if (!logits || !dlogits || !in->ids || !in->weights || !in->counts || !in->tokens)
        return GEMM_ERR_INVALID_ARG;
    if ((uintptr_t)logits % size_of(dtype) || (uintptr_t)dlogits % size_of(dtype) ||
        (uintptr_t)grad_weights % 4 || (uintptr_t)grad_loss % 4 || (uintptr_t)in->ids % 4 ||
        (uintptr_t)in->weights % 4 || (uintptr_t)in->counts % 4 || (uintptr_t)in->tokens % 4)
        return GEMM_ERR_MISALIGNED;
    RouteArgs a{};
    a.logits = logits;
    a.T = T;
    a.ld = ld;
    a.E = (int)E;
    a.k = (int)top_k;
    a.renorm = renormalize != 0;
    a.vec = rows_vectorize(logits, ld, dtype);
    a.ids = in->ids;
    a.weights = in->weights;
    a.counts = in->counts;
    a.tokens = in->tokens;
    a.grad_w = grad_weights;
    a.grad_loss = grad_loss;
    a.dlogits = dlogits;
    a.ldd = ldd;
    a.vec_d = rows_vectorize(dlogits, ldd, dtype);
    return by_type(dtype, a.E, [&](auto dt, auto lpr, auto q) {
        constexpr int rows = 4 * 64 / lpr.value;       // of a block and pass
        const unsigned grid = (unsigned)std::min<int64_t>(cdiv(T, rows), 2048);
        hipLaunchKernelGGL((route_backward<dt.value, lpr.value, q.value>), dim3(grid), dim3(256), 0, stream, a);
    });
}

}  // extern "C"
