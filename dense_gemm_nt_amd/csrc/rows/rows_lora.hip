// rows_lora.hip -- a shared projection with low-rank adapters picked per row:
// the low-rank products, the adapters' gradients, and the host side.  (The
// product with the up matrices is part of the projection's own kernel:
// lora_add in rows_common.hpp.)
#include "rows_group.hpp"
#include "rows_host.hpp"
#include "rows_index.hpp"
#include "rows_launch.hpp"

namespace gnt {
namespace {

constexpr int kShrinkWaves = 8;
constexpr int kMaxLowSplits = 16;

struct ShrinkArgs {
    const uint16_t *x;        // [M][K]
    const uint16_t *down;     // adapter a: rank rows of down_ld at a * down_stride
    const int32_t *ids;
    float *low;               // [splits][M][rank_pad]
    int64_t down_stride;
    int M, K, ldx, down_ld, adapters, rank, rank_pad;
    int k_per_split;          // a multiple of the kernel's K step
};

// One or two low-rank products of the same rows and adapters in one launch (a
// training step's two: x with A, dy with B transposed): K splits z < first of the
// one, the rest of the other.
struct ShrinkPair {
    ShrinkArgs a[2];
    int first;
    int lanes_j;              // blocks sharing a row tile's adapters (gridDim.y)
    unsigned *counters;       // zeroed here for the projection's split reduction
    int num_counters;
};

__device__ __forceinline__ void clear_counters(const ShrinkPair &pair)
{
    const Walk w = clear_walk(blockIdx.x, blockIdx.y, blockIdx.z, gridDim.x, gridDim.y, gridDim.z, blockDim.x, threadIdx.x);
    for (int64_t i = w.first; i < pair.num_counters; i += w.step)
        pair.counters[i] = 0;
}

// low[s][m][r] = sum over split s of K of x[m][k] down_a[r][k], a = ids[m].
//
// One block takes 16 rows and one K split; its eight waves take K in steps
// of 128 in turn (a wave reads 256 contiguous bytes of each row and of each
// rank's row per step) and add up through LDS in wave order.  For each adapter
// among the tile's rows all the rows are multiplied and the adapter's own kept:
// MFMA work is free here (the bytes of x and of the adapters bound the kernel),
// and no sorting of rows is needed.  A decode batch puts the adapters of a row
// tile on different blocks (lanes_j), and K splits over more of them.
// 1 x 4096, rank 16: 3.6 us; 64 x 8192, rank 16, 48 adapters 7.5 us (16 MB: the
// round trips bound it, not the bytes); 836 x 5952, rank 16, 61 adapters 48 us (every row tile
// reads about 14 adapters: 280 MB out of the caches).
template <int IN, int RT>
__global__ __launch_bounds__(kShrinkWaves * 64) void lora_shrink(ShrinkPair pair)
{
    const bool second = (int)blockIdx.z >= pair.first;
    const ShrinkArgs &p = pair.a[second];
    const int z = blockIdx.z - (second ? pair.first : 0);
    constexpr int W = kShrinkWaves, ROWS = 16, COLS = 16 * RT;
    __shared__ float part[W][ROWS][COLS + 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    clear_counters(pair);

    const int r0 = blockIdx.x * ROWS;
    const int m = r0 + (lane & (ROWS - 1));
    const int a_in = m < p.M ? p.ids[m] : -1;
    const int id = (uint32_t)a_in < (uint32_t)p.adapters ? a_in : -1;
    uint64_t left = __builtin_amdgcn_ballot_w64(id >= 0) & ((1ull << ROWS) - 1);
    const int kb = z * p.k_per_split;
    const int ke = min(p.K, kb + p.k_per_split);
    const int rows = min(ROWS, p.M - r0);
    const __amdgpu_buffer_rsrc_t rs_x =
        make_rsrc(p.x + (int64_t)r0 * p.ldx, (uint32_t)rows * (uint32_t)p.ldx * 2u);
    const int li = lane & 15, kq = 8 * (lane >> 4);
    float *out = p.low + (int64_t)z * p.M * p.rank_pad;

    for (int nth = 0; left; ++nth) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        left &= ~__builtin_amdgcn_ballot_w64(id == a);
        if (nth % pair.lanes_j != (int)blockIdx.y)
            continue;
        for (int c0 = 0; c0 < p.rank_pad; c0 += COLS) {
            const uint32_t d_bytes = __builtin_amdgcn_readfirstlane(
                (uint32_t)max(0, min(COLS, p.rank - c0)) * (uint32_t)p.down_ld * 2u);
            const __amdgpu_buffer_rsrc_t rs_d =
                make_rsrc(p.down + a * p.down_stride + (int64_t)c0 * p.down_ld, d_bytes);
            f32x4 acc[RT];
#pragma unroll
            for (int j = 0; j < RT; ++j)
                acc[j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
            for (int k0 = kb + wave * 128; k0 < ke; k0 += W * 128) {
                u32x4 xf[4], df[4][RT];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int k = k0 + 32 * s + kq;
                    const bool in = k < ke;         // K is a multiple of 8
                    xf[s] = __builtin_bit_cast(
                        u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                   rs_x, in && li < rows ? ((uint32_t)li * (uint32_t)p.ldx + (uint32_t)k) * 2u : kOutOfRange,
                                   0, 0));
#pragma unroll
                    for (int j = 0; j < RT; ++j)
                        df[s][j] = __builtin_bit_cast(
                            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                       rs_d,
                                       in && c0 + 16 * j + li < p.rank
                                           ? ((uint32_t)(16 * j + li) * (uint32_t)p.down_ld + (uint32_t)k) * 2u
                                           : kOutOfRange,
                                       0, 0));
                }
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int j = 0; j < RT; ++j)
                        acc[j] = mfma16x16x32<IN>(xf[s], df[s][j], acc[j]);
            }
            mfma_settle();
            __syncthreads();          // the last adapter's sums have been read
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    part[wave][4 * (lane >> 4) + e][16 * j + li] = acc[j][e];
            __syncthreads();
            for (int t = tid; t < ROWS * COLS; t += W * 64) {
                const int row = t / COLS, col = t % COLS;
                if (r0 + row < p.M && c0 + col < p.rank_pad && p.ids[r0 + row] == a) {
                    float v = 0.0f;
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        v += part[w][row][col];
                    out[(int64_t)(r0 + row) * p.rank_pad + c0 + col] = v;
                }
            }
        }
    }
}

// The same product for many rows.  A block takes 64 rows and one K split, and
// walks K in 64-deep slabs through an LDS ring filled by direct-to-LDS loads (1 KB a
// wave: 8 rows of 128 bytes, whole cache lines, where the kernel above reads 64
// bytes of 16 rows an instruction into registers and every 16 rows read all of
// an adapter).  A slab holds 64 rows of x and 64 rank rows: those of one
// adapter of up to 64 ranks, or of two or four adapters of up to 32 or 16, so
// that a tile's adapters take few passes over its rows; a higher rank takes two
// passes.  Wave w multiplies rows 16 w .. +16 with all 64 ranks, and keeps each row's
// own adapter's.  Bytes bound it: 8 slabs, 64 KB of x, are in flight a compute unit.
// In calls whose projection's operands pass in between: 5001 x 8192, rank 64, 4 adapters
// 47 to 49 us (138 MB); 8192 x 4096 and 8192 x 8192 in one launch, rank 32 53 to 55 us
// (208 MB, 3.9 TB/s; a device copy moves 4.85).
template <int IN>
__global__ __launch_bounds__(256) void lora_shrink_rows(ShrinkPair pair)
{
    const bool second = (int)blockIdx.z >= pair.first;
    const ShrinkArgs &p = pair.a[second];
    const int z = blockIdx.z - (second ? pair.first : 0);
    constexpr int STAGES = 8, X_BYTES = 64 * 128, STAGE = 2 * X_BYTES, NL = 4;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    clear_counters(pair);

    const int r0 = blockIdx.x * 64, rows = min(64, p.M - r0);
    const int a_in = lane < rows ? p.ids[r0 + lane] : -1;
    const int id = (uint32_t)a_in < (uint32_t)p.adapters ? a_in : -1;
    uint64_t left = __builtin_amdgcn_ballot_w64(id >= 0);
    const int kb = z * p.k_per_split;
    const int ke = min(p.K, kb + p.k_per_split);
    const int slabs = (ke - kb + 63) / 64;
    // (blocks start at different slabs: rows a power of two apart, read in step,
    // would share their memory channels)
    const int rot = slabs > 0 ? (int)(blockIdx.x * 8) % slabs : 0;
    const __amdgpu_buffer_rsrc_t rs_x =
        make_rsrc(p.x + (int64_t)r0 * p.ldx, (uint32_t)rows * (uint32_t)p.ldx * 2u);
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
    // load row of this lane within 8 rows, and the chunk that the swizzle puts here
    const int lr = lane >> 3;
    const int per = p.rank <= 16 ? 16 : p.rank <= 32 ? 32 : 64;     // rank rows of an adapter
    float *out = p.low + (int64_t)z * p.M * p.rank_pad;

    while (left) {
        // up to 64 / per adapters for this pass; slot s holds ranks from per s on
        int slot[4];
        uint64_t mine[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            slot[s] = s ? slot[s - 1] : -1;         // (an empty slot reads the last one's again)
            mine[s] = 0;
            if (s * per < 64 && left) {
                slot[s] = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
                mine[s] = __builtin_amdgcn_ballot_w64(id == slot[s]);
                left &= ~mine[s];
            }
        }
        for (int rank0 = 0; rank0 < p.rank; rank0 += 64) {
            // the rank rows 8 (4 j + wave) .. +8, j = 0, 1, that this wave loads
            __amdgpu_buffer_rsrc_t rs_d[2];
            uint32_t d_off[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = 8 * (4 * j + wave), s = row / per;
                const int a = s == 0 ? slot[0] : s == 1 ? slot[1] : s == 2 ? slot[2] : slot[3];
                rs_d[j] = make_rsrc(p.down + a * p.down_stride, (uint32_t)p.rank * (uint32_t)p.down_ld * 2u);
                // (rows past the rank read its last row again: their sums are not kept)
                d_off[j] = (uint32_t)min(rank0 + row % per + lr, p.rank - 1) * (uint32_t)p.down_ld * 2u;
            }
            auto issue = [&](int i) {
                const int r = i + rot;
                const int k0 = kb + (r < slabs ? r : r - slabs) * 64;
                const uint32_t at = lds0 + (uint32_t)(i % STAGES) * STAGE;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = 8 * (4 * j + wave) + lr;
                    const int c = (lane & 7) ^ row_key<8>(row);
                    const bool in = k0 + 8 * c < ke;
                    const uint32_t koff = (uint32_t)k0 * 2u, cb = (uint32_t)c * 16u;
                    const uint32_t xo = (uint32_t)min(row, rows - 1) * (uint32_t)p.ldx * 2u + cb;
                    load_lds16(rs_x, in ? xo : kOutOfRange, koff, at + (uint32_t)(4 * j + wave) * 1024u);
                    load_lds16(rs_d[j], in ? d_off[j] + cb : kOutOfRange, koff,
                               at + X_BYTES + (uint32_t)(4 * j + wave) * 1024u);
                }
            };
            f32x4 acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
            wg_barrier();                   // the last pass's slabs have been read
#pragma unroll 1
            for (int i = 0; i < STAGES - 1 && i < slabs; ++i)
                issue(i);
            for (int i = 0; i < slabs; ++i) {
                // slab i has landed once at most the loads of the slabs after it are out
                if (i + STAGES - 2 < slabs)
                    wait_vmcnt<(STAGES - 2) * NL>();
                else
                    wait_vmcnt<0>();
                wait_lgkmcnt0();
                wg_barrier();
                if (i + STAGES - 1 < slabs)
                    issue(i + STAGES - 1);
                const uint8_t *sx = smem + (i % STAGES) * STAGE, *sd = sx + X_BYTES;
                const int li = lane & 15;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const int c = 4 * ks + (lane >> 4);
                    const int xr = 16 * wave + li;
                    const u32x4 xf = *reinterpret_cast<const u32x4 *>(sx + xr * 128 + ((c ^ row_key<8>(xr)) * 16));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int dr = 16 * j + li;
                        const u32x4 df = *reinterpret_cast<const u32x4 *>(sd + dr * 128 + ((c ^ row_key<8>(dr)) * 16));
                        acc[j] = mfma16x16x32<IN>(xf, df, acc[j]);
                    }
                }
            }
            wait_lgkmcnt0();
            mfma_settle();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int s = 16 * j / per, rank = rank0 + 16 * j % per + (lane & 15);
                const uint64_t keep = s == 0 ? mine[0] : s == 1 ? mine[1] : s == 2 ? mine[2] : mine[3];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 16 * wave + 4 * (lane >> 4) + e;
                    if ((keep >> row) & 1 && rank < p.rank_pad)
                        out[(int64_t)(r0 + row) * p.rank_pad + rank] = rank < p.rank ? acc[j][e] : 0.0f;
                }
            }
        }
    }
}

// Zeros (a kernel, so that a captured call replays it like any other).
__global__ void clear_words(uint32_t *p, int64_t words)
{
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += step)
        p[i] = 0;
}

// ---- gradients ----

struct Stretch {
    int adapter, first, end;    // places [first, end) of the sorted rows
    int packed;                 // where the stretch's packed low-rank values begin, of 64
};

struct GradArgs {
    const int32_t *ids;
    int M, adapters, rank, rank_pad, N, K;
    // grouping of the rows by adapter
    int *hist;
    int64_t per_block;
    int blocks;
    int32_t *counts, *offsets, *order;
    int chunk;                  // rows of a stretch, at most
    int max_stretches;
    Stretch *stretches;         // [max_stretches]; adapter -1 past the last
    int *first_stretch;         // [adapters + 1]
    // dA: z = x [M][K] with v = the gradient of the low-rank values; dB: z = dy
    // [M][N] with v = the low-rank values.  v is [v_splits][M][rank_pad], scaled here.
    const uint16_t *z[2];
    const float *v[2];
    int ldz[2], cols[2], v_splits[2];
    u32x4 *pack[2];             // v scaled, split and transposed, as fragments (lora_pack)
    float *part[2];             // [stretch][rank_pad][cols]
    const float *scale;
    void *out[2];               // dA [adapter][rank][K], dB [adapter][N][rank]
    int out_dtype;
};

// The rows' order by adapter, and (a block of its own) the stretches: each
// adapter's rows in runs of at most `chunk`, so that a stretch is one unit of
// work with one adapter.
__global__ __launch_bounds__(kGroupThreads) void lora_place(GradArgs a)
{
    __shared__ PlaceLds l;
    if ((int)blockIdx.x < a.blocks) {
        place_block<false>(l, a.ids, a.M, a.adapters, a.per_block, a.hist, nullptr, blockIdx.x, a.blocks, a.counts,
                           a.offsets, a.order);
        return;
    }
    const int tid = threadIdx.x, L = a.adapters;
    for (int e = tid; e < L; e += kGroupThreads) {
        int c = 0;
#pragma unroll 8
        for (int i = 0; i < a.blocks; ++i)
            c += a.hist[(int64_t)i * (L + 1) + e];
        l.wave[0][e] = l.wave[1][e] = c;
        l.start[e] = (c + a.chunk - 1) / a.chunk;
    }
    if (tid == 0)
        l.start[L] = l.wave[0][L] = 0;
    __syncthreads();
    scan_lds(l.start, L + 1, l.part);       // stretches before adapter e
    scan_lds(l.wave[0], L + 1, l.part);     // rows before it
    for (int e = tid; e <= L; e += kGroupThreads) {
        a.first_stretch[e] = l.start[e];
        if (e < L) {
            const int rows = l.wave[0][e], end = rows + l.wave[1][e];
            // (64 places a piece: the chunk is a multiple of 64, so pieces before
            // this adapter's are those of the rows before it, and one at most for
            // each adapter before it)
            int packed = (rows / 64 + e) * 64;
            for (int s = l.start[e], at = rows; at < end; ++s, at += a.chunk, packed += a.chunk)
                a.stretches[s] = Stretch{e, at, min(end, at + a.chunk), packed};
        }
    }
    for (int s = l.start[L] + tid; s < a.max_stretches; s += kGroupThreads)
        a.stretches[s] = Stretch{-1, 0, 0, 0};
}

// [adapter][rows][cols] (rows of ld) to [adapter][cols][rows], so that the
// gradients' products read the adapters as the forward kernels do.
struct FlipArgs {
    const uint16_t *src[2];
    uint16_t *dst[2];
    int64_t stride[2];
    int ld[2], rows[2], cols[2];
    int tiles[2];               // 64 x 64 tiles of one adapter's matrix
};

// The first launch of a training step: the adapters transposed, and (the first
// a.blocks blocks of row y = 0 past the tiles') the rows of each adapter counted.
__global__ __launch_bounds__(256) void lora_prepare(FlipArgs p, GradArgs a)
{
    __shared__ uint16_t t[64][66];
    const int block = (int)blockIdx.x - p.tiles[0] - p.tiles[1];
    if (block >= 0) {
        __shared__ int hist[kMaxGroups + 1];
        if (blockIdx.y != 0)
            return;
        for (int e = threadIdx.x; e <= a.adapters; e += 256)
            hist[e] = 0;
        __syncthreads();
        const int64_t t0 = block * a.per_block;
        const int64_t t1 = t0 + a.per_block < a.M ? t0 + a.per_block : a.M;
        for (int64_t i = t0 + threadIdx.x; i < t1; i += 256) {
            const int g = a.ids[i];
            atomicAdd(&hist[(uint32_t)g < (uint32_t)a.adapters ? g : a.adapters], 1);
        }
        __syncthreads();
        for (int e = threadIdx.x; e <= a.adapters; e += 256)
            a.hist[(int64_t)block * (a.adapters + 1) + e] = hist[e];
        return;
    }
    const int w = (int)blockIdx.x >= p.tiles[0];
    const int tile = blockIdx.x - (w ? p.tiles[0] : 0);
    const int tc = (p.cols[w] + 63) / 64;
    const int r0 = tile / tc * 64, c0 = tile % tc * 64;
    const uint16_t *src = p.src[w] + blockIdx.y * p.stride[w];
    uint16_t *dst = p.dst[w] + (int64_t)blockIdx.y * p.rows[w] * p.cols[w];
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
    // (rows and columns are multiples of 8: whole pieces)
    u32x4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (r0 + y + 32 * i < p.rows[w] && c0 + 8 * x < p.cols[w])
            v[i] = *reinterpret_cast<const u32x4 *>(src + (int64_t)(r0 + y + 32 * i) * p.ld[w] + c0 + 8 * x);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint32_t *>(&t[y + 32 * i][8 * x + 2 * e]) = v[i][e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = y + 32 * i;
        if (c0 + c < p.cols[w] && r0 + 8 * x < p.rows[w]) {
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = (uint32_t)t[8 * x + 2 * e][c] | (uint32_t)t[8 * x + 2 * e + 1][c] << 16;
            *reinterpret_cast<u32x4 *>(dst + (int64_t)(c0 + c) * p.rows[w] + r0 + 8 * x) = o;
        }
    }
}

// v's rows of a piece of 64 places of a stretch, scaled, split in bf16 parts and
// transposed (zeros behind the stretch) to fragments as they go into the MFMA,
// [piece][16 ranks][32 rows][part][lane] of 16 bytes: done once, where each column
// tile of the gradient's kernel would do it again.
__global__ __launch_bounds__(256) void lora_pack(GradArgs p)
{
    __shared__ float t[64][64 + 1];
    __shared__ int row_of[64];
    const int w = blockIdx.z, tid = threadIdx.x;
    const Stretch st = p.stretches[blockIdx.y];
    const int at = st.first + blockIdx.x * 64;
    if (st.adapter < 0 || at >= st.end)
        return;
    const float sc = p.scale[st.adapter];
    const int64_t v_split = (int64_t)p.M * p.rank_pad;
    if (tid < 64)
        row_of[tid] = at + tid < st.end ? p.order[at + tid] : -1;
    const int64_t piece = st.packed / 64 + blockIdx.x;
    for (int r0 = 0; r0 < p.rank_pad; r0 += 64) {
        const int ranks = min(64, p.rank_pad - r0), quads = ranks / 4;
        __syncthreads();
        for (int i = tid; i < 64 * quads; i += 256) {
            const int row = i / quads, r = i % quads * 4;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            if (row_of[row] >= 0) {
                const float *src = p.v[w] + (int64_t)row_of[row] * p.rank_pad + r0 + r;
                for (int s = 0; s < p.v_splits[w]; ++s)
                    v += *reinterpret_cast<const f32x4 *>(src + s * v_split);
                v *= sc;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[row][r + e] = v[e];
        }
        __syncthreads();
        constexpr int NP = kParts;
        u32x4 *out = p.pack[w] + (piece * (p.rank_pad / 16) + r0 / 16) * (NP * 128);
        // lane l of a fragment: rank l % 16, rows 8 (l / 16) .. +8 of its 32
        for (int i = tid; i < ranks * 8; i += 256) {
            const int lane = i % 64, ks = i / 64 % 2, g = i / 128;
            u32x4 f[NP];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const float *src = &t[32 * ks + 8 * (lane >> 4) + 2 * d][16 * g + (lane & 15)];
                uint16_t a[NP], b[NP];
                split_parts(src[0], a);
                split_parts(src[65], b);
#pragma unroll
                for (int h = 0; h < NP; ++h)
                    f[h][d] = (uint32_t)a[h] | (uint32_t)b[h] << 16;
            }
#pragma unroll
            for (int h = 0; h < NP; ++h)
                out[((g * 2 + ks) * NP + h) * 64 + lane] = f[h];
        }
    }
}

// A z tile of the gradients' products in LDS: 64 rows of 128 columns, 256 bytes a
// row; 32-byte pieces of a row are permuted by the row, so that the 16 rows of
// a transposing read fall into different banks.
constexpr int kGradRows = 64, kGradCols = 128;

__device__ __forceinline__ int z_key(int row) { return (row & 3) | ((row >> 3) & 1) << 2; }

// This thread's four pieces of a tile: row tid / 16 + 16 i, chunk tid % 16 of 16 bytes.
__device__ __forceinline__ void store_z(uint8_t *zs, const u32x4 (&zr)[4], int tid)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (tid >> 4) + 16 * i, c = tid & 15;
        *reinterpret_cast<u32x4 *>(zs + row * 256 + ((((c >> 1) ^ z_key(row)) << 1) | (c & 1)) * 16) = zr[i];
    }
}

// acc += v z over a tile's rows 32 ks .. +32, read transposed (ds_read_b64_tr_b16):
// acc[r][j] holds ranks 16 r .. +16 of columns 32 wave + 16 j .. +16.  vf: rank
// 16 r + lane % 16, rows 32 ks + 8 (lane / 16) .. +8, of every part.
template <int IN, int RT>
__device__ __forceinline__ void multiply_z(const uint8_t *zs, int ks, const u32x4 (&vf)[RT][kParts],
                                           f32x4 (&acc)[RT][2], int wave, int lane)
{
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    u32x4 zf[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        v4s got[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = 32 * ks + 8 * (lane >> 4) + 4 * half + ((lane & 15) >> 2);
            const uint8_t *a = zs + row * 256 + ((2 * wave + j) ^ z_key(row)) * 32 + (lane & 3) * 8;
            got[half] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)a);
        }
        const u32x2 lo = __builtin_bit_cast(u32x2, got[0]), hi = __builtin_bit_cast(u32x2, got[1]);
        zf[j] = (u32x4){lo[0], lo[1], hi[0], hi[1]};
    }
    // z's finite values in one bf16 part or two, the second without v's last part
    constexpr int ZP = IN == IN_FP16 ? 2 : 1;
    auto parts_of = [](u32x4 x, u32x4 (&z)[2]) {
        z[0] = x;
        if constexpr (IN == IN_FP16)
            bf16_halves(x, z[0], z[1]);
    };
    // (an infinity in z times a value's later part, 0 or of the other sign, would
    // be a NaN: such pieces are taken apart)
    if (__builtin_amdgcn_ballot_w64((has_special<IN>(zf[0]) | has_special<IN>(zf[1])) != 0)) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                add_special<IN>(
                    zf[j], first_part(vf[r]), true,
                    [&](u32x4 x) {
                        u32x4 z[2];
                        parts_of(x, z);
#pragma unroll
                        for (int i = 0; i < ZP; ++i)
#pragma unroll
                            for (int h = 0; h < kParts - i; ++h)
                                acc[r][j] = mfma16x16x32<IN_BF16>(vf[r][h], z[i], acc[r][j]);
                    },
                    [&](u32x4 x, u32x4 y) { acc[r][j] = mfma16x16x32<IN_BF16>(y, x, acc[r][j]); });
        return;
    }
    u32x4 z[2][2];
    parts_of(zf[0], z[0]);
    parts_of(zf[1], z[1]);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < ZP; ++i)
#pragma unroll
            for (int h = 0; h < kParts - i; ++h) {
                acc[r][0] = mfma16x16x32<IN_BF16>(vf[r][h], z[0][i], acc[r][0]);
                acc[r][1] = mfma16x16x32<IN_BF16>(vf[r][h], z[1][i], acc[r][1]);
            }
}

// part[stretch][r][c] = sum over the stretch's rows m of s_a v[m][r] z[m][c]:
// the contraction runs over rows, so z's tile (64 rows of 128 columns, gathered
// by the rows' order) is staged in LDS as it lies and read back transposed, v's
// fragments (lora_pack) beside it for all four waves.  Bytes bound it: z is read
// once, in whole 256-byte row pieces, the next tile's loads in flight while a
// tile is multiplied, the order of the one after that already there.  Sorted into
// stretches of one adapter, partial sums need no atomics.  8192 rows, 12288
// columns, rank 32, bf16 50 us (236 MB, 4.8 TB/s); 70 while each wave read v's parts for
// itself, in 64-byte pieces.
template <int IN, int RT>
__global__ __launch_bounds__(256) void lora_grad(GradArgs p)
{
    __shared__ __attribute__((aligned(16))) uint8_t zs[2][kGradRows * 256];
    constexpr int NP = kParts, FRAGS = RT * NP * 128, VL = (FRAGS + 255) / 256;
    __shared__ u32x4 vs[2][VL * 256];
    const int w = blockIdx.z, tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c0 = blockIdx.x * kGradCols;
    if (c0 >= p.cols[w])
        return;
    const Stretch st = p.stretches[blockIdx.y];
    if (st.adapter < 0)
        return;
    const bool col_in = c0 + 8 * (tid & 15) < p.cols[w];            // cols is a multiple of 8
    const int col = col_in ? c0 + 8 * (tid & 15) : c0;
    const int last = st.first + (st.end - 1 - st.first) / kGradRows * kGradRows;   // the last tile
    const int groups = p.rank_pad / 16;

    for (int rg = 0; rg < p.rank_pad; rg += 16 * RT) {
        f32x4 acc[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            acc[r][0] = acc[r][1] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        // In flight while tile t is multiplied: the rows and fragments of t + 1 and t + 2,
        // the order of t + 3.  A turn's loads are issued in the order in which they are
        // waited for, and none is under a condition (what lies behind the stretch
        // re-reads its last row or tile; rows are zeroed on their way to LDS): the waits
        // are then for some of the loads, not all.
        int row_at[2][4];
        u32x4 zr[2][4], vr[2][VL];
        auto load_order = [&](int (&rows)[4], int at) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                rows[i] = p.order[min(at + (tid >> 4) + 16 * i, st.end - 1)];
        };
        auto load = [&](u32x4 (&z)[4], const int (&rows)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                z[i] = *reinterpret_cast<const u32x4 *>(p.z[w] + (int64_t)rows[i] * p.ldz[w] + col);
        };
        auto load_v = [&](u32x4 (&v)[VL], int at) {
            const int64_t piece = (st.packed + min(at, last) - st.first) / 64;
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const int f = min(i * 256 + tid, FRAGS - 1), r = f / (NP * 128);       // (past rank_pad: not kept)
                v[i] = p.pack[w][(piece * groups + min(rg / 16 + r, groups - 1)) * (NP * 128) + f % (NP * 128)];
            }
        };
        auto turn = [&](auto parity, int at) {
            constexpr int P = decltype(parity)::value;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!col_in || at + (tid >> 4) + 16 * i >= st.end)
                    zr[P][i] = (u32x4){0u, 0u, 0u, 0u};
            store_z(zs[P], zr[P], tid);
#pragma unroll
            for (int i = 0; i < VL; ++i)
                vs[P][i * 256 + tid] = vr[P][i];
            load_order(row_at[1 - P], at + 3 * kGradRows);
            load(zr[P], row_at[P]);
            load_v(vr[P], at + 2 * kGradRows);
            // (a tile's buffers are written again two turns later, after the barrier
            // of the turn between, which follows this turn's reads)
            wait_lgkmcnt0();
            wg_barrier();
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                u32x4 vf[RT][NP];
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int h = 0; h < NP; ++h)
                        vf[r][h] = vs[P][((r * 2 + ks) * NP + h) * 64 + lane];
                multiply_z<IN, RT>(zs[P], ks, vf, acc, wave, lane);
            }
        };
        load_order(row_at[0], st.first);
        load_order(row_at[1], st.first + kGradRows);
        load(zr[0], row_at[0]);
        load_v(vr[0], st.first);
        load_order(row_at[0], st.first + 2 * kGradRows);
        load(zr[1], row_at[1]);
        load_v(vr[1], st.first + kGradRows);
        for (int at = st.first;; at += 2 * kGradRows) {
            turn(std::integral_constant<int, 0>{}, at);
            if (at >= last)
                break;
            turn(std::integral_constant<int, 1>{}, at + kGradRows);
            if (at + kGradRows >= last)
                break;
        }
        mfma_settle();
        float *out = p.part[w] + (int64_t)blockIdx.y * p.rank_pad * p.cols[w];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int rank = rg + 16 * r + 4 * (lane >> 4) + e;
                    const int c = c0 + 32 * wave + 16 * j + (lane & 15);
                    if (rank < p.rank && c < p.cols[w])
                        out[(int64_t)rank * p.cols[w] + c] = acc[r][j][e];
                }
        __syncthreads();
    }
}

__device__ __forceinline__ void store_grad(void *out, int64_t at, float v, int dtype)
{
    if (dtype == GEMM_FP32)
        static_cast<float *>(out)[at] = v;
    else
        static_cast<uint16_t *>(out)[at] = dtype == GEMM_BF16 ? to16<IN_BF16>(v) : to16<IN_FP16>(v);
}

// The gradients for few rows (few_rows), in one launch where grouping the rows,
// packing v, the products and their sums are four: a block finds the rows of its
// adapter itself and takes them all.  v is staged for as many rows as kFewStage
// values hold, scaled, in FP32; a lane splits what it multiplies.
constexpr int kFewRows = 1024, kFewStage = 8192;

// A backward call without dX, in us, against four launches (BF16, rank 16; dy and x of 4096
// and 2048 columns): 300 rows of 1, 3, 16, 64 adapters 22 / 21 / 32 / 70 against 29 / 29 / 41 /
// 78; 1000 rows 47 / 33 / 58 / 102 against 30 / 38 / 69 / 109.  So one adapter of more than
// about 500 rows, whose blocks are few and long, would be faster in four launches (at
// 600 rows 33 against 30); the rule does not ask for it.  Past the bound on rows times
// rank: 731 rows, 4448 columns, rank 24, 3 adapters 26 us of kernels against 22.
__host__ __device__ constexpr bool few_rows(int64_t M, int64_t rank_pad)
{
    return M <= kFewRows && M * rank_pad <= 16 * kFewRows;
}

template <int IN, int RT>
__global__ __launch_bounds__(256) void lora_grad_few(GradArgs p)
{
    constexpr int RANKS = 16 * RT, GROUP = kFewStage / RANKS, PITCH = RANKS + 1;
    __shared__ __attribute__((aligned(16))) uint8_t zs[2][kGradRows * 256];
    __shared__ float vs[GROUP * PITCH];
    __shared__ int rows[kFewRows];
    __shared__ int found[4];
    const int w = blockIdx.z, a = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c0 = blockIdx.x * kGradCols;
    if (c0 >= p.cols[w])
        return;
    // the adapter's rows, in order: each wave's stretch of the ids, then put together
    constexpr int STEPS = kFewRows / 256;
    const int per = (p.M + 255) / 256 * 64;
    int mine[STEPS];
    int n = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int m = wave * per + 64 * i + lane;
        mine[i] = 64 * i < per && m < p.M ? p.ids[m] : -1;
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(mine[i] == a));
    if (lane == 0)
        found[wave] = n;
    __syncthreads();
    int at = 0, total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        at += i < wave ? found[i] : 0;
        total += found[i];
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const uint64_t has = __builtin_amdgcn_ballot_w64(mine[i] == a);
        if (mine[i] == a)
            rows[at + __builtin_popcountll(has & ((1ull << lane) - 1))] = wave * per + 64 * i + lane;
        at += __builtin_popcountll(has);
    }
    __syncthreads();

    const int col = c0 + 8 * (tid & 15);               // cols is a multiple of 8
    const bool col_in = col < p.cols[w];
    const float sc = p.scale[a];
    const int64_t v_split = (int64_t)p.M * p.rank_pad;
    for (int rg = 0; rg < p.rank_pad; rg += RANKS) {
        f32x4 acc[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            acc[r][0] = acc[r][1] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        u32x4 zr[4];
        auto load = [&](int t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int place = t + (tid >> 4) + 16 * i;
                zr[i] = (u32x4){0u, 0u, 0u, 0u};
                if (col_in && place < total)
                    zr[i] = *reinterpret_cast<const u32x4 *>(p.z[w] + (int64_t)rows[place] * p.ldz[w] + col);
            }
        };
        load(0);
        int turn = 0;
        for (int g0 = 0; g0 < total; g0 += GROUP) {
            __syncthreads();                           // the last group's values have been read
            for (int i = tid; i < GROUP * (RANKS / 4); i += 256) {
                const int row = i / (RANKS / 4), r = i % (RANKS / 4) * 4;
                if (row >= (total - g0 + 63) / 64 * 64)
                    break;
                f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
                if (g0 + row < total && rg + r < p.rank_pad) {
                    const float *src = p.v[w] + (int64_t)rows[g0 + row] * p.rank_pad + rg + r;
#pragma unroll 4
                    for (int s = 0; s < p.v_splits[w]; ++s)
                        v += *reinterpret_cast<const f32x4 *>(src + s * v_split);
                    v *= sc;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    vs[row * PITCH + r + e] = v[e];
            }
            const int end = min(total, g0 + GROUP);
            for (int t = g0; t < end; t += kGradRows, turn ^= 1) {
                store_z(zs[turn], zr, tid);
                load(t + kGradRows);
                // (a tile's buffer is written again two turns later, after the barrier
                // of the turn between, which follows this turn's reads)
                __syncthreads();
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    u32x4 vf[RT][kParts];
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const float *src = vs + (t - g0 + 32 * ks + 8 * (lane >> 4) + 2 * d) * PITCH + 16 * r + (lane & 15);
                            uint16_t a[kParts], b[kParts];
                            split_parts(src[0], a);
                            split_parts(src[PITCH], b);
#pragma unroll
                            for (int h = 0; h < kParts; ++h)
                                vf[r][h][d] = (uint32_t)a[h] | (uint32_t)b[h] << 16;
                        }
                    multiply_z<IN, RT>(zs[turn], ks, vf, acc, wave, lane);
                }
            }
        }
        mfma_settle();
        // dA [adapter][rank][K], dB [adapter][N][rank]
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int rank = rg + 16 * r + 4 * (lane >> 4) + e;
                    const int c = c0 + 32 * wave + 16 * j + (lane & 15);
                    if (rank < p.rank && c < p.cols[w])
                        store_grad(p.out[w], w == 0 ? ((int64_t)a * p.rank + rank) * p.cols[w] + c
                                                    : ((int64_t)a * p.cols[w] + c) * p.rank + rank,
                                   acc[r][j][e], p.out_dtype);
                }
        __syncthreads();
    }
}

// The stretches' sums, in order: dA as it lies, dB transposed.  A block takes 32
// columns of 16 ranks; a thread four columns of one rank and one half of the
// stretches, so that a few loads of a thread cover them (24 stretches of 64 ranks,
// 2256 columns: 6.2 us against 16.6 with a column of two ranks a thread).
__global__ __launch_bounds__(256) void lora_grad_sum(GradArgs p)
{
    __shared__ float t[16][33];
    __shared__ f32x4 second[128];
    const int w = blockIdx.z & 1, a = blockIdx.y, r0 = (blockIdx.z >> 1) * 16;
    if (blockIdx.x * 32 >= (unsigned)p.cols[w])
        return;
    const int x = (threadIdx.x & 7) * 4, y = (threadIdx.x >> 3) & 15, half = threadIdx.x >> 7;
    const int col = blockIdx.x * 32 + x;
    const bool in = col < p.cols[w] && r0 + y < p.rank;          // cols is a multiple of 8
    const int s0 = p.first_stretch[a], s1 = p.first_stretch[a + 1], mid = (s0 + s1) / 2;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in)
#pragma unroll 8
        for (int s = half ? mid : s0; s < (half ? s1 : mid); ++s)
            v += *reinterpret_cast<const f32x4 *>(p.part[w] + ((int64_t)s * p.rank_pad + r0 + y) * p.cols[w] + col);
    if (half)
        second[threadIdx.x & 127] = v;
    __syncthreads();
    if (!half) {
        v += second[threadIdx.x];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (w == 0 && in)
                store_grad(p.out[w], ((int64_t)a * p.rank + r0 + y) * p.cols[w] + col + i, v[i], p.out_dtype);
            t[y][x + i] = v[i];
        }
    }
    if (w == 0)
        return;
    __syncthreads();
    const int r = threadIdx.x & 15;
#pragma unroll
    for (int c = threadIdx.x >> 4; c < 32; c += 16) {
        const int n = blockIdx.x * 32 + c;
        if (n < p.cols[w] && r0 + r < p.rank)
            store_grad(p.out[w], ((int64_t)a * p.cols[w] + n) * p.rank + r0 + r, t[r][c], p.out_dtype);
    }
}

// ---- host ----

constexpr int64_t kPartialBytes = (int64_t)64 << 20;   // bound on a plan's K-split partials

// How a low-rank product is spread over the machine.
struct ShrinkPlan {
    int rt, lanes_j, splits, k_per_split, tiles;
    bool rows;              // lora_shrink_rows
};

ShrinkPlan plan_shrink(int64_t M, int64_t K, int64_t adapters, int64_t rank)
{
    ShrinkPlan s{};
    const int64_t pad = cdiv(rank, 16);
    s.rt = pad >= 4 ? 4 : pad >= 2 ? 2 : 1;
    // Past 2048 rows 64-row tiles: there are enough of them, with K splits, for
    // every compute unit, and they take an adapter for fewer reads of its ranks.  The
    // kernel alone in us, 16-row against 64-row tiles, x of three calls in turn:
    //   8192 x 8192, rank 64: 1 adapter 85 / 37, 4 in runs 86 / 37, 64 in runs 154 / 58, 4
    //   mixed 299 / 120, 64 mixed 1676 / 1588; rank 16: 1 adapter 43 / 35
    //   4096 x 4096, rank 16: 1 adapter 11.0 / 11.4, 4 mixed 32 / 11, 64 mixed 125 / 108
    // Up to 2048 rows neither always: 2048 x 4096, rank 16: 1 adapter 7.4 / 9.6, 64 mixed
    // 62 / 84, but 4 mixed 17.8 / 10.7; 1024 x 4096, rank 16: 6.0 / 9.7, 33 / 82, 11.1 / 10.6.
    s.rows = M > 2048;
    if (s.rows) {
        s.tiles = (int)cdiv(M, 64);
        s.lanes_j = 1;
        const int64_t slabs = cdiv(K, 64);
        const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(kNumCUs / s.tiles, slabs / 16));
        s.k_per_split = (int)std::max<int64_t>(64, cdiv(slabs, splits) * 64);
    } else {
        s.tiles = (int)std::max<int64_t>(1, cdiv(M, 16));
        // a row tile's adapters on blocks of their own while there are few row tiles
        s.lanes_j = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(adapters, std::min<int64_t>(M, 16)),
                                                                2 * kNumCUs / s.tiles));
        const int64_t blocks = (int64_t)s.tiles * s.lanes_j;
        const int64_t steps = cdiv(K, 128);
        int64_t splits = std::max<int64_t>(1, std::min<int64_t>(2 * kNumCUs / blocks, cdiv(steps, kShrinkWaves)));
        splits = std::min<int64_t>(splits, kMaxLowSplits);
        s.k_per_split = (int)std::max<int64_t>(128, cdiv(steps, splits) * 128);
    }
    s.splits = (int)std::max<int64_t>(1, cdiv(K, s.k_per_split));
    return s;
}

// Adds a product to a launch (at most two, of the same rows and adapters: their
// plans then differ in K alone).
void add_shrink(ShrinkPair &pair, const ShrinkPlan &s, ShrinkArgs p)
{
    p.k_per_split = s.k_per_split;
    pair.lanes_j = s.lanes_j;
    pair.a[pair.first > 0] = p;
    if (pair.first == 0)
        pair.first = s.splits;
}

hipError_t run_shrink(const ShrinkPlan &s, const ShrinkPair &p, int splits, int in_dtype, hipStream_t stream)
{
    const dim3 grid(s.tiles, s.lanes_j, splits);
    auto launch = [&](auto in) {
        if (s.rows)
            hipLaunchKernelGGL(lora_shrink_rows<in.value>, grid, dim3(256), 0, stream, p);
        else if (s.rt == 1)
            hipLaunchKernelGGL((lora_shrink<in.value, 1>), grid, dim3(kShrinkWaves * 64), 0, stream, p);
        else if (s.rt == 2)
            hipLaunchKernelGGL((lora_shrink<in.value, 2>), grid, dim3(kShrinkWaves * 64), 0, stream, p);
        else
            hipLaunchKernelGGL((lora_shrink<in.value, 4>), grid, dim3(kShrinkWaves * 64), 0, stream, p);
    };
    if (in_dtype == GEMM_BF16)
        launch(std::integral_constant<int, IN_BF16>{});
    else
        launch(std::integral_constant<int, IN_FP16>{});
    return hipGetLastError();
}

// The projection's plan: the library's own, without stream-K (whose partials
// leave in segments that are not whole tiles).
Plan plan_projection(int64_t M, int64_t N, int64_t K)
{
    // ... but for 33 to 64 rows where two rows of 32 x 128 tiles, too many to
    // split K, leave compute units idle that one row of 128 x 128 tiles with K
    // splits does not.  The plain product on either tile, in us, where the rule takes the
    // latter: 64 x 10240 x 8192 (160 blocks against 240) 52 / 38, 64 x 8704 x 8192 51 / 34,
    // 40 x 8704 x 4096 28 / 22, 64 x 6144 x 8192 32 / 28, 64 x 6144 x 4096 18.5 / 19.7; and where
    // not: 64 x 8192 x 4096 19 / 22, 40 x 8192 x 8192 31 / 33, 64 x 16384 x 4096 30 / 31, but 64 x
    // 12288 x 8192 (as many blocks on both) 52 / 44.
    if (M > 32 && M <= 64) {
        const Plan p = make_plan(M, N, K, kPartialBytes, -1, -1, 0);
        const Plan q = make_plan(M, N, K, kPartialBytes, CFG_T128x128, -1, 0);
        auto idle = [](const Plan &x) { return cdiv(x.grid, kNumCUs) * kNumCUs - x.grid; };
        return p.cfg == CFG_T32x128 && idle(q) + kNumCUs / 8 < idle(p) ? q : p;
    }
    return make_plan(M, N, K, kPartialBytes, -1, -1, 0);
}
// A product's rows in one launch, or in two: where the ping-pong tiles' last pass
// over the machine is at most half full, the rows of the full passes, and then the
// rest, with K splits that give the idle units a share.  5001 x 8192 x 8192 (640
// tiles: two passes and a half) 642 us in one launch, 458 + 144 in two.
struct Pieces {
    Plan plan[2];
    int64_t rows[2];
    int count;
};

Pieces plan_pieces(int64_t M, int64_t N, int64_t K)
{
    Pieces s{};
    s.plan[0] = plan_projection(M, N, K);
    s.rows[0] = M;
    s.count = 1;
    const Plan &p = s.plan[0];
    if (p.cfg != CFG_PP2_256x256 || p.splits != 1 || p.grid <= kNumCUs)
        return s;
    // passes of the machine, in k-slabs; a tile's start and end cost about 8
    auto cost = [](const Plan &x) { return cdiv(x.grid, kNumCUs) * (x.kt_per_split + 8); };
    const int64_t full = p.grid / kNumCUs * kNumCUs / p.tiles_n * 256;      // rows
    if (full == 0 || full >= M)
        return s;
    Pieces t{};
    t.plan[0] = make_plan(full, N, K, kPartialBytes, CFG_PP2_256x256, 1, 0);
    t.plan[1] = plan_projection(M - full, N, K);
    t.rows[0] = full;
    t.rows[1] = M - full;
    t.count = 2;
    return t.plan[1].cfg == CFG_PP2_256x256 && cost(t.plan[0]) + cost(t.plan[1]) + 8 < cost(p) ? t : s;
}

lora_fn projection_fn(const Plan &p, int64_t M, int in_dtype, int out_dtype)
{
    const bool rot = rotate_slabs(1, M);
    switch (p.cfg) {
    case CFG_T128x128: return (rot ? kLora_128_s4_rot : kLora_128_s4)[in_dtype][out_dtype];
    case CFG_T128x128_S2: return kLora_128_s2[in_dtype][out_dtype];
    case CFG_T32x128: return kLora_32_rot[in_dtype][out_dtype];
    case CFG_W4_256x128: return kLora_w4[in_dtype][out_dtype];
    default: return kLora_pp2[in_dtype][out_dtype];
    }
}

struct ProjectionWs {
    float *partials;
    unsigned *counters;
    int num_counters;
};

ProjectionWs carve_projection(Carver &c, const Plan &p)
{
    ProjectionWs w;
    w.num_counters = p.inreduce ? p.tiles_m * p.tiles_n : 0;
    w.partials = c.take<float>(p.splits > 1 ? p.ws_bytes / 4 : 0);
    w.counters = c.take<unsigned>(w.num_counters);
    return w;
}

// The arguments of the projection's tile from its plan (operands set by the caller).
void fill_projection(LoraArgs &a, const Plan &p, const ProjectionWs &w, void *C, int64_t M, int64_t N, int64_t K,
                     int64_t ldc, int out_dtype, const gemm_epilogue_t *epi)
{
    a.C = C;
    a.M = (int)M, a.N = (int)N, a.K = (int)K;
    a.ldc = (int)ldc;
    a.tiles_m = p.tiles_m, a.tiles_n = p.tiles_n;
    a.k_tiles = p.k_tiles;
    a.splits = p.splits;
    a.kt_per_split = p.kt_per_split;
    a.group_m = p.group_m;
    const int64_t size = size_of(out_dtype);
    a.vec_store = ldc % 4 == 0 && (uintptr_t)C % (4 * size) == 0;
    a.rows16 = (ldc * size) % 16 == 0 && (uintptr_t)C % 16 == 0;
    a.nt_b = p.tiles_m <= 2;
    a.partials = w.partials;
    a.counters = w.counters;
    a.inreduce = p.inreduce;
    a.alpha = 1.0f;
    if (epi) {
        a.alpha = epi->alpha;
        a.beta = epi->beta;
        a.bias = epi->bias_along != GEMM_BIAS_NONE ? epi->bias : nullptr;
        a.bias_along = epi->bias_along;
        a.act = epi->activation;
        a.bias_vec = (uintptr_t)a.bias % 16 == 0;
        a.epi = !(a.alpha == 1.0f && a.beta == 0.0f && a.bias_along == GEMM_BIAS_NONE && a.act == GEMM_ACT_NONE);
    }
}

hipError_t run_projection(lora_fn fn, const Plan &p, const LoraArgs &a, int out_dtype, hipStream_t stream)
{
    hipError_t e = fn(a, (unsigned)p.grid, stream);
    if (e != hipSuccess || p.splits <= 1 || p.inreduce)
        return e;
    const KernelArgs &k = a;
    const unsigned grid = (unsigned)cdiv((int64_t)a.M * ((a.N + 3) / 4), 256);
    if (out_dtype == GEMM_BF16)
        hipLaunchKernelGGL(splitk_sum<OUT_BF16>, dim3(grid), dim3(256), 0, stream, k);
    else if (out_dtype == GEMM_FP16)
        hipLaunchKernelGGL(splitk_sum<OUT_FP16>, dim3(grid), dim3(256), 0, stream, k);
    else
        hipLaunchKernelGGL(splitk_sum<OUT_FP32>, dim3(grid), dim3(256), 0, stream, k);
    return hipGetLastError();
}

// `count` zeros of `size` bytes (rank is a multiple of 8, so a count of them fills
// whole words)
hipError_t zero_fill(void *p, int64_t count, int64_t size, hipStream_t stream)
{
    const int64_t words = count * size / 4;
    if (words == 0)
        return hipSuccess;
    hipLaunchKernelGGL(clear_words, dim3((unsigned)std::min<int64_t>(cdiv(words, 256), 4096)), dim3(256), 0, stream,
                       static_cast<uint32_t *>(p), words);
    return hipGetLastError();
}

gemm_status_t check_sizes(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank)
{
    if (M < 0 || N < 0 || K < 0 || adapters < 0 || rank < 0)
        return GEMM_ERR_INVALID_ARG;
    if (M >= kMaxRows || N >= kMaxSize || K >= kMaxSize || adapters >= kMaxSize || rank > 128 || rank % 8 || K % 8)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

gemm_status_t check_adapters(const gemm_adapters_t *ad, int64_t N, int64_t K)
{
    if (ad->num_adapters == 0 || ad->rank == 0)
        return GEMM_OK;
    if (!ad->scale || !ad->ids || ad->a_stride < 0 || ad->b_stride < 0)
        return GEMM_ERR_INVALID_ARG;
    if ((uintptr_t)ad->scale % 4 || (uintptr_t)ad->ids % 4)
        return GEMM_ERR_MISALIGNED;
    gemm_status_t st;
    if ((st = check_operand(ad->A, K, ad->a_ld)) != GEMM_OK ||
        (st = check_operand(ad->B, ad->rank, ad->b_ld)) != GEMM_OK)
        return st;
    if (ad->a_stride % 8 || ad->b_stride % 8)
        return GEMM_ERR_MISALIGNED;
    const int64_t most = (int64_t)1 << 30;
    return ad->rank * ad->a_ld >= most || N * ad->b_ld >= most ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

bool has_adapters(int64_t adapters, int64_t rank) { return adapters > 0 && rank > 0; }

struct ForwardWs {
    float *low;
    ProjectionWs proj[2];
};

ForwardWs carve_forward(Carver &c, const Pieces &p, const ShrinkPlan &s, int64_t M, int64_t adapters, int64_t rank)
{
    ForwardWs w;
    w.low = c.take<float>(has_adapters(adapters, rank) ? (int64_t)s.splits * M * cdiv(rank, 16) * 16 : 0);
    w.proj[0] = carve_projection(c, p.plan[0]);
    w.proj[1] = w.proj[0];
    if (p.count > 1)
        w.proj[1] = carve_projection(c, p.plan[1]);
    return w;
}

void set_adapters(LoraArgs &a, const gemm_adapters_t *ad, const float *low, int low_splits, int64_t M,
                  const uint16_t *up, int64_t up_stride, int64_t up_ld)
{
    a.low = low;
    a.low_splits = low_splits;
    a.low_stride = M * cdiv(ad->rank, 16) * 16;
    a.up = up;
    a.up_stride = up_stride;
    a.up_ld = (int)up_ld;
    a.scale = ad->scale;
    a.ids = ad->ids;
    a.adapters = (int)ad->num_adapters;
    a.rank = (int)ad->rank;
    a.rank_pad = (int)cdiv(ad->rank, 16) * 16;
}

ShrinkArgs shrink_args(const gemm_adapters_t *ad, const void *x, int64_t M, int64_t K, int64_t ldx,
                       const void *down, int64_t down_stride, int64_t down_ld, float *low)
{
    ShrinkArgs p{};
    p.x = static_cast<const uint16_t *>(x);
    p.down = static_cast<const uint16_t *>(down);
    p.ids = ad->ids;
    p.low = low;
    p.down_stride = down_stride;
    p.M = (int)M, p.K = (int)K, p.ldx = (int)ldx;
    p.down_ld = (int)down_ld;
    p.adapters = (int)ad->num_adapters;
    p.rank = (int)ad->rank;
    p.rank_pad = (int)cdiv(ad->rank, 16) * 16;
    return p;
}

// Everything a backward call keeps in its workspace.
struct BackwardWs {
    ShrinkPlan t, u;
    GradPlan dx;
    float *low_t, *low_u;
    uint16_t *flip_a, *flip_b;
    GradArgs g;
    ProjectionWs proj;
};

BackwardWs carve_backward(Carver &c, int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank)
{
    BackwardWs w{};
    const int64_t pad = cdiv(rank, 16) * 16;
    w.t = plan_shrink(M, K, adapters, rank);
    w.u = plan_shrink(M, N, adapters, rank);
    if (M > 0 && K > 0)
        w.dx = plan_mn_major(M, K, N, kPartialBytes);
    w.proj = carve_projection(c, w.dx.plan);
    if (!has_adapters(adapters, rank) || M == 0 || N == 0 || K == 0)
        return w;      // nothing but a product, or less
    w.low_t = c.take<float>(w.t.splits * M * pad);
    w.low_u = c.take<float>(w.u.splits * M * pad);
    w.flip_a = c.take<uint16_t>(adapters * rank * K);
    w.flip_b = c.take<uint16_t>(adapters * rank * N);
    GradArgs &g = w.g;
    g.M = (int)M, g.N = (int)N, g.K = (int)K;
    g.adapters = (int)adapters, g.rank = (int)rank, g.rank_pad = (int)pad;
    g.cols[0] = (int)K, g.cols[1] = (int)N;
    if (few_rows(M, pad))
        return w;
    g.per_block = std::max<int64_t>(cdiv(cdiv(M, 32), kGroupThreads) * kGroupThreads, kGroupThreads);
    g.blocks = (int)cdiv(M, g.per_block);
    g.hist = c.take<int>((int64_t)g.blocks * (adapters + 1));
    g.counts = c.take<int32_t>(adapters);
    g.offsets = c.take<int32_t>(adapters + 1);
    g.order = c.take<int32_t>(M);
    // stretches so long that column tiles x stretches give about two blocks a
    // compute unit, and no longer: each stretch writes a partial sum (gradients and
    // their sums with two against four, v in two parts: 8192 rows, 12288 columns, rank
    // 32 48 us against 52; 5918, 2256, 64 26 against 36; 2048, 4096, 16 12 against 13; but
    // 7164, 10328, 24 48 against 45)
    const int64_t tiles = cdiv(K, 128) + cdiv(N, 128);
    const int64_t want = std::max<int64_t>(1, 2 * kNumCUs / tiles);
    g.chunk = (int)std::max<int64_t>(64, cdiv(cdiv(M, want), 64) * 64);
    g.max_stretches = (int)(M / g.chunk + std::min<int64_t>(adapters, M));
    g.stretches = c.take<Stretch>(g.max_stretches);
    g.first_stretch = c.take<int>(adapters + 1);
    const int64_t pieces = cdiv(M, 64) + adapters;     // each adapter's rows end inside one
    for (int i = 0; i < 2; ++i) {
        g.pack[i] = c.take<u32x4>(pieces * (pad / 16) * (kParts * 128));
        g.part[i] = c.take<float>((int64_t)g.max_stretches * pad * g.cols[i]);
    }
    return w;
}

}  // namespace
}  // namespace gnt

using namespace gnt;

extern "C" {

gemm_status_t gemm_lora_workspace(int64_t M, int64_t N, int64_t K, int64_t num_adapters,
                                  int64_t rank, int64_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_INVALID_ARG;
    *bytes = 0;
    const gemm_status_t st = check_sizes(M, N, K, num_adapters, rank);
    if (st != GEMM_OK || M == 0 || N == 0)
        return st;
    Carver c{nullptr};
    carve_forward(c, plan_pieces(M, N, K), plan_shrink(M, K, num_adapters, rank), M, num_adapters, rank);
    *bytes = c.used;
    return GEMM_OK;
}

gemm_status_t gemm_run_lora(const void *X, const void *W, void *Y, int64_t M, int64_t N, int64_t K,
                            int64_t ldx, int64_t ldw, int64_t ldy, int in_dtype, int out_dtype,
                            const gemm_adapters_t *adapters, const gemm_epilogue_t *epi,
                            void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    if (!adapters)
        return GEMM_ERR_INVALID_ARG;
    if (!is_16bit(in_dtype) || !is_out(out_dtype))
        return GEMM_ERR_UNSUPPORTED;
    gemm_status_t st = check_sizes(M, N, K, adapters->num_adapters, adapters->rank);
    if (st != GEMM_OK || (st = check_epilogue(epi)) != GEMM_OK)
        return st;
    if (M == 0 || N == 0)
        return GEMM_OK;
    if ((st = check_output(Y, N, ldy, out_dtype)) != GEMM_OK)
        return st;
    if (K > 0 && ((st = check_operand(X, K, ldx)) != GEMM_OK || (st = check_operand(W, K, ldw)) != GEMM_OK ||
                  (st = check_adapters(adapters, N, K)) != GEMM_OK))
        return st;
    const Pieces p = plan_pieces(M, N, K);
    const ShrinkPlan s = plan_shrink(M, K, adapters->num_adapters, adapters->rank);
    for (int i = 0; i < p.count; ++i)
        if (p.plan[i].grid <= 0 || p.plan[i].grid >= kMaxBlocks)
            return GEMM_ERR_UNSUPPORTED;
    Carver c{static_cast<uint8_t *>(workspace)};
    const ForwardWs w = carve_forward(c, p, s, M, adapters->num_adapters, adapters->rank);
    if ((st = check_workspace(workspace, workspace_bytes, c.used)) != GEMM_OK)
        return st;
    // (of two pieces only the second splits K)
    const ProjectionWs &counted = w.proj[p.count - 1];
    LoraArgs a{};
    hipError_t e;
    if (K > 0 && has_adapters(adapters->num_adapters, adapters->rank)) {
        set_adapters(a, adapters, w.low, s.splits, M, static_cast<const uint16_t *>(adapters->B), adapters->b_stride,
                     adapters->b_ld);
        ShrinkPair q{};
        q.counters = counted.counters;
        q.num_counters = counted.num_counters;
        add_shrink(q, s, shrink_args(adapters, X, M, K, ldx, adapters->A, adapters->a_stride, adapters->a_ld, w.low));
        e = run_shrink(s, q, s.splits, in_dtype, stream);
    } else {
        e = zero_fill(counted.counters, counted.num_counters, 4, stream);
    }
    int64_t row = 0;
    for (int i = 0; i < p.count && e == hipSuccess; ++i) {
        LoraArgs b = a;
        b.A = static_cast<const uint16_t *>(X) + row * ldx;
        b.B = static_cast<const uint16_t *>(W);
        b.lda = (int)ldx;
        b.ldb = (int)ldw;
        if (b.adapters) {
            b.ids += row;
            b.low += row * b.rank_pad;
        }
        fill_projection(b, p.plan[i], w.proj[i], static_cast<uint8_t *>(Y) + row * ldy * size_of(out_dtype), p.rows[i], N,
                        K, ldy, out_dtype, epi);
        if (b.bias_along == GEMM_BIAS_M)
            b.bias += row;
        e = run_projection(projection_fn(p.plan[i], p.rows[i], in_dtype, out_dtype), p.plan[i], b, out_dtype, stream);
        row += p.rows[i];
    }
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

static gemm_status_t check_backward(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank)
{
    const gemm_status_t st = check_sizes(M, N, K, adapters, rank);
    if (st != GEMM_OK)
        return st;
    return N % 8 || adapters > kMaxGroups ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

gemm_status_t gemm_lora_backward_workspace(int64_t M, int64_t N, int64_t K, int64_t num_adapters,
                                           int64_t rank, int64_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_INVALID_ARG;
    *bytes = 0;
    const gemm_status_t st = check_backward(M, N, K, num_adapters, rank);
    if (st != GEMM_OK || M == 0 || K == 0)
        return st;
    Carver c{nullptr};
    carve_backward(c, M, N, K, num_adapters, rank);
    *bytes = c.used;
    return GEMM_OK;
}

gemm_status_t gemm_run_lora_backward(const void *dY, const void *X, const void *W, void *dX,
                                     void *dA, void *dB, int64_t M, int64_t N, int64_t K,
                                     int64_t lddy, int64_t ldx, int64_t ldw, int64_t lddx,
                                     int in_dtype, int dx_dtype, int grad_dtype,
                                     const gemm_adapters_t *adapters, void *workspace,
                                     int64_t workspace_bytes, hipStream_t stream)
{
    if (!adapters)
        return GEMM_ERR_INVALID_ARG;
    if (!is_16bit(in_dtype) || !is_out(dx_dtype) || !is_out(grad_dtype))
        return GEMM_ERR_UNSUPPORTED;
    const int64_t L = adapters->num_adapters, R = adapters->rank;
    gemm_status_t st = check_backward(M, N, K, L, R);
    if (st != GEMM_OK)
        return st;
    // both or neither (an array without elements may be null)
    const bool grads = dA || dB;
    if (grads && ((!dA && L * R * K > 0) || (!dB && L * R * N > 0)))
        return GEMM_ERR_INVALID_ARG;
    const bool some = M > 0 && N > 0 && K > 0;
    if (some && ((st = check_operand(dY, N, lddy)) != GEMM_OK || (st = check_operand(X, K, ldx)) != GEMM_OK ||
                 (st = check_operand(W, K, ldw)) != GEMM_OK || (st = check_adapters(adapters, N, K)) != GEMM_OK))
        return st;
    const bool want_dx = dX && M > 0 && K > 0;
    if (want_dx && (st = check_output(dX, K, lddx, dx_dtype)) != GEMM_OK)
        return st;
    // (zero_fill writes words)
    if ((uintptr_t)dA % 4 || (uintptr_t)dB % 4)
        return GEMM_ERR_MISALIGNED;
    Carver c{static_cast<uint8_t *>(workspace)};
    BackwardWs w = carve_backward(c, M, N, K, L, R);
    if ((want_dx || (some && grads)) && (st = check_workspace(workspace, workspace_bytes, c.used)) != GEMM_OK)
        return st;
    if (want_dx && (w.dx.plan.grid <= 0 || w.dx.plan.grid >= kMaxBlocks))
        return GEMM_ERR_UNSUPPORTED;

    hipError_t e = hipSuccess;
    const bool adapt = some && has_adapters(L, R) && (want_dx || grads);
    if (!adapt && grads) {
        e = zero_fill(dA, L * R * K, size_of(grad_dtype), stream);
        if (e == hipSuccess)
            e = zero_fill(dB, L * R * N, size_of(grad_dtype), stream);
    }
    LoraArgs a{};
    if (adapt) {
        // B_a transposed: the low-rank gradients are then products like the forward's
        FlipArgs f{};
        f.src[0] = static_cast<const uint16_t *>(adapters->A);
        f.src[1] = static_cast<const uint16_t *>(adapters->B);
        f.dst[0] = w.flip_a, f.dst[1] = w.flip_b;
        f.stride[0] = adapters->a_stride, f.stride[1] = adapters->b_stride;
        f.ld[0] = (int)adapters->a_ld, f.ld[1] = (int)adapters->b_ld;
        f.rows[0] = (int)R, f.cols[0] = (int)K;
        f.rows[1] = (int)N, f.cols[1] = (int)R;
        for (int i = 0; i < 2; ++i)
            f.tiles[i] = (int)(cdiv(f.rows[i], 64) * cdiv(f.cols[i], 64));
        w.g.ids = adapters->ids;
        w.g.scale = adapters->scale;
        hipLaunchKernelGGL(lora_prepare, dim3(f.tiles[0] + f.tiles[1] + (grads ? w.g.blocks : 0), (unsigned)L), dim3(256),
                           0, stream, f, w.g);
        e = hipGetLastError();
        // dy with B transposed, and for the adapters' gradients x with A
        ShrinkPair u{};
        u.counters = w.proj.counters;
        u.num_counters = w.proj.num_counters;
        add_shrink(u, w.u, shrink_args(adapters, dY, M, N, lddy, w.flip_b, R * N, N, w.low_u));
        if (grads)
            add_shrink(u, w.t, shrink_args(adapters, X, M, K, ldx, adapters->A, adapters->a_stride, adapters->a_ld,
                                           w.low_t));
        if (e == hipSuccess)
            e = run_shrink(w.u, u, w.u.splits + (grads ? w.t.splits : 0), in_dtype, stream);
        set_adapters(a, adapters, w.low_u, w.u.splits, M, w.flip_a, R * K, R);
    } else if (want_dx && e == hipSuccess) {
        e = zero_fill(w.proj.counters, w.proj.num_counters, 4, stream);
    }
    if (want_dx && e == hipSuccess) {
        a.A = static_cast<const uint16_t *>(dY);
        a.B = static_cast<const uint16_t *>(W);
        a.lda = (int)lddy;
        a.ldb = (int)ldw;
        fill_projection(a, w.dx.plan, w.proj, dX, M, K, N, lddx, dx_dtype, nullptr);
        e = run_projection((w.dx.tile ? kLora_tile_km : kLora_pp2_km)[in_dtype][dx_dtype], w.dx.plan, a, dx_dtype,
                           stream);
    }
    if (adapt && grads && e == hipSuccess) {
        GradArgs &g = w.g;
        g.z[0] = static_cast<const uint16_t *>(X), g.z[1] = static_cast<const uint16_t *>(dY);
        g.ldz[0] = (int)ldx, g.ldz[1] = (int)lddy;
        g.v[0] = w.low_u, g.v[1] = w.low_t;
        g.v_splits[0] = w.u.splits, g.v_splits[1] = w.t.splits;
        g.out[0] = dA, g.out[1] = dB;
        g.out_dtype = grad_dtype;
        const unsigned widest = (unsigned)std::max(g.cols[0], g.cols[1]);
        const dim3 grid((widest + 127) / 128, g.max_stretches, 2);
        const int pad = g.rank_pad / 16;
        auto grad = [&](auto in) {
            if (few_rows(M, g.rank_pad)) {
                const dim3 few((widest + 127) / 128, (unsigned)L, 2);
                if (pad == 1)
                    hipLaunchKernelGGL((lora_grad_few<in.value, 1>), few, dim3(256), 0, stream, g);
                else if (pad <= 3)
                    hipLaunchKernelGGL((lora_grad_few<in.value, 2>), few, dim3(256), 0, stream, g);
                else
                    hipLaunchKernelGGL((lora_grad_few<in.value, 4>), few, dim3(256), 0, stream, g);
                return;
            }
            hipLaunchKernelGGL(lora_place, dim3(g.blocks + 1), dim3(kGroupThreads), 0, stream, g);
            hipLaunchKernelGGL(lora_pack, dim3(g.chunk / 64, g.max_stretches, 2), dim3(256), 0, stream, g);
            if (pad == 1)
                hipLaunchKernelGGL((lora_grad<in.value, 1>), grid, dim3(256), 0, stream, g);
            else if (pad <= 3)
                hipLaunchKernelGGL((lora_grad<in.value, 2>), grid, dim3(256), 0, stream, g);
            else
                hipLaunchKernelGGL((lora_grad<in.value, 4>), grid, dim3(256), 0, stream, g);
            hipLaunchKernelGGL(lora_grad_sum, dim3((widest + 31) / 32, (unsigned)L, 2 * pad), dim3(256), 0, stream, g);
        };
        if (in_dtype == GEMM_BF16)
            grad(std::integral_constant<int, IN_BF16>{});
        else
            grad(std::integral_constant<int, IN_FP16>{});
        e = hipGetLastError();
    }
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // extern "C"
