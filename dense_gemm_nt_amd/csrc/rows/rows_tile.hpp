// rows_tile.hpp -- a 128 x 128 tile for products whose B is MN-major (B as
// [K][ldb], element (n, k) at B[k ldb + n]) and whose A is K-major: the input
// gradients' form, where few rows leave most compute units without a 256 x 256
// ping-pong tile.  Two blocks share a compute unit, so one's stores and first
// loads run under the other's multiplications.  777 x 2048 x 4096 with four K splits
// and adapters 34 us; 1000 rows of 8 experts, 2048 x 1408 27 us.  (Where the
// ping-pong tiles fill the machine they are faster by a third.)
//
// Four waves, each a 64 x 64 block (2 x 2 MFMA blocks of 32 x 32).  32-deep slabs,
// 8 KB an operand, in a ring of five (80 KB a block) filled by direct-to-LDS loads:
//   K-major A: 128 rows of 64 bytes, a load 16 rows; the 16-byte chunk c of row r at
//     chunk c ^ row_key<4>(r)
//   MN-major B: 32 k-rows of 128 columns (256 bytes), a load 4 k-rows; chunk c of
//     k-row r at chunk c ^ 4 (r mod 4), read back transposed (ds_read_b64_tr_b16)
// Rows and columns past the operand re-read its last ones (their outputs are never
// stored); k past K reads zeros.  A load out of range in every lane may count
// as done ahead of those issued before it, and the last slab of a K that is no
// multiple of 32 holds such loads: the waits that count loads are not used with
// it in flight.
#pragma once

#include <type_traits>

#include "rows_common.hpp"

namespace gnt {

constexpr int kTileStages = 5, kTileOperand = 8192;

// What a tile's argument block brings: LoraArgs a plan's tile and K split, to whose sums adapters
// are added (add), RoutedArgs an expert's tile; others (outside this folder) specialize it.
//   kLookup  finds the block's tile (false: none) without K splits, in place of the plan's map
//   kPaired  B's k-rows alternate in groups of eight between two arrays
//   map, tile  the block's tile and split (false: none), and its number in the launch
//   kStore   store(p, acc, r0, c0, stage, lane) in place of a whole sum's store
template <typename Args>
struct PlanTile {
    static constexpr bool kLookup = false, kPaired = false, kStore = false;
    static __device__ __forceinline__ const uint16_t *b(const Args &p, int) { return p.B; }
    static __device__ __forceinline__ int ldb(const Args &p, int) { return p.ldb; }
    static __device__ __forceinline__ int cols(const Args &) { return 0; }
    static __device__ __forceinline__ int tile(const Args &p, int tm, int tn) { return tm * p.tiles_n + tn; }
    static __device__ __forceinline__ bool map(Args &p, int &tm, int &tn, int &split)
    {
        if (p.inreduce)
            map_block_split_minor(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, p.group_m, p.splits, tm, tn, split);
        else
            map_block(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, p.group_m, tm, tn, split);
        return true;
    }
};

template <typename Args>
struct TileHooks;

template <>
struct TileHooks<LoraArgs> : PlanTile<LoraArgs> {
    template <int IN, int OUT>
    static __device__ __forceinline__ void add(LoraArgs &p, f32x16 (&acc)[2][2], int r0, int c0, int split, int lane)
    {
        lora_add<IN, 4, true, low_parts<IN, OUT>>(p, acc, r0, c0, split, lane);
    }
};

template <>
struct TileHooks<RoutedArgs> : PlanTile<RoutedArgs> {
    static constexpr bool kLookup = true;
};

template <int IN, int OUT, typename Args>
__global__ __launch_bounds__(256, 2) void rows_tile(Args p)
{
    using Hooks = TileHooks<Args>;
    constexpr bool ROUTED = Hooks::kLookup, PAIRED = Hooks::kPaired;
    constexpr int BM = 128, BN = 128, BK = 32, ST = kTileStages, OPER = kTileOperand, NL = 4;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[ST * 2 * OPER];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;

    int tm, tn, split = 0;
    if constexpr (ROUTED) {
        if (!routed_lookup(p, tm, tn))
            return;
    } else if (!Hooks::map(p, tm, tn, split)) {
        return;
    }
    const int m0 = tm * BM, n0 = tn * BN;
    // (k_tiles and kt_per_split count 64-deep slabs, as the plans do)
    const int k_begin = split * p.kt_per_split * 64;
    const int k_end = min(p.K, k_begin + p.kt_per_split * 64);
    const int nk = (k_end - k_begin + BK - 1) / BK;
    const bool whole = (k_end - k_begin) % BK == 0 && (!PAIRED || Hooks::cols(p) % (BK / 2) == 0);
    const int rows_a = min(BM, p.M - m0), rows_b = min(BN, p.N - n0);

    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
    const __amdgpu_buffer_rsrc_t rs_a =
        make_rsrc(p.A + (int64_t)m0 * p.lda, (uint32_t)rows_a * (uint32_t)p.lda * 2u);
    const int kr = lane >> 4, chunk = (lane & 15) ^ (4 * kr);      // MN-major: k-row of 4, logical chunk
    const int ar = lane >> 2;                                      // K-major: row of 16
    auto issue = [&](int i) {
        const int k0 = k_begin + i * BK;
        const uint32_t at = lds0 + (uint32_t)(i % ST) * (2u * OPER);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = 64 * j + 16 * wave + ar;
            const int c = (lane & 3) ^ row_key<4>(row);
            const uint32_t v = k0 + 8 * c < k_end
                ? (uint32_t)min(row, rows_a - 1) * (uint32_t)p.lda * 2u + (uint32_t)c * 16u : kOutOfRange;
            load_lds16(rs_a, v, (uint32_t)k0 * 2u, at + (uint32_t)(64 * j + 16 * wave) * 64u);
        }
        // B's k-rows of the slab as whole rows of ldb elements, from the tile's
        // first column
        const int k_rows = PAIRED ? min(BK / 2, Hooks::cols(p) - k0 / 2) : min(BK, k_end - k0);
        const int ldb = Hooks::ldb(p, wave >> 1);
        const __amdgpu_buffer_rsrc_t rs_b =
            make_rsrc(Hooks::b(p, wave >> 1) + (int64_t)(PAIRED ? k0 / 2 : k0) * ldb + n0,
                      (uint32_t)(((int64_t)k_rows * ldb - n0) * 2));
        const int col = min(8 * chunk, (rows_b - 1) & ~7);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = PAIRED ? 8 * j + 4 * (wave & 1) + kr : 16 * j + 4 * wave + kr;
            const uint32_t v = row < k_rows ? (uint32_t)row * (uint32_t)ldb * 2u + (uint32_t)col * 2u : kOutOfRange;
            load_lds16(rs_b, v, 0, at + OPER + (uint32_t)(16 * j + 4 * wave) * 256u);
        }
    };

    // Fragments of k 16 ks .. +16: the 8 k from 8 (lane / 32) of B's column cb + lane % 32,
    // of A's row rb + lane % 32.
    const int tr_kq = (lane & 15) >> 2;
    const int tr_lp = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int tr_base = (8 * (lane >> 5) + tr_kq) * 256 + 8 * (lane & 1);
    auto read_mn = [&](const uint8_t *base, int ks, int cb) -> u32x4 {
        typedef short v4s __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4s lds_v4s;
        const int c = 4 * ((cb >> 5) ^ tr_kq) + tr_lp;
        const uint8_t *at = base + tr_base + (16 * ks) * 256 + c * 16;
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)at));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(at + 4 * 256)));
        return (u32x4){a[0], a[1], b[0], b[1]};
    };
    auto read_a = [&](const uint8_t *base, int ks, int rb) -> u32x4 {
        const int r = rb + (lane & 31);
        return *reinterpret_cast<const u32x4 *>(base + r * 64 + (((2 * ks + (lane >> 5)) ^ row_key<4>(r)) * 16));
    };

    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.0f;
#pragma unroll 1
    for (int i = 0; i < ST - 1 && i < nk; ++i)
        issue(i);
    for (int i = 0; i < nk; ++i) {
        // slab i has landed for this wave once at most the loads of the ST - 2
        // slabs after it are out
        if (i + ST - 2 < nk - (whole ? 0 : 1))
            wait_vmcnt<(ST - 2) * NL>();
        else
            wait_vmcnt<0>();
        wait_lgkmcnt0();
        wg_barrier();
        if (i + ST - 1 < nk)
            issue(i + ST - 1);
        const uint8_t *sa = smem + (i % ST) * (2 * OPER), *sb = sa + OPER;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            u32x4 af[2], bf[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                af[f] = read_a(sa, ks, wm + 32 * f);
                bf[f] = read_mn(sb, ks, wn + 32 * f);
            }
#pragma unroll
            for (int fn = 0; fn < 2; ++fn)
#pragma unroll
                for (int fm = 0; fm < 2; ++fm)
                    acc[fn][fm] = mfma32x32x16<IN>(bf[fn], af[fm], acc[fn][fm]);
        }
    }
    mfma_settle();
    if constexpr (!ROUTED) {
        Hooks::template add<IN, OUT>(p, acc, m0 + wm, n0 + wn, split, lane);
        if (p.inreduce) {
            // (the ring is behind the barrier's last reader once the partials are out)
            if (!splitk_arrive<4>(p, acc, Hooks::tile(p, tm, tn), split, wave, lane,
                                        reinterpret_cast<uint32_t *>(smem)))
                return;
            p.splits = 1;
        }
    }

    // Each wave's block through its own 16 KB of the ring as FP32 rows of 64, the
    // 16-byte chunk c of row r at c ^ (r mod 16), and out in 16-byte pieces of
    // rows where C allows it.
    wait_lgkmcnt0();
    wg_barrier();
    const int r0 = m0 + wm, c0 = n0 + wn;
    if constexpr (Hooks::kStore) {
        Hooks::store(p, acc, r0, c0, smem + wave * 16384, lane);
        return;
    }
    const bool partial = !ROUTED && p.splits > 1;
    const bool wide = !partial && p.rows16 && !p.epi && r0 + 64 <= p.M && c0 + 64 <= p.N;
    if (!wide) {
#pragma unroll
        for (int fm = 0; fm < 2; ++fm) {
            const int m = r0 + fm * 32 + (lane & 31);
            if (m >= p.M)
                continue;
#pragma unroll
            for (int fn = 0; fn < 2; ++fn)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = c0 + fn * 32 + 8 * q + 4 * (lane >> 5);
                    if (n >= p.N)
                        continue;
                    const f32x4 x = {acc[fn][fm][4 * q], acc[fn][fm][4 * q + 1], acc[fn][fm][4 * q + 2],
                                     acc[fn][fm][4 * q + 3]};
                    store_result<OUT>(p, split, m, n, x);
                }
        }
        return;
    }
    uint8_t *stage = smem + wave * 16384;
#pragma unroll
    for (int fn = 0; fn < 2; ++fn)
#pragma unroll
        for (int fm = 0; fm < 2; ++fm)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = fm * 32 + (lane & 31), c = fn * 8 + 2 * q + (lane >> 5);
                const f32x4 v = {acc[fn][fm][4 * q], acc[fn][fm][4 * q + 1], acc[fn][fm][4 * q + 2],
                                 acc[fn][fm][4 * q + 3]};
                *reinterpret_cast<f32x4 *>(stage + r * 256 + ((c ^ (r & 15)) * 16)) = v;
            }
    wait_lgkmcnt0();
    if constexpr (OUT == OUT_FP32) {
        float *out = static_cast<float *>(p.C) + (int64_t)r0 * p.ldc + c0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int r = 4 * j + (lane >> 4), c = lane & 15;
            const f32x4 v = *reinterpret_cast<const f32x4 *>(stage + r * 256 + ((c ^ (r & 15)) * 16));
            __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(out + (int64_t)r * p.ldc + 4 * c));
        }
    } else {
        uint16_t *out = static_cast<uint16_t *>(p.C) + (int64_t)r0 * p.ldc + c0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = 8 * j + (lane >> 3), c = 2 * (lane & 7);
            const f32x4 a = *reinterpret_cast<const f32x4 *>(stage + r * 256 + ((c ^ (r & 15)) * 16));
            const f32x4 b = *reinterpret_cast<const f32x4 *>(stage + r * 256 + (((c + 1) ^ (r & 15)) * 16));
            constexpr int T = OUT == OUT_BF16 ? IN_BF16 : IN_FP16;
            u32x4 v;
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                v[d] = (uint32_t)to16<T>(a[2 * d]) | (uint32_t)to16<T>(a[2 * d + 1]) << 16;
                v[2 + d] = (uint32_t)to16<T>(b[2 * d]) | (uint32_t)to16<T>(b[2 * d + 1]) << 16;
            }
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(out + (int64_t)r * p.ldc + 4 * c));
        }
    }
}

}  // namespace gnt
