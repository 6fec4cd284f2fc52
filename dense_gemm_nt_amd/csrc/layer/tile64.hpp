// tile64.hpp -- a 64 x 64 tile for small products with an MN-major B (B as [K][ldb], element
// (n, k) at B[k ldb + n]; of paired arrays in turn groups of eight k-rows), which leave most
// compute units without a larger one: A K-major, [M][lda].
//
// Four waves (2 x 2 blocks of 32 x 32), two blocks a compute unit; a ring of four stages of
// 64-deep slabs (8 KB an operand) filled by direct-to-LDS loads, and all of a slab's fragments
// read before its first MFMA.  Of few blocks a launch's beginning and end (its first loads, the
// stores) take 6 to 8 us and a slab 0.15; of 416 blocks of 44 slabs (23 us) a slab 0.37, its
// loads from the L2s at 17 TB/s.  Level with this: fragments read a slab ahead, loads between the
// MFMAs, eight stages.  Slower: two groups of four waves a tile with half of K each (one block a
// compute unit; 1000 x 2047's update 202 us, 189 with this), and a K-major B the same way (191,
// 178 with the plan tile's order of reads and loads).
//
//   A: 64 rows of 128 bytes, a load 8 rows; chunk c of row r at c ^ row_key<8>(r)
//   B: 64 k-rows of 64 columns, a load 8 k-rows; chunk c of k-row r at c ^ 4 (r / 2 mod 2), so
//      that the four k-rows that half a wave's transposing read touches, 64 bytes of each,
//      are in different banks
// Rows and columns past the operand re-read its last ones (their outputs are never stored); k past
// K reads zeros.  A load out of range in every lane may count as done ahead of those issued
// before it, and the last slab of a B whose k-rows are no multiple of the slab's may hold such
// loads: the waits that count loads are not used with it in flight.
#pragma once

#include <type_traits>

#include "../rows/rows_tile.hpp"

namespace gnt {

template <int IN, int OUT, typename Args>
__global__ __launch_bounds__(256, 2) void tile64(Args p)
{
    using Hooks = TileHooks<Args>;
    constexpr bool PAIRED = Hooks::kPaired;
    constexpr int ST = 4, OPER = 8192, NL = 4;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[ST * 2 * OPER];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;

    int tm, tn, split;
    if (!Hooks::map(p, tm, tn, split))
        return;
    const int m0 = tm * 64, n0 = tn * 64;
    const int rows_a = min(64, p.M - m0), rows_b = min(64, p.N - n0);
    const int first = split * p.kt_per_split, nk = min(p.k_tiles - first, p.kt_per_split);
    const bool whole = PAIRED ? Hooks::cols(p) % 32 == 0 : p.K % 64 == 0;

    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
    const __amdgpu_buffer_rsrc_t rs_a =
        make_rsrc(p.A + (int64_t)m0 * p.lda, (uint32_t)rows_a * (uint32_t)p.lda * 2u);
    const int ldb = Hooks::ldb(p, wave & 1);
    const uint16_t *B = Hooks::b(p, wave & 1);
    // load j of wave w: rows (k-rows) 32 j + 8 w .. +8
    const int lr = lane >> 3;
    const int lc = (lane & 7) ^ row_key<8>(8 * wave + lr);
    const int mc = (lane & 7) ^ (4 * ((lr >> 1) & 1));
    auto issue = [&](int i) {
        const int k0 = (first + i) * 64;
        const uint32_t at = lds0 + (uint32_t)(i % ST) * (2u * OPER);
        const bool kin = lc * 8 < p.K - k0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = 32 * j + 8 * wave + lr;
            const uint32_t v = kin ? (uint32_t)min(row, rows_a - 1) * (uint32_t)p.lda * 2u + (uint32_t)lc * 16u : kOutOfRange;
            load_lds16(rs_a, v, (uint32_t)k0 * 2u, at + (uint32_t)(32 * j + 8 * wave) * 128u);
        }
        const int k_rows = PAIRED ? min(32, Hooks::cols(p) - k0 / 2) : min(64, p.K - k0);
        const __amdgpu_buffer_rsrc_t rs_b =
            make_rsrc(B + (int64_t)(PAIRED ? k0 / 2 : k0) * ldb + n0, (uint32_t)(((int64_t)k_rows * ldb - n0) * 2));
        const int col = min(8 * mc, (rows_b - 1) & ~7);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = PAIRED ? 16 * j + 8 * (wave >> 1) + lr : 32 * j + 8 * wave + lr;
            const uint32_t v = row < k_rows ? (uint32_t)row * (uint32_t)ldb * 2u + (uint32_t)col * 2u : kOutOfRange;
            load_lds16(rs_b, v, 0, at + OPER + (uint32_t)(32 * j + 8 * wave) * 128u);
        }
    };

    // Fragments of k 16 ks .. +16: the 8 k from 8 (lane / 32) of row (column) rb + lane % 32.
    const int fr = lane & 31, h = lane >> 5;
    auto read_a = [&](const uint8_t *base, int ks, int rb) -> u32x4 {
        const int r = rb + fr;
        return *reinterpret_cast<const u32x4 *>(base + r * 128 + (((2 * ks + h) ^ row_key<8>(r)) * 16));
    };
    // (ds_read_b64_tr_b16 gives lane i of a 16-lane group element i % 4 of the 8-byte pieces that
    // lanes i / 4 + 4 e address: lane j addresses k-row 8 (j / 32) + (j % 16) / 4, and four on,
    // columns 16 (j / 16 mod 2) + 4 (j % 4) .. +4)
    const int kq = (lane & 15) >> 2, piece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    auto read_mn = [&](const uint8_t *base, int ks, int cb) -> u32x4 {
        typedef short v4s __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4s lds_v4s;
        const int c = (cb / 8 + piece) ^ (4 * ((kq >> 1) & 1));
        const uint8_t *at = base + (16 * ks + 8 * h + kq) * 128 + c * 16 + 8 * (lane & 1);
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)at));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(at + 4 * 128)));
        return (u32x4){a[0], a[1], b[0], b[1]};
    };

    f32x16 acc[1][1];
#pragma unroll
    for (int e = 0; e < 16; ++e)
        acc[0][0][e] = 0.0f;
#pragma unroll 1
    for (int i = 0; i < ST - 1 && i < nk; ++i)
        issue(i);
    for (int i = 0; i < nk; ++i) {
        // slab i has landed for this wave once at most the loads of the ST - 2 slabs after it are out
        if (i + ST - 2 < nk - (whole ? 0 : 1))
            wait_vmcnt<(ST - 2) * NL>();
        else
            wait_vmcnt<0>();
        wait_lgkmcnt0();
        wg_barrier();
        if (i + ST - 1 < nk)
            issue(i + ST - 1);
        const uint8_t *sa = smem + (i % ST) * (2 * OPER), *sb = sa + OPER;
        u32x4 af[4], bf[4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            af[ks] = read_a(sa, ks, wm);
            bf[ks] = read_mn(sb, ks, wn);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            acc[0][0] = mfma32x32x16<IN>(bf[ks], af[ks], acc[0][0]);
    }
    mfma_settle();
    wait_lgkmcnt0();
    wg_barrier();                          // the ring is idle
    Hooks::template add<IN, OUT>(p, acc, m0 + wm, n0 + wn, split, lane);
    if (p.inreduce) {
        if (!splitk_arrive<4>(p, acc, Hooks::tile(p, tm, tn), split, wave, lane, reinterpret_cast<uint32_t *>(smem)))
            return;
        p.splits = 1;
    }
    uint8_t *stage = smem + wave * 4096;
    if constexpr (Hooks::kStore) {
        Hooks::store(p, acc, m0 + wm, n0 + wn, stage, lane);
    } else {
        const int r0 = m0 + wm, c0 = n0 + wn;
        constexpr int SIZE = OUT == OUT_FP32 ? 4 : 2;
        store_block_rows<OUT>(acc, stage, static_cast<uint8_t *>(p.C) + ((int64_t)r0 * p.ldc + c0) * SIZE, p.ldc,
                              p.M - r0, p.N - c0, lane);
    }
}

}  // namespace gnt
