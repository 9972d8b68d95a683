// w4_tile.h -- the matrix-instruction core of the products with many token rows:
// C[i, j] = sum_l A(i, l) B(j, l) on BM x BN tiles of LDS, 64 summation indices a step.
//
// An operand tile lies in LDS in one of two layouts, both in 16-byte chunks of
// eight bfloat16:
//   by rows  [row][64 l], 8 chunks a row, chunk c of row r at c ^ (r / 2 & 7);
//   by steps [64 l][row], chunk c of line l at by_steps(c, l): the source holds its
//            rows as columns, and ds_read_b64_tr_b16 turns 4 x 16 blocks on the way
//            to the matrix instruction.
// Both permutations spread the 256 bytes of a read cycle over all banks.
// Dense operands arrive by buffer_load ... lds (no registers, out-of-range chunks
// arrive as zeros); stored 4-bit weights pass through registers, where they
// become bfloat16.  Two stages: the next one fills while the present one is used.
//
// v_mfma_f32_32x32x16_bf16: lane l gives row l % 32, indices 8 (l / 32) .. + 7 of
// each operand; sum e of a lane is row 8 (e / 4) + 4 (l / 32) + e % 4 of the first
// operand and row l % 32 of the second.
#pragma once

#include "w4_mfma.h"

namespace fqw {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;

constexpr int kDeep = 64;             // summation indices per step
constexpr uint32_t kOut = 0x80000000u;  // an offset beyond every buffer: reads as zeros

template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int MS = BM / WM / 32, NS = BN / WN / 32;  // 32 x 32 tiles of a wave
};

__device__ __forceinline__ int by_rows(int row, int chunk) { return row * 64 + ((chunk ^ (row / 2 & 7)) * 8); }
// position of chunk c in line l, and the chunk at a position
__device__ __forceinline__ int by_steps(int c, int l) {
    return c ^ ((l & 1) << 2) ^ (l & 2) ^ ((l & 2) << 2) ^ ((c >> 3) & 3);
}
__device__ __forceinline__ int by_steps_at(int p, int l) {
    const int c = p ^ ((l & 1) << 2) ^ ((l & 2) << 2);
    return c ^ (l & 2) ^ ((c >> 3) & 3);
}

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A buffer of `bytes` bytes from p on: loads beyond its end give zeros.  Uniform over the wave.
__device__ __forceinline__ u32x4 buffer(const void* p, uint32_t bytes) {
    const uint64_t a = (uint64_t)p;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)a),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32) & 0xFFFF),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}
// 16 bytes a lane from offset `off` of a buffer to 1 KiB of LDS at dst (one address per
// wave, in M0, which nothing else here uses).  Written out, because the compiler's own
// form makes every later LDS read wait for it; wait_dma() ends such loads.  There is
// no destination register that could be reused meanwhile.  The wait states cover a
// descriptor or address that the vector unit has just put into scalar registers (5).
__device__ __forceinline__ void dma16(u32x4 b, uint16_t* dst, uint32_t off) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_void*)dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(b)
                 : "memory");
}
__device__ __forceinline__ void wait_dma() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A dense operand, rows of `ld` elements with `cols` summation indices each, that
// fills tiles by rows.  Base 16-byte aligned, ld and cols multiples of 8, ROWS * ld
// * 2 bytes under 2^31.
template <int ROWS, int THREADS>
struct DenseRows {
    static constexpr int kLoads = ROWS * 8 / THREADS, kWaveRows = kLoads * 8;
    const uint16_t* base;
    static_assert(kLoads % 2 == 0, "8 rows a load: even and odd loads differ in row / 2 & 4");
    uint32_t bytes, off, step;
    int64_t cols;
    int col, wave;
    __device__ __forceinline__ DenseRows(const uint16_t* p, int64_t row0, int64_t rows, int64_t ld, int64_t cols_,
                                         int wave_, int lane)
        : cols(cols_), wave(wave_) {
        const int64_t left = rows - row0 < ROWS ? rows - row0 : ROWS;
        base = p + row0 * ld;
        bytes = (uint32_t)(left * ld * 2);
        col = ((lane % 8) ^ (lane / 16)) * 8;
        off = (uint32_t)((wave * kWaveRows + lane / 8) * ld) * 2;
        step = (uint32_t)(8 * ld * 2);
    }
    __device__ __forceinline__ void fill(uint16_t* tile, int64_t l0) const {
        const u32x4 b = buffer(base + l0, bytes);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = i % 2 ? col ^ 32 : col;
            dma16(b, tile + (wave * kWaveRows + i * 8) * 64, c < cols - l0 ? off + i * step + 2 * c : kOut);
        }
    }
};

// A dense operand whose summation index runs over its `lines` lines of `ld`
// elements, columns col0 .. col0 + ROWS - 1 (of `cols`): fills tiles by steps.  Base
// 16-byte aligned, ld and cols multiples of 8, 64 * ld * 2 bytes under 2^31.
template <int ROWS, int THREADS>
struct DenseSteps {
    static constexpr int kChunks = ROWS / 8, kLoads = kDeep * kChunks / THREADS, kLines = 64 / kChunks;
    static_assert(kLines == 2 || kLines == 4, "a wave's 64 chunks are whole lines");
    const uint16_t* base;
    int64_t lines, ld;
    uint32_t off[2];  // even and odd loads differ in l & 2 where a load is 2 lines
    int wave;
    __device__ __forceinline__ DenseSteps(const uint16_t* p, int64_t col0, int64_t cols, int64_t lines_, int64_t ld_,
                                          int wave_, int lane)
        : base(p + col0), lines(lines_), ld(ld_), wave(wave_) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int l = lane / kChunks + (kLines == 2 ? 2 * h : 0);
            const int c = by_steps_at(lane % kChunks, l) * 8;
            off[h] = c < cols - col0 ? (uint32_t)((lane / kChunks) * ld + c) * 2 : kOut;
        }
    }
    __device__ __forceinline__ void fill(uint16_t* tile, int64_t l0) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int l = (wave * kLoads + i) * kLines;  // kLoads is even: i & 1 is the parity of l / kLines
            const int64_t left = lines - l0 - l;
            const int64_t n = left < 0 ? 0 : left < kLines ? left : kLines;
            dma16(buffer(base + (l0 + l) * ld, (uint32_t)(n * ld * 2)), tile + l * ROWS, off[i & 1]);
        }
    }
};

// operand registers for v_mfma_f32_32x32x16_bf16: 32 rows from `row`, indices 16 s .. + 15
__device__ __forceinline__ bf16x8 frag_rows(const uint16_t* tile, int row, int s, int lane) {
    return *reinterpret_cast<const bf16x8*>(tile + by_rows(row + lane % 32, 2 * s + lane / 32));
}
template <int ROWS>
__device__ __forceinline__ bf16x8 frag_steps(uint16_t* tile, int row, int s, int lane) {
    const int l = 16 * s + 8 * (lane / 32) + (lane % 16) / 4, c = row / 8 + 2 * (lane / 16 % 2) + lane % 4 / 2;
    const int h = lane % 2 * 4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tile + l * ROWS + by_steps(c, l) * 8 + h));
    const s16x4 b =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tile + (l + 4) * ROWS + by_steps(c, l) * 8 + h));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Tiles of C in the order that the 8 dies' caches like: workgroup b runs on die
// b % 8, which gets a run of consecutive tiles, and runs go down bands of `band`
// tile rows so that a die holds few distinct tiles of either operand.
__device__ __forceinline__ void tile_at(uint32_t b, uint32_t ni, uint32_t nj, uint32_t& ti, uint32_t& tj) {
    const uint32_t all = ni * nj, die = b % 8, q = all / 8, r = all % 8;
    const uint32_t t = die * q + (die < r ? die : r) + b / 8;
    constexpr uint32_t kBand = 4;
    const uint32_t first = t / (kBand * nj) * kBand, rows = ni - first < kBand ? ni - first : kBand;
    const uint32_t in = t - first * nj;
    ti = first + in % rows;
    tj = in / rows;
}

}  // namespace fqw
