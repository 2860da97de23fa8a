// The 4-bit weights' layout and the pieces that their products share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "device_common.hpp"
#include "grinqh.h"
#include "internal.h"
#include "kv_common.hpp"

namespace grinqh {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTileOut = 16, kTileIn = 128;        // a tile of codes: 1024 bytes, one 16-byte load of a wave
constexpr int kMaxRows = 1 << 20, kMaxExperts = 1024;

// A product's operands, for the kernels (ends NULL: one expert has all rows).
struct FourbitArgs {
    const void* x;
    const int32_t* rows;
    const int32_t* ends;
    const uint8_t* codes;
    const uint16_t* grid;
    void* y;
    int64_t x_stride;
    int n_x, n_rows, d_in, d_out, k_tiles, row_tiles, n_experts, y_dtype;
};

// Eight codes (one word of a tile) as the bf16 values 16 + q, in the order of the
// inputs: between 16 and 32 a bf16 steps by 1/8, so a code's four bits, put at
// bit 3, add q to 16 exactly.  Seven instructions for eight codes.
// (seven, if the constants are in registers: 16 in a vector register, which the
// compiler has to be kept from folding, and the mask in a scalar one.)
__device__ __forceinline__ uint32_t bf16_sixteens() {
    uint32_t v = 0x41804180u;
    asm("" : "+v"(v));                             // no instruction: one that wrote a register here would need waits of its own
    return v;
}
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t w, uint32_t sixteens) {
    constexpr uint32_t kMask = 0x00780078u;
    const u32x4 v{(w & kMask) | sixteens, ((w >> 4) & kMask) | sixteens, ((w >> 8) & kMask) | sixteens,
                  (__builtin_amdgcn_alignbit(w, w, 12) & kMask) | sixteens};
    return __builtin_bit_cast(bf16x8, v);
}
constexpr float kCodeBias = 15.5f;                 // 16 + q - kCodeBias = q + 1/2

// Rows of one expert's run that a tile of TM rows works on.
struct RunTile {
    int expert, row, count;                        // count 0: no such tile
};

__device__ __forceinline__ int run_sum_up_to(int x, int lane) {                // over lanes 0 .. lane
#pragma unroll
    for (int k = 1; k < kWave; k <<= 1) {
        const int y = __shfl_up(x, k);
        if (lane >= k) x += y;
    }
    return x;
}

// Tile `number` of all experts' tiles, in order; every lane of the wave comes here.
__device__ __forceinline__ RunTile find_run_tile(const FourbitArgs& a, int tm, int number, int lane) {
    if (a.ends == nullptr) return RunTile{0, number * tm, min(tm, a.n_rows - number * tm)};
    const auto end_of = [&](int e) { return min(max(a.ends[e], 0), a.n_rows); };
    int first = 0, count = a.n_experts, before = 0;
    while (true) {
        const int run = (count + kWave - 1) / kWave;
        const int e0 = min(first + lane * run, first + count), e1 = min(e0 + run, first + count);
        int tiles = 0;
        int begin = end_of(e0);
        for (int e = e0; e < e1; ++e) {
            const int end = end_of(e + 1);
            tiles += (max(end - begin, 0) + tm - 1) / tm;
            begin = end;
        }
        const int sum = run_sum_up_to(tiles, lane);
        const uint64_t over = __ballot(before + sum > number);
        if (over == 0) return RunTile{0, 0, 0};
        const int at = __builtin_ctzll(over);
        before += __builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(tiles, at);
        first = __builtin_amdgcn_readlane(e0, at);
        count = __builtin_amdgcn_readlane(e1, at) - first;
        if (run == 1) break;
    }
    const int begin = end_of(first), end = end_of(first + 1);
    const int row = begin + (number - before) * tm;
    return RunTile{first, row, min(tm, end - row)};
}

// The row of x that row r of the result takes, or -1: none, it counts as zeros.
__device__ __forceinline__ int source_row(const FourbitArgs& a, int r) {
    const int s = a.rows == nullptr ? r : a.rows[r];
    return static_cast<unsigned>(s) < static_cast<unsigned>(a.n_x) ? s : -1;
}

// 16 (4) bytes per lane from memory straight into LDS, lane after lane from `lds`
// (uniform).  Written out because the compiler, not knowing which buffer an LDS
// read is from, would wait for every such load before it; the kernels wait for
// them themselves.
__device__ __forceinline__ void load_to_lds(const void* from, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(from)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_word_to_lds(const void* from, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tglobal_load_lds_dword %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(from)
                 : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)p));
}

// Chunk c (16 bytes) of row r of 128 bf16 lies at c ^ (r & 15): the 16 rows of an
// operand's read fall on different banks.
__device__ __forceinline__ int chunk_at(int r, int c) { return r * 256 + ((c ^ (r & 15)) * 16); }

bool valid_fourbit_layout(const grinqh_fourbit_layout* L);

// Tiles of tm rows that a call can have: at most one more for every expert that can have rows.
inline int64_t most_row_tiles(const FourbitArgs& a, int tm) {
    return a.ends == nullptr ? (a.n_rows + tm - 1) / tm : a.n_rows / tm + std::min(a.n_rows, a.n_experts);
}

// The kernel for many rows (fourbit_tile.hip; bf16 activations), in tiles of 64 or
// 128 rows x kTileColumns outputs, up to kMaxTileGroups of them (a launch has less than 2^32 work items).
constexpr int kTileColumns = 256;
constexpr int64_t kMaxTileGroups = (int64_t{1} << 23) - 16;
grinqh_status launch_fourbit_tile(const FourbitArgs& a, int group, int rows, hipStream_t stream);

}  // namespace grinqh
