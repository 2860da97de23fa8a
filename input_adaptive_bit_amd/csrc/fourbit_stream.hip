// Products of few rows with 4-bit weights: the weights are streamed once, on
// the matrix cores.  Here too: the host's checks, and which kernel a call takes.
//
//   y[t][j] = sum_g s_jg * A_tjg + (z_jg - 15.5 s_jg) * S_tg,
//   A_tjg = sum_{i in g} x_ti (16 + q_ji),   S_tg = sum_{i in g} x_ti.
//
// A workgroup makes 16 R outputs of some rows; its waves take the tiles of 128
// inputs in turn and add their sums up through LDS, so nothing is split across
// workgroups, nothing needs a workspace, and the order of the sums is fixed.  A
// tile of 16 x 128 codes is one 16-byte load a lane, straight in the matrix
// operand's order, and a word of it becomes eight bf16 values 16 + q in seven
// instructions (codes_to_bf16); products of those with bf16 activations are
// exact.  With the weights as the first operand a lane holds four outputs of one
// row (16x16x32 MFMA), and S comes from the same instruction with a first operand
// of ones, in the same place.  Scales and zero points: each lane loads one pair
// of the tile's (up to four groups x four outputs a quad of lanes), and LDS or a
// broadcast within 16 lanes (DPP) hands them out.
//
// fp32 activations are split into three bf16 (8 + 8 + 8 bits, exact but for what
// lies below the smallest bf16): each part a product of its own, or for few rows and
// outputs three neighbouring columns of one.
#include <math.h>

#include <algorithm>

#include "fourbit_common.hpp"

namespace grinqh {
namespace {

constexpr int kStreamTilesY = 1 << 15;             // row tiles in a launch's second dimension
constexpr int kDepth = 4;                          // tiles of codes that a wave has under way (and fp32 tiles split at a time)

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int N>
__device__ __forceinline__ uint32_t row_bcast(uint32_t v) {                    // lane N of each 16
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x150 + N, 0xF, 0xF, true));
}

// Eight floats as the sum of three bf16 each, cut off one after another: the upper
// halves of x, of what is left, and of what is left then.
__device__ __forceinline__ void split_eight(const f32x4& low, const f32x4& high, bf16x8& a, bf16x8& b, bf16x8& c) {
    u32x4 part[3];
    uint32_t word[3][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = i < 4 ? low[i & 3] : high[i & 3];
        const float rest = x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
        word[0][i & 1] = __float_as_uint(x);
        word[1][i & 1] = __float_as_uint(rest);
        word[2][i & 1] = __float_as_uint(rest - __uint_as_float(__float_as_uint(rest) & 0xFFFF0000u));
        if (i & 1)
#pragma unroll
            for (int p = 0; p < 3; ++p) part[p][i >> 1] = __builtin_amdgcn_perm(word[p][1], word[p][0], 0x07060302u);
    }
    a = __builtin_bit_cast(bf16x8, part[0]);
    b = __builtin_bit_cast(bf16x8, part[1]);
    c = __builtin_bit_cast(bf16x8, part[2]);
}

// Codes of a tile of R x 16 outputs, and this lane's (s, z) pair of each.
template <int R>
struct Codes {
    u32x4 code[R];
    uint32_t grid[R];
};

template <int R>
struct WeightAt {
    const uint8_t* codes[R];
    const uint16_t* grid[R];
};

template <int GROUP, int R>
__device__ __forceinline__ WeightAt<R> weight_at(const FourbitArgs& a, int expert, int tile0, int lane) {
    constexpr int NG = kTileIn / GROUP;
    const int col = lane & 15, quad = lane >> 4;
    WeightAt<R> at;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t tile = (static_cast<int64_t>(expert) * a.row_tiles + min(tile0 + r, a.row_tiles - 1)) * a.k_tiles;
        at.codes[r] = a.codes + tile * 1024 + lane * 16;
        at.grid[r] = a.grid + (tile * NG * 16 + min(col >> 2, NG - 1) * 16 + 4 * quad + (col & 3)) * 2;
    }
    return at;
}

template <int GROUP, int R>
__device__ __forceinline__ void load_codes(Codes<R>& c, const WeightAt<R>& at, int kt) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        c.code[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(at.codes[r] + static_cast<int64_t>(kt) * 1024));
        c.grid[r] = *reinterpret_cast<const uint32_t*>(at.grid[r] + static_cast<int64_t>(kt) * (kTileIn / GROUP * 32));
    }
}

// Adds a tile's products to y[row tile]: lane 16 q + c has outputs 4 q .. 4 q + 3 of
// row c.  A group's sum begins at -15.5 S, so what is left is s times it and z
// times S, with s and z as they are packed (`grid` gives the four pairs): mixed
// multiply-adds take fp16 operands.
// P: bf16 that an activation is the sum of, the largest first.
template <int GROUP, int R, int P, typename Grid>
__device__ __forceinline__ void multiply(f32x4 (&y)[R], const u32x4 (&code)[R], const bf16x8 (&x)[P][4], Grid grid) {
    constexpr int NG = kTileIn / GROUP, STEPS = 4 / NG;
    const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    const uint32_t sixteens = bf16_sixteens();
    f32x4 sum[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        sum[g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = P * g * STEPS; i < P * (g + 1) * STEPS; ++i)
            sum[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, x[P - 1 - i % P][i / P], sum[g], 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        bf16x8 w[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) w[m] = codes_to_bf16(code[r][m], sixteens);
        const auto of_group = [&](auto group) {
            constexpr int G = decltype(group)::value;
            const u32x4 pairs = grid(r, group);
            f32x4 t = sum[G] * -kCodeBias;
#pragma unroll
            for (int i = P * G * STEPS; i < P * (G + 1) * STEPS; ++i)
                t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i / P], x[P - 1 - i % P][i / P], t, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f16x2 sz = __builtin_bit_cast(f16x2, static_cast<uint32_t>(pairs[i]));
                y[r][i] = __builtin_fmaf(static_cast<float>(sz[0]), t[i], __builtin_fmaf(static_cast<float>(sz[1]), sum[G][0], y[r][i]));
            }
        };
        of_group(std::integral_constant<int, 0>());
        if constexpr (NG > 1) of_group(std::integral_constant<int, 1>());
        if constexpr (NG > 2) {
            of_group(std::integral_constant<int, 2>());
            of_group(std::integral_constant<int, 3>());
        }
    }
}

// Four outputs j .. j + 3 of a row.
__device__ __forceinline__ void store_outputs(const FourbitArgs& a, int vector_store, int row, int j, const f32x4& y) {
    const int64_t to = static_cast<int64_t>(row) * a.d_out + j;
    if (vector_store) {
        if (a.y_dtype == GRINQH_F32)
            *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + to) = y;
        else
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + to) =
                u32x2{f32_to_bf16(y[0]) | static_cast<uint32_t>(f32_to_bf16(y[1])) << 16,
                      f32_to_bf16(y[2]) | static_cast<uint32_t>(f32_to_bf16(y[3])) << 16};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (j + i >= a.d_out) break;
        if (a.y_dtype == GRINQH_F32)
            static_cast<float*>(a.y)[to + i] = y[i];
        else
            static_cast<uint16_t*>(a.y)[to + i] = f32_to_bf16(y[i]);
    }
}

// bf16 activations.  What a wave works on goes through a piece of LDS of its own:
// rows read in the operand's order would ask for 16 lines an instruction, lane
// after lane in another one (64 rows 4096 to 14336 took 37 us so, 23 through LDS); brought into
// LDS four whole lines at a time, and with them the codes, D tiles are under way
// without a register held.  XR: rows in fours (4 XR of them).
template <int R, int XR>
struct WaveStage {
    static constexpr int kCodes = XR * 1024, kGrid = kCodes + R * 1024, kBytes = kGrid + R * 256, kLoads = XR + 2 * R;
};

template <int GROUP, typename T, int R, int XR, int W, int D>
__global__ __launch_bounds__(W * kWave, 2) void fourbit_wave_kernel(FourbitArgs a, int vector_store) {
    using S = WaveStage<R, XR>;
    constexpr int kRed = W * R * 1024;
    __shared__ __attribute__((aligned(1024))) char lds[W * D * S::kBytes > kRed ? W * D * S::kBytes : kRed];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr bool kF32 = sizeof(T) == 4;
    constexpr int kLineLanes = kF32 ? 32 : 16, kPiece = 16 / sizeof(T);        // lanes that bring a row's 128 inputs, of a lane
    constexpr int kRows = XR * kWave / kLineLanes;
    static_assert(kRows <= 16 && (kRows & (kRows - 1)) == 0, "rows that divide the columns of a matrix tile");
    const RunTile run = find_run_tile(a, kRows, blockIdx.z * kStreamTilesY + blockIdx.y, lane);
    if (run.count <= 0) return;
    const int col = lane & 15, quad = lane >> 4, tile0 = blockIdx.x * R;
    const WeightAt<R> at = weight_at<GROUP, R>(a, run.expert, tile0, lane);
    // Rows past the run read its last one, rows gathered from nowhere the first of
    // x (and are stored as zeros); inputs past the last read the row's last
    // ones, and the padded groups' s and z of zero take them out.
    const T* from[XR];
    int piece[XR];
#pragma unroll
    for (int i = 0; i < XR; ++i) {
        const int r = i * (kWave / kLineLanes) + lane / kLineLanes;
        from[i] = static_cast<const T*>(a.x) + max(source_row(a, run.row + min(r, run.count - 1)), 0) * a.x_stride;
        piece[i] = kPiece * (lane % kLineLanes ^ (r & 15));
    }
    char* mine = lds + wave * (D * S::kBytes);
    const uint32_t lds0 = lds_address(mine);
    const auto bring = [&](int stage, int kt) {
        kt = min(kt, a.k_tiles - 1);
        const uint32_t to = lds0 + stage * S::kBytes;
#pragma unroll
        for (int i = 0; i < XR; ++i)
            load_to_lds(from[i] + min(kt * kTileIn + piece[i], a.d_in - kPiece), to + i * 1024);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            load_to_lds(at.codes[r] + static_cast<int64_t>(kt) * 1024, to + S::kCodes + r * 1024);
            load_word_to_lds(at.grid[r] + static_cast<int64_t>(kt) * (kTileIn / GROUP * 32), to + S::kGrid + r * 256);
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) bring(d, wave + d * W);
    f32x4 y[R];
#pragma unroll
    for (int r = 0; r < R; ++r) y[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    int stage = 0;
    for (int kt = wave; kt < a.k_tiles; kt += W) {
        constexpr int kUnderWay = (D - 1) * S::kLoads;             // loads that may be: those of the stages behind this one
        static_assert(kUnderWay < 64, "a count that the wait can name");
        __builtin_amdgcn_s_waitcnt(0x0F70 | (kUnderWay & 15) | (kUnderWay >> 4) << 14);
        asm volatile("" ::: "memory");
        const char* from_lds = mine + stage * S::kBytes;
        constexpr int NG = kTileIn / GROUP;
        u32x4 code[R], grid[R][NG];
        bf16x8 x[kF32 ? 3 : 1][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            code[r] = *reinterpret_cast<const u32x4*>(from_lds + S::kCodes + r * 1024 + lane * 16);
#pragma unroll
            for (int g = 0; g < NG; ++g) grid[r][g] = *reinterpret_cast<const u32x4*>(from_lds + S::kGrid + r * 256 + quad * 64 + g * 16);
        }
        const int row = col & (kRows - 1);                         // the rows again in the columns past them
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if constexpr (kF32) {
                const char* at = from_lds + row * 512;
                const f32x4 low = *reinterpret_cast<const f32x4*>(at + (8 * m + 2 * quad ^ row) * 16);
                const f32x4 high = *reinterpret_cast<const f32x4*>(at + (8 * m + 2 * quad + 1 ^ row) * 16);
                split_eight(low, high, x[0][m], x[1][m], x[2][m]);
            } else {
                x[0][m] = *reinterpret_cast<const bf16x8*>(from_lds + chunk_at(row, 4 * m + quad));
            }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);                        // lgkmcnt(0): the stage has been read and may be filled again
        asm volatile("" ::: "memory");
        bring(stage, kt + D * W);
        stage = stage + 1 == D ? 0 : stage + 1;
        multiply<GROUP, R, kF32 ? 3 : 1>(y, code, x, [&](int r, auto g) { return grid[r][decltype(g)::value]; });
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);                            // vmcnt(0): nothing is brought into LDS any more
    __syncthreads();
    f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int r = 0; r < R; ++r) red[(wave * R + r) * kWave + lane] = y[r];
    __syncthreads();
    for (int r = wave; r < R; r += W) {
        f32x4 sum = red[r * kWave + lane];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += red[(w * R + r) * kWave + lane];
        const int j = (tile0 + r) * kTileOut + 4 * quad;
        if (col >= run.count || j >= a.d_out) continue;
        if (source_row(a, run.row + col) < 0) sum = f32x4{0.f, 0.f, 0.f, 0.f};
        store_outputs(a, vector_store, run.row + col, j, sum);
    }
}

// What some lanes of a wave wrote to LDS is there for its other lanes to read, and
// what they read for others to overwrite.  The wave's LDS operations are carried out in
// their order, so this keeps the compiler from changing it and is no instruction.
__device__ __forceinline__ void between_lanes() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// fp32 activations of up to MT rows: the three parts of a row take three
// neighbouring columns.  A wave splits the activations of kDepth of its tiles at a
// time (eight values a lane) and passes them to the operand's order through a
// piece of LDS of its own.
template <int GROUP, int MT, int W>
__global__ __launch_bounds__(W * kWave, 2) void fourbit_stream_f32_kernel(FourbitArgs a, int vector_store) {
    constexpr int kCols = 3 * MT;
    __shared__ u32x4 parts[W][kDepth * 16 * kCols];        // [tile][16-byte chunk of its inputs][column]
    __shared__ f32x4 red[W][kWave];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const RunTile run = find_run_tile(a, MT, blockIdx.z * kStreamTilesY + blockIdx.y, lane);
    if (run.count <= 0) return;
    const int col = lane & 15, quad = lane >> 4;
    const WeightAt<1> at = weight_at<GROUP, 1>(a, run.expert, blockIdx.x, lane);
    Codes<1> ring[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if (wave + d * W < a.k_tiles) load_codes<GROUP>(ring[d], at, wave + d * W);

    // This lane splits chunk `col` of tile `quad` of the kDepth.
    const float* from[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int src = t < run.count ? source_row(a, run.row + t) : -1;
        from[t] = src < 0 ? nullptr : static_cast<const float*>(a.x) + src * a.x_stride + 8 * col;
    }
    f32x4 raw[MT][2];
    const auto load_x = [&](int kt) {
        const int k = (kt + quad * W) * kTileIn;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            raw[t][0] = raw[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (from[t] != nullptr && k + 8 * col < a.d_in) {
                raw[t][0] = *reinterpret_cast<const f32x4*>(from[t] + k);
                raw[t][1] = *reinterpret_cast<const f32x4*>(from[t] + k + 4);
            }
        }
    };
    load_x(wave);

    f32x4 y[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
    for (int kt = wave; kt < a.k_tiles; kt += kDepth * W) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            bf16x8 part[3];
            split_eight(raw[t][0], raw[t][1], part[0], part[1], part[2]);
#pragma unroll
            for (int p = 0; p < 3; ++p) parts[wave][lane * kCols + 3 * t + p] = __builtin_bit_cast(u32x4, part[p]);
        }
        between_lanes();
        load_x(kt + kDepth * W);
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            const int now = kt + d * W;
            if (now < a.k_tiles) {
                bf16x8 x[1][4];
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    x[0][m] = __builtin_bit_cast(bf16x8, parts[wave][(16 * d + 4 * m + quad) * kCols + min(col, kCols - 1)]);
                const uint32_t mine = ring[d].grid[0];
                multiply<GROUP, 1, 1>(y, ring[d].code, x, [&](int, auto g) {
                    constexpr int at = 4 * decltype(g)::value;
                    return u32x4{row_bcast<at>(mine), row_bcast<at + 1>(mine), row_bcast<at + 2>(mine), row_bcast<at + 3>(mine)};
                });
                if (now + kDepth * W < a.k_tiles) load_codes<GROUP>(ring[d], at, now + kDepth * W);
            }
        }
        between_lanes();                                       // all of it has been read: the next tiles may go there
    }
    red[wave][lane] = y[0];
    __syncthreads();
    if (wave != 0) return;
    f32x4 sum = red[0][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) sum += red[w][lane];
    f32x4 mid, low;                                                            // the row's other parts, two and one columns on
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mid[i] = __shfl_down(sum[i], 1, 16);
        low[i] = __shfl_down(sum[i], 2, 16);
    }
    sum = low + mid + sum;
    const int j = blockIdx.x * kTileOut + 4 * quad;
    if (col % 3 == 0 && col / 3 < run.count && j < a.d_out) store_outputs(a, vector_store, run.row + col / 3, j, sum);
}

dim3 stream_grid(const FourbitArgs& a, int rows, int outputs) {
    const int64_t tiles = most_row_tiles(a, rows);
    return dim3((a.row_tiles + outputs - 1) / outputs, static_cast<unsigned>(std::min<int64_t>(tiles, kStreamTilesY)),
                static_cast<unsigned>((tiles + kStreamTilesY - 1) / kStreamTilesY));
}

template <int GROUP, int R, int XR, int W, int D>
grinqh_status wave_launch(const FourbitArgs& a, int vector_store, hipStream_t stream) {
    return launch_kernel(fourbit_wave_kernel<GROUP, uint16_t, R, XR, W, D>, stream_grid(a, 4 * XR, R), W * kWave, 0, stream, a, vector_store);
}
template <int GROUP, int R, int XR, int W, int D>
grinqh_status wave_f32_launch(const FourbitArgs& a, int vector_store, hipStream_t stream) {
    return launch_kernel(fourbit_wave_kernel<GROUP, float, R, XR, W, D>, stream_grid(a, 2 * XR, R), W * kWave, 0, stream, a, vector_store);
}

template <int GROUP, int MT, int W>
grinqh_status stream_f32_launch(const FourbitArgs& a, int vector_store, hipStream_t stream) {
    return launch_kernel(fourbit_stream_f32_kernel<GROUP, MT, W>, stream_grid(a, MT, 1), W * kWave, 0, stream, a, vector_store);
}

// Tiles of tm rows that a call has, about: half of an expert's last one is empty.
int64_t expected_tiles(const FourbitArgs& a, int tm) {
    if (a.ends == nullptr) return (a.n_rows + tm - 1) / tm;
    return a.n_rows / tm + std::max(1, std::min(a.n_rows, a.n_experts) / 2);
}

// Which kernel, by the sizes that the host knows.  Times in us on 256 CUs, groups
// of 128, of codes that come from memory:
//                          wave kernel   64-row tiles   128-row tiles
//   4096 to 4096, 512 rows     37             41             61
//   4096 to 4096, 1024 rows    73             47             63
//   4096 to 14336, 128 rows    36             40             61
//   4096 to 14336, 192 rows    55             41             62
//   4096 to 14336, 1024 rows   267            157            131
// A step of 128 inputs takes a 64-row tile 1.25 us and a 128-row tile 2, whether
// few of them run or one on every CU; the wave kernel takes 0.15 ns for 16 rows x
// 16 outputs x 128 inputs where there are enough of them to fill the card.  Smaller
// groups cost all of them 8 and 35 % more.  Tiles that would be more than a launch
// holds (results of well over 100 GB) are not taken: the wave kernel's grid has three dimensions.
//
// Of the wave kernels, the wider and taller one where it leaves work for every CU (us;
// R W: outputs in sixteens and waves of a workgroup):
//                                  tiles   1 8    2 8    2 4    4 4
//   1 row 4096 to 4096               256   3.9    5.0    5.3    7.3
//   8 rows 4096 to 8192              512   6.4    5.6    5.8    7.6
//   8 rows 4096 to 14336             896   10.7   8.7    8.2    8.3
//   8 rows 8192 to 28672, g 64      1792   37     29     28.7   27.5
//   16 rows 4096 to 4096             256   4.6    5.7    5.9    7.8
//   16 rows 4096 to 8192             512   8.3    6.2    6.3    8.0
//   16 rows 2048 to 11008, g 64      688   9.2    7.9    6.3    6.2
//   16 rows 8192 to 28672, g 64     1792   51     39     35     30
//   64 rows 4096 to 4096            1024          9.7    8.0    7.7
// and of four, eight and sixteen rows the fewest that hold a call's: one row 4096 to
// 4096 takes 3.9, 4.0 and 4.3 us, 16 rows to 64 experts 4096 to 1024 9.3 us in
// eights and 9.9 in sixteens, 516 rows to 64 experts 73 in eights and 51 in sixteens.
//
// fp32 (us): the kernel that splits in few lanes where a CU's waves work on one tile
// of outputs, else the wave kernel, of 8 or 16 rows, one or four sixteens of outputs wide.
//                                  tiles   few lanes   1 wide   4 wide
//   1 row 4096 to 4096               256   4.3         7.5      11.6
//   1 row 4096 to 8192               512   7.7         13.1     11.7
//   1 row 4096 to 14336              896   12.7        23.8     12.3
//   5 rows 4096 to 4096              256   5.5         7.4      11.4
//   5 rows 4096 to 8192              512   10.6        12.9     11.6
//   5 rows 4096 to 14336             896   19.3        23.9     12.0
//   16 rows 4096 to 4096             256               8.6      13.0
//   16 rows 4096 to 14336            896               27       13.3
template <int GROUP>
grinqh_status stream_group(const FourbitArgs& a, int x_dtype, int vector_store, hipStream_t stream) {
    const int64_t rows = a.n_rows / a.n_experts;                   // of an expert, on average
    const auto tiles = [&](int tm) { return expected_tiles(a, tm) * a.row_tiles; };
    if (x_dtype == GRINQH_F32) {
        if (rows <= 1 && tiles(1) <= 640) return stream_f32_launch<GROUP, 1, 16>(a, vector_store, stream);
        if (rows <= 5 && tiles(5) <= 640) return stream_f32_launch<GROUP, 5, 8>(a, vector_store, stream);
        if (a.ends == nullptr ? rows <= 8 : rows <= 2) {
            if (tiles(8) <= 400) return wave_f32_launch<GROUP, 1, 4, 8, 2>(a, vector_store, stream);
            return wave_f32_launch<GROUP, 4, 4, 4, 2>(a, vector_store, stream);
        }
        if (tiles(16) <= 400) return wave_f32_launch<GROUP, 1, 8, 8, 2>(a, vector_store, stream);
        return wave_f32_launch<GROUP, 4, 8, 4, 2>(a, vector_store, stream);
    }
    const int64_t columns = (a.d_out + kTileColumns - 1) / kTileColumns;
    const auto steps = [&](int tm, double step) {
        return most_row_tiles(a, tm) * columns > kMaxTileGroups ? INFINITY : step * ((expected_tiles(a, tm) * columns + 255) / 256);
    };
    const double waves = 0.15e-3 * tiles(16), small = steps(64, 1.25), large = steps(128, 2.0);
    if (std::min(small, large) < waves) return launch_fourbit_tile(a, GROUP, small <= large ? 64 : 128, stream);
    if (a.ends == nullptr ? rows <= 8 : rows <= 2) {
        if (a.ends == nullptr && rows <= 4 && tiles(4) <= 320) return wave_launch<GROUP, 1, 1, 8, 4>(a, vector_store, stream);
        if (tiles(8) <= 320) return wave_launch<GROUP, 1, 2, 8, 3>(a, vector_store, stream);
        if (tiles(8) <= 576) return wave_launch<GROUP, 2, 2, 8, 2>(a, vector_store, stream);
        return wave_launch<GROUP, 2, 2, 4, 2>(a, vector_store, stream);
    }
    if (tiles(16) <= 320) return wave_launch<GROUP, 1, 4, 8, 2>(a, vector_store, stream);
    if (tiles(16) <= 576) return wave_launch<GROUP, 2, 4, 8, 2>(a, vector_store, stream);
    return wave_launch<GROUP, 4, 4, 4, 2>(a, vector_store, stream);
}

// Host checks of a product, and its kernel.
grinqh_status product(const grinqh_fourbit_layout* L, const grinqh_expert_args& p, bool plain, void* stream) {
    if (!valid_fourbit_layout(L) || (plain && L->n_experts != 1)) return GRINQH_EINVAL;
    if ((p.x_dtype != GRINQH_BF16 && p.x_dtype != GRINQH_F32) || (p.y_dtype != GRINQH_BF16 && p.y_dtype != GRINQH_F32))
        return GRINQH_EINVAL;
    if (p.n_rows < 0 || p.n_rows > kMaxRows) return GRINQH_EINVAL;
    if (p.n_rows == 0) return GRINQH_OK;
    if (p.n_x < 1 || p.n_x > kMaxRows || p.x == nullptr || p.codes == nullptr || p.grid == nullptr || p.y == nullptr ||
        (!plain && p.ends == nullptr))
        return GRINQH_EINVAL;
    if (p.x_stride < L->d_in || p.x_stride > kMaxStride) return GRINQH_EINVAL;
    const size_t xb = p.x_dtype == GRINQH_BF16 ? 2 : 4, yb = p.y_dtype == GRINQH_BF16 ? 2 : 4;
    if (!aligned_to(p.x, 16) || p.x_stride * xb % 16 != 0 || !aligned_to(p.codes, 16) || !aligned_to(p.grid, 16) ||
        !aligned_to(p.y, yb) || !aligned_to(p.rows, 4) || !aligned_to(p.ends, 4))
        return GRINQH_EALIGN;
    const size_t rows = static_cast<size_t>(p.n_rows);
    if (written_overlaps({{p.y, rows * L->d_out * yb}},
                         {{p.x, (static_cast<size_t>(p.n_x - 1) * p.x_stride + L->d_in) * xb},
                          {p.rows, p.rows == nullptr ? 0 : rows * 4},
                          {p.ends, p.ends == nullptr ? 0 : (static_cast<size_t>(L->n_experts) + 1) * 4},
                          {p.codes, grinqh_fourbit_code_bytes(L)}, {p.grid, grinqh_fourbit_grid_bytes(L)}}))
        return GRINQH_EINVAL;
    const FourbitArgs a{p.x, p.rows, p.ends, p.codes, p.grid, p.y, p.x_stride, p.n_x, p.n_rows, L->d_in, L->d_out,
                        L->k_tiles, L->row_tiles, L->n_experts, p.y_dtype};
    const int vector_store = L->d_out % 4 == 0 && aligned_to(p.y, 4 * yb);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (L->group == 32) return stream_group<32>(a, p.x_dtype, vector_store, st);
    if (L->group == 64) return stream_group<64>(a, p.x_dtype, vector_store, st);
    return stream_group<128>(a, p.x_dtype, vector_store, st);
}

}  // namespace
}  // namespace grinqh

using namespace grinqh;

extern "C" {

grinqh_status grinqh_fourbit_linear(const grinqh_fourbit_layout* L, const void* x, grinqh_dtype x_dtype,
                                    int64_t x_stride, int32_t n_tokens, const uint8_t* codes,
                                    const uint16_t* grid, void* y, grinqh_dtype y_dtype, void* stream) {
    return product(L, grinqh_expert_args{x, x_stride, x_dtype, n_tokens, nullptr, nullptr, n_tokens, codes, grid, y, y_dtype},
                   true, stream);
}

grinqh_status grinqh_expert_linear(const grinqh_fourbit_layout* L, const grinqh_expert_args* args, void* stream) {
    if (args == nullptr) return GRINQH_EINVAL;
    return product(L, *args, false, stream);
}

}  // extern "C"
