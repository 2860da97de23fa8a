// Products of few rows with 4-bit weights: the weights are streamed once, on
// the matrix cores.
//
//   y[t][j] = sum_g s_jg * (A_tjg - 15.5 S_tg) + z_jg * S_tg,
//   A_tjg = sum_{i in g} x_ti (16 + q_ji),   S_tg = sum_{i in g} x_ti.
//
// A workgroup makes 16 R outputs of up to 16 NB rows; its waves take the tiles of
// 128 inputs in turn and add their sums up through LDS, so nothing is split
// across workgroups, nothing needs a workspace, and the order of the sums is
// fixed.  A wave loads a tile of 16 x 128 codes with one 16-byte load a lane,
// straight in the matrix operand's order, and makes eight bf16 values 16 + q of a
// word in seven instructions (codes_to_bf16); products of those with bf16
// activations are exact.  With the weights as the first operand a lane holds four
// outputs of one row (16x16x32 MFMA), and S comes from the same instruction with
// a first operand of ones, in the same place.  Scales and zero points: each lane
// loads one pair of the tile's (up to four groups x four outputs a quad of lanes),
// and a broadcast within the 16 lanes of a row (DPP) hands them out.
//
// fp32 activations are split into three bf16 (8 + 8 + 8 bits, exact but for
// what lies below the smallest bf16), which take three neighbouring columns: five rows a pass.
#include <algorithm>

#include "fourbit_common.hpp"

namespace grinqh {
namespace {

constexpr int kStreamTilesY = 1 << 15;             // row tiles in a launch's second dimension
template <bool F32, int NB>
constexpr int kStreamRows = F32 ? 5 : 16 * NB;     // rows of a workgroup

template <int N>
__device__ __forceinline__ float row_bcast(float v) {                          // lane N of each 16
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + N, 0xF, 0xF, false));
}

// The PART-th of the three bf16 that add up to x, as the upper half of a word.  Truncation:
// no part rounds up past the largest float.  What is not finite is all in the first.
__device__ __forceinline__ uint32_t bf16_part(float x, int part) {
    const uint32_t hi = __float_as_uint(x) & 0xFFFF0000u;
    const float rest = x - __uint_as_float(hi);
    const uint32_t mid = __float_as_uint(rest) & 0xFFFF0000u;
    const uint32_t lo = __float_as_uint(rest - __uint_as_float(mid)) & 0xFFFF0000u;
    if ((__float_as_uint(x) & 0x7F800000u) == 0x7F800000u)                     // a NaN's bits may all lie in the lower half
        return part != 0 ? 0u : x != x ? 0x7FC00000u : hi;
    return part == 0 ? hi : part == 1 ? mid : lo;
}

template <bool F32, int R, int NB>
struct Stage {
    u32x4 code[R];
    uint32_t grid[R];
    u32x4 x[NB][4][F32 ? 2 : 1];
};

template <int GROUP, bool F32, int R, int NB, int W, int DEPTH>
__global__ __launch_bounds__(W * kWave) void fourbit_stream_kernel(FourbitArgs a, int vector_store) {
    constexpr int NG = kTileIn / GROUP, STEPS = 4 / NG;
    __shared__ f32x4 red[W][R * NB][kWave];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const RunTile run = find_run_tile(a, kStreamRows<F32, NB>, blockIdx.z * kStreamTilesY + blockIdx.y, lane);
    if (run.count <= 0) return;
    const int col = lane & 15, quad = lane >> 4;
    const int tile0 = blockIdx.x * R;

    // This lane's rows of x: a column of every block of 16 (rows past the run's
    // last take it again; what comes out is not stored).
    const char* from[NB];
    bool there[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int t = F32 ? min(col / 3, run.count - 1) : min(16 * b + col, run.count - 1);
        const int src = source_row(a, run.row + t);
        there[b] = src >= 0;
        from[b] = static_cast<const char*>(a.x) + (max(src, 0) * a.x_stride + 8 * quad) * (F32 ? 4 : 2);
    }
    const uint8_t* codes[R];
    const uint16_t* grid[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t tile = (static_cast<int64_t>(run.expert) * a.row_tiles + min(tile0 + r, a.row_tiles - 1)) * a.k_tiles;
        codes[r] = a.codes + tile * 1024 + lane * 16;
        grid[r] = a.grid + (tile * NG * 16 + min(col >> 2, NG - 1) * 16 + 4 * quad + (col & 3)) * 2;
    }
    const auto load = [&](Stage<F32, R, NB>& st, int kt) {
        kt = min(kt, a.k_tiles - 1);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            st.code[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes[r] + static_cast<int64_t>(kt) * 1024));
            st.grid[r] = *reinterpret_cast<const uint32_t*>(grid[r] + static_cast<int64_t>(kt) * (NG * 32));
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int k = kt * kTileIn + 32 * m;
                const u32x4* p = reinterpret_cast<const u32x4*>(from[b] + static_cast<int64_t>(k < a.d_in ? k : 0) * (F32 ? 4 : 2));
                st.x[b][m][0] = p[0];
                if constexpr (F32) st.x[b][m][1] = p[1];
            }
    };

    f32x4 total[R][NB];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b) total[r][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

    const auto work = [&](const Stage<F32, R, NB>& st, int kt) {
        bf16x8 x[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                u32x4 v;
                if constexpr (F32) {
                    const int part = col % 3;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const u32x4 w = st.x[b][m][i >> 1];
                        v[i] = bf16_part(__uint_as_float(w[2 * (i & 1)]), part) >> 16 |
                               bf16_part(__uint_as_float(w[2 * (i & 1) + 1]), part);
                    }
                } else {
                    v = st.x[b][m][0];
                }
                const bool in = there[b] && kt * kTileIn + 32 * m < a.d_in;
                x[b][m] = __builtin_bit_cast(bf16x8, in ? v : u32x4{0u, 0u, 0u, 0u});
            }
        bf16x8 w[R][4];
        float s[R], z[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int m = 0; m < 4; ++m) w[r][m] = codes_to_bf16(st.code[r][m]);
            s[r] = f16_to_f32(static_cast<uint16_t>(st.grid[r]));
            z[r] = __builtin_fmaf(-kCodeBias, s[r], f16_to_f32(static_cast<uint16_t>(st.grid[r] >> 16)));
        }
        const auto of_group = [&](auto group) {
            constexpr int G = decltype(group)::value;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                f32x4 sum{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int m = G * STEPS; m < (G + 1) * STEPS; ++m)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, x[b][m], sum, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    f32x4 t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int m = G * STEPS; m < (G + 1) * STEPS; ++m)
                        t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[r][m], x[b][m], t, 0, 0, 0);
                    f32x4& y = total[r][b];
                    y[0] = __builtin_fmaf(row_bcast<4 * G>(s[r]), t[0], __builtin_fmaf(row_bcast<4 * G>(z[r]), sum[0], y[0]));
                    y[1] = __builtin_fmaf(row_bcast<4 * G + 1>(s[r]), t[1], __builtin_fmaf(row_bcast<4 * G + 1>(z[r]), sum[1], y[1]));
                    y[2] = __builtin_fmaf(row_bcast<4 * G + 2>(s[r]), t[2], __builtin_fmaf(row_bcast<4 * G + 2>(z[r]), sum[2], y[2]));
                    y[3] = __builtin_fmaf(row_bcast<4 * G + 3>(s[r]), t[3], __builtin_fmaf(row_bcast<4 * G + 3>(z[r]), sum[3], y[3]));
                }
            }
        };
        of_group(std::integral_constant<int, 0>());
        if constexpr (NG > 1) of_group(std::integral_constant<int, 1>());
        if constexpr (NG > 2) {
            of_group(std::integral_constant<int, 2>());
            of_group(std::integral_constant<int, 3>());
        }
    };

    // A ring of DEPTH tiles under way.
    Stage<F32, R, NB> ring[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(ring[d], wave + d * W);
    for (int kt = wave; kt < a.k_tiles; kt += DEPTH * W) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (kt + d * W < a.k_tiles) {
                work(ring[d], kt + d * W);
                if (kt + (d + DEPTH) * W < a.k_tiles) load(ring[d], kt + (d + DEPTH) * W);
            }
        }
    }

#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int b = 0; b < NB; ++b) red[wave][r * NB + b][lane] = total[r][b];
    __syncthreads();
    for (int at = threadIdx.x; at < R * NB * kWave; at += W * kWave) {
        const int rb = at >> 6;
        f32x4 y = red[0][rb][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) y += red[w][rb][lane];
        int t = 16 * (rb % NB) + col;
        if constexpr (F32) {                                                   // three parts of a row, the largest last
            f32x4 up = y;
#pragma unroll
            for (int i = 0; i < 4; ++i) up[i] = __shfl_down(y[i], 2, 16);
            f32x4 mid = y;
#pragma unroll
            for (int i = 0; i < 4; ++i) mid[i] = __shfl_down(y[i], 1, 16);
            y = up + mid + y;
            t = col % 3 == 0 && col < 15 ? col / 3 : run.count;
        }
        const int j = (tile0 + rb / NB) * kTileOut + 4 * quad;
        if (t >= run.count || j >= a.d_out) continue;
        const int64_t to = static_cast<int64_t>(run.row + t) * a.d_out + j;
        if (vector_store) {
            if (a.y_dtype == GRINQH_F32)
                *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + to) = y;
            else
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + to) =
                    u32x2{f32_to_bf16(y[0]) | static_cast<uint32_t>(f32_to_bf16(y[1])) << 16,
                          f32_to_bf16(y[2]) | static_cast<uint32_t>(f32_to_bf16(y[3])) << 16};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (j + i >= a.d_out) break;
                if (a.y_dtype == GRINQH_F32)
                    static_cast<float*>(a.y)[to + i] = y[i];
                else
                    static_cast<uint16_t*>(a.y)[to + i] = f32_to_bf16(y[i]);
            }
        }
    }
}

template <int GROUP, bool F32, int R, int NB, int W, int DEPTH>
grinqh_status stream_launch(const FourbitArgs& a, int vector_store, hipStream_t stream) {
    constexpr int kRows = kStreamRows<F32, NB>;
    // at most a tile more for every expert that can have rows
    const int64_t tiles = a.ends == nullptr ? (a.n_rows + kRows - 1) / kRows
                                            : a.n_rows / kRows + std::min(a.n_rows, a.n_experts);
    const unsigned y = static_cast<unsigned>(std::min<int64_t>(tiles, kStreamTilesY));
    const dim3 grid((a.row_tiles + R - 1) / R, y, static_cast<unsigned>((tiles + kStreamTilesY - 1) / kStreamTilesY));
    return launch_kernel(fourbit_stream_kernel<GROUP, F32, R, NB, W, DEPTH>, grid, W * kWave, 0, stream, a, vector_store);
}

template <int GROUP>
grinqh_status stream_group(const FourbitArgs& a, int x_dtype, int vector_store, hipStream_t stream) {
    if (x_dtype == GRINQH_F32) return stream_launch<GROUP, true, 1, 1, 8, 2>(a, vector_store, stream);
    const int rows = a.n_rows / a.n_experts;       // of an expert, on average
    if (rows <= 16) return stream_launch<GROUP, false, 1, 1, 8, 4>(a, vector_store, stream);
    return stream_launch<GROUP, false, 2, 2, 8, 2>(a, vector_store, stream);
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
