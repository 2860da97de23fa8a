// Products of many rows with 4-bit weights: tiles of rows x outputs on the
// matrix cores.
//
//   y[t][j] = sum_g s_jg * A_tjg + (z_jg - 15.5 s_jg) * S_tg,
//   A_tjg = sum_{i in g} x_ti (16 + q_ji),   S_tg = sum_{i in g} x_ti.
//
// A workgroup of eight waves makes a tile of 64 or 128 rows x 256 outputs and walks
// the inputs in steps of 128.  Rows are brought straight into LDS two steps ahead
// and summed up one ahead; codes go from memory into the wave that owns their
// outputs, which makes the second operand of them itself (codes_to_bf16), so no
// code is unpacked twice.  A group's products are summed in accumulators of their
// own, exact codes with bf16 activations, and scaled into the fp32 sums while the
// next products run.  z S is one more matrix instruction a group, of z and S
// cut into bf16 parts.
//
// 2048 rows 4096 to 14336: 266 us, 0.90 PFLOP/s, where a large bf16 product of the
// library reaches 1.37.  A step of 128 rows takes 2.1 us, 1.0 of them matrix
// instructions: scaling, unpacking and LDS reads share the issue of waves that meet
// at every step's barrier.
// Tried, before results were stored in whole stretches: rows through registers
// 289 us, twice the outputs a wave with half the rows 301 us.
#include "fourbit_common.hpp"

namespace grinqh {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileWaves = 8, kTileThreads = kTileWaves * kWave;
constexpr int kXcds = 8;

// TM rows (TB blocks of 32) x 256 outputs, 32 to a wave.
template <int GROUP, int TB>
struct TileShape {
    static constexpr int TM = TB * 32, TN = kTileWaves * 32, NG = kTileIn / GROUP;
    static constexpr int kSteps = TM * 16 / kTileThreads;          // steps of 32 inputs that a wave sums up of 16 rows
    static constexpr int kParts = GROUP / 32 > kSteps ? GROUP / 32 / kSteps : 1;   // waves that a group's sums of x come from
    static constexpr int kSums = kSteps > GROUP / 32 ? kSteps / (GROUP / 32) : 1;  // groups that a wave has sums of
    static constexpr int kEntries = NG * kParts;                   // sums of a row in a step
    static constexpr int kBytes = TM * 256;                        // of a step's rows
};

// A float as the sum of three bf16, cut off one after another (24 bits).
struct Cut {
    uint32_t a, b, c;                                              // in the upper halves of words
};
__device__ __forceinline__ Cut cut(float v) {
    const uint32_t a = __float_as_uint(v) & 0xFFFF0000u;
    const float r = v - __uint_as_float(a);
    const uint32_t b = __float_as_uint(r) & 0xFFFF0000u;
    return Cut{a, b, __float_as_uint(r - __uint_as_float(b))};
}
// The upper halves of two words, `low` in the lower half.
__device__ __forceinline__ uint32_t upper_halves(uint32_t low, uint32_t high) {
    return __builtin_amdgcn_perm(high, low, 0x07060302u);
}
// Operands whose eight products add up to u * v to 2^-24 of it: every product of
// two parts but the smallest.
__device__ __forceinline__ u32x4 left_parts(float u) {
    const Cut s = cut(u);
    const uint32_t bc = upper_halves(s.b, s.c);
    return u32x4{upper_halves(s.a, s.a), upper_halves(s.b, s.a), bc, bc};
}
__device__ __forceinline__ u32x4 right_parts(float v) {
    const Cut z = cut(v);
    return u32x4{upper_halves(z.a, z.b), upper_halves(z.a, z.c), upper_halves(z.b, z.a), upper_halves(z.c, z.b)};
}

// Eight outputs of a row (fewer at its end), 16 bytes at a time where the result
// allows it.
__device__ __forceinline__ void store_eight(const FourbitArgs& a, int whole, int64_t to, const f32x4 (&v)[2], int count) {
    if (whole) {
        if (a.y_dtype == GRINQH_F32) {
            f32x4* y = reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + to);
            y[0] = v[0];
            if (count > 4) y[1] = v[1];
        } else {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = f32_to_bf16(v[i >> 1][2 * (i & 1)]) | static_cast<uint32_t>(f32_to_bf16(v[i >> 1][2 * (i & 1) + 1])) << 16;
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.y) + to) = w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= count) break;
        if (a.y_dtype == GRINQH_F32)
            static_cast<float*>(a.y)[to + i] = v[i >> 2][i & 3];
        else
            static_cast<uint16_t*>(a.y)[to + i] = f32_to_bf16(v[i >> 2][i & 3]);
    }
}

template <int GROUP, int TB>
__global__ __launch_bounds__(kTileThreads) void fourbit_tile_kernel(FourbitArgs a, int m_tiles, int n_tiles, int whole_stores) {
    using S = TileShape<GROUP, TB>;
    constexpr int NG = S::NG, STEPS = 8 / NG, TC = TB / 2;         // steps of 16 inputs in a group; row blocks in half a tile
    __shared__ __attribute__((aligned(1024))) char xs[3][S::kBytes];
    __shared__ u32x4 sums[3][S::kEntries][S::TM];                  // sums of rows, as left_parts
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    // Consecutive workgroups run on different XCDs: each takes a stretch of tiles
    // of its own, rows first, so that its L2 serves the same weights to all of them.
    const int tiles = m_tiles * n_tiles, stretch = (tiles + kXcds - 1) / kXcds;
    const int tile = (blockIdx.x % kXcds) * stretch + blockIdx.x / kXcds;
    if (static_cast<int>(blockIdx.x) / kXcds >= stretch || tile >= tiles) return;
    const RunTile run = find_run_tile(a, S::TM, tile % m_tiles, lane);
    if (run.count <= 0) return;
    const int out0 = (tile / m_tiles) * S::TN + wave * 32;         // first output of the wave

    // A wave brings TM / 8 rows of x, four whole lines at a time, straight into LDS:
    // lane after lane, so a lane asks for the chunk whose place it is.  Rows that
    // are not there (past the run, or gathered from nowhere) read another row and
    // are not stored, or stored as zeros; inputs past the last read the row's
    // last ones, and the padded groups' s and z of zero take them out.
    const uint16_t* from[S::kSteps];
    int chunk[S::kSteps];
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i) {
        const int r = wave * (4 * S::kSteps) + 4 * i + (lane >> 4), t = min(r, run.count - 1);
        from[i] = static_cast<const uint16_t*>(a.x) + max(source_row(a, run.row + t), 0) * a.x_stride;
        chunk[i] = 8 * ((lane & 15) ^ (r & 15));
    }
    const uint32_t lds0 = lds_address(&xs[0][0]) + wave * (S::kSteps * 1024);
    const auto bring_x = [&](int buffer, int kt) {
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i)
            load_to_lds(from[i] + min(kt * kTileIn + chunk[i], a.d_in - 8), lds0 + buffer * S::kBytes + i * 1024);
    };
    // 16 rows as an operand, 32 kSteps inputs of each: with ones as the other their
    // sums come out, four rows to each 16 lanes, of which each lane keeps one.
    const int row16 = (wave % (S::TM / 16)) * 16, my_step = wave / (S::TM / 16) * S::kSteps;
    const auto sum_x = [&](int buffer) {
        const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
#pragma unroll
        for (int g = 0; g < S::kSums; ++g) {
            f32x4 sum{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = g * (S::kSteps / S::kSums); i < (g + 1) * (S::kSteps / S::kSums); ++i) {
                const bf16x8 mine = *reinterpret_cast<const bf16x8*>(&xs[buffer][chunk_at(row16 + (lane & 15), 4 * (my_step + i) + (lane >> 4))]);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mine, ones, sum, 0, 0, 0);
            }
            const float even = lane & 2 ? sum[2] : sum[0], odd = lane & 2 ? sum[3] : sum[1];
            // which of the step's sums: its group, and the wave's part of it
            sums[buffer][my_step * S::kSums / S::kSteps + g][row16 + 4 * (lane >> 4) + (lane & 3)] = left_parts(lane & 1 ? odd : even);
        }
    };

    // Codes: 32 outputs are two packed tiles; a lane takes the words of its output
    // for inputs 32 m + 8 half and 16 further.
    const uint8_t* codes;
    const uint16_t* grid;
    {
        const int j = min(out0 / kTileOut + ((lane >> 4) & 1), a.row_tiles - 1);
        const int64_t at = (static_cast<int64_t>(run.expert) * a.row_tiles + j) * a.k_tiles;
        codes = a.codes + at * 1024 + ((lane & 15) + 16 * half) * 16;
        grid = a.grid + (at * NG * 16 + (lane & 15)) * 2;
    }
    u32x4 code[2], code_next[2];
    uint32_t scale[NG], scale_next[NG];
    const auto load_w = [&](u32x4 (&c)[2], uint32_t (&s)[NG], int kt) {
        const uint8_t* p = codes + static_cast<int64_t>(kt) * 1024;
        c[0] = *reinterpret_cast<const u32x4*>(p);
        c[1] = *reinterpret_cast<const u32x4*>(p + 512);
#pragma unroll
        for (int g = 0; g < NG; ++g) s[g] = *reinterpret_cast<const uint32_t*>(grid + (static_cast<int64_t>(kt) * NG + g) * 32);
    };

    // y: the sums; p: products of a group and half the rows, two sets in turn.
    f32x16 y[TB], p[2][TC];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
        for (int t = 0; t < TB; ++t) y[t][i] = 0.f;
#pragma unroll
        for (int t = 0; t < TC; ++t) p[1][t][i] = 0.f;
    }

    const uint32_t sixteens = bf16_sixteens();
    // Tiles that run beside one another begin at different inputs, so that they
    // do not all ask the same few channels of memory for their rows.
    const int first = (tile / m_tiles + tile % m_tiles) % a.k_tiles;
    const auto place = [&](int kt) {                               // the last tile again past the end
        kt = min(kt, a.k_tiles - 1) + first;
        return kt < a.k_tiles ? kt : kt - a.k_tiles;
    };
    bring_x(0, place(0));
    bring_x(1, place(1));
    load_w(code, scale, place(0));
    // All loads have come in before the loop (the compiler, seeing some under way on
    // one path into it, would wait at every step's start for that step's own).
    __builtin_amdgcn_s_waitcnt(0x0F70);                            // vmcnt(0)
    __syncthreads();
    sum_x(0);
    __syncthreads();

    const auto x_at = [&](int buffer, int t, int step) {
        return *reinterpret_cast<const bf16x8*>(xs[buffer] + chunk_at(t * 32 + (lane & 31), 2 * step + half));
    };
    const auto w_at = [&](const u32x4 (&c)[2], int step) { return codes_to_bf16(c[step & 1][step >> 1], sixteens); };
    bf16x8 x[2][TC], w[STEPS];
#pragma unroll
    for (int t = 0; t < TC; ++t) {
        x[0][t] = x_at(0, t, 0);
        x[1][t] = x_at(0, t, 1);
    }
    w[0] = w_at(code, 0);
    float s = 0.f;                                                 // of the products that wait
    constexpr int kEvery = 4 * TC >= STEPS ? 1 : STEPS / (4 * TC), kPieces = 4 * TC >= STEPS ? 4 * TC / STEPS : 1;

    int turn = 0;                                                  // kt % 3
    for (int kt = 0; kt < a.k_tiles; ++kt) {
        // No branch: behind one the compiler would put all that is added meanwhile.
        // Past the last step the last tile is brought again, for nobody.  Rows are
        // brought two steps ahead and summed one ahead, so that a step's first
        // operands are there before the barrier that ends the step before.
        const int next_turn = turn == 2 ? 0 : turn + 1, last_turn = turn == 0 ? 2 : turn - 1;
        load_w(code_next, scale_next, place(kt + 1));
        bring_x(last_turn, place(kt + 2));
        bf16x8 z{};
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int st = 0; st < STEPS; ++st) {
                    const int q = (g * 2 + h) * STEPS + st;                     // of 16 in all
                    // z S of two sums of x, into the rows whose products do not wait
                    constexpr int kPairs = (S::kEntries + 1) / 2, kApart = NG / kPairs;
                    if (st == 0 && g % kApart == 0) {
                        const int e = 2 * (g / kApart);
                        if (h == 0) {
                            const uint32_t low = scale[e / S::kParts], high = S::kEntries == 1 ? 0u : scale[(e + 1) / S::kParts % NG];
                            const uint32_t sz = half ? high : low;
                            z = __builtin_bit_cast(bf16x8, right_parts(__builtin_fmaf(-kCodeBias, f16_to_f32(static_cast<uint16_t>(sz)),
                                                                                      f16_to_f32(static_cast<uint16_t>(sz >> 16)))));
                        }
#pragma unroll
                        for (int t = 0; t < TC; ++t) {
                            const u32x4 sum = sums[turn][S::kEntries == 1 ? 0 : e + half][(h * TC + t) * 32 + (lane & 31)];
                            y[h * TC + t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, sum), z, y[h * TC + t], 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < TC; ++t) {
                        f32x16 zero{};
                        p[h][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[q & 1][t], w[st], st == 0 ? zero : p[h][t], 0, 0, 0);
                    }
                    // the next step's weights, and rows two steps ahead: an LDS read takes longer than one
                    if (h == 0 && st + 1 < STEPS) w[st + 1] = w_at(code, g * STEPS + st + 1);
                    const int q2 = (q + 2) % 16, g2 = q2 / (2 * STEPS), h2 = q2 / STEPS % 2, st2 = q2 % STEPS;
#pragma unroll
                    for (int t = 0; t < TC; ++t) x[q & 1][t] = x_at(q + 2 < 16 ? turn : next_turn, h2 * TC + t, g2 * STEPS + st2);
                    // a piece of the products that wait: rows 8 i + 4 half + 0 .. 3 of block t
                    if (st % kEvery == 0) {
#pragma unroll
                        for (int k = 0; k < kPieces; ++k) {
                            const int piece = st / kEvery * kPieces + k, t = piece / 4, i = piece % 4;
#pragma unroll
                            for (int n = 4 * i; n < 4 * i + 4; ++n)
                                y[(h ^ 1) * TC + t][n] = __builtin_fmaf(s, p[h ^ 1][t][n], y[(h ^ 1) * TC + t][n]);
                        }
                    }
                    if (st == STEPS - 1) {                                      // these are the ones that wait now
                        s = f16_to_f32(static_cast<uint16_t>(scale[g]));
                        asm volatile("" : "+v"(s));                              // else each use converts it, in a longer instruction
                        if (h == 1) w[0] = g + 1 < NG ? w_at(code, (g + 1) * STEPS) : w_at(code_next, 0);
                    }
                    if (q == 3) sum_x(next_turn);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
        for (int i = 0; i < 2; ++i) code[i] = code_next[i];
#pragma unroll
        for (int g = 0; g < NG; ++g) scale[g] = scale_next[g];
        turn = next_turn;
        // Before the others may go on: the rows that this step brought are in LDS
        // (the next step sums them up and reads its last operands from them), and so
        // are the sums (of the LDS operations only the last four may be under way,
        // all of them reads).
        asm volatile("" ::: "memory");
        static_assert(2 * TC <= 4, "reads at the end of a step");
        __builtin_amdgcn_s_waitcnt(0x0070 | 4 << 8);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
#pragma unroll
    for (int t = 0; t < TC; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) y[TC + t][i] = __builtin_fmaf(s, p[1][t][i], y[TC + t][i]);

    // Out: 32 rows at a time through LDS, so that a wave stores whole stretches of
    // them (2048 rows 4096 to 14336: 266 us, 288 element by element).  The rows lie 32 bytes apart from multiples of 256: a lane
    // pair's rows, 4 apart, fall on different banks.  No rows are brought any more:
    // the last step has waited for them.
    constexpr int kOutStride = S::TN * 4 + 32;
    static_assert(32 * kOutStride <= 3 * S::kBytes, "the rows' buffers hold 32 rows of the result");
    char* out = &xs[0][0];
    const int block0 = (tile / m_tiles) * S::TN, columns = min(S::TN, a.d_out - block0);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            *reinterpret_cast<float*>(out + (8 * (i >> 2) + 4 * half + (i & 3)) * kOutStride + (wave * 32 + (lane & 31)) * 4) = y[t][i];
        __syncthreads();
        for (int at = threadIdx.x; at < 32 * (S::TN / 8); at += kTileThreads) {
            const int r = at / (S::TN / 8), c = at % (S::TN / 8) * 8, row = t * 32 + r;
            if (row >= run.count || c >= columns) continue;
            f32x4 v[2];
            v[0] = *reinterpret_cast<const f32x4*>(out + r * kOutStride + c * 4);
            v[1] = *reinterpret_cast<const f32x4*>(out + r * kOutStride + c * 4 + 16);
            if (source_row(a, run.row + row) < 0) v[0] = v[1] = f32x4{0.f, 0.f, 0.f, 0.f};
            store_eight(a, whole_stores, static_cast<int64_t>(run.row + row) * a.d_out + block0 + c, v, columns - c);
        }
    }
}

template <int GROUP, int TB>
grinqh_status tile_launch(const FourbitArgs& a, hipStream_t stream) {
    using S = TileShape<GROUP, TB>;
    static_assert(S::TN == kTileColumns && kTileThreads * (kMaxTileGroups + kXcds) < int64_t{1} << 32, "what the caller has counted");
    const int64_t m = most_row_tiles(a, S::TM), n = (a.d_out + S::TN - 1) / S::TN, groups = (m * n + kXcds - 1) / kXcds * kXcds;
    const bool f32 = a.y_dtype == GRINQH_F32;
    const int whole_stores = a.d_out % (f32 ? 4 : 8) == 0 && aligned_to(a.y, 16);
    return launch_kernel(fourbit_tile_kernel<GROUP, TB>, dim3(static_cast<unsigned>(groups)), kTileThreads, 0, stream, a,
                         static_cast<int>(m), static_cast<int>(n), whole_stores);
}

}  // namespace

template <int GROUP>
static grinqh_status tile_group(const FourbitArgs& a, int rows, hipStream_t stream) {
    return rows == 64 ? tile_launch<GROUP, 2>(a, stream) : tile_launch<GROUP, 4>(a, stream);
}

grinqh_status launch_fourbit_tile(const FourbitArgs& a, int group, int rows, hipStream_t stream) {
    if (group == 32) return tile_group<32>(a, rows, stream);
    if (group == 64) return tile_group<64>(a, rows, stream);
    return tile_group<128>(a, rows, stream);
}

}  // namespace grinqh
