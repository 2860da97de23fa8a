// Attention of one new token of every sequence over its paged key-value cache.
//
// For query head h with key-value head g = h / group,
//   o = sum_t p_t v_t,  p_t = exp(a_t - m) / l,  a_t = scale * q . k_t.
//
// One pass over the cache with a running maximum and sum, on the bf16 matrix
// cores.  A workgroup takes one part of one sequence's tokens for up to 16 query
// heads of one key-value head; its waves (plan_decode says how many) take tiles
// of 32 tokens in turn, each with its own maximum, sum and output, joined at the
// end.
//
// Scores.  S = K Q^T as 16 tokens x 16 heads (v_mfma_f32_16x16x32_bf16).  Any
// order of the head's dimensions serves as the contraction's as long as K and
// Q agree, so a lane loads its token's row in 16-byte pieces as they lie and
// Q is laid out to match.  Keys enter as their integer codes (exact in bf16):
// q . k = s (sum q c + sum q / 2) + z sum q.
//
// Values.  O^T = V^T P^T as 16 dimensions x 16 heads over the 32 tokens.  The
// lane that holds a head's scores of 8 tokens (rows 4 g .. 4 g + 3 of both score
// tiles, g = lane / 16) takes just these tokens as its share of the contraction,
// so the weights never leave their lane; and any dimension may stand for a row
// of the product, so a lane loads D / 16 neighbouring dimensions of its 8 tokens
// and has the transposed operand in its own registers.  The codes' scale goes
// into the weights, p' = p s, and
//   sum p v = sum p' (c - mid) + sum p (z + s (mid + 1/2)),
// with the products sum p' c - mid sum p' (mid = 2^(bits - 1): the rounding of
// p' then weighs the distance from the grid's middle only).  p' (p at 16 bits)
// is used as the sum of two bf16, a relative error of 2^-16: the matrix cores
// have the time, and outputs keep the precision of fp32 weights.
//
// Long caches are cut into parts (plan_decode); each part's output, maximum
// and sum go to the workspace and the part that arrives last joins them in
// their order.
//
// What bounds it.  The cache's bytes: 32 sequences of 17 .. 8192 tokens at 8
// bits (278 MB) take 62 us, 4.5 TB/s, and past 64 K tokens each further one costs
// its bytes at 5.8 TB/s.  One sequence of 32768 (69 MB) takes 20 us, 13 of them
// the cache at 5.3 TB/s; the rest is a chain of trips to memory: 1 us for the
// length, 2 for the queries and the first tile, 1.5 to store a part and count
// its arrival, 2 to 3 to join.  At 4 bits unpacking is half of the vector
// instructions (380 for a tile), which take half of the cycles: 131071 tokens and 64
// heads (143 MB) in 39 us.  All of these with the longest length as max_len (the
// times of kernels alone, as the others in this paragraph).
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "kv_common.hpp"

namespace grinqh {
namespace {

constexpr int kTileTokens = 32;                        // tokens of a wave's tile
constexpr int kBatch = 16;                             // parts joined at a time
constexpr int kHeadTile = 16;                          // query heads of a workgroup
constexpr int64_t kMaxDecodeGroups = 1 << 23;          // workgroups of a launch
constexpr int kCounters = 4096;                        // arrival counters at the start of the workspace
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct DecodeArgs {
    KvDims d;
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const uint16_t* k_grid;
    const uint16_t* v_grid;
    const void* q;
    const int32_t* page_table;
    const int32_t* seq_lens;
    void* out;
    float* lse;
    unsigned* counters;
    float* parts;            // [item][split][heads_here][D], then the statistics
    int64_t q_stride, table_stride;
    int n_q_heads, group, head_tiles, items, splits, chunk, max_pages;
    int longest;             // min(max_len, max_pages * page_size)
    int q_dtype, out_dtype;
    float scale_log2;        // scale * log2(e): exponents are of base 2
};

// Bytes at p, `N` a power of two, as dwords (16 bits in the low half for N = 2).
template <int N>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t* r) {
    if constexpr (N == 2) {
        r[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (N == 4) {
        r[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 8) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p);
        r[0] = v.x;
        r[1] = v.y;
    } else {
#pragma unroll
        for (int n = 0; n < N / 16; ++n) {
            const u32x4 v = reinterpret_cast<const u32x4*>(p)[n];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[4 * n + i] = v[i];
        }
    }
}

template <int D, int BITS>
struct Shape {
    static constexpr int kRow = D * BITS / 8;                        // bytes of a row
    static constexpr int kKBytes = kRow / 4;                         // of a key row in one lane
    static constexpr int kPiece = kKBytes < 16 ? kKBytes : 16;       // loaded at a time
    static constexpr int kPieces = kKBytes / kPiece;
    static constexpr int kPerPiece = kPiece * 8 / BITS;              // dimensions of a piece
    static constexpr int kSteps = D / 32;                            // contraction steps of a score tile
    static constexpr int kVBytes = kRow / 16;                        // of a value row in one lane
    static constexpr int kVDwords = kVBytes < 4 ? 1 : kVBytes / 4;
    static constexpr int kVDims = D / 16;
};

// At 4 bits the heads of groups of up to 8 have two columns of the score tile each
// (COPIES 2): column i and column i + 8 hold the same scores, and the lanes of the
// first weigh the tokens of the tile's first half, those of the second the others,
// as states of their own until the end.  Half the softmax work for each lane: in a
// captured graph 131071 tokens take 42 us instead of 44 (and 41 with the waves that
// the registers then allow), 32 sequences of 2048 22 instead of 24.  At 8 bits it
// gained nothing.
__device__ __forceinline__ bool second_copy(int lane) { return (lane & 8) != 0; }

// A wave's 32 tokens as loaded: keys of two score tiles, values of this lane's
// 8 tokens, grids of the tokens that it weighs.
template <int D, int BITS, int COPIES>
struct Tile {
    uint32_t k[2][D * BITS / 128];
    uint32_t v[8][Shape<D, BITS>::kVDwords];
    u32x4 kg[2 / COPIES], vg[2 / COPIES];
};

// The grids of a lane's tokens.
template <int COPIES>
__device__ __forceinline__ void load_grids(u32x4 (&to)[2 / COPIES], const uint16_t* grid, const int64_t (&row)[2], int lane) {
    const int g = lane >> 4;
    if constexpr (COPIES == 2) {
        const int64_t first = row[0], other = row[1];
        to[0] = *reinterpret_cast<const u32x4*>(grid + (second_copy(lane) ? other : first) * 2 + 8 * g);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) to[h] = *reinterpret_cast<const u32x4*>(grid + row[h] * 2 + 8 * g);
    }
}

// Row of the first token of each half of the tile at t0 (pages that are not
// there read page 0, and nothing of it is used).
__device__ __forceinline__ void tile_rows(int64_t (&row)[2], const DecodeArgs& a, int t0, const int (&page)[2], int head) {
#pragma unroll
    for (int h = 0; h < 2; ++h) row[h] = page_row(a.d, page[h], head, t0 + 16 * h);
}

template <int D, int BITS, int COPIES>
__device__ __forceinline__ void load_keys(Tile<D, BITS, COPIES>& T, const DecodeArgs& a, const int64_t (&row)[2], int lane) {
    using S = Shape<D, BITS>;
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t* k = a.k_codes + row[h] * S::kRow;
#pragma unroll
        for (int n = 0; n < S::kPieces; ++n)
            load_bytes<S::kPiece>(k + static_cast<uint32_t>(i * S::kRow + (4 * n + g) * S::kPiece),
                                  &T.k[h][n * S::kPiece / 4]);
    }
    if constexpr (BITS < 16) load_grids<COPIES>(T.kg, a.k_grid, row, lane);
}

template <int D, int BITS, int COPIES>
__device__ __forceinline__ void load_values(Tile<D, BITS, COPIES>& T, const DecodeArgs& a, const int64_t (&row)[2], int lane) {
    using S = Shape<D, BITS>;
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t* v = a.v_codes + row[h] * S::kRow;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            load_bytes<S::kVBytes>(v + static_cast<uint32_t>((4 * g + j) * S::kRow + i * S::kVBytes), T.v[4 * h + j]);
    }
    if constexpr (BITS < 16) load_grids<COPIES>(T.vg, a.v_grid, row, lane);
}

__device__ __forceinline__ uint32_t pack_high(float lo, float hi) {   // bf16 of two floats that have one exactly
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

__device__ __forceinline__ float ubyte(uint32_t w, int b) { return static_cast<float>((w >> (8 * b)) & 0xFFu); }

// Four codes 0 .. 15, one to a byte, as bf16: read as FP8 E4M3 a byte c is
// c * 2^-9 (the subnormals and the first binade are evenly spaced).
__device__ __forceinline__ void nibbles_bf16(uint32_t bytes, uint32_t& lo, uint32_t& hi) {
    lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, 512.f, false));
    hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, 512.f, true));
}

// Contraction step `st` of a key row's share as 8 bf16.  At 4 bits the 8
// dimensions of a dword come as 0, 2, 4, 6, 1, 3, 5, 7 (q_order).
template <int BITS>
__device__ __forceinline__ bf16x8 key_step(const uint32_t* k, int st) {
    u32x4 f;
    if constexpr (BITS == 16) {
        f = u32x4{k[4 * st], k[4 * st + 1], k[4 * st + 2], k[4 * st + 3]};
    } else if constexpr (BITS == 8) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t w = k[2 * st + x];
            f[2 * x] = pack_high(ubyte(w, 0), ubyte(w, 1));
            f[2 * x + 1] = pack_high(ubyte(w, 2), ubyte(w, 3));
        }
    } else {
        const uint32_t w = k[st];
        uint32_t r[4];
        nibbles_bf16(w & 0x0F0F0F0Fu, r[0], r[1]);
        nibbles_bf16((w >> 4) & 0x0F0F0F0Fu, r[2], r[3]);
        f = u32x4{r[0], r[1], r[2], r[3]};
    }
    return __builtin_bit_cast(bf16x8, f);
}

template <int BITS>
__device__ __forceinline__ constexpr int q_order(int e) {
    return BITS == 4 ? (e < 4 ? 2 * e : 2 * (e - 4) + 1) : e;
}

// Two rows of the transposed operand (dimensions 2 m2 and 2 m2 + 1 of this
// lane's D / 16): its 8 tokens' values (codes below 16 bits) as bf16.
template <int D, int BITS, int COPIES>
__device__ __forceinline__ void value_pair(const Tile<D, BITS, COPIES>& T, int m2, bf16x8 (&f)[2]) {
    u32x4 r[2];
    if constexpr (BITS == 16) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            r[0][x] = __builtin_amdgcn_perm(T.v[2 * x + 1][m2], T.v[2 * x][m2], 0x05040100u);
            r[1][x] = __builtin_amdgcn_perm(T.v[2 * x + 1][m2], T.v[2 * x][m2], 0x07060302u);
        }
    } else if constexpr (BITS == 8) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                r[y][x] = pack_high(ubyte(T.v[2 * x][m2 / 2], 2 * (m2 % 2) + y), ubyte(T.v[2 * x + 1][m2 / 2], 2 * (m2 % 2) + y));
    } else {
        const int w = m2 / 4, b = m2 % 4;                         // dword and byte
        const uint32_t two = b == 0 ? 0x0C0C0400u : b == 1 ? 0x0C0C0501u : b == 2 ? 0x0C0C0602u : 0x0C0C0703u;
#pragma unroll
        for (int half = 0; half < 2; ++half) {                    // tokens 0 .. 3, 4 .. 7: byte b of each
            const uint32_t t01 = __builtin_amdgcn_perm(T.v[4 * half + 1][w], T.v[4 * half][w], two);
            const uint32_t t23 = __builtin_amdgcn_perm(T.v[4 * half + 3][w], T.v[4 * half + 2][w], two);
            const uint32_t by = t01 | t23 << 16;
            uint32_t lo, hi;
            nibbles_bf16(by & 0x0F0F0F0Fu, lo, hi);
            r[0][2 * half] = lo;
            r[0][2 * half + 1] = hi;
            nibbles_bf16((by >> 4) & 0x0F0F0F0Fu, lo, hi);
            r[1][2 * half] = lo;
            r[1][2 * half + 1] = hi;
        }
    }
    f[0] = __builtin_bit_cast(bf16x8, r[0]);
    f[1] = __builtin_bit_cast(bf16x8, r[1]);
}

// Maximum (or sum) over the four lanes that hold one head's tokens (lane,
// lane ^ 16, lane ^ 32, lane ^ 48).
__device__ __forceinline__ float over_groups_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float over_groups_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// A wave's state: the output sums of its head (lane % 16), the head's maximum,
// this lane's share of the sum and of the constant part.
template <int D>
struct State {
    f32x4 o[D / 16];
    float m, l, konst;
};

// The scores of a tile (exponents of base 2) of the tokens that this lane weighs.
template <int D, int BITS, int QP, int COPIES>
__device__ __forceinline__ void tile_scores(float (&a)[8 / COPIES], const Tile<D, BITS, COPIES>& T,
                                            const bf16x8 (&qf)[QP][D / 32], float q_sum, float scale_log2, int lane) {
    f32x4 sc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bf16x8 kf = key_step<BITS>(T.k[h], s);
#pragma unroll
            for (int x = 0; x < QP; ++x) sc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[x][s], sc[h], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
    for (int e = 0; e < 8 / COPIES; ++e) {
        const int h = e / 4, r = e % 4;
        const float x = COPIES == 2 && second_copy(lane) ? sc[1][r] : sc[h][r];
        if constexpr (BITS < 16) {
            const float s = f16_to_f32(static_cast<uint16_t>(T.kg[h][r])), z = f16_to_f32(static_cast<uint16_t>(T.kg[h][r] >> 16));
            a[e] = scale_log2 * __builtin_fmaf(s, x, __builtin_fmaf(0.5f, s, z) * q_sum);
        } else {
            a[e] = scale_log2 * x;
        }
    }
}

// Folds a tile's scores and values into the state.
template <int D, int BITS, int COPIES>
__device__ __forceinline__ void use_values(State<D>& st, Tile<D, BITS, COPIES>& T, float (&a)[8 / COPIES], int t0, int end,
                                           const int (&page)[2], int lane) {
    static_assert(COPIES == 1 || BITS < 16, "values of 16 bits are cleared token by token, whoever weighs them");
    constexpr int E = 8 / COPIES;                        // tokens that a lane weighs
    const int g = lane >> 4;
    const bool second = COPIES == 2 && second_copy(lane);
    float vs[E], vz[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        if constexpr (BITS < 16) {
            vs[e] = f16_to_f32(static_cast<uint16_t>(T.vg[e / 4][e % 4]));
            vz[e] = f16_to_f32(static_cast<uint16_t>(T.vg[e / 4][e % 4] >> 16));
        }
    // A tile with tokens that are not there: no score, no value, whatever the memory holds.
    if (t0 + kTileTokens > end || page[0] < 0 || page[1] < 0) {
        const auto seen = [&](int half, int r) { return page[half] >= 0 && t0 + 16 * half + 4 * g + r < end; };
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const bool is = second ? seen(1, e % 4) : seen(e / 4, e % 4);
            a[e] = is ? a[e] : -INFINITY;
            if constexpr (BITS < 16) {
                vs[e] = is ? vs[e] : 0.f;
                vz[e] = is ? vz[e] : 0.f;
            } else {
#pragma unroll
                for (int w = 0; w < Shape<D, BITS>::kVDwords; ++w) T.v[e][w] = is ? T.v[e][w] : 0u;
            }
        }
    }
    float top = a[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(top, a[e]);
    const float m_new = fmaxf(st.m, over_groups_max(top));
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float keep = __builtin_amdgcn_exp2f(st.m - base);
    st.m = m_new;
    constexpr float mid = static_cast<float>(1 << (BITS - 1));
    float p[E], l = 0.f, konst = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        p[e] = __builtin_amdgcn_exp2f(a[e] - base);
        l += p[e];
        if constexpr (BITS < 16) {
            konst = __builtin_fmaf(p[e], __builtin_fmaf(mid + 0.5f, vs[e], vz[e]), konst);
            p[e] *= vs[e];
        }
    }
    u32x4 hi, lo;
#pragma unroll
    for (int x = 0; x < E / 2; ++x) {
        hi[x] = pack_bf16(p[2 * x], p[2 * x + 1]);
        const float r0 = __uint_as_float(hi[x] << 16), r1 = __uint_as_float(hi[x] & 0xFFFF0000u);
        lo[x] = pack_bf16(p[2 * x] - r0, p[2 * x + 1] - r1);
        if constexpr (BITS < 16) {
            const float s0 = r0 + __uint_as_float(lo[x] << 16), s1 = r1 + __uint_as_float(lo[x] & 0xFFFF0000u);
            konst = __builtin_fmaf(-mid, s0 + s1, konst);
        }
    }
    if constexpr (COPIES == 2) {                         // the other copy's tokens weigh nothing here
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            hi[2 + x] = second ? hi[x] : 0u;
            lo[2 + x] = second ? lo[x] : 0u;
            hi[x] = second ? 0u : hi[x];
            lo[x] = second ? 0u : lo[x];
        }
    }
    st.l = __builtin_fmaf(st.l, keep, l);
    st.konst = __builtin_fmaf(st.konst, keep, konst);
    if (__any(keep != 1.f)) {
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) st.o[m][r] *= keep;
    }
#pragma unroll
    for (int m2 = 0; m2 < D / 32; ++m2) {
        bf16x8 vf[2];
        value_pair<D, BITS, COPIES>(T, m2, vf);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            f32x4& o = st.o[2 * m2 + y];
            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[y], __builtin_bit_cast(bf16x8, hi), o, 0, 0, 0);
            o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[y], __builtin_bit_cast(bf16x8, lo), o, 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Two neighbouring values of an output row.
__device__ __forceinline__ void store_pair(void* out, int dtype, int64_t at, float x, float y) {
    if (dtype == GRINQH_F32)
        *reinterpret_cast<float2*>(static_cast<float*>(out) + at) = make_float2(x, y);
    else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + at) = pack_bf16(x, y);
}

__device__ __forceinline__ float2 agent_load(const float* p) {
    const uint64_t w = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __builtin_bit_cast(float2, w);
}
__device__ __forceinline__ void agent_store(float* p, float2 v) {
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

// Columns of the score tile that a head has.
__host__ __device__ constexpr int copies_of(int bits, int group) { return bits == 4 && group <= kHeadTile / 2 ? 2 : 1; }

// Waves of a workgroup that has a CU to itself, by its registers (fp32 queries:
// twelve at 128 dimensions; the plan does not know the type).  Most fit; in
// scratch are 9 registers of a wave at 16 bits and 256 dimensions, and with fp32
// queries 71 there, 21 at 8 bits and 256 dimensions and 11 at 8 bits and 128.
__host__ __device__ constexpr int big_waves(int D, int copies, int qp = 1) {
    return D == 256 ? 8 : copies == 2 && (D == 64 || qp == 1) ? 16 : 12;
}

__host__ __device__ constexpr int waves_per_simd(int D, int qp, int waves) {
    return waves > 4 ? waves / 4 : D == 256 || qp == 2 ? 2 : 3;
}

// x of the lane 8 further round the row of 16.
__device__ __forceinline__ float other_copy(float x) {
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x128, 0xF, 0xF, true));   // row_ror:8
}

template <int D, int BITS, int QP, int W, int COPIES>
__global__ __launch_bounds__(W * kWave, waves_per_simd(D, QP, W)) void decode_kernel(DecodeArgs a) {
    using S = Shape<D, BITS>;
    constexpr int kDecWaves = W, kDecThreads = W * kWave, kUnit = W * kTileTokens;   // tokens of one round
    constexpr int kStride = D + 4;                       // floats of a head's row in LDS
    extern __shared__ __attribute__((aligned(16))) float lds[];                       // [wave][head][kStride], then m and l [wave][head]
    __shared__ int is_last;
    // Parts are the slow index: workgroups go to the 8 XCDs in turn, and with
    // the items as the fast one every XCD gets early and late parts alike (late
    // parts of short sequences are empty).
    const int item = blockIdx.x % a.items, split = blockIdx.x / a.items;
    const int tile = item % a.head_tiles, bg = item / a.head_tiles;
    const int b = bg / a.d.heads, head = bg % a.d.heads;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int here = min(kHeadTile, a.group - tile * kHeadTile);      // query heads of this workgroup
    const int column = COPIES == 2 ? i & 7 : i;                       // this lane's among them
    const int h0 = head * a.group + tile * kHeadTile;                 // first query head
    const int begin = split * a.chunk;
    int t = begin + wave * kTileTokens;

    // What does not hang on the sequence's length is asked for with it: the
    // first tile's pages and the queries.
    const int32_t* table = a.page_table + b * a.table_stride;
    const auto raw_pages = [&](int t0, int (&page)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) page[h] = table[min((t0 + 16 * h) >> a.d.page_shift, a.max_pages - 1)];
    };
    int page[2];
    raw_pages(t, page);
    u32x4 raw_q[S::kSteps][QP];
    {
        const int64_t q0 = b * a.q_stride + static_cast<int64_t>(h0 + (column < here ? column : 0)) * D;
#pragma unroll
        for (int s = 0; s < S::kSteps; ++s) {
            constexpr int kPer = S::kPerPiece / 8;                    // steps of a piece
            const int64_t at = q0 + (4 * (s / kPer) + g) * S::kPerPiece + 8 * (s % kPer);
#pragma unroll
            for (int x = 0; x < QP; ++x)
                raw_q[s][x] = QP == 1 ? *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + at)
                                      : *reinterpret_cast<const u32x4*>(static_cast<const float*>(a.q) + at + 4 * x);
        }
    }
    // Pages of the two halves of the tile at t0; -1 past the end or absent.
    const auto check_pages = [&](int t0, int end, int (&page)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            page[h] = t0 + 16 * h < end ? page_or_absent(page[h], a.d.n_pages) : -1;
    };
    Tile<D, BITS, COPIES> T;
    int64_t row[2];
    const int len = min(max(a.seq_lens[b], 0), a.longest);
    const int parts = max(1, (len + a.chunk - 1) / a.chunk);
    if (split >= parts) return;
    const int end = min(len, begin + a.chunk);
    check_pages(t, end, page);
    if (t < end) {
        tile_rows(row, a, t, page, head);
        load_keys(T, a, row, lane);
        load_values(T, a, row, lane);
    }

    // Q, in the order of the key pieces; heads that are not there are zeros.
    bf16x8 qf[QP][S::kSteps];
    float q_sum = 0.f;
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = QP == 2 ? __uint_as_float(raw_q[s][QP == 2 ? e / 4 : 0][e % 4])
                           : __uint_as_float(e % 2 ? raw_q[s][0][e / 2] & 0xFFFF0000u : raw_q[s][0][e / 2] << 16);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = column < here ? w[q_order<BITS>(e)] : 0.f;
            const __bf16 part = static_cast<__bf16>(x);
            qf[0][s][e] = part;
            q_sum += x;
            if constexpr (QP == 2) qf[1][s][e] = static_cast<__bf16>(x - static_cast<float>(part));
        }
    }
    q_sum = over_groups_sum(q_sum);

    State<D> st;
    st.m = -INFINITY;
    st.l = st.konst = 0.f;
#pragma unroll
    for (int m = 0; m < D / 16; ++m) st.o[m] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (t < end) {
        // A tile's keys are free once its scores are formed, its values once
        // they are added: the next tile's are loaded into the same registers.
        for (;;) {
            const bool more = t + kUnit < end;
            int next[2];
            raw_pages(t + kUnit, next);
            float sc[8 / COPIES];
            tile_scores<D, BITS, QP, COPIES>(sc, T, qf, q_sum, a.scale_log2, lane);
            __builtin_amdgcn_sched_barrier(0);
            check_pages(t + kUnit, end, next);
            if (more) {
                tile_rows(row, a, t + kUnit, next, head);
                load_keys(T, a, row, lane);
            }
            __builtin_amdgcn_sched_barrier(0);
            use_values<D, BITS, COPIES>(st, T, sc, t, end, page, lane);
            if (!more) break;
            load_values(T, a, row, lane);
            t += kUnit;
            page[0] = next[0];
            page[1] = next[1];
        }
    }

    // Join a head's columns, then the waves.
    if constexpr (COPIES == 2) {
        const float m = fmaxf(st.m, other_copy(st.m)), f = __builtin_amdgcn_exp2f(st.m - (m == -INFINITY ? 0.f : m));
        const auto both = [&](float x) {
            x *= f;
            return x + other_copy(x);
        };
        st.m = m;
        st.l = both(st.l);
        st.konst = both(st.konst);
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) st.o[x][r] = both(st.o[x][r]);
    }
    st.l = over_groups_sum(st.l);
    st.konst = over_groups_sum(st.konst);
    float* stats = lds + kDecWaves * here * kStride;
    if (i < here) {
        float* o = lds + (wave * here + i) * kStride;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int m = 0; m < D / 16; ++m) o[(4 * g + r) * (D / 16) + m] = st.o[m][r] + st.konst;
        if (g == 0) {
            stats[(wave * here + i) * 2] = st.m;
            stats[(wave * here + i) * 2 + 1] = st.l;
        }
    }
    __syncthreads();
    const bool whole = parts == 1;
    float* part = a.parts + (static_cast<int64_t>(item) * a.splits + split) * min(a.group, kHeadTile) * (D + 2);
    for (int e = threadIdx.x * 2; e < here * D; e += kDecThreads * 2) {
        const int h = e / D, x = e % D;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) m = fmaxf(m, stats[(w * here + h) * 2]);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(stats[(w * here + h) * 2] - base);
            const float* o = lds + (w * here + h) * kStride + x;
            l = __builtin_fmaf(f, stats[(w * here + h) * 2 + 1], l);
            y0 = __builtin_fmaf(f, o[0], y0);
            y1 = __builtin_fmaf(f, o[1], y1);
        }
        if (whole) {
            const float r = l == 0.f ? 0.f : 1.f / l;
            store_pair(a.out, a.out_dtype, (static_cast<int64_t>(b) * a.n_q_heads + h0 + h) * D + x, y0 * r, y1 * r);
            if (a.lse != nullptr && x == 0)
                a.lse[static_cast<int64_t>(b) * a.n_q_heads + h0 + h] = kLn2 * (m + __builtin_amdgcn_logf(l));
        } else {
            agent_store(part + h * D + x, make_float2(y0, y1));
            if (x == 0) agent_store(part + here * D + 2 * h, make_float2(m, l));
        }
    }
    if (whole) return;

    // The part that arrives last joins all of them.  Every access to the parts
    // and the counter is an agent-scope atomic, performed past the XCDs' own
    // caches; a wave's stores are done when its memory counter says so, the
    // barrier waits for every wave's, and the arrival is counted after it, so
    // the last arrival's loads, issued after the count, find every part.  (No
    // fence: at agent scope it would write back the XCD's whole L2.)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned prev = __hip_atomic_fetch_add(a.counters + item, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        is_last = prev == static_cast<unsigned>(parts - 1);
    }
    __syncthreads();
    if (!is_last) return;
    if (threadIdx.x == 0) __hip_atomic_store(a.counters + item, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // Every thread weighs the parts by itself: a batch's statistics and values
    // are asked for at once, one trip to memory.  Where two outputs to a thread
    // leave threads over, `sets` of them share the parts.
    const int64_t step = static_cast<int64_t>(min(a.group, kHeadTile)) * (D + 2);
    const float* first = a.parts + static_cast<int64_t>(item) * a.splits * step;
    const int pairs = here * (D / 2);
    const int sets = max(1, kDecThreads / pairs);
    const auto finish = [&](int h, int x, f32x4 r) {      // r: m, l and two outputs
        const float inv = r[1] == 0.f ? 0.f : 1.f / r[1];
        store_pair(a.out, a.out_dtype, (static_cast<int64_t>(b) * a.n_q_heads + h0 + h) * D + x, r[2] * inv, r[3] * inv);
        if (a.lse != nullptr && x == 0)
            a.lse[static_cast<int64_t>(b) * a.n_q_heads + h0 + h] = kLn2 * (r[0] + __builtin_amdgcn_logf(r[1]));
    };
    const auto fold = [](f32x4& r, float m, float l, float y0, float y1) {
        const float top = fmaxf(r[0], m), base = top == -INFINITY ? 0.f : top;
        const float f = __builtin_amdgcn_exp2f(r[0] - base), g = __builtin_amdgcn_exp2f(m - base);
        r = f32x4{top, r[1] * f + l * g, r[2] * f + y0 * g, r[3] * f + y1 * g};
    };
    f32x4* shared = reinterpret_cast<f32x4*>(lds);        // [set][pair]
    for (int u = threadIdx.x; u < sets * pairs; u += kDecThreads) {
        const int e = u % pairs, set = u / pairs, h = e / (D / 2), x = e % (D / 2) * 2;
        f32x4 r{-INFINITY, 0.f, 0.f, 0.f};
        for (int s0 = set; s0 < parts; s0 += kBatch * sets) {
            float2 ml[kBatch], v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                v[k] = make_float2(0.f, 0.f);
                if (s0 + k * sets < parts) {
                    const float* p = first + (s0 + k * sets) * step;
                    ml[k] = agent_load(p + here * D + 2 * h);
                    v[k] = agent_load(p + h * D + x);
                }
            }
            float top = r[0];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
            const float base = top == -INFINITY ? 0.f : top;
            r *= __builtin_amdgcn_exp2f(r[0] - base);
            r[0] = top;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float f = __builtin_amdgcn_exp2f(ml[k].x - base);
                r[1] = __builtin_fmaf(f, ml[k].y, r[1]);
                r[2] = __builtin_fmaf(f, v[k].x, r[2]);
                r[3] = __builtin_fmaf(f, v[k].y, r[3]);
            }
        }
        if (sets == 1)
            finish(h, x, r);
        else
            shared[u] = r;
    }
    if (sets == 1) return;
    __syncthreads();
    for (int e = threadIdx.x; e < pairs; e += kDecThreads) {
        f32x4 r = shared[e];
        for (int k = 1; k < sets; ++k) {
            const f32x4 y = shared[k * pairs + e];
            fold(r, y[0], y[1], y[2], y[3]);
        }
        finish(e / (D / 2), e % (D / 2) * 2, r);
    }
}

// How a call is cut up (host arithmetic on its sizes alone, so by max_len and not
// by the lengths: 4000 tokens take 11.4 us with that as max_len and 31.9 with
// 131072, whose parts are of 4224 tokens).  Measured in us a call in a captured
// graph, 8 bits, 8 key-value heads of 128, groups of 4, max_len the longest length:
//   one sequence, four waves and eight: 500 tokens 8.3, 10.2; 2000 10.0, 10.6; 4000
//   12.8, 11.8; 32768 24, 22; eight waves and twelve: 8192 15.2, 14.3; 131071 at 4
//   bits, groups of 8, 46.6, 43.5; twelve and sixteen there, with two columns a head:
//   42.2, 40.5;
//   32 sequences of 17 .. 8192 tokens, four waves: one workgroup to a CU 79, twelve
//   66 (eight waves, one to a CU 73); 32 of 2048 each: 34, 37.
constexpr int kCus = 256, kFewItems = 48, kOneRound = 128;

struct DecodePlan {
    int waves, head_tiles, splits, chunk;
    int64_t items;
    size_t ws_bytes;
};

size_t workspace_of(const grinqh_kv_layout& L, int group, int64_t parts) {
    const size_t part = static_cast<size_t>(std::min(group, kHeadTile)) * (L.head_dim + 2) * sizeof(float);
    return (kCounters * sizeof(unsigned) + parts * part + 255) / 256 * 256;
}

DecodePlan plan_decode(const grinqh_kv_layout& L, int n_q_heads, int batch, int max_len) {
    DecodePlan p;
    const int group = n_q_heads / L.n_kv_heads;
    p.head_tiles = (group + kHeadTile - 1) / kHeadTile;
    p.items = static_cast<int64_t>(batch) * L.n_kv_heads * p.head_tiles;
    // Few sequences and heads: parts for one round of a short cache (four waves,
    // 128 tokens), else one workgroup to a CU.  Many: workgroups
    // of four waves, three to a CU, of 512 tokens and more, enough of them that
    // sequences of different lengths fill the card evenly.
    const bool few = p.items <= kFewItems;
    const auto units_of = [&](int waves) { return (static_cast<int64_t>(max_len) + waves * kTileTokens - 1) / (waves * kTileTokens); };
    p.waves = few && p.items * units_of(4) > kOneRound ? big_waves(L.head_dim, copies_of(L.bits, group)) : 4;
    const int64_t units = units_of(p.waves);
    const auto at_most = [&](int64_t groups) {          // units of a part, for that many workgroups in all
        const int64_t parts = std::max<int64_t>(1, groups / std::max<int64_t>(p.items, 1));
        return (units + parts - 1) / parts;
    };
    int64_t per = few ? at_most(kCus) : std::max<int64_t>(at_most(12 * kCus), 4);
    if (!few && p.items * ((units + per - 1) / per) < 3 * kCus) per = std::min(per, at_most(3 * kCus));
    // Joining is one workgroup's work: more than 32 parts only of four rounds each.
    per = std::max(per, std::min<int64_t>((units + 31) / 32, 4));
    if (p.items > kCounters) per = units;
    p.chunk = static_cast<int>(per * p.waves * kTileTokens);
    p.splits = static_cast<int>((units + per - 1) / per);
    p.ws_bytes = workspace_of(L, group, p.splits > 1 ? p.items * p.splits : 0);
    return p;
}

// The workspace of a program's largest call, enough for every smaller one: the
// parts that plan_decode makes, at most, for up to these items and tokens.  (Its
// own count falls where a longer cache or a larger batch gives rounder parts.)
// at_most(g) leaves no more than g workgroups in all, a part has a unit or more,
// and four of them where there are many items and no part was made smaller for
// want of 3 * kCus workgroups.
size_t most_workspace(const grinqh_kv_layout& L, int n_q_heads, int batch, int max_len) {
    const DecodePlan p = plan_decode(L, n_q_heads, batch, max_len);
    const int64_t units = (static_cast<int64_t>(max_len) + 4 * kTileTokens - 1) / (4 * kTileTokens);
    int64_t parts = 0;                                   // one unit is one part, which stores nothing
    if (units > 1)
        parts = p.items <= kFewItems ? std::min<int64_t>(kCus, p.items * units)
                                     : std::max(std::min<int64_t>(12 * kCus, p.items * ((units + 3) / 4)),
                                                std::min<int64_t>(3 * kCus, p.items * units));
    return workspace_of(L, n_q_heads / L.n_kv_heads, parts);
}

template <int D, int BITS, int COPIES>
grinqh_status launch_queries(const DecodeArgs& a, int waves, unsigned n, hipStream_t stream) {
    const int here = a.group < kHeadTile ? a.group : kHeadTile;
    const auto launch = [&](auto kernel, int w) {
        const size_t lds = static_cast<size_t>(w) * std::max<size_t>(here * (D + 4 + 2) * sizeof(float), kWave * sizeof(f32x4));
        return launch_kernel(kernel, dim3(n), w * kWave, lds, stream, a);
    };
    if (waves > 4) {
        constexpr int W1 = big_waves(D, COPIES, 1), W2 = big_waves(D, COPIES, 2);
        return a.q_dtype == GRINQH_BF16 ? launch(decode_kernel<D, BITS, 1, W1, COPIES>, W1) : launch(decode_kernel<D, BITS, 2, W2, COPIES>, W2);
    }
    return a.q_dtype == GRINQH_BF16 ? launch(decode_kernel<D, BITS, 1, 4, COPIES>, 4) : launch(decode_kernel<D, BITS, 2, 4, COPIES>, 4);
}

template <int D, int BITS>
grinqh_status launch_copies(const DecodeArgs& a, int waves, unsigned n, hipStream_t stream) {
    if constexpr (BITS == 4)
        if (copies_of(BITS, a.group) == 2) return launch_queries<D, BITS, 2>(a, waves, n, stream);
    return launch_queries<D, BITS, 1>(a, waves, n, stream);
}

template <int D>
grinqh_status launch_bits(const DecodeArgs& a, int bits, int waves, unsigned n, hipStream_t stream) {
    if (bits == 4) return launch_copies<D, 4>(a, waves, n, stream);
    if (bits == 8) return launch_copies<D, 8>(a, waves, n, stream);
    return launch_copies<D, 16>(a, waves, n, stream);
}

bool valid_heads(const grinqh_kv_layout* L, int n_q_heads, int batch, int max_len) {
    return valid_kv_layout(L) && n_q_heads >= 1 && n_q_heads <= kMaxQHeads && n_q_heads % L->n_kv_heads == 0 &&
           batch >= 0 && batch <= kMaxBatch && max_len >= 1 && max_len <= kMaxCacheLen;
}

}  // namespace
}  // namespace grinqh

using namespace grinqh;

extern "C" {

size_t grinqh_attention_workspace_bytes(const grinqh_kv_layout* L, int32_t n_q_heads, int32_t batch,
                                        int32_t max_len) {
    return valid_heads(L, n_q_heads, batch, max_len) ? most_workspace(*L, n_q_heads, batch, max_len) : 0;
}

grinqh_status grinqh_decode_attention(const grinqh_kv_layout* L, const grinqh_kv_pools* pools, const void* q,
                                      grinqh_dtype q_dtype, int64_t q_stride, int32_t n_q_heads,
                                      const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                      const int32_t* seq_lens, int32_t batch, int32_t max_len, float scale,
                                      void* out, grinqh_dtype out_dtype, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    const grinqh_status st = check_kv_pools(L, pools);
    if (st != GRINQH_OK) return st;
    if (!valid_heads(L, n_q_heads, batch, max_len) || !(fabsf(scale) <= kMaxScale)) return GRINQH_EINVAL;
    if ((q_dtype != GRINQH_BF16 && q_dtype != GRINQH_F32) || (out_dtype != GRINQH_BF16 && out_dtype != GRINQH_F32))
        return GRINQH_EINVAL;
    if (batch == 0) return GRINQH_OK;
    if (q == nullptr || page_table == nullptr || seq_lens == nullptr || out == nullptr || workspace == nullptr)
        return GRINQH_EINVAL;
    const int64_t width = static_cast<int64_t>(n_q_heads) * L->head_dim;
    if (q_stride < width || q_stride > kMaxStride || max_pages < 1 || table_stride < max_pages ||
        table_stride > kMaxStride)
        return GRINQH_EINVAL;
    const int64_t qb = q_dtype == GRINQH_BF16 ? 2 : 4, ob = out_dtype == GRINQH_BF16 ? 2 : 4;
    if (!aligned_to(q, 16) || q_stride * qb % 16 != 0 || !aligned_to(page_table, 4) || !aligned_to(seq_lens, 4) ||
        !aligned_to(out, 16) || !aligned_to(lse, 4) || !aligned_to(workspace, 256))
        return GRINQH_EALIGN;
    const DecodePlan plan = plan_decode(*L, n_q_heads, batch, max_len);
    if (workspace_bytes < plan.ws_bytes) return GRINQH_ENOSPACE;
    if (plan.items * plan.splits > kMaxDecodeGroups) return GRINQH_EINVAL;
    const size_t code_bytes = grinqh_kv_code_bytes(L), grid_bytes = grinqh_kv_grid_bytes(L);
    if (written_overlaps({{out, static_cast<size_t>(batch * width * ob)},
                          {lse, lse == nullptr ? 0 : static_cast<size_t>(batch) * n_q_heads * sizeof(float)},
                          {workspace, plan.ws_bytes}},
                         {{q, static_cast<size_t>(((batch - 1) * q_stride + width) * qb)},
                          {page_table, static_cast<size_t>((batch - 1) * table_stride + max_pages) * sizeof(int32_t)},
                          {seq_lens, static_cast<size_t>(batch) * sizeof(int32_t)},
                          {pools->k_codes, code_bytes}, {pools->v_codes, code_bytes},
                          {pools->k_grid, grid_bytes}, {pools->v_grid, grid_bytes}}))
        return GRINQH_EINVAL;
    const int64_t reach = static_cast<int64_t>(max_pages) * L->page_size;
    DecodeArgs a;
    a.d = kv_dims(*L);
    a.k_codes = pools->k_codes;
    a.v_codes = pools->v_codes;
    a.k_grid = pools->k_grid;
    a.v_grid = pools->v_grid;
    a.q = q;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.out = out;
    a.lse = lse;
    a.counters = static_cast<unsigned*>(workspace);
    a.parts = reinterpret_cast<float*>(a.counters + kCounters);
    a.q_stride = q_stride;
    a.table_stride = table_stride;
    a.n_q_heads = n_q_heads;
    a.group = n_q_heads / L->n_kv_heads;
    a.head_tiles = plan.head_tiles;
    a.items = static_cast<int>(plan.items);
    a.splits = plan.splits;
    a.max_pages = max_pages;
    a.chunk = plan.chunk;
    a.longest = static_cast<int>(reach < max_len ? reach : max_len);
    a.q_dtype = q_dtype;
    a.out_dtype = out_dtype;
    a.scale_log2 = scale * kLog2e;
    const unsigned n = static_cast<unsigned>(plan.items * plan.splits);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (L->head_dim == 64) return launch_bits<64>(a, L->bits, plan.waves, n, s);
    if (L->head_dim == 128) return launch_bits<128>(a, L->bits, plan.waves, n, s);
    return launch_bits<256>(a, L->bits, plan.waves, n, s);
}

}  // extern "C"
