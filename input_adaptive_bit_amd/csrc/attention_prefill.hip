// Attention over whole prompts, packed behind one another, with grouped heads.
//
// For query i of a sequence with n queries and m keys, and key-value head
// g = h / group,
//   o = sum_j p_j v_j,  p_j = exp(a_j - max) / sum,  a_j = scale * q . k_j,
// over the keys j <= i + m - n (all keys where not causal).
//
// One pass over the keys with a running maximum and sum.  The rows of a
// key-value head are its (query, head of the group) pairs, query by query, so a
// tile of rows spans few queries: short prompts fill tiles, and little of a
// causal tile is masked.  A workgroup of four waves takes 128 rows, 32 to a
// wave; tiles of keys and values go through LDS for all of them, the next
// tile's loads under way while this one is used.
//
// Scores.  S^T = K Q^T (32 keys x 32 rows, v_mfma_f32_32x32x16_bf16): a lane
// holds 16 of a row's 32 scores, the lane 32 further the others, so maximum and
// sum need one exchange between the two.  The exponent is one fused
// multiply-add, exp2(s c - max c) with c = scale log2 e; the rounding of max c
// multiplies all of a row's weights alike.  Past kFar it would not be small
// any more (past 2^30 it alone makes weights 0 or infinite): the tiles of such
// rows are used outside the inner loop, with (s - max) c.  At 8192 tokens, 32
// heads of 128, the test for them takes 533 us from 530 (one card, in a captured
// graph); with every row so, 2830.
//
// Values.  O^T = V^T P^T.  The scores a lane holds are its share of the
// contraction as they are (the contraction's order is free), rounded to bf16
// in place; V^T comes from LDS with transposing reads (ds_read_b64_tr_b16).
//
// The maximum is the first tile's until a score exceeds it by 30 (as powers of
// two): weights up to 2^30 lose nothing in fp32 and bf16, and the sums are
// hardly ever rescaled.
//
// What bounds it.  Matrix and vector instructions together: at 8192 tokens, 32
// heads of 128 (525 - 547 us in a program, by the card, 1005 - 1047 TFLOP/s; 550 - 602
// under the kernel trace), the matrix cores are busy for 51% of the cycles and the
// vector units for 52%, 41% of the matrix cycles with vector work beside them, at
// 1.8 - 1.9 GHz; LDS reads take 26% and have no bank conflicts.  A wave's own
// overlap (the halves of a tile) took it from 594 us; 64 rows to a wave would
// halve the LDS reads but leave one wave per SIMD.  Heads of
// 64 have half the matrix work for the same exponentials: 720 TFLOP/s at 4096
// tokens, the vector units busy for 60% of the cycles, the matrix cores for 32%.
// Short prompts: a workgroup takes 2 us to find its rows, 3 to its first tile,
// 1.2 a tile (two to a CU: 1.6) and 2 for its output.
#include <math.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "kv_common.hpp"

namespace grinqh {
namespace {

typedef grinqh_prefill_attention_args Args;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kPreWaves = 4;
constexpr int kPreThreads = kPreWaves * kWave;
constexpr int64_t kMaxPreGroups = 1 << 23;              // workgroups of a launch
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 30.f;                          // log2 by which scores may exceed the maximum in use
// Largest |max c| that is rounded: half a step there, 2^-9, changes weights by
// 2^-9 ln 2, so that sums of different maxima (before and after a rescaling, of
// two parts) fit together to less than the weights' own rounding to bf16, 2^-8.
constexpr float kFar = 65536.f;

template <int D>
struct PreShape {
    static constexpr int kRows = kPreWaves * 32;        // rows of a workgroup
    static constexpr int kTK = 64;                      // keys of a tile
    static constexpr int kChunks = D / 8;               // 16-byte chunks of a key
    static constexpr int kBytes = kTK * D * 2;          // of a tile of keys (or values)
};

typedef int i32x4 __attribute__((ext_vector_type(4)));

// 16 bytes per lane from a buffer straight into LDS, lane after lane from
// `lds` + AT (uniform).  Written out because the compiler, not knowing which tile
// an LDS read is from, would wait for every such load before it; the kernel waits
// for all of them itself, before the barrier that hands a tile over.
template <int AT>
__device__ __forceinline__ void load_to_lds(i32x4 rsrc, uint32_t off, uint32_t lds) {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 1\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(rsrc), "i"(AT)
                 : "memory", "m0", "scc");
}

// A tile lies in LDS as rows of 2 D bytes, chunk c (16 bytes) of row r at
// c ^ swizzle(r): the 16 rows that one step of a key operand's read touches fall
// on different banks, and so do the 4 rows x 4 chunks of a value operand's.
template <int D, bool VALUES>
__device__ __forceinline__ constexpr int swizzle(int r) {
    if (VALUES) return D == 64 ? (r & 2) << 1 : (r & 3) << 2;
    return D == 64 ? (r & 7) ^ (r >> 3 & 1) : r & 15;
}

// Loads a tile into LDS in the order of LDS.  The lane's
// chunk changes from one load to the next where they are 8 rows apart (keys of
// head_dim 256).
template <int D, bool VALUES>
struct TileLoad {
    static constexpr int kRowsAtOnce = kPreThreads / PreShape<D>::kChunks, kOffsets = kRowsAtOnce < 16 && !VALUES ? 2 : 1;
    uint32_t off[kOffsets];
    __device__ __forceinline__ TileLoad(int64_t stride) {
        const int r = threadIdx.x / PreShape<D>::kChunks, slot = threadIdx.x % PreShape<D>::kChunks;
#pragma unroll
        for (int x = 0; x < kOffsets; ++x)
            off[x] = r * static_cast<uint32_t>(stride) * 2 + (slot ^ swizzle<D, VALUES>(r + x * kRowsAtOnce)) * 16;
    }
    // A tile at `from`; what lies `bytes` behind it and further reads as zeros.
    __device__ __forceinline__ void operator()(uint64_t from, uint32_t bytes, uint32_t stride_bytes, uint32_t lds) const {
        const i32x4 rs{static_cast<int>(from), static_cast<int>(from >> 32) & 0xFFFF, static_cast<int>(bytes), 0x00020000};
        uint32_t at[kOffsets];
#pragma unroll
        for (int x = 0; x < kOffsets; ++x) {
            at[x] = off[x] + x * kRowsAtOnce * stride_bytes;
            asm volatile("" : "+v"(at[x]));             // one register each, not one for every load of the loop
        }
        load<0>(rs, at, stride_bytes, lds);
    }
    template <int N>
    __device__ __forceinline__ void load(i32x4 rs, uint32_t (&at)[kOffsets], uint32_t stride_bytes, uint32_t lds) const {
        if constexpr (N < PreShape<D>::kTK / kRowsAtOnce) {
            load_to_lds<N * kPreThreads * 16>(rs, at[N % kOffsets], lds);
            at[N % kOffsets] += kOffsets * kRowsAtOnce * stride_bytes;
            load<N + 1>(rs, at, stride_bytes, lds);
        }
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

__device__ __forceinline__ void store_four(const Args& a, int64_t at, float y0, float y1, float y2, float y3) {
    if (a.out_dtype == GRINQH_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(y0, y1, y2, y3);
    else
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) = u32x2{pack_bf16(y0, y1), pack_bf16(y2, y3)};
}

// Of weights 2^(s c - round(max c)), so with the same product; past kFar of
// 2^((s - max) c), and the score itself may be close to the largest float.
__device__ __forceinline__ float lse_of(float top, float sum, float c, float scale) {
    if (sum == 0.f) return -INFINITY;
    const float log_sum = __builtin_amdgcn_logf(sum);
    return fabsf(top * c) > kFar ? __builtin_fmaf(top, fabsf(scale), kLn2 * log_sum) : kLn2 * (top * c + log_sum);
}

// Where the workspace holds a part: its rows' sums, then their (maximum, weight).
template <int D>
__device__ __forceinline__ int64_t part_at(int number, int head, int part, int heads, int most_parts) {
    return ((static_cast<int64_t>(number) * heads + head) * most_parts + part) * PreShape<D>::kRows * (D + 2);
}

// x of this lane and of the lane 32 further.
__device__ __forceinline__ float max_halves(float x) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
__device__ __forceinline__ float sum_halves(float x) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// Where a flat tile number lies: its sequence, the tile in it, and how many
// tiles the sequence has; seq -1 past the last.  Up to 64 sequences are taken
// from the longest to the shortest, so that the launch ends on short ones; more
// are narrowed down by 64 runs of sequences at a time.
struct Place {
    int seq, tile, tiles;
};
__device__ __forceinline__ int tiles_of(const Args& a, int group, int rows, int seq) {
    const int q0 = min(max(a.cu_q[seq], 0), a.total_q), q1 = min(max(a.cu_q[seq + 1], 0), a.total_q);
    return static_cast<int>((static_cast<int64_t>(max(q1 - q0, 0)) * group + rows - 1) / rows);
}
__device__ __forceinline__ int sum_up_to(int x, int lane) {                    // over lanes 0 .. lane
#pragma unroll
    for (int k = 1; k < kWave; k <<= 1) {
        const int y = __shfl_up(x, k);
        if (lane >= k) x += y;
    }
    return x;
}
__device__ __forceinline__ Place find_tile(const Args& a, int group, int rows, int number, int lane) {
    int first = 0, count = a.batch, before = 0;
    while (count > kWave) {
        const int run = (count + kWave - 1) / kWave;
        const int r0 = min(first + lane * run, first + count), r1 = min(r0 + run, first + count);
        int tiles = 0;
        for (int seq = r0; seq < r1; ++seq) tiles += tiles_of(a, group, rows, seq);
        const int sum = sum_up_to(tiles, lane);
        const uint64_t over = __ballot(before + sum > number);
        if (over == 0) return Place{-1, -1, 0};
        const int at = __builtin_ctzll(over);
        before += __builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(tiles, at);
        count = __builtin_amdgcn_readlane(r1 - r0, at);
        first = __builtin_amdgcn_readlane(r0, at);
    }
    int seq = first + lane, tiles = lane < count ? tiles_of(a, group, rows, seq) : 0;
    if (a.batch > 1 && a.batch <= kWave) {
        int rank = 0;
        for (int b = 0; b < a.batch; ++b) {
            const int other = __builtin_amdgcn_readlane(tiles, b);
            rank += other > tiles || (other == tiles && b < lane);
        }
        // lane -> lane of its rank (lanes past the last sequence keep their place)
        const int to = 4 * (lane < a.batch ? rank : lane);
        tiles = __builtin_amdgcn_ds_permute(to, tiles);
        seq = __builtin_amdgcn_ds_permute(to, seq);
    }
    const int sum = sum_up_to(tiles, lane);
    const uint64_t over = __ballot(before + sum > number);
    if (over == 0) return Place{-1, -1, 0};
    const int at = __builtin_ctzll(over);
    const int upto = __shfl(sum, at), mine = __shfl(tiles, at);
    return Place{__shfl(seq, at), number - (before + upto - mine), mine};
}

// How a call is cut up (host arithmetic on its sizes alone).
struct PrePlan {
    int64_t tiles;          // row tiles of a key-value head, at most
    int parts;              // parts of a tile's keys, at most
    size_t ws_bytes;
};

// Parts of a tile that sees `keys` keys: whole tiles of at least kMinPart keys.
constexpr int kMinPart = 256, kMaxParts = 32, kCus = 256;
__device__ __forceinline__ int parts_of(int keys, int most) { return max(1, min(most, keys / kMinPart)); }

template <int D>
__global__ __launch_bounds__(kPreThreads, D == 256 ? 1 : D == 64 ? 3 : 2) void prefill_attention_kernel(Args a, float c, int most_parts) {
    using S = PreShape<D>;
    constexpr int TK = S::kTK, KK = D / 16, DT = D / 32;
    __shared__ __attribute__((aligned(1024))) char lds[2][2][S::kBytes];       // [buffer][keys, values]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = a.n_q_heads / a.n_kv_heads;
    // Heads are the fast index, so that with eight of them each XCD's L2 keeps one head's keys.
    const int head = blockIdx.x % a.n_kv_heads;
    const int flat = blockIdx.x / a.n_kv_heads;             // and parts within a tile the next
    // Short tiles have few parts.  The first part's place among a tile's moves on
    // from tile to tile: otherwise, with a power of two of parts, some XCDs or
    // shader engines would get all first parts and others all that are not there
    // (1024 tokens, 32 heads of 128 in four parts: 41 us, 34 so).
    const int number = flat / most_parts, part = (flat + number) % most_parts;
    const Place at = find_tile(a, group, S::kRows, number, lane);
    if (at.seq < 0 || at.tile < 0 || at.tile >= at.tiles) return;   // (a tile outside: ends that do not ascend)
    const int seq = __builtin_amdgcn_readfirstlane(at.seq);
    // The last tiles of a causal sequence see the most keys and go first.
    const int tile = __builtin_amdgcn_readfirstlane(a.causal ? at.tiles - 1 - at.tile : at.tile);
    const int q_begin = min(max(a.cu_q[seq], 0), a.total_q), q_end = min(max(a.cu_q[seq + 1], 0), a.total_q);
    const int k_begin = min(max(a.cu_k[seq], 0), a.total_k);
    const int n = q_end - q_begin, m = max(min(max(a.cu_k[seq + 1], 0), a.total_k) - k_begin, 0);

    // Rows: first query and head of the tile, then this lane's.
    const int64_t row0 = static_cast<int64_t>(tile) * S::kRows;
    const int i0 = static_cast<int>(row0 / group), rem0 = static_cast<int>(row0 % group);
    const auto query_of = [&](int local) { return i0 + (rem0 + local) / group; };
    const auto seen_by = [&](int i) { return a.causal ? min(max(i + m - n + 1, 0), m) : m; };   // keys 0 .. that - 1
    const int local0 = wave * 32;
    const int all_end = seen_by(min(query_of(S::kRows - 1), n - 1));           // keys any row of the workgroup sees
    const int wave_end = seen_by(min(query_of(local0 + 31), n - 1));  // any row of the wave
    const int wave_full = seen_by(query_of(local0));                           // all rows of the wave
    const bool idle = query_of(local0) >= n;                                   // no row of the wave exists

    // This workgroup's part of the tile's keys, in whole tiles of keys.
    const int parts = parts_of(all_end, most_parts);
    if (part >= parts) return;
    const int all_tiles = (all_end + TK - 1) / TK;
    const int first = part * all_tiles / parts, tiles = (part + 1) * all_tiles / parts;

    // This lane's row.
    const int local = local0 + (lane & 31), i = query_of(local), h = head * group + (rem0 + local) % group;
    const bool there = i < n;
    const int seen = there ? seen_by(i) : 0;
    const int64_t out_row = there ? static_cast<int64_t>(q_begin + i) * a.n_q_heads + h : -1;
    bf16x8 qf[KK];
    {
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + (q_begin + (there ? i : 0)) * a.q_stride + (there ? h : 0) * D;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            u32x4 x = *reinterpret_cast<const u32x4*>(q + 16 * kk + 8 * (lane >> 5));
            if (a.scale < 0.f) x ^= 0x80008000u;                               // c is |scale| log2 e
            if (a.scale == 0.f) x = u32x4{0u, 0u, 0u, 0u};
            qf[kk] = __builtin_bit_cast(bf16x8, x);
        }
    }

    f32x16 o[DT];
    float top = -INFINITY, l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] = 0.f;

    const uint16_t* keys = static_cast<const uint16_t*>(a.k) + k_begin * a.k_stride + head * D;
    const uint16_t* values = static_cast<const uint16_t*>(a.v) + k_begin * a.v_stride + head * D;
    const TileLoad<D, false> load_keys(a.k_stride);
    const TileLoad<D, true> load_values(a.v_stride);
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)&lds[0][0][0]));
    // The next tile to load: where it is, and the bytes that exist of it.
    const uint32_t k_bytes = static_cast<uint32_t>(a.k_stride) * 2, v_bytes = static_cast<uint32_t>(a.v_stride) * 2;
    const int last = (m - 1) / TK, last_rows = (m - 1) % TK;
    const uint32_t k_last = last_rows * k_bytes + 2 * D, v_last = last_rows * v_bytes + 2 * D;
    uint64_t k_next = reinterpret_cast<uint64_t>(keys + static_cast<int64_t>(first * TK) * a.k_stride);
    uint64_t v_next = reinterpret_cast<uint64_t>(values + static_cast<int64_t>(first * TK) * a.v_stride);
    const uint32_t lds_wave = lds0 + wave * kWave * 16;
    const auto load = [&](int t) {
        const uint32_t at = lds_wave + (t & 1) * 2 * S::kBytes;
        load_keys(k_next, t == last ? k_last : (TK - 1) * k_bytes + 2 * D, k_bytes, at);
        load_values(v_next, t == last ? v_last : (TK - 1) * v_bytes + 2 * D, v_bytes, at + S::kBytes);
        k_next += static_cast<uint64_t>(TK) * k_bytes;
        v_next += static_cast<uint64_t>(TK) * v_bytes;
    };
    // Operand reads: this lane's place in a tile; steps and dimension tiles only
    // flip bits of the chunk.
    const uint32_t k_at = (lane & 31) * D * 2 + (((lane >> 5) ^ swizzle<D, false>(lane & 31)) * 16);
    uint32_t v_at;
    {
        const int x = lane & 15, r = 4 * (lane >> 5) + (x >> 2);
        v_at = r * D * 2 + (((2 * ((lane >> 4) & 1) + ((x & 3) >> 1)) ^ swizzle<D, true>(r)) * 16) + (x & 1) * 8;
    }
    const auto key_frag = [&](uint32_t kb, int half, int kk) {                 // 32 keys of a half, 16 dimensions
        return *reinterpret_cast<const bf16x8 __attribute__((address_space(3)))*>((kb ^ (kk * 32)) + half * 32 * D * 2);
    };
    const auto value_frag = [&](uint32_t vb, int step, int d) {                // 16 keys from 16 step, 32 dimensions
        const uint32_t at = (vb ^ (d * 64)) + step * 16 * D * 2;
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 8 * D * 2));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    const auto mma = [](bf16x8 x, bf16x8 y, f32x16 z) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, z, 0, 0, 0); };
    const auto zero = [] {
        f32x16 z;
#pragma unroll
        for (int r = 0; r < 16; ++r) z[r] = 0.f;
        return z;
    };
    const auto top_of = [](const f32x16& s) {
        float x = s[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) x = fmaxf(x, s[r]);
        return max_halves(x);
    };
    const auto mask = [&](f32x16& s, int key0) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = key0 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4 < seen ? s[r] : -INFINITY;
    };
    // Weights of the score pair e (0 .. 7) of a half, into its operands.
    const auto weigh = [&](const f32x16& s, int e, float mc, u32x4 (&p)[2], float& sum) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * e], c, -mc));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * e + 1], c, -mc));
        sum += p0;
        sum += p1;
        uint32_t w = pack_bf16(p0, p1);
        asm volatile("" : "+v"(w));                     // here, between the products, not where it is used
        p[e / 4][e % 4] = w;
    };

    if (first < tiles) load(first);
    __builtin_amdgcn_s_waitcnt(0);                      // the queries too: nothing but tiles is waited for below
    // The inner loop never touches the output sums but to add to them.  A row whose
    // scores pass its maximum by too much leaves it and comes back to the same
    // tile with the new maximum; a tile with values that are not finite where some
    // row does not see them, or with a row whose maximum is far from zero, is used
    // outside.
    float mx = 0.f;
    bool again = false;
    for (int t = first;;) {
      bool passed = false, odd = false;
      for (; t < tiles; ++t) {
        const int t0 = t * TK;
        if (!again) {
            __builtin_amdgcn_s_waitcnt(0);              // this wave's share of the tile has arrived
            __syncthreads();                            // everyone's has; and the other buffer is free
            if (t + 1 < tiles) load(t + 1);
        }
        again = false;
        const uint32_t kb = lds0 + (t & 1) * 2 * S::kBytes + k_at, vb = lds0 + (2 * (t & 1) + 1) * S::kBytes + v_at;
        if (idle || t0 >= wave_end) continue;           // no row here sees any of it
        // The second half's scores are formed between the first's weights, the
        // first's values added between the second's.
        const bool masked = t0 + TK > wave_full;        // some row sees a part of the tile
        f32x16 s0 = zero(), s1 = zero();
        u32x4 p0[2], p1[2];
        float sum = 0.f;
        bf16x8 kf[3], vf[2][DT];
        kf[0] = key_frag(kb, 0, 0);
        kf[1] = key_frag(kb, 0, 1);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            kf[(kk + 2) % 3] = kk + 2 < KK ? key_frag(kb, 0, kk + 2) : key_frag(kb, 1, kk + 2 - KK);
            s0 = mma(kf[kk % 3], qf[kk], s0);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (masked) mask(s0, t0);
        mx = top_of(s0);
        top = top == -INFINITY ? mx : top;              // nothing summed yet
        const float mc0 = top == -INFINITY ? 0.f : top * c;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            if (kk + 2 < KK) kf[(KK + kk + 2) % 3] = key_frag(kb, 1, kk + 2);
            if (kk >= KK - DT) vf[0][kk - (KK - DT)] = value_frag(vb, 0, kk - (KK - DT));
            s1 = mma(kf[(KK + kk) % 3], qf[kk], s1);
#pragma unroll
            for (int e = 8 * kk / KK; e < 8 * (kk + 1) / KK; ++e) weigh(s0, e, mc0, p0, sum);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (masked) mask(s1, t0 + 32);
        const float mx1 = top_of(s1);
        top = top == -INFINITY ? mx1 : top;
        const float mc1 = top == -INFINITY ? 0.f : top * c;
        mx = fmaxf(mx, mx1);
        passed = __any((mx - top) * c > kSlack);        // (no if both are infinite: NaN)
        odd = __any(fabsf(mc1) > kFar);
        if (masked) {                                   // a value that is not finite where some row does not see it
            uint32_t high = 0;
#pragma unroll
            for (int st = 0; st < 4; ++st)
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const u32x4 w = __builtin_bit_cast(u32x4, value_frag(vb, st, d));
#pragma unroll
                    for (int x = 0; x < 4; ++x) high |= ((w[x] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                    __builtin_amdgcn_sched_barrier(0);
                }
            odd |= __any(high != 0);
        }
        if (passed || odd) break;
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                vf[(st + 1) & 1][d] = value_frag(vb, st + 1, d);
                o[d] = mma(vf[st & 1][d], __builtin_bit_cast(bf16x8, p0[st]), o[d]);
                const int x = st * DT + d;
#pragma unroll
                for (int e = 4 * x / DT; e < 4 * (x + 1) / DT; ++e) weigh(s1, e, mc1, p1, sum);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
        for (int st = 2; st < 4; ++st)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                if (st == 2) vf[1][d] = value_frag(vb, 3, d);
                o[d] = mma(vf[st & 1][d], __builtin_bit_cast(bf16x8, p1[st - 2]), o[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        l += sum;
      }
      if (!passed && !odd) break;
      if (passed) {
          const float m_new = (mx - top) * c > kSlack ? mx : top;
          const float keep = m_new == top ? 1.f : __builtin_amdgcn_exp2f((top - m_new) * c);
          top = m_new;
          l *= keep;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int r = 0; r < 16; ++r) o[d][r] *= keep;
          again = true;
      } else {
          const int t0 = t * TK;
          const uint32_t kb = lds0 + (t & 1) * 2 * S::kBytes + k_at, vb = lds0 + (2 * (t & 1) + 1) * S::kBytes + v_at;
          f32x16 s0 = zero(), s1 = zero();
          u32x4 p0[2], p1[2];
          float sum = 0.f;
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) {
              s0 = mma(key_frag(kb, 0, kk), qf[kk], s0);
              s1 = mma(key_frag(kb, 1, kk), qf[kk], s1);
              __builtin_amdgcn_sched_barrier(0);
          }
          mask(s0, t0);
          mask(s1, t0 + 32);
          float mc = top == -INFINITY ? 0.f : top * c, shift = 0.f;
          if (fabsf(mc) > kFar) {
              shift = top;
              mc = 0.f;
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) {
              s0[r] -= shift;
              s1[r] -= shift;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) weigh(s0, e, mc, p0, sum);
          // The product would carry 0 * Inf into rows that do not see the
          // value.  The finite values go the same way; what is not finite is
          // counted, up and down (NaN both ways), over the seen keys.
#pragma unroll
          for (int e = 0; e < 8; ++e) weigh(s1, e, mc, p1, sum);
          const u32x4 p[4] = {p0[0], p0[1], p1[0], p1[1]};
#pragma unroll
          for (int d = 0; d < DT; ++d) {
              f32x16 up = zero(), down = zero();
#pragma unroll
              for (int st = 0; st < 4; ++st) {
                  const u32x4 w = __builtin_bit_cast(u32x4, value_frag(vb, st, d));
                  u32x4 fin, pos, neg, one;
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                      fin[x] = pos[x] = neg[x] = 0;
#pragma unroll
                      for (int y = 0; y < 32; y += 16) {
                          const uint32_t v = (w[x] >> y) & 0xFFFFu;
                          const bool bad = (v & 0x7F80u) == 0x7F80u, nan = bad && (v & 0x7Fu) != 0;
                          fin[x] |= (bad ? 0u : v) << y;
                          pos[x] |= (bad && (nan || v < 0x8000u) ? 0x3F80u : 0u) << y;
                          neg[x] |= (bad && (nan || v >= 0x8000u) ? 0x3F80u : 0u) << y;
                      }
                      const int key = t0 + 16 * st + 8 * (x / 2) + 4 * (lane >> 5) + 2 * (x % 2);
                      one[x] = (key < seen ? 0x3F80u : 0u) | (key + 1 < seen ? 0x3F800000u : 0u);
                  }
                  o[d] = mma(__builtin_bit_cast(bf16x8, fin), __builtin_bit_cast(bf16x8, p[st]), o[d]);
                  up = mma(__builtin_bit_cast(bf16x8, pos), __builtin_bit_cast(bf16x8, one), up);
                  down = mma(__builtin_bit_cast(bf16x8, neg), __builtin_bit_cast(bf16x8, one), down);
                  __builtin_amdgcn_sched_barrier(0);
              }
#pragma unroll
              for (int r = 0; r < 16; ++r) o[d][r] += (up[r] > 0.f ? INFINITY : 0.f) + (down[r] > 0.f ? -INFINITY : 0.f);
          }
          l += sum;
          ++t;
          again = false;
      }
    }

    const float sum = sum_halves(l);
    if (parts > 1) {        // sums, maximum and weight for join_kernel
        float* to = static_cast<float*>(a.workspace) + part_at<D>(number, head, part, a.n_kv_heads, most_parts);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<float4*>(to + local * D + 32 * d + 8 * x + 4 * (lane >> 5)) =
                    make_float4(o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]);
        if (lane < 32) *reinterpret_cast<float2*>(to + S::kRows * D + 2 * local) = make_float2(top, sum);
        return;
    }
    if (out_row < 0) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
        const auto y = [&](int r) { return o[d][r] * inv; };
        if (a.out_dtype == GRINQH_F32) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + out_row * D + 32 * d + 8 * x + 4 * (lane >> 5)) =
                    make_float4(y(4 * x), y(4 * x + 1), y(4 * x + 2), y(4 * x + 3));
            continue;
        }
        // Two lanes hold a row: they swap quads, so that each has 8 neighbours of it
        // and 16 bytes to store (six prompts of 33 .. 1200 tokens: 50 us with 8, 46 so).
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const u32x2 z = __builtin_amdgcn_permlane32_swap(pack_bf16(y(4 * x + 2 * e), y(4 * x + 2 * e + 1)),
                                                                 pack_bf16(y(4 * x + 4 + 2 * e), y(4 * x + 5 + 2 * e)), false, false);
                w[e] = z.x;
                w[2 + e] = z.y;
            }
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + out_row * D + 32 * d + 8 * x + 8 * (lane >> 5)) = w;
        }
    }
    if (a.lse != nullptr && lane < 32) a.lse[out_row] = lse_of(top, sum, c, a.scale);
}

// Joins the parts of every tile that has several.  A workgroup takes
// kJoinRows rows of a tile; D / 4 lanes hold a row, four values each.
constexpr int kJoinRows = 32, kJoinBatch = 8;           // rows of a workgroup; parts asked for at a time

template <int D>
__global__ __launch_bounds__(kPreThreads) void join_kernel(Args a, float c, int most_parts) {
    using S = PreShape<D>;
    const int lane = threadIdx.x & 63, group = a.n_q_heads / a.n_kv_heads;
    const int head = blockIdx.x % a.n_kv_heads, number = blockIdx.x / a.n_kv_heads;
    const Place at = find_tile(a, group, S::kRows, number, lane);
    if (at.seq < 0 || at.tile < 0 || at.tile >= at.tiles) return;
    const int seq = at.seq, tile = a.causal ? at.tiles - 1 - at.tile : at.tile;
    const int q_begin = min(max(a.cu_q[seq], 0), a.total_q), q_end = min(max(a.cu_q[seq + 1], 0), a.total_q);
    const int k_begin = min(max(a.cu_k[seq], 0), a.total_k);
    const int n = q_end - q_begin, m = max(min(max(a.cu_k[seq + 1], 0), a.total_k) - k_begin, 0);
    const int64_t row0 = static_cast<int64_t>(tile) * S::kRows;
    const int i0 = static_cast<int>(row0 / group), rem0 = static_cast<int>(row0 % group);
    const int last = min(i0 + (rem0 + S::kRows - 1) / group, n - 1);
    const int parts = parts_of(a.causal ? min(max(last + m - n + 1, 0), m) : m, most_parts);
    if (parts == 1) return;
    const float* from = static_cast<const float*>(a.workspace) + part_at<D>(number, head, 0, a.n_kv_heads, most_parts);
    const int64_t step = part_at<D>(0, 0, 1, a.n_kv_heads, most_parts);
    constexpr int kPerRow = D / 4;
    for (int u = threadIdx.x; u < kJoinRows * kPerRow; u += kPreThreads) {
        const int local = blockIdx.y * kJoinRows + u / kPerRow, x = u % kPerRow * 4;
        const int i = i0 + (rem0 + local) / group, h = head * group + (rem0 + local) % group;
        if (i >= n) continue;
        // A batch of parts is asked for at once: 2 us less than one after the other.
        float top = -INFINITY, l = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = 0; p0 < parts; p0 += kJoinBatch) {
            float2 ml[kJoinBatch];
            float4 v[kJoinBatch];
#pragma unroll
            for (int p = 0; p < kJoinBatch; ++p) {
                ml[p] = make_float2(-INFINITY, 0.f);
                v[p] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p0 + p < parts) {
                    const float* part = from + (p0 + p) * step;
                    ml[p] = *reinterpret_cast<const float2*>(part + S::kRows * D + 2 * local);
                    v[p] = *reinterpret_cast<const float4*>(part + local * D + x);
                }
            }
            float next = top;
#pragma unroll
            for (int p = 0; p < kJoinBatch; ++p) next = fmaxf(next, ml[p].x);
            const float base = next == -INFINITY ? 0.f : next;
            const float keep = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((top - base) * c);
            top = next;
            l *= keep;
            y = make_float4(y.x * keep, y.y * keep, y.z * keep, y.w * keep);
#pragma unroll
            for (int p = 0; p < kJoinBatch; ++p) {
                if (p0 + p >= parts) continue;
                const float f = __builtin_amdgcn_exp2f((ml[p].x - base) * c);
                l = __builtin_fmaf(f, ml[p].y, l);
                y = make_float4(__builtin_fmaf(f, v[p].x, y.x), __builtin_fmaf(f, v[p].y, y.y), __builtin_fmaf(f, v[p].z, y.z),
                                __builtin_fmaf(f, v[p].w, y.w));
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t row = static_cast<int64_t>(q_begin + i) * a.n_q_heads + h;
        store_four(a, row * D + x, y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        if (a.lse != nullptr && x == 0) a.lse[row] = lse_of(top, l, c, a.scale);
    }
}

template <int D>
PrePlan plan_prefill(const Args& a) {
    PrePlan p;
    const int64_t group = a.n_q_heads / a.n_kv_heads;
    const int64_t rows = PreShape<D>::kRows, dense = (a.total_q * group + rows - 1) / rows;
    const int64_t some = std::min(a.batch, a.total_q);                         // sequences that have queries, at most
    p.tiles = a.total_q * group / rows + some;                                 // at most, whatever the lengths
    // Parts where they make the call shorter, by a model of what was measured. A
    // tile of keys takes a workgroup alone on its CU kTime us, two on one CU 1.35 and
    // three 1.8 times that (where there is room for them); a call takes as long as
    // its longest piece or as all pieces together; the parts cost a second launch
    // and their way through memory. Sequences are taken to be alike, and a tile's
    // keys to lie evenly between `least` and `most`. In us, the model's pick in
    // brackets: 512 queries after 7680 keys, 32 heads of 128, in 1, 2, 3, [4], 5, 8
    // parts: 158, 103, 103, 93, 108, 108; 4096 tokens, 4 heads of 128, 1, 2, [3], 4, 5,
    // 8: 81, 54, 47, 42, 48, 54; 1024 tokens, 32 heads of 128, [1], 2, 3: 28, 34, 34;
    // 1300 tokens, 6 heads of 256, 1, 2, 3, [4], 5: 51, 43, 39, 39, 40; 170 queries
    // after 12806 keys, 6 heads of 64, 1, 4, 8, 16, [25]: 184, 57, 35, 27, 27.
    constexpr int kFit = D == 64 ? 3 : D == 128 ? 2 : 1;
    constexpr double kTime = D == 64 ? 0.95 : D == 128 ? 1.2 : 2.1;            // us
    constexpr double kJoin = 4.0, kRate = D == 64 ? 3.5e6 : D == 128 ? 3.0e6 : 1.8e6;   // us, bytes per us
    constexpr double kTogether[4] = {0.0, 1.0, 1.35, 1.8};
    // Every sequence leaves half a tile, and has one.
    const int64_t groups = std::max(dense + (some - 1) / 2, some) * a.n_kv_heads;
    const double most = static_cast<double>(a.total_k) / std::max<int64_t>(1, some);
    const double least = a.causal ? std::max(0.0, most - static_cast<double>(a.total_q) / std::max<int64_t>(1, some)) : most;
    const auto share = [&](double keys) {               // of the tiles, with that many keys or more
        return keys <= least ? 1.0 : keys > most ? 0.0 : (most - keys) / (most - least);
    };
    const auto cost = [&](int parts, double pieces) {   // pieces of a tile on average
        const double per_cu = groups * pieces / kCus, full = std::min<double>(kFit, std::max(1.0, per_cu));
        const int64_t deep = static_cast<int64_t>(std::max(1.0, std::ceil(per_cu))), at = static_cast<int64_t>(full);
        const double all = (least + most) / 2 / pieces * (deep / kFit * kTogether[kFit] + kTogether[deep % kFit]);
        double longest = most / parts;
        if (parts > 1 && least < parts * kMinPart)      // a tile with keys for one part less
            longest = std::max(longest, static_cast<double>(parts * kMinPart) / (parts - 1));
        longest *= kTogether[at] + (at < kFit ? (full - at) * (kTogether[at + 1] - kTogether[at]) : 0.0);
        const double bytes = 2.0 * groups * (pieces - 1 + share(2 * kMinPart)) * rows * (D + 2) * sizeof(float);
        return kTime / PreShape<D>::kTK * std::max(all, longest) + (parts > 1 ? kJoin + bytes / kRate : 0.0);
    };
    p.parts = 1;
    if (groups < 3 * kCus) {
        double pieces = 1.0, best = cost(1, 1.0);
        for (int parts = 2; parts <= kMaxParts && parts * kMinPart <= most; ++parts) {
            pieces += share(parts * kMinPart);
            const double c = cost(parts, pieces);
            if (c < 0.97 * best) {
                best = c;
                p.parts = parts;
            }
        }
    }
    p.ws_bytes = p.parts > 1 ? static_cast<size_t>(p.tiles) * a.n_kv_heads * p.parts * PreShape<D>::kRows * (D + 2) * sizeof(float) : 0;
    return p;
}

template <int D>
size_t prefill_workspace(const Args& a) {
    return plan_prefill<D>(a).ws_bytes;
}

bool writes_what_it_reads(const Args& a, size_t ws_bytes) {
    const int64_t q_width = static_cast<int64_t>(a.n_q_heads) * a.head_dim, width = static_cast<int64_t>(a.n_kv_heads) * a.head_dim;
    const auto rows = [](int64_t n, int64_t stride, int64_t of) { return n > 0 ? static_cast<size_t>((n - 1) * stride + of) * 2 : 0; };
    const size_t ends = (static_cast<size_t>(a.batch) + 1) * sizeof(int32_t);
    const size_t out = static_cast<size_t>(a.total_q) * q_width * (a.out_dtype == GRINQH_BF16 ? 2 : 4);
    const size_t lse = a.lse == nullptr ? 0 : static_cast<size_t>(a.total_q) * a.n_q_heads * sizeof(float);
    return written_overlaps({{a.out, out}, {a.lse, lse}, {a.workspace, ws_bytes}},
                            {{a.q, rows(a.total_q, a.q_stride, q_width)}, {a.k, rows(a.total_k, a.k_stride, width)},
                             {a.v, rows(a.total_k, a.v_stride, width)}, {a.cu_q, ends}, {a.cu_k, ends}});
}

template <int D>
grinqh_status launch_prefill_attention(const Args& a, hipStream_t stream) {
    PrePlan p = plan_prefill<D>(a);
    if (p.tiles * a.n_kv_heads > kMaxPreGroups) return GRINQH_EINVAL;
    if (a.workspace == nullptr) p = PrePlan{p.tiles, 1, 0};
    if (a.workspace_bytes < p.ws_bytes) return GRINQH_ENOSPACE;
    if (writes_what_it_reads(a, p.ws_bytes)) return GRINQH_EINVAL;
    const float c = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
    const unsigned n = static_cast<unsigned>(p.tiles * a.n_kv_heads);
    const grinqh_status st = launch_kernel(prefill_attention_kernel<D>, dim3(n * p.parts), kPreThreads, 0, stream, a, c, p.parts);
    if (p.parts == 1 || st != GRINQH_OK) return st;
    return launch_kernel(join_kernel<D>, dim3(n, PreShape<D>::kRows / kJoinRows), kPreThreads, 0, stream, a, c, p.parts);
}

}  // namespace
}  // namespace grinqh

using namespace grinqh;

namespace {

// Sizes and types: what the workspace depends on.
grinqh_status check_sizes(const Args& a) {
    if (a.batch < 0 || a.batch > kMaxBatch || a.total_q < 0 || a.total_q > kMaxPacked || a.total_k < 0 ||
        a.total_k > kMaxPacked)
        return GRINQH_EINVAL;
    if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return GRINQH_EINVAL;
    if (a.n_kv_heads < 1 || a.n_kv_heads > kMaxKvHeads || a.n_q_heads < 1 || a.n_q_heads > kMaxQHeads ||
        a.n_q_heads % a.n_kv_heads != 0 || !(fabsf(a.scale) <= kMaxScale))
        return GRINQH_EINVAL;
    if (a.out_dtype != GRINQH_BF16 && a.out_dtype != GRINQH_F32) return GRINQH_EINVAL;
    return GRINQH_OK;
}

}  // namespace

extern "C" size_t grinqh_prefill_attention_workspace_bytes(const grinqh_prefill_attention_args* args) {
    if (args == nullptr || check_sizes(*args) != GRINQH_OK) return 0;
    if (args->head_dim == 64) return prefill_workspace<64>(*args);
    if (args->head_dim == 128) return prefill_workspace<128>(*args);
    return prefill_workspace<256>(*args);
}

extern "C" grinqh_status grinqh_prefill_attention(const grinqh_prefill_attention_args* args, void* stream) {
    if (args == nullptr) return GRINQH_EINVAL;
    const Args& a = *args;
    const grinqh_status st = check_sizes(a);
    if (st != GRINQH_OK) return st;
    if (a.batch == 0 || a.total_q == 0) return GRINQH_OK;
    if (a.q == nullptr || a.cu_q == nullptr || a.cu_k == nullptr || a.out == nullptr) return GRINQH_EINVAL;
    if (a.total_k > 0 && (a.k == nullptr || a.v == nullptr)) return GRINQH_EINVAL;
    const int64_t qw = static_cast<int64_t>(a.n_q_heads) * a.head_dim, kw = static_cast<int64_t>(a.n_kv_heads) * a.head_dim;
    if (a.q_stride < qw || a.k_stride < kw || a.v_stride < kw || a.q_stride > kMaxStride || a.k_stride > kMaxStride ||
        a.v_stride > kMaxStride)
        return GRINQH_EINVAL;
    if (!aligned_to(a.q, 16) || !aligned_to(a.k, 16) || !aligned_to(a.v, 16) || a.q_stride % 8 != 0 ||
        a.k_stride % 8 != 0 || a.v_stride % 8 != 0 || !aligned_to(a.cu_q, 4) || !aligned_to(a.cu_k, 4) ||
        !aligned_to(a.out, 16) || !aligned_to(a.lse, 4) || !aligned_to(a.workspace, 256))
        return GRINQH_EALIGN;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.head_dim == 64) return launch_prefill_attention<64>(a, s);
    if (a.head_dim == 128) return launch_prefill_attention<128>(a, s);
    return launch_prefill_attention<256>(a, s);
}
