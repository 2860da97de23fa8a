// Norms of queries and keys for each head, the rotation by position, and the
// cache's write, in one pass over the rows.
//
//   x <- x * weight / sqrt(mean(x^2) + eps)
//   (a, b) <- (a cos t - b sin t, b cos t + a sin t),  t = position * freq
//
// D / 8 neighbouring lanes hold a row, 8 values each (one 16-byte load of bf16,
// two of fp32): the mean comes from exchanges between them, the other half of a
// rotated pair from the lane that holds it, and a row of the cache is quantised
// from the same registers (kv_store.hpp).  Angles are the same for all heads of a
// token: a workgroup takes some tokens, or a part of the heads of one, and works
// its angles out once, one a thread, into LDS.
// An angle's turns are counted in fp64 and only the fraction of a turn is
// rounded to fp32 (at position 10^5 a 32-bit product would be off by 0.01
// radian); sine and cosine are of that fraction.
//
// Memory bounds it: 16381 tokens of 64 + 8 heads of 128 bf16, normed, into an 8-bit
// cache, 670 MB, take 129 us (5.2 TB/s, a large copy's rate), with 150 vector
// instructions for a row of queries.  At 230 (addresses in 64 bits, signs of sines
// by choice, copies around lane permutations) it was 145 us, with angles worked out
// by the lanes that use them, IEEE roots and divisions 194.
#include <algorithm>

#include "internal.h"
#include "kv_common.hpp"
#include "kv_store.hpp"

namespace grinqh {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kRopeThreads = 256;
constexpr int kMostAngles = 512;                   // of a workgroup: 4 to 16 tokens
constexpr int kMostGroups = 1 << 22;               // of a launch
constexpr int kFill = 2048;                        // workgroups that fill the card: eight to a CU

struct RopeArgs {
    KvDims d;
    const void* src[3];                            // queries, keys, values
    int64_t src_stride[3];
    void* dst[2];
    int64_t dst_stride[2];
    uint8_t* codes[2];
    uint16_t* grid[2];
    const int64_t* slots;
    const int32_t* positions;
    const double* freqs;
    const void* weight[2];
    int64_t n_tokens;
    int n_q, n_kv, rows;                           // rows: of a token
    int tokens, step_tokens, step_rows;            // of a workgroup; to a lane group's next row
    int rope_dim, neighbours, weight_dtype;
    float eps;
};

template <typename T>
struct RawRow {
    u32x4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void widen(const RawRow<T>& raw, float (&w)[kPerLane]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[2 * i] = __uint_as_float(raw.v[0][i] << 16);
            w[2 * i + 1] = __uint_as_float(raw.v[0][i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __uint_as_float(raw.v[i >> 2][i & 3]);
    }
}

// Rounds to T (a choice of the caller's: the type of queries and keys), and
// leaves in w what that stands for.
template <typename T>
__device__ __forceinline__ RawRow<T> narrow(float (&w)[kPerLane]) {
    RawRow<T> raw;
    if constexpr (sizeof(T) == 2) {
        typedef float two __attribute__((ext_vector_type(2)));
        typedef __bf16 two_bf16 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i)                            // one instruction, to nearest even
            raw.v[0][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((two{w[2 * i], w[2 * i + 1]}), two_bf16));
        widen<T>(raw, w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw.v[i >> 2][i & 3] = __float_as_uint(w[i]);
    }
    return raw;
}

template <typename T>
__device__ __forceinline__ RawRow<T> load_raw(const void* at) {
    RawRow<T> raw;
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) raw.v[i] = static_cast<const u32x4*>(at)[i];
    return raw;
}

// Turns of an angle and weights, as a lane of a row reads them: its 8 values' first
// four from one stretch and its last four from another, lane after lane.
__device__ __forceinline__ int in_halves(int i, int count) { return (i & 4 ? count / 2 : 0) + (i >> 3) * 4 + (i & 3); }
__device__ __forceinline__ void read_eight(const float* halves, int count, int lane, float (&v)[kPerLane]) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    const f32x4 a = reinterpret_cast<const f32x4*>(halves)[lane], b = reinterpret_cast<const f32x4*>(halves + count / 2)[lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}

// One of three values that are there already: a choice between what they are read
// from would become an address that differs between lanes.
template <typename V>
__device__ __forceinline__ V pick(bool first, bool second, V a, V b, V c) { return first ? a : second ? b : c; }

template <int D, typename T, int BITS>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    constexpr int kLanes = D / kPerLane, kItems = kRopeThreads / kLanes, kTokens = kMostAngles / (D / 2);
    // sines[1]: negative, for the lanes that hold a pair's first half
    __shared__ __attribute__((aligned(16))) float cosines[kMostAngles], sines[2][kMostAngles], weights[2][D];
    __shared__ int64_t slots[kTokens];
    const int lane = threadIdx.x % kLanes, pairs = a.rope_dim / 2;
    const int64_t token0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tokens), a.n_tokens - token0));
    // The group's rows: (t, r), every kItems gridDim.y-th of the workgroup's.
    const int rows = a.rows;
    int r = threadIdx.x / kLanes + kItems * blockIdx.y, t = r / rows;
    r -= t * rows;
    // Places within the workgroup's tokens: 16 strides of 2^24 floats fit 32 bits.
    struct Rows {
        char* at;
        uint32_t stride;
    };
    const auto rows_of = [&](const void* base, int64_t stride) {
        return Rows{static_cast<char*>(const_cast<void*>(base)) + token0 * stride * static_cast<int>(sizeof(T)), static_cast<uint32_t>(stride)};
    };
    const Rows q = rows_of(a.src[0], a.src_stride[0]), k = rows_of(a.src[1], a.src_stride[1]), v = rows_of(a.src[2], a.src_stride[2]);
    const Rows q_out = rows_of(a.dst[0], a.dst_stride[0]), k_out = rows_of(a.dst[1], a.dst_stride[1]);
    const auto place = [&](int t, int head, uint32_t stride) {
        return (static_cast<uint32_t>(t) * stride + static_cast<uint32_t>(head * D + lane * kPerLane)) * static_cast<uint32_t>(sizeof(T));
    };
    const int first_v = a.n_q + a.n_kv;
    const auto load = [&](int t, int r) {
        const bool is_q = r < a.n_q, is_v = r >= first_v;
        const char* at = pick(is_q, is_v, q.at, v.at, k.at);
        const uint32_t stride = pick(is_q, is_v, q.stride, v.stride, k.stride);
        return load_raw<T>(at + place(t, r - pick(is_q, is_v, 0, first_v, a.n_q), stride));
    };
    RawRow<T> next;
    if (t < tokens) next = load(t, r);                         // under way while the angles are worked out
    for (int i = threadIdx.x; i < tokens * pairs; i += kRopeThreads) {
        const int of = i / pairs, j = i - of * pairs;
        const double turns = a.positions[token0 + of] * a.freqs[j] * 0.15915494309189533577;          // 1 / (2 pi)
        float s, c;
        sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
        const int at = of * pairs + (a.neighbours ? j : in_halves(j, pairs));
        sines[0][at] = s;
        sines[1][at] = -s;
        cosines[at] = c;
    }
    if (threadIdx.x < D) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
            if (a.weight[w] != nullptr)
                weights[w][in_halves(threadIdx.x, D)] = a.weight_dtype == GRINQH_BF16
                    ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.weight[w])[threadIdx.x]) << 16)
                    : static_cast<const float*>(a.weight[w])[threadIdx.x];
    }
    if (BITS != 0 && threadIdx.x < tokens) slots[threadIdx.x] = a.slots[token0 + threadIdx.x];
    __syncthreads();

    // Where the other half of this lane's pairs is, and its sign.
    const int across = a.rope_dim / (2 * kPerLane);
    const bool turned = lane * kPerLane < a.rope_dim, second = lane >= across;
    const int partner_at = ((threadIdx.x & 63) + (!turned ? 0 : second ? -across : across)) * 4;
    while (t < tokens) {
        RawRow<T> raw = next;
        int next_t = t + a.step_tokens, next_r = r + a.step_rows;
        if (next_r >= rows) {
            next_r -= rows;
            ++next_t;
        }
        if (next_t < tokens) next = load(next_t, next_r);
        const bool is_q = r < a.n_q, is_v = r >= first_v;
        float w[kPerLane];
        widen<T>(raw, w);
        if (!is_v) {
            if (pick(is_q, false, a.weight[0] != nullptr, a.weight[1] != nullptr, a.weight[1] != nullptr)) {
                float sum = 0.f, g[kPerLane];
                read_eight(weights[is_q ? 0 : 1], D, lane, g);
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) sum = __builtin_fmaf(w[i], w[i], sum);
                sum = over_row<D>(sum, [](float x, float y) { return x + y; });
                const float scale = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) w[i] = w[i] * scale * g[i];
            }
            if (a.neighbours) {
                if (turned) {
                    typedef float f32x4 __attribute__((ext_vector_type(4)));
                    const f32x4 c = reinterpret_cast<const f32x4*>(cosines + t * pairs)[lane], s = reinterpret_cast<const f32x4*>(sines[0] + t * pairs)[lane];
#pragma unroll
                    for (int i = 0; i < kPerLane; i += 2) {
                        const float x = w[i], y = w[i + 1];
                        w[i] = __builtin_fmaf(x, c[i / 2], -(y * s[i / 2]));
                        w[i + 1] = __builtin_fmaf(y, c[i / 2], x * s[i / 2]);
                    }
                }
            } else {
                // The other half's value times the sine.  Eight lanes on (heads of
                // 128, all turned): a rotation within 16 lanes, without LDS.
                float c[kPerLane], s[kPerLane];
                const int of = t * pairs, at = !turned ? 0 : second ? lane - across : lane;
                read_eight(cosines + of, pairs, at, c);
                read_eight(sines[second ? 0 : 1] + of, pairs, at, s);
                if (across == 8) {
#pragma unroll
                    for (int i = 0; i < kPerLane; ++i) s[i] *= dpp<0x128>(w[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < kPerLane; ++i)
                        s[i] *= __int_as_float(__builtin_amdgcn_ds_bpermute(partner_at, __float_as_int(w[i])));
                }
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) w[i] = turned ? __builtin_fmaf(w[i], c[i], s[i]) : w[i];
            }
            raw = narrow<T>(w);
            if (is_q || a.dst[1] != nullptr) {
                char* to = pick(is_q, false, q_out.at, k_out.at, k_out.at) +
                           place(t, is_q ? r : r - a.n_q, pick(is_q, false, q_out.stride, k_out.stride, k_out.stride));
#pragma unroll
                for (unsigned i = 0; i < sizeof(T) / 2; ++i) reinterpret_cast<u32x4*>(to)[i] = raw.v[i];
            }
        }
        if constexpr (BITS != 0) {
            const int which = is_v ? 1 : 0;
            const int64_t row = is_q ? -1 : kv_row(a.d, slots[t], r - a.n_q - which * a.n_kv);
            if (row >= 0) {
                uint8_t* codes = pick(is_v, false, a.codes[1], a.codes[0], a.codes[0]);
                if constexpr (BITS == 16) {
                    if constexpr (sizeof(T) == 4) raw.v[0] = narrow<uint16_t>(w).v[0];
                    *reinterpret_cast<u32x4*>(codes + row * (D * 2) + lane * 16) = raw.v[0];
                } else {
                    store_quantised_row<D, BITS>(w, codes, pick(is_v, false, a.grid[1], a.grid[0], a.grid[0]), row, lane);
                }
            }
        }
        t = next_t;
        r = next_r;
    }
}

template <int D, typename T, int BITS>
grinqh_status rope_launch(RopeArgs& a, hipStream_t stream) {
    constexpr int kItems = kRopeThreads / (D / kPerLane), kTokens = kMostAngles / (D / 2);
    // About five rows to a group of lanes: a workgroup's tokens where there are
    // many, a token's heads over several workgroups where those leave CUs idle.
    static_assert(int64_t{kTokens} * kMostGroups >= kMaxPacked, "a launch holds every call's tokens");
    a.tokens = static_cast<int>(std::max({int64_t{1}, (a.n_tokens + kMostGroups - 1) / kMostGroups,
                                          std::min<int64_t>({kTokens, 5 * kItems / a.rows, a.n_tokens / kFill})}));
    const int64_t groups = (a.n_tokens + a.tokens - 1) / a.tokens;
    const int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((a.rows + kItems - 1) / kItems, kFill / groups)));
    a.step_tokens = parts * kItems / a.rows;
    a.step_rows = parts * kItems % a.rows;
    return launch_kernel(rope_kernel<D, T, BITS>, dim3(static_cast<unsigned>(groups), parts), kRopeThreads, 0, stream, a);
}

template <int D, typename T>
grinqh_status rope_bits(RopeArgs& a, int bits, hipStream_t stream) {
    if (bits == 0) return rope_launch<D, T, 0>(a, stream);
    if (bits == 4) return rope_launch<D, T, 4>(a, stream);
    if (bits == 8) return rope_launch<D, T, 8>(a, stream);
    return rope_launch<D, T, 16>(a, stream);
}

template <typename T>
grinqh_status rope_dim(RopeArgs& a, int head_dim, int bits, hipStream_t stream) {
    if (head_dim == 64) return rope_bits<64, T>(a, bits, stream);
    if (head_dim == 128) return rope_bits<128, T>(a, bits, stream);
    return rope_bits<256, T>(a, bits, stream);
}

bool valid_type(int dtype) { return dtype == GRINQH_BF16 || dtype == GRINQH_F32; }

}  // namespace
}  // namespace grinqh

using namespace grinqh;

extern "C" {

grinqh_status grinqh_qk_rope(const grinqh_rope_args* p, void* stream) {
    if (p == nullptr) return GRINQH_EINVAL;
    const bool cached = p->cache != nullptr;
    if (cached) {
        const grinqh_status st = check_kv_pools(p->cache, p->pools);
        if (st != GRINQH_OK) return st;
        if (p->cache->n_kv_heads != p->n_kv_heads || p->cache->head_dim != p->head_dim) return GRINQH_EINVAL;
    }
    if (!valid_type(p->dtype) || p->n_tokens < 0 || p->n_tokens > kMaxPacked) return GRINQH_EINVAL;
    if (p->n_q_heads < 1 || p->n_q_heads > kMaxQHeads || p->n_kv_heads < 1 || p->n_kv_heads > kMaxKvHeads) return GRINQH_EINVAL;
    if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return GRINQH_EINVAL;
    if (p->rope_dim < 0 || p->rope_dim > p->head_dim || p->rope_dim % 16 != 0) return GRINQH_EINVAL;
    const bool normed = p->q_weight != nullptr || p->k_weight != nullptr;
    if (normed && (!valid_type(p->weight_dtype) || !(p->eps >= 0.f && p->eps < INFINITY))) return GRINQH_EINVAL;
    if (p->n_tokens == 0) return GRINQH_OK;
    if (p->q == nullptr || p->k == nullptr || p->q_out == nullptr || (p->k_out == nullptr && !cached)) return GRINQH_EINVAL;
    if (p->rope_dim > 0 && (p->positions == nullptr || p->freqs == nullptr)) return GRINQH_EINVAL;
    if (cached && (p->v == nullptr || p->slots == nullptr)) return GRINQH_EINVAL;
    const int64_t n = p->n_tokens, eb = p->dtype == GRINQH_BF16 ? 2 : 4;
    const int64_t q_width = static_cast<int64_t>(p->n_q_heads) * p->head_dim, k_width = static_cast<int64_t>(p->n_kv_heads) * p->head_dim;
    const auto bad_stride = [](int64_t stride, int64_t width) { return stride < width || stride > kMaxStride; };
    if (bad_stride(p->q_stride, q_width) || bad_stride(p->k_stride, k_width) || bad_stride(p->q_out_stride, q_width) ||
        (p->k_out != nullptr && bad_stride(p->k_out_stride, k_width)) || (cached && bad_stride(p->v_stride, k_width)))
        return GRINQH_EINVAL;
    const auto off = [&](const void* at, int64_t stride) { return at != nullptr && (!aligned_to(at, 16) || stride * eb % 16 != 0); };
    if (off(p->q, p->q_stride) || off(p->k, p->k_stride) || off(p->q_out, p->q_out_stride) || off(p->k_out, p->k_out_stride) ||
        (cached && off(p->v, p->v_stride)) || !aligned_to(p->q_weight, 16) || !aligned_to(p->k_weight, 16) ||
        !aligned_to(p->positions, 4) || !aligned_to(p->freqs, 8) || (cached && !aligned_to(p->slots, 8)))
        return GRINQH_EALIGN;
    const auto rows = [&](int64_t stride, int64_t width) { return static_cast<size_t>(((n - 1) * stride + width) * eb); };
    const size_t q_bytes = rows(p->q_stride, q_width), k_bytes = rows(p->k_stride, k_width);
    const size_t weight_bytes = p->head_dim * (p->weight_dtype == GRINQH_BF16 ? 2u : 4u);
    const size_t code_bytes = cached ? grinqh_kv_code_bytes(p->cache) : 0, grid_bytes = cached ? grinqh_kv_grid_bytes(p->cache) : 0;
    const grinqh_kv_pools none{nullptr, nullptr, nullptr, nullptr};
    const grinqh_kv_pools& pools = cached ? *p->pools : none;
    const Span q_out{p->q_out, rows(p->q_out_stride, q_width)};
    const Span k_out{p->k_out, p->k_out == nullptr ? 0 : rows(p->k_out_stride, k_width)};
    // an output may be its input itself
    const bool q_same = p->q_out == p->q && p->q_out_stride == p->q_stride, k_same = p->k_out == p->k && p->k_out_stride == p->k_stride;
    const Span more[] = {{p->v, cached ? rows(p->v_stride, k_width) : 0},
                         {p->slots, cached ? static_cast<size_t>(n) * 8 : 0},
                         {p->positions, p->rope_dim > 0 ? static_cast<size_t>(n) * 4 : 0},
                         {p->freqs, static_cast<size_t>(p->rope_dim) * 4},
                         {p->q_weight, p->q_weight == nullptr ? 0 : weight_bytes},
                         {p->k_weight, p->k_weight == nullptr ? 0 : weight_bytes}};
    // Rows of one fused projection lie between one another: what is shared there is
    // a stretch of memory, not a value, so an output that is its input is held
    // against the other inputs row by row.
    const auto apart = [&](const void* out, int64_t out_stride, int64_t out_width, const void* in, int64_t in_stride, int64_t in_width) {
        const uintptr_t o = reinterpret_cast<uintptr_t>(out), i = reinterpret_cast<uintptr_t>(in);
        if (!overlaps(out, rows(out_stride, out_width), in, rows(in_stride, in_width))) return true;
        if (out_stride != in_stride) return false;
        const int64_t period = out_stride * eb, gap = static_cast<int64_t>(i - o), at = ((gap % period) + period) % period;
        return at >= out_width * eb && at + in_width * eb <= period;                // the same place between two tokens' rows
    };
    if (!q_same && !apart(p->q_out, p->q_out_stride, q_width, p->q, p->q_stride, q_width)) return GRINQH_EINVAL;
    if (!apart(p->q_out, p->q_out_stride, q_width, p->k, p->k_stride, k_width)) return GRINQH_EINVAL;
    if (cached && !apart(p->q_out, p->q_out_stride, q_width, p->v, p->v_stride, k_width)) return GRINQH_EINVAL;
    if (p->k_out != nullptr) {
        if (!apart(p->k_out, p->k_out_stride, k_width, p->q, p->q_stride, q_width)) return GRINQH_EINVAL;
        if (!k_same && !apart(p->k_out, p->k_out_stride, k_width, p->k, p->k_stride, k_width)) return GRINQH_EINVAL;
        if (cached && !apart(p->k_out, p->k_out_stride, k_width, p->v, p->v_stride, k_width)) return GRINQH_EINVAL;
        if (!apart(p->k_out, p->k_out_stride, k_width, p->q_out, p->q_out_stride, q_width)) return GRINQH_EINVAL;
    }
    for (int i = 1; i < 6; ++i)                                                     // the values were held against the outputs above
        if (overlaps(q_out.at, q_out.bytes, more[i].at, more[i].bytes) || overlaps(k_out.at, k_out.bytes, more[i].at, more[i].bytes))
            return GRINQH_EINVAL;
    if (cached && written_overlaps({{pools.k_codes, code_bytes}, {pools.v_codes, code_bytes}, {pools.k_grid, grid_bytes}, {pools.v_grid, grid_bytes}},
                                   {q_out, k_out, {p->q, q_bytes}, {p->k, k_bytes}, more[0], more[1], more[2], more[3], more[4], more[5]}))
        return GRINQH_EINVAL;
    RopeArgs a{};
    if (cached) a.d = kv_dims(*p->cache);
    a.src[0] = p->q;
    a.src[1] = p->k;
    a.src[2] = p->v;
    a.src_stride[0] = p->q_stride;
    a.src_stride[1] = p->k_stride;
    a.src_stride[2] = p->v_stride;
    a.dst[0] = p->q_out;
    a.dst[1] = p->k_out;
    a.dst_stride[0] = p->q_out_stride;
    a.dst_stride[1] = p->k_out_stride;
    a.codes[0] = pools.k_codes;
    a.codes[1] = pools.v_codes;
    a.grid[0] = pools.k_grid;
    a.grid[1] = pools.v_grid;
    a.slots = p->slots;
    a.positions = p->positions;
    a.freqs = p->freqs;
    a.weight[0] = p->q_weight;
    a.weight[1] = p->k_weight;
    a.n_tokens = n;
    a.n_q = p->n_q_heads;
    a.n_kv = p->n_kv_heads;
    a.rows = p->n_q_heads + p->n_kv_heads * (cached ? 2 : 1);
    a.rope_dim = p->rope_dim;
    a.neighbours = p->neighbours != 0;
    a.weight_dtype = p->weight_dtype;
    a.eps = p->eps;
    const int bits = cached ? p->cache->bits : 0;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return p->dtype == GRINQH_BF16 ? rope_dim<uint16_t>(a, p->head_dim, bits, st) : rope_dim<float>(a, p->head_dim, bits, st);
}

}  // extern "C"
