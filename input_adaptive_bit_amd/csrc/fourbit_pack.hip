// Packing of 4-bit codes and their groups' scales and zero points into the order
// in which the products load them (offline).
//
// A thread makes one word: eight codes of an output and eight neighbouring inputs
// (one 8-byte load; d_in is a multiple of 32, so they lie in one group of
// eight or past the end).  A wave writes 256 consecutive bytes.  Memory bounds
// it: 4096 to 14336 in 27 us (92 MB, 3.4 TB/s; rows are read in pieces of 32 bytes).
#include "fourbit_common.hpp"

namespace grinqh {
namespace {

constexpr int kPackThreads = 256;
constexpr int64_t kMaxPackGroups = 1 << 20;        // more words than these hold go round again

__global__ __launch_bounds__(kPackThreads) void fourbit_codes_kernel(const uint8_t* q, uint32_t* codes, int d_in, int d_out,
                                                                     int k_tiles, int row_tiles, int64_t words) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPackThreads;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x; at < words; at += step) {
        const int m = at & 3, lane = (at >> 2) & 63;
        const int64_t tile = at >> 8;
        const int k_tile = tile % k_tiles;
        const int64_t er = tile / k_tiles, e = er / row_tiles;
        const int j = static_cast<int>(er % row_tiles) * kTileOut + (lane & 15);
        const int i = k_tile * kTileIn + 32 * m + 8 * (lane >> 4);
        uint32_t w = 0;
        if (j < d_out && i < d_in) {
            const uint64_t eight = *reinterpret_cast<const uint64_t*>(q + (e * d_out + j) * d_in + i);
#pragma unroll
            for (int x = 0; x < 8; ++x) w |= static_cast<uint32_t>((eight >> (8 * x)) & 15u) << (4 * (x >> 1) + 16 * (x & 1));
            w = w << 3 | w >> 29;
        }
        codes[at] = w;
    }
}

__global__ __launch_bounds__(kPackThreads) void fourbit_grid_kernel(const uint16_t* s, const uint16_t* z, uint32_t* grid,
                                                                    int groups, int d_out, int padded, int row_tiles,
                                                                    int64_t pairs) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPackThreads;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x; at < pairs; at += step) {
        const int64_t tile = at >> 4, er = tile / padded, e = er / row_tiles;
        const int g = tile % padded, j = static_cast<int>(er % row_tiles) * kTileOut + static_cast<int>(at & 15);
        uint32_t pair = 0;
        if (j < d_out && g < groups) {
            const int64_t from = (e * d_out + j) * groups + g;
            pair = s[from] | static_cast<uint32_t>(z[from]) << 16;
        }
        grid[at] = pair;
    }
}

unsigned groups_for(int64_t n) {
    const int64_t g = (n + kPackThreads - 1) / kPackThreads;
    return static_cast<unsigned>(g < kMaxPackGroups ? g : kMaxPackGroups);
}

}  // namespace

bool valid_fourbit_layout(const grinqh_fourbit_layout* L) {
    if (L == nullptr) return false;
    if (L->group != 32 && L->group != 64 && L->group != 128) return false;
    if (L->d_in < L->group || L->d_in > (1 << 20) || L->d_in % L->group != 0) return false;
    if (L->d_out < 1 || L->d_out > (1 << 20) || L->n_experts < 1 || L->n_experts > kMaxExperts) return false;
    if (L->k_tiles != (L->d_in + kTileIn - 1) / kTileIn || L->row_tiles != (L->d_out + kTileOut - 1) / kTileOut) return false;
    return static_cast<int64_t>(L->n_experts) * L->row_tiles * L->k_tiles <= int64_t{1} << 30;
}

}  // namespace grinqh

using namespace grinqh;

extern "C" {

grinqh_status grinqh_fourbit_layout_init(int32_t d_in, int32_t d_out, int32_t group, int32_t n_experts,
                                         grinqh_fourbit_layout* out) {
    if (out == nullptr || d_in < 1 || d_in > (1 << 20) || d_out < 1 || d_out > (1 << 20)) return GRINQH_EINVAL;
    const grinqh_fourbit_layout L{d_in, d_out, group, n_experts, (d_in + kTileIn - 1) / kTileIn,
                                  (d_out + kTileOut - 1) / kTileOut};
    if (!valid_fourbit_layout(&L)) return GRINQH_EINVAL;
    *out = L;
    return GRINQH_OK;
}

size_t grinqh_fourbit_code_bytes(const grinqh_fourbit_layout* L) {
    if (!valid_fourbit_layout(L)) return 0;
    return static_cast<size_t>(L->n_experts) * L->row_tiles * L->k_tiles * 1024u;
}

size_t grinqh_fourbit_grid_bytes(const grinqh_fourbit_layout* L) {
    if (!valid_fourbit_layout(L)) return 0;
    return static_cast<size_t>(L->n_experts) * L->row_tiles * L->k_tiles * (kTileIn / L->group) * 64u;
}

grinqh_status grinqh_fourbit_pack(const grinqh_fourbit_layout* L, const uint8_t* q, const uint16_t* s,
                                  const uint16_t* z, uint8_t* codes, uint16_t* grid, void* stream) {
    if (!valid_fourbit_layout(L) || q == nullptr || s == nullptr || z == nullptr || codes == nullptr || grid == nullptr)
        return GRINQH_EINVAL;
    if (!aligned_to(q, 8) || !aligned_to(s, 2) || !aligned_to(z, 2) || !aligned_to(codes, 16) || !aligned_to(grid, 16))
        return GRINQH_EALIGN;
    const size_t n = static_cast<size_t>(L->n_experts) * L->d_out, groups = L->d_in / L->group;
    const size_t code_bytes = grinqh_fourbit_code_bytes(L), grid_bytes = grinqh_fourbit_grid_bytes(L);
    if (written_overlaps({{codes, code_bytes}, {grid, grid_bytes}}, {{q, n * L->d_in}, {s, n * groups * 2}, {z, n * groups * 2}}))
        return GRINQH_EINVAL;
    const int64_t words = static_cast<int64_t>(code_bytes / 4), pairs = static_cast<int64_t>(grid_bytes / 4);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const grinqh_status status = launch_kernel(fourbit_codes_kernel, groups_for(words), kPackThreads, 0, st, q,
                                               reinterpret_cast<uint32_t*>(codes), L->d_in, L->d_out, L->k_tiles,
                                               L->row_tiles, words);
    if (status != GRINQH_OK) return status;
    return launch_kernel(fourbit_grid_kernel, groups_for(pairs), kPackThreads, 0, st, s, z, reinterpret_cast<uint32_t*>(grid),
                         static_cast<int>(groups), L->d_out, L->k_tiles * (kTileIn / L->group), L->row_tiles, pairs);
}

}  // extern "C"
