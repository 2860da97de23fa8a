// The page plan of a batch's step: pages for the new tokens, their slots and
// positions, the new lengths and the ends of the packed sequences.
//
// With h = ceil(len / page) pages held, t = ceil((len + new) / page) needed and
// need = t - h, sequence b takes the pages
//   free[n_free - 1 - (sum_{c < b, served} need_c + i)],  i = 0 .. need - 1,
// if the sum of need over all up to b, served or not, is no more than n_free.  So one scan over the sequences decides all
// of it (fourfold: pages, new tokens, granted pages, lengths), and then every new token can be
// worked on alone: its sequence by a search in the ends, its page from the table
// (the page that was begun before) or from the list.  The token that begins a
// page writes the table's entry.
//
// A workgroup scans 1024 sequences at a time, with sums that stop at the type's end:
// what counts is whether they pass a bound of 2^24, and the largest int32 stands for
// all beyond it.  Nothing here is more than a few kB a workgroup, and what
// bounds a call is the chain: the lengths' loads, the scan, a token's search, its
// page's load.  So for up to 1024 sequences every workgroup scans them all for itself
// and keeps the result in LDS for its own tokens: one launch.  Lengths that are updated in
// place cannot be read by other workgroups meanwhile, and of more sequences the
// scan itself takes longer than a launch: then one workgroup scans, and a second
// launch does the tokens (up to 4096 of few sequences: that same workgroup).
// 48 sequences of a token each take 3.2 us, 700 of 512 tokens 6.8 in one launch and
// 7.5 in two, 3000 of 100 tokens 11 (a captured launch of nothing takes 2.4).
#include <algorithm>

#include "internal.h"
#include "kv_common.hpp"

namespace grinqh {
namespace {

constexpr int kPageThreads = 1024, kPageWaves = kPageThreads / kWave, kSpreadThreads = 256;
constexpr int kOneGroup = 4096;                    // tokens up to which one workgroup does the scan and them
constexpr int kMostGroups = 512;                   // of a launch whose workgroups all scan: two to a CU

struct PagesArgs {
    grinqh_extend_args p;
    int page_shift;
};

// What the scan leaves of a sequence for its tokens: its length before, and the
// place of its first new page among all that are taken (-1: refused).
struct Sequence {
    int32_t before, first;
};

// Sums that stop at 2^32 - 1, in any order the same.
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// x of the lane that CTRL names (0 where there is none or the row is not among ROWS).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t from_lane(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, ROWS, 0xF, false));
}

// Sums up to and with a lane: of its row of 16, of the wave.
__device__ __forceinline__ uint32_t row_sum_up_to(uint32_t x) {
    x = add(x, from_lane<0x111, 0xF>(x));                     // row_shr 1, 2, 4, 8
    x = add(x, from_lane<0x112, 0xF>(x));
    x = add(x, from_lane<0x114, 0xF>(x));
    return add(x, from_lane<0x118, 0xF>(x));
}
__device__ __forceinline__ uint32_t wave_sum_up_to(uint32_t x) {
    x = row_sum_up_to(x);
    x = add(x, from_lane<0x142, 0xA>(x));                     // row_bcast 15: rows 1 and 3
    return add(x, from_lane<0x143, 0xC>(x));                  // row_bcast 31: rows 2 and 3
}

struct Pair {
    uint32_t a, b;
};
__device__ __forceinline__ Pair add(Pair x, Pair y) { return Pair{add(x.a, y.a), add(x.b, y.b)}; }

// Sums up to and with a thread of the workgroup; `all` is what they come to.  One
// barrier: `waves` is another one at the next call, and free again at the one after.
template <int WAVES>
__device__ __forceinline__ Pair group_sum_up_to(Pair x, Pair* waves, Pair& all) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    x = Pair{wave_sum_up_to(x.a), wave_sum_up_to(x.b)};
    if (lane == kWave - 1) waves[wave] = x;
    __syncthreads();
    const Pair of = waves[lane & (WAVES - 1)];
    const uint32_t a = row_sum_up_to(of.a), b = row_sum_up_to(of.b);
    const auto at = [](uint32_t v, int l) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l)); };
    all = Pair{at(a, WAVES - 1), at(b, WAVES - 1)};
    return wave == 0 ? x : add(x, Pair{at(a, wave - 1), at(b, wave - 1)});
}

__device__ __forceinline__ int32_t clamp32(uint32_t x) { return static_cast<int32_t>(min(x, 0x7FFFFFFFu)); }

// New token t of sequence b, whose new tokens begin at `begin`.
__device__ __forceinline__ void place_token(const PagesArgs& a, const Sequence& s, int n_free, int b, int t, int begin) {
    const auto& p = a.p;
    const int64_t position = static_cast<int64_t>(s.before) + (t - begin);
    p.positions[t] = static_cast<int32_t>(min(position, int64_t{0x7FFFFFFF}));
    int64_t slot = -1;
    if (s.first >= 0) {
        const int64_t at = position >> a.page_shift, held = (static_cast<int64_t>(s.before) + p.page_size - 1) >> a.page_shift;
        int32_t* entry = p.page_table + b * p.table_stride + at;
        int page;
        if (at < held) {
            page = *entry;
        } else {
            page = p.free_pages[n_free - 1 - (s.first + (at - held))];
            if ((position & (p.page_size - 1)) == 0) *entry = page;
        }
        page = page_or_absent(page, p.n_pages);
        if (page >= 0) slot = (static_cast<int64_t>(page) << a.page_shift) + (position & (p.page_size - 1));
    }
    p.slots[t] = slot;
}
__device__ __forceinline__ void no_token(const PagesArgs& a, int t) {
    a.p.slots[t] = -1;
    a.p.positions[t] = 0;
}

// The sequence of token t: the last whose new tokens begin at t or before (those
// without new tokens end where the next begins).  lo .. hi bound it.
__device__ __forceinline__ int sequence_of(const int32_t* begins, int t, int lo, int hi) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (begins[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}
// The same for a wave's one token, 64 places at a time.
__device__ __forceinline__ int sequence_of_wave(const int32_t* begins, int t, int count, int lane) {
    int lo = 0;
    while (count > 1) {
        const int step = (count + kWave - 1) / kWave;
        const int passed = __popcll(__ballot(lane * step < count && begins[lo + min(lane * step, count - 1)] <= t)) - 1;
        lo += passed * step;
        count = min(step, count - passed * step);
    }
    return lo;
}

// TOKENS: the tokens too (of up to THREADS sequences; every workgroup scans, the
// first one's results are written); else one workgroup, which leaves the
// sequences in the workspace.
template <bool TOKENS, int THREADS>
__global__ __launch_bounds__(THREADS) void extend_scan_kernel(PagesArgs a) {
    constexpr int WAVES = THREADS / kWave;
    __shared__ Pair waves[2][WAVES];
    __shared__ int refused;
    __shared__ Sequence here[TOKENS ? THREADS : 1];
    __shared__ int32_t begins[TOKENS ? THREADS : 1];
    const auto& p = a.p;
    Sequence* seqs = static_cast<Sequence*>(p.workspace);
    if (threadIdx.x == 0) refused = 0;
    const uint32_t n_free = min(max(p.n_free[0], 0), p.n_pages), page = p.page_size;
    const bool writes = !TOKENS || blockIdx.x == 0;
    const auto pages_of = [&](uint32_t tokens) { return (tokens >> a.page_shift) + ((tokens & (page - 1)) != 0); };
    Pair asked{0u, 0u}, given{0u, 0u};                        // pages and new tokens; pages and lengths
    for (int base = 0; base < p.batch; base += THREADS) {
        const int b = base + threadIdx.x;
        const bool there = b < p.batch;
        const uint32_t old = there ? max(p.seq_lens[b], 0) : 0, fresh = there ? max(p.n_new[b], 0) : 0;
        const uint32_t held = pages_of(old), wanted = pages_of(old + fresh), need = wanted - held;
        // What no step could serve asks for no pages: else the sequences behind it
        // would be refused for its sake, step after step.
        const bool possible = wanted <= static_cast<uint32_t>(p.max_pages) && need <= static_cast<uint32_t>(p.n_pages);
        Pair all;
        const Pair upto = add(asked, group_sum_up_to<WAVES>(Pair{possible ? need : 0u, fresh}, waves[0], all));
        asked = add(asked, all);
        const bool granted = fresh == 0 || (possible && upto.a <= n_free && upto.b <= static_cast<uint32_t>(p.capacity));
        // Pages are taken by their place among those of all sequences, served or
        // not: the pages of one that is refused for its own sake stay unused in
        // the list only if none behind it are taken, so places are counted again
        // over what is granted.
        const uint32_t mine = granted ? need : 0u, len = granted ? old + fresh : old;
        const Pair to = add(given, group_sum_up_to<WAVES>(Pair{mine, len}, waves[1], all));
        given = add(given, all);
        const Sequence s{static_cast<int32_t>(old), granted ? static_cast<int32_t>(to.a - mine) : -1};
        if (TOKENS) {
            here[threadIdx.x] = s;
            begins[threadIdx.x] = clamp32(upto.b - fresh);
        }
        if (there && writes) {
            if (!TOKENS) seqs[b] = s;
            p.new_lens[b] = clamp32(len);
            p.cu_q[b + 1] = clamp32(upto.b);
            p.cu_k[b + 1] = clamp32(to.b);
            if (!granted) atomicAdd(&refused, 1);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && writes) {
        p.cu_q[0] = p.cu_k[0] = 0;
        p.refused[0] = refused;
        p.n_free_out[0] = static_cast<int>(n_free - given.a);
        if (!TOKENS) reinterpret_cast<uint32_t*>(seqs + p.batch)[0] = n_free;
    }
    if (!TOKENS) return;
    for (int t = blockIdx.x * THREADS + threadIdx.x; t < p.capacity; t += gridDim.x * THREADS) {
        if (static_cast<uint32_t>(t) >= asked.b) {
            no_token(a, t);
        } else {
            const int b = sequence_of(begins, t, 0, p.batch - 1);
            place_token(a, here[b], static_cast<int>(n_free), b, t, begins[b]);
        }
    }
}

__global__ __launch_bounds__(kSpreadThreads) void extend_tokens_kernel(PagesArgs a) {
    const auto& p = a.p;
    const Sequence* seqs = static_cast<const Sequence*>(p.workspace);
    const int n_free = reinterpret_cast<const int32_t*>(seqs + p.batch)[0];
    const int lane = threadIdx.x & 63, first = __builtin_amdgcn_readfirstlane(blockIdx.x * kSpreadThreads + (threadIdx.x & ~63));
    const int t = first + lane, all = p.batch == 0 ? 0 : p.cu_q[p.batch];
    int lo = 0, hi = 0;
    if (first < all) {
        lo = sequence_of_wave(p.cu_q, first, p.batch, lane);
        hi = sequence_of_wave(p.cu_q, min(first + kWave, all) - 1, p.batch, lane);
    }
    if (t >= p.capacity) return;
    if (t >= all) {
        no_token(a, t);
    } else {
        const int b = sequence_of(p.cu_q, t, lo, hi);
        place_token(a, seqs[b], n_free, b, t, p.cu_q[b]);
    }
}

// One workgroup.  Of every 1024 sequences the finished ones are listed, in order;
// then a wave takes one at a time, in two rounds for every kPageWaves of them:
// how many of its entries name a page, then where they go.  A chain of trips to
// memory for every 16 sequences: 48 of 128 pages each take 8 us, 70 of 700 15.
__global__ __launch_bounds__(kPageThreads) void release_kernel(int32_t* table, int64_t stride, int32_t* lens, const uint8_t* finished,
                                                               int batch, int max_pages, int page_shift, int32_t* free_pages,
                                                               int32_t* n_free, int n_pages) {
    __shared__ int list[kPageThreads], listed_of[kPageWaves], counts[2][kPageWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t listed = min(max(n_free[0], 0), n_pages);
    for (int base = 0; base < batch; base += kPageThreads) {
        const int mine = base + threadIdx.x;
        const uint64_t over = __ballot(mine < batch && finished[min(mine, batch - 1)] != 0);
        if (lane == 0) listed_of[wave] = __popcll(over);
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < kPageWaves; ++w) {
            before += w < wave ? listed_of[w] : 0;
            all += listed_of[w];
        }
        if (over >> lane & 1) list[before + __popcll(over & ((uint64_t{1} << lane) - 1))] = mine;
        __syncthreads();
        for (int first = 0, turn = 0; first < all; first += kPageWaves, turn ^= 1) {
            const bool done = first + wave < all;
            const int b = done ? list[first + wave] : 0;
            const int64_t len = done ? max(lens[b], 0) : 0;
            const int held = static_cast<int>(min((len + (int64_t{1} << page_shift) - 1) >> page_shift, static_cast<int64_t>(max_pages)));
            int32_t* row = table + static_cast<int64_t>(b) * stride;
            int count = 0;
            for (int i = 0; i < held; i += kWave)
                count += __popcll(__ballot(i + lane < held && page_or_absent(row[min(i + lane, held - 1)], n_pages) >= 0));
            if (lane == 0) counts[turn][wave] = count;
            __syncthreads();
            int64_t to = listed;
            for (int w = 0; w < kPageWaves; ++w) {
                to += w < wave ? counts[turn][w] : 0;
                listed += counts[turn][w];
            }
            for (int i = 0; i < held; i += kWave) {
                const int page = i + lane < held ? page_or_absent(row[i + lane], n_pages) : -1;
                const uint64_t there = __ballot(page >= 0);
                const int64_t at = to + __popcll(there & ((uint64_t{1} << lane) - 1));
                if (page >= 0 && at < n_pages) free_pages[at] = page;
                if (i + lane < held) row[i + lane] = -1;
                to += __popcll(there);
            }
            if (done && lane == 0) lens[b] = 0;
        }
        __syncthreads();                                      // the list has been read
    }
    if (threadIdx.x == 0) n_free[0] = static_cast<int32_t>(min(listed, static_cast<int64_t>(n_pages)));
}

bool valid_pages(int batch, int max_pages, int64_t table_stride, int page_size, int n_pages) {
    if (batch < 0 || batch > kMaxBatch || max_pages < 1 || max_pages > (1 << 24)) return false;
    if (table_stride < max_pages || table_stride > kMaxStride || n_pages < 1 || n_pages > (1 << 24)) return false;
    return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 || page_size == 256;
}

size_t table_bytes(int batch, int max_pages, int64_t stride) {
    return batch == 0 ? 0 : static_cast<size_t>((batch - 1) * stride + max_pages) * 4;
}

}  // namespace
}  // namespace grinqh

using namespace grinqh;

extern "C" {

size_t grinqh_kv_extend_workspace_bytes(int32_t batch) {
    if (batch < 0 || batch > kMaxBatch) return 0;
    return static_cast<size_t>(batch) * sizeof(Sequence) + 16;
}

grinqh_status grinqh_kv_extend(const grinqh_extend_args* args, void* stream) {
    if (args == nullptr) return GRINQH_EINVAL;
    const grinqh_extend_args& p = *args;
    if (!valid_pages(p.batch, p.max_pages, p.table_stride, p.page_size, p.n_pages)) return GRINQH_EINVAL;
    if (p.capacity < 0 || p.capacity > kMaxPacked) return GRINQH_EINVAL;
    if (p.n_free == nullptr || p.n_free_out == nullptr || p.refused == nullptr || p.cu_q == nullptr || p.cu_k == nullptr ||
        p.free_pages == nullptr || p.workspace == nullptr)
        return GRINQH_EINVAL;
    if (p.batch > 0 && (p.page_table == nullptr || p.seq_lens == nullptr || p.n_new == nullptr || p.new_lens == nullptr))
        return GRINQH_EINVAL;
    if (p.capacity > 0 && (p.slots == nullptr || p.positions == nullptr)) return GRINQH_EINVAL;
    for (const void* at : {static_cast<const void*>(p.page_table), static_cast<const void*>(p.seq_lens), static_cast<const void*>(p.n_new),
                           static_cast<const void*>(p.free_pages), static_cast<const void*>(p.n_free), static_cast<const void*>(p.new_lens),
                           static_cast<const void*>(p.n_free_out), static_cast<const void*>(p.refused), static_cast<const void*>(p.cu_q),
                           static_cast<const void*>(p.cu_k), static_cast<const void*>(p.positions)})
        if (!aligned_to(at, 4)) return GRINQH_EALIGN;
    if (!aligned_to(p.slots, 8) || !aligned_to(p.workspace, 16)) return GRINQH_EALIGN;
    const size_t ws = grinqh_kv_extend_workspace_bytes(p.batch);
    if (p.workspace_bytes < ws) return GRINQH_ENOSPACE;
    const size_t batch = static_cast<size_t>(p.batch) * 4, ends = batch + 4, room = static_cast<size_t>(p.capacity);
    const bool lens_same = p.new_lens == p.seq_lens, free_same = p.n_free_out == p.n_free;
    if (written_overlaps({{p.page_table, table_bytes(p.batch, p.max_pages, p.table_stride)}, {p.new_lens, batch}, {p.n_free_out, 4},
                          {p.refused, 4}, {p.cu_q, ends}, {p.cu_k, ends}, {p.slots, room * 8}, {p.positions, room * 4}, {p.workspace, ws}},
                         {{p.n_new, batch}, {p.free_pages, static_cast<size_t>(p.n_pages) * 4},
                          {p.seq_lens, lens_same ? 0 : batch}, {p.n_free, free_same ? size_t{0} : size_t{4}}}))
        return GRINQH_EINVAL;
    const PagesArgs a{p, log2_of(p.page_size)};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool shared = !lens_same && !free_same;             // others may scan while one workgroup writes
    if (p.batch <= 256 && p.capacity <= 256) return launch_kernel(extend_scan_kernel<true, 256>, dim3(1), 256, 0, st, a);
    if (p.batch <= kPageThreads && (shared || p.capacity <= kOneGroup)) {
        const int groups = std::min((p.capacity + kPageThreads - 1) / kPageThreads, kMostGroups);
        return launch_kernel(extend_scan_kernel<true, kPageThreads>, dim3(shared ? std::max(groups, 1) : 1), kPageThreads, 0, st, a);
    }
    const grinqh_status status = launch_kernel(extend_scan_kernel<false, kPageThreads>, dim3(1), kPageThreads, 0, st, a);
    if (status != GRINQH_OK) return status;
    if (p.capacity == 0) return GRINQH_OK;
    return launch_kernel(extend_tokens_kernel, dim3((p.capacity + kSpreadThreads - 1) / kSpreadThreads), kSpreadThreads, 0, st, a);
}

grinqh_status grinqh_kv_release(int32_t* page_table, int64_t table_stride, int32_t* seq_lens,
                                const uint8_t* finished, int32_t batch, int32_t max_pages, int32_t page_size,
                                int32_t* free_pages, int32_t* n_free, int32_t n_pages, void* stream) {
    if (!valid_pages(batch, max_pages, table_stride, page_size, n_pages)) return GRINQH_EINVAL;
    if (batch == 0) return GRINQH_OK;
    if (page_table == nullptr || seq_lens == nullptr || finished == nullptr || free_pages == nullptr || n_free == nullptr)
        return GRINQH_EINVAL;
    if (!aligned_to(page_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(free_pages, 4) || !aligned_to(n_free, 4))
        return GRINQH_EALIGN;
    const size_t n = static_cast<size_t>(batch);
    if (written_overlaps({{page_table, table_bytes(batch, max_pages, table_stride)}, {seq_lens, n * 4},
                          {free_pages, static_cast<size_t>(n_pages) * 4}, {n_free, 4}}, {{finished, n}}))
        return GRINQH_EINVAL;
    return launch_kernel(release_kernel, dim3(1), kPageThreads, 0, static_cast<hipStream_t>(stream), page_table, table_stride,
                         seq_lens, finished, static_cast<int>(batch), static_cast<int>(max_pages), log2_of(page_size), free_pages,
                         n_free, static_cast<int>(n_pages));
}

}  // extern "C"
