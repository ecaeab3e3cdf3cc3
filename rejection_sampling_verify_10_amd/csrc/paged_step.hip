// Pages for a step: how many each sequence needs, taken from the head of a ring of
// free pages in the order of the sequences, given back at its tail; and the slots
// of the step's tokens.
//
// Every workgroup sums the whole batch's needs for itself (three small arrays, from
// the L2; a row a thread) and then serves its own sequences, so nothing passes
// between workgroups and one launch does.  Where a call writes the arrays that it
// reads, what others still read (pages held, the ring's ends) is written by the last
// workgroup that has read them.  Taken pages lie between the ring's head and its
// tail, pages given back behind the tail: no entry is both read and written.
//
// Bound by latency: three dependent loads, a sum, a store, and a ticket where it
// writes in place.  512 sequences of 8 tokens 5.0 us (10.5 with 64-bit sums by
// shuffles), 16 prompts of up to 8192 tokens 4.4.  Whole calls in place: 512 rows of 8
// tokens 7.4 us, 2048 of 64 10.0, 65536 of 32 270, 1024 prompts of 8192 26.

#include <algorithm>
#include <type_traits>

#include "paged.hpp"

namespace sv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kPart = 1024;         // least tokens of a row that a workgroup finds the slots of, where there are several for it
constexpr int kRowsMax = 128;       // rows of a workgroup
constexpr int kMostWorkgroups = 1024;

struct Need {
    int len, cnt, held, need;
    bool ok;                        // the row's numbers make sense and fit its table
    __device__ __forceinline__ unsigned grow() const { return ok ? static_cast<unsigned>(max(need - held, 0)) : 0u; }
    __device__ __forceinline__ unsigned drop() const { return ok ? static_cast<unsigned>(max(held - need, 0)) : 0u; }
};
__device__ __forceinline__ Need read_need(const PageStepArgs& a, int t) {
    Need n;
    n.len = a.lengths[t];
    n.cnt = a.counts ? a.counts[t] : a.N;
    n.held = a.held[t];
    const bool live = n.len >= 0;
    const long long end = live ? static_cast<long long>(n.len) + n.cnt : 0;
    const long long need = (end + (1 << a.page_log2) - 1) >> a.page_log2;
    // (more pages than there are would wrap around the ring twice)
    n.ok = n.held >= 0 && n.held <= min(a.width, a.pages) && (!live || (n.cnt >= 0 && n.cnt <= a.N)) && need <= a.width;
    n.need = n.ok ? static_cast<int>(need) : 0;
    if (!live) n.cnt = 0;
    return n;
}

// Sums stop at 2^30, which no pool's pages reach: only whether they fit counts past that.
__device__ __forceinline__ unsigned add(unsigned a, unsigned b) { return min(a + b, 1u << 30); }
__device__ __forceinline__ unsigned wave_inclusive(unsigned v) {
    const int lane = threadIdx.x & (kWave - 1);
    const auto shifted = [](unsigned x, auto ctl) {
        return static_cast<unsigned>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctl)::value, 0xf, 0xf, true));
    };
    v = add(v, shifted(v, std::integral_constant<int, 0x111>()));       // row_shr:1, 2, 4, 8
    v = add(v, shifted(v, std::integral_constant<int, 0x112>()));
    v = add(v, shifted(v, std::integral_constant<int, 0x114>()));
    v = add(v, shifted(v, std::integral_constant<int, 0x118>()));
    const unsigned r0 = bcast(static_cast<int>(v), 15), r1 = add(r0, bcast(static_cast<int>(v), 31)),
                   r2 = add(r1, bcast(static_cast<int>(v), 47));
    const int row = lane >> 4;
    return add(v, row == 0 ? 0u : row == 1 ? r0 : row == 2 ? r1 : r2);
}
// Sums over the block's threads up to this one, and over all of them.
struct Pair {
    unsigned grow, drop;
};
__device__ __forceinline__ Pair block_inclusive(Pair v, Pair& total, Pair (&sh)[kWaves]) {
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    const Pair i = {wave_inclusive(v.grow), wave_inclusive(v.drop)};
    __syncthreads();
    if (lane == kWave - 1) sh[wave] = i;
    __syncthreads();
    Pair before = {0, 0};
    total = {0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) before = total;
        total.grow = add(total.grow, sh[w].grow);
        total.drop = add(total.drop, sh[w].drop);
    }
    return {add(before.grow, i.grow), add(before.drop, i.drop)};
}

struct Served {                     // a row of this workgroup's, in LDS
    int len, cnt, held, need, row;  // cnt -1: not served
    int take, give;                 // places in the ring of its first new page, and of the first one it gives back
};
// x mod pages for x below twice as many.
__device__ __forceinline__ int wrap(unsigned x, int pages) {
    return static_cast<int>(x >= static_cast<unsigned>(pages) ? x - pages : x);
}

__global__ __launch_bounds__(kThreads) void page_step_kernel(PageStepArgs a, int rows_wg, int parts, int part_n) {
    __shared__ Pair sh[kWaves];
    __shared__ Served mine[kRowsMax];
    __shared__ unsigned most[kWaves];
    __shared__ unsigned ticket;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int part = blockIdx.x % parts;
    const int first = blockIdx.x / parts * rows_wg, end = min(a.T, first + rows_wg);
    const int head = a.state[0], free_pages = a.state[1];
    const bool ring_ok = head >= 0 && head < a.pages && free_pages >= 0 && free_pages <= a.pages;
    const unsigned supply = ring_ok ? free_pages : 0;

    Pair base = {0, 0};
    unsigned taken = 0;             // the sum of the rows that grow and are served: the last one that fits
    Need n{};
    bool served = false;
    for (int t0 = 0; t0 < a.T; t0 += kThreads) {
        const int t = t0 + tid;
        n = Need{};
        if (t < a.T) n = read_need(a, t);
        n.ok = n.ok && ring_ok;
        Pair total, upto = block_inclusive({n.grow(), n.drop()}, total, sh);
        upto.grow = add(base.grow, upto.grow), upto.drop = add(base.drop, upto.drop);
        served = n.ok && (n.grow() == 0 || upto.grow <= supply);
        if (served && n.grow() > 0) taken = upto.grow;
        if (t >= first && t < end) {
            Served s;
            s.len = n.len, s.cnt = served ? n.cnt : -1, s.held = n.held, s.need = served ? n.need : n.held;
            s.take = served ? static_cast<int>((head + upto.grow - n.grow()) % a.pages) : 0;
            s.give = served ? static_cast<int>((head + supply + upto.drop - n.drop()) % a.pages) : 0;
            s.row = t;
            mine[t - first] = s;
            if (part == 0) {
                a.out_granted[t] = s.cnt;
                if (a.apart) a.out_held[t] = s.need;
            }
        }
        base.grow = add(base.grow, total.grow), base.drop = add(base.drop, total.drop);
    }
    __syncthreads();

    // a row's new pages, the ones it gives back (its first part), and its tokens' slots
    const auto serve = [&](const Served& s, int at, int step) {
        int32_t* table = a.tables + s.row * a.table_stride;
        int32_t* slots = a.out_slots + static_cast<long long>(s.row) * a.N;
        const auto fresh = [&](int j) { return a.ring[wrap(static_cast<unsigned>(s.take) + (j - s.held), a.pages)]; };
        if (part == 0) {
            for (int j = s.held + at; j < s.need; j += step) table[j] = fresh(j);
            for (int j = s.need + at; j < s.held; j += step)
                a.ring[wrap(static_cast<unsigned>(s.give) + (j - s.need), a.pages)] = table[j];
        }
        const int last = min(a.N, (part + 1) * part_n);
        for (int i = part * part_n + at; i < last; i += step) {
            int slot = -1;
            if (i < s.cnt) {
                const int pos = s.len + i, j = pos >> a.page_log2;
                const int page = j < s.held ? table[j] : fresh(j);
                if (page >= 0 && page < a.pages) slot = (page << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
            }
            slots[i] = slot;
        }
    };
    if (rows_wg == 1) {
        serve(mine[0], tid, kThreads);
    } else {
        for (int i = wave_id(); i < end - first; i += kWaves) serve(mine[i], lane, kWave);
    }

    // the ring's ends, and the pages held: in place by the last workgroup, which knows that the others have read them
    if (a.apart) {
        if (blockIdx.x != 0) return;
    } else {
        __syncthreads();
        if (tid == 0) ticket = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (ticket != gridDim.x - 1) return;
        if (tid == 0) __hip_atomic_store(a.done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    const unsigned w = wave_max_u32(taken);
    if (lane == 0) most[wave_id()] = w;
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < kWaves; ++i) taken = max(taken, most[i]);
        taken = max(taken, most[0]);
        a.out_state[0] = ring_ok ? static_cast<int>((head + taken) % a.pages) : head;
        a.out_state[1] = ring_ok ? static_cast<int>(free_pages - taken + base.drop) : free_pages;
    }
    if (a.apart) return;
    if (a.T <= kThreads) {
        if (tid < a.T) a.out_held[tid] = served ? n.need : n.held;
        return;
    }
    unsigned grown = 0;
    for (int t0 = 0; t0 < a.T; t0 += kThreads) {
        const int t = t0 + tid;
        n = Need{};
        if (t < a.T) n = read_need(a, t);
        n.ok = n.ok && ring_ok;
        Pair total;
        const Pair upto = block_inclusive({n.grow(), 0}, total, sh);
        if (t < a.T) a.out_held[t] = n.ok && (n.grow() == 0 || add(grown, upto.grow) <= supply) ? n.need : n.held;
        grown = add(grown, total.grow);
    }
}

}  // namespace

hipError_t launch_page_step(const PageStepArgs& a, hipStream_t s, Timing t) {
    // A wave a row, or a workgroup for one or for each 1024 tokens of it; about a thousand workgroups at most, since each reads all
    // rows (4096 rows of 8192 tokens in 32768 of them: 967 us, 52 so).
    const int parts = std::min((a.N + kPart - 1) / kPart, std::max(1, kMostWorkgroups / a.T));
    const int rows_wg = a.N > kPart && a.T <= kMostWorkgroups ? 1 : a.T <= 512 * kWaves ? kWaves : (a.T + 511) / 512;
    const int part_n = (a.N + parts - 1) / parts;
    const dim3 grid(static_cast<unsigned>((a.T + rows_wg - 1) / rows_wg) * parts);
    launch_timed(t, page_step_kernel, grid, dim3(kThreads), 0, s, a, rows_wg, parts, part_n);
    return hipGetLastError();
}

}  // namespace sv
