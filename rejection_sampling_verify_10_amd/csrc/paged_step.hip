// Pages for a step: how many each sequence needs, taken from the head of a ring of
// free pages in the order of the sequences, given back at its tail; and the slots
// of the step's tokens.
//
// Every workgroup sums the whole batch's needs for itself (three small arrays, from
// the L2) and then serves its own sequences, so nothing passes between workgroups
// and one launch does.  The arrays a call reads may be the ones it writes, so what
// others still read (pages held, the ring's ends) is written by the last workgroup
// that has read them.  Taken pages lie between the ring's head and its tail, pages
// given back behind the tail: no entry is both read and written.

#include "paged.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kPart = 1024;         // tokens of a row that a workgroup finds the slots of

struct Need {
    int len, cnt, held, need;
    bool ok;                        // the row's numbers make sense and fit its table
    __device__ __forceinline__ int grow() const { return ok ? max(need - held, 0) : 0; }
    __device__ __forceinline__ int drop() const { return ok ? max(held - need, 0) : 0; }
};
__device__ __forceinline__ Need read_need(const PageStepArgs& a, int t) {
    Need n;
    n.len = a.lengths[t];
    n.cnt = a.counts ? a.counts[t] : a.N;
    n.held = a.held[t];
    const bool live = n.len >= 0;
    const long long end = live ? static_cast<long long>(n.len) + n.cnt : 0;
    const long long need = (end + (1 << a.page_log2) - 1) >> a.page_log2;
    n.ok = n.held >= 0 && n.held <= a.width && (!live || (n.cnt >= 0 && n.cnt <= a.N)) && need <= a.width;
    n.need = n.ok ? static_cast<int>(need) : 0;
    if (!live) n.cnt = 0;
    return n;
}

// Exclusive sums over the block's threads, and their totals.
struct Pair {
    long long grow, drop;
};
__device__ __forceinline__ long long shift_up(long long v, int o) { return __shfl_up(v, o, kWave); }
__device__ __forceinline__ Pair block_exclusive(Pair v, Pair& total, Pair (&sh)[kWaves]) {
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    Pair i = v;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const long long g = shift_up(i.grow, o), d = shift_up(i.drop, o);
        if (lane >= o) i.grow += g, i.drop += d;
    }
    __syncthreads();
    if (lane == kWave - 1) sh[wave] = i;
    __syncthreads();
    Pair before = {0, 0};
    total = {0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before.grow += sh[w].grow, before.drop += sh[w].drop;
        total.grow += sh[w].grow, total.drop += sh[w].drop;
    }
    return {before.grow + i.grow - v.grow, before.drop + i.drop - v.drop};
}

struct Served {                     // a row of this workgroup's, in LDS
    int len, cnt, held, need, row;  // cnt -1: not served
    int take, give;                 // places in the ring of its first new page, and of the first one it gives back
};
// x mod pages for x below twice as many.
__device__ __forceinline__ int wrap(unsigned x, int pages) {
    return static_cast<int>(x >= static_cast<unsigned>(pages) ? x - pages : x);
}

__global__ __launch_bounds__(kThreads) void page_step_kernel(PageStepArgs a, int rows_wg, int parts) {
    __shared__ Pair sh[kWaves];
    __shared__ Served mine[kThreads];
    __shared__ unsigned ticket;
    const int tid = threadIdx.x;
    const int part = blockIdx.x % parts;
    const int first = blockIdx.x / parts * rows_wg, end = min(a.T, first + rows_wg);
    const int head = a.state[0], free_pages = a.state[1];
    const bool ring_ok = head >= 0 && head < a.pages && free_pages >= 0 && free_pages <= a.pages;
    const long long supply = ring_ok ? free_pages : 0;

    Pair base = {0, 0};
    long long taken = 0;            // pages of the rows that are served: they are the first ones
    for (int t0 = 0; t0 < a.T; t0 += kThreads) {
        const int t = t0 + tid;
        Need n{};
        if (t < a.T) n = read_need(a, t);
        n.ok = n.ok && ring_ok;
        Pair total, at = block_exclusive({t < a.T ? n.grow() : 0, t < a.T ? n.drop() : 0}, total, sh);
        at.grow += base.grow, at.drop += base.drop;
        const bool served = n.ok && (n.grow() == 0 || at.grow + n.grow() <= supply);
        if (t >= first && t < end) {
            Served s;
            s.len = n.len, s.cnt = served ? n.cnt : -1, s.held = n.held, s.need = served ? n.need : n.held;
            s.take = served ? static_cast<int>((head + at.grow) % a.pages) : 0;
            s.give = served ? static_cast<int>((head + supply + at.drop) % a.pages) : 0;
            s.row = t;
            mine[t - first] = s;
            if (part == 0) a.out_granted[t] = s.cnt;
        }
        base.grow += total.grow, base.drop += total.drop;
        // a row that grows is served while the sum up to it fits, so the last sum that fits is what is taken
        const long long fits = t < a.T && served && n.grow() > 0 ? at.grow + n.grow() : 0;
        long long most = fits;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const long long other = __shfl_xor(most, o, kWave);
            most = other > most ? other : most;
        }
        __syncthreads();
        if ((tid & (kWave - 1)) == 0) sh[wave_id()].grow = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) taken = sh[w].grow > taken ? sh[w].grow : taken;
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
        const int last = min(a.N, (part + 1) * kPart);
        for (int n = part * kPart + at; n < last; n += step) {
            int slot = -1;
            if (n < s.cnt) {
                const int pos = s.len + n, j = pos >> a.page_log2;
                const int page = j < s.held ? table[j] : fresh(j);
                if (page >= 0 && page < a.pages) slot = (page << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
            }
            slots[n] = slot;
        }
    };
    if (rows_wg == 1) {
        serve(mine[0], tid, kThreads);
    } else {
        for (int i = wave_id(); i < end - first; i += kWaves) serve(mine[i], tid & (kWave - 1), kWave);
    }

    // the last workgroup writes what the others read
    __syncthreads();
    if (tid == 0) ticket = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (ticket != gridDim.x - 1) return;
    if (tid == 0) {
        __hip_atomic_store(a.done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        a.out_state[0] = ring_ok ? static_cast<int>((head + taken) % a.pages) : head;
        a.out_state[1] = ring_ok ? static_cast<int>(free_pages - taken + base.drop) : free_pages;
    }
    Pair sum = {0, 0};
    for (int t0 = 0; t0 < a.T; t0 += kThreads) {
        const int t = t0 + tid;
        Need n{};
        if (t < a.T) n = read_need(a, t);
        n.ok = n.ok && ring_ok;
        Pair total, at = block_exclusive({t < a.T ? n.grow() : 0, 0}, total, sh);
        const bool served = n.ok && (n.grow() == 0 || sum.grow + at.grow + n.grow() <= supply);
        if (t < a.T) a.out_held[t] = served ? n.need : n.held;
        sum.grow += total.grow;
    }
}

}  // namespace

hipError_t launch_page_step(const PageStepArgs& a, hipStream_t s, Timing t) {
    // a workgroup a row up to 256 of them, and one for each 1024 tokens of it
    const int rows_wg = (a.T + 255) / 256, parts = (a.N + kPart - 1) / kPart;
    const dim3 grid(static_cast<unsigned>((a.T + rows_wg - 1) / rows_wg) * parts);
    launch_timed(t, page_step_kernel, grid, dim3(kThreads), 0, s, a, rows_wg, parts);
    return hipGetLastError();
}

}  // namespace sv
