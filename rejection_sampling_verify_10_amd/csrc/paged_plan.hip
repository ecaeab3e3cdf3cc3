// How a step's attention is cut up, from the lengths on the GPU: once a step, for
// every layer.
//
// Consecutive batch rows with the same prefix are a run: all their query rows form
// one matrix against the prefix, in tiles of 128 (32, where there are no more), so
// each tile's keys are read once for all of them.  A batch row's own slots are met
// by its own query rows.  A job, one tile against its key axis, is cut into equal
// units; a unit is a workgroup for each head.  The size that no unit passes is the
// least for which the units of more than half of it find places at once, or a few
// steps above; the smaller ones fill the gaps, because units are launched the
// longest first (in 64 classes of length).  The tiles that read the same keys stay
// side by side.
//
// One workgroup, since everything goes by the sum over the batch.  Bound by latency:
// the rows' lengths and their prefixes' (two dependent loads), a dozen barriers, the
// stores: 9-11 us up to 1024 rows.  Units of several sizes are tried at once, two waves
// a size; reading the rows again for every size in turn took 18-27 us.

#include <algorithm>

#include "paged.hpp"

namespace sv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kClasses = kWave;         // of length, the longest first
constexpr int kSteps = 8;               // sizes of a unit that are tried, each a sixteenth above the one before

__device__ __forceinline__ unsigned wave_add(unsigned v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += xshfl(v, o);
    return v;
}
__device__ __forceinline__ unsigned wave_inclusive(unsigned v) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const unsigned t = __shfl_up(v, o, kWave);
        if (lane >= o) v += t;
    }
    return v;
}
// Sum over the block's threads below this one, and over all (fewer than 2^31 rows of parts).
__device__ __forceinline__ unsigned block_exclusive(unsigned v, unsigned& total, unsigned (&sh)[kWaves]) {
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    const unsigned i = wave_inclusive(v);
    __syncthreads();
    if (lane == kWave - 1) sh[wave] = i;
    __syncthreads();
    unsigned before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += sh[w];
        total += sh[w];
    }
    return before + i - v;
}

struct Row {                        // an error row: no new tokens, no prefix
    int pre, cnt, prefix, shared;   // own committed slots, new tokens, table row and slots of its prefix
    __device__ __forceinline__ int run() const { return shared > 0 && cnt > 0 ? prefix : -1; }
};
__device__ __forceinline__ Row read_row(const PagedPlanArgs& a, int b) {
    Row r;
    const long long capacity = static_cast<long long>(a.width) << a.page_log2;
    r.pre = a.lengths[b];
    r.cnt = a.counts ? a.counts[b] : a.N;
    r.prefix = a.prefix_row ? a.prefix_row[b] : -1;
    bool ok = r.pre >= 0 && r.cnt >= 0 && r.cnt <= a.N && static_cast<long long>(r.pre) + r.cnt <= capacity && r.prefix < a.T;
    r.shared = 0;
    if (r.prefix >= 0 && r.prefix < a.T) {
        r.shared = a.lengths[r.prefix];
        ok = ok && r.shared >= 0 && r.shared <= capacity;
    }
    if (!ok) r.pre = r.cnt = r.shared = 0;
    return r;
}
// Slots of its own that the i-th tile of a batch row's query rows looks at (windows that may have a mask: all of them).
__device__ __forceinline__ int own_limit(const PagedPlanArgs& a, const Row& r, int i) {
    if (a.own_tiles == 1) return r.cnt > 0 ? r.pre + r.cnt : 0;
    const int first = i * a.own_rows / a.G, last = (min((i + 1) * a.own_rows, a.M) - 1) / a.G;     // tokens
    if (first >= r.cnt) return 0;
    return r.pre + (a.N <= kPgMaskN ? r.cnt : min(last + 1, r.cnt));
}
__device__ __forceinline__ int chunks(int slots) { return (slots + kPgChunk - 1) / kPgChunk; }

// ceil(n / d) for n < 2^24: the float quotient is off by less than one.
__device__ __forceinline__ int ceil_div(int n, int d) {
    const int q = static_cast<int>(static_cast<float>(n) * __builtin_amdgcn_rcpf(static_cast<float>(d)));
    const int r = n - q * d;                            // -d < r < 2d
    return q + (r > 0 ? 1 : 0) + (r > d ? 1 : 0);
}
// A job of `n` chunks for units of at most `most`: its parts, and the chunks of each but the last. (Whether 128 query rows meet
// them or 32: the few take as long, waiting for memory.)
struct Cut {
    int parts, each;
    __device__ __forceinline__ Cut(int n, int most) {
        each = max(ceil_div(n, max(ceil_div(n, most), 1)), 1);
        parts = max(ceil_div(n, each), 1);
    }
};

struct Run {
    int b0, rows, prefix, shared, tile, tiles;  // tile: query rows of a unit
    int unit, part;                             // its first ones
};

__device__ __forceinline__ void write_unit(PagedUnit* to, const PagedUnit& u) {
    static_assert(sizeof(PagedUnit) == 48, "three vectors");
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    const i32x4 w[3] = {{u.b0, u.row0, u.rows, u.table}, {u.k0, u.k1, u.pre, u.cnt}, {u.part, u.wide, 0, 0}};
#pragma unroll
    for (int i = 0; i < 3; ++i) reinterpret_cast<i32x4*>(to)[i] = w[i];
}

__global__ __launch_bounds__(kThreads) void paged_plan_kernel(PagedPlanArgs a) {
    __shared__ unsigned sh[kWaves];
    __shared__ Row rows[kThreads];
    __shared__ Run run[kThreads + 1];
    __shared__ unsigned long long cost;                 // chunks of all jobs
    __shared__ unsigned large[kSteps];
    __shared__ int place[kClasses];                     // where the next unit of a class goes
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    if (tid == 0) cost = 0;
    if (tid < kSteps) large[tid] = 0;
    if (tid < kClasses) place[tid] = 0;

    // Batch rows are looked at 1024 at a time, a row a thread (a run ends there too); where there are no more, once.
    int runs = 0, mine = 0;                             // of these rows; this thread's row's
    const auto look = [&](int b0) {
        if (b0 > 0 || a.B > kThreads) __syncthreads();  // the rows before have been used
        const int b = b0 + tid;
        Row r = {0, 0, -1, 0};
        if (b < a.B) r = read_row(a, b);
        rows[tid] = r;
        __syncthreads();
        if (!a.prefix_row) return;
        const bool first = b < a.B && (tid == 0 || r.run() != rows[tid - 1].run());
        const unsigned long long leads = __ballot(first);
        if (lane == 0) sh[wave] = __popcll(leads);
        __syncthreads();
        unsigned before = 0, count = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) before += sh[w];
            count += sh[w];
        }
        runs = static_cast<int>(count);
        mine = static_cast<int>(before) + __popcll(leads & (~0ull >> (kWave - 1 - lane))) - 1;
        if (first) run[mine].b0 = b, run[mine].prefix = r.run(), run[mine].shared = r.run() >= 0 ? r.shared : 0;
        if (tid == 0) run[count].b0 = min(a.B, b0 + kThreads);
        __syncthreads();
        if (tid < runs) {
            Run& to = run[tid];
            to.rows = (run[tid + 1].b0 - to.b0) * a.M;
            to.tile = to.rows <= kPgNarrow ? kPgNarrow : kPgWide;
            to.tiles = to.shared > 0 ? (to.rows + to.tile - 1) / to.tile : 0;
        }
        __syncthreads();
    };
    const auto items = [&](int b0) { return (min(a.B, b0 + kThreads) - b0) * a.own_tiles; };
    // f(chunks, tiles) for every stride-th job among these rows (all tiles of a run are one)
    const auto each_job = [&](int b0, int from, int stride, const auto& f) {
        for (int k = from; k < runs; k += stride)
            if (run[k].tiles) f(chunks(run[k].shared), run[k].tiles);
        const int n = items(b0);
        for (int j = from; j < n; j += stride) {
            const int row = a.own_tiles == 1 ? j : j / a.own_tiles;
            f(chunks(own_limit(a, rows[row], j - row * a.own_tiles)), 1);
        }
    };
    const bool several = a.B > kThreads;
    look(0);

    // the chunks that no unit passes
    int most = 1 << 29;
    if (a.target > 0) {
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            if (b0 > 0) look(b0);
            unsigned long long sum = 0;                 // below 2^23 chunks * 2^19 tiles a job
            each_job(b0, tid, kThreads, [&](int n, int tiles) { sum += static_cast<unsigned long long>(n) * tiles; });
            const unsigned lo = wave_add(static_cast<unsigned>(sum) & 0xffffffu), hi = wave_add(static_cast<unsigned>(sum >> 24));
            if (lane == 0 && (lo | hi)) atomicAdd(&cost, (static_cast<unsigned long long>(hi) << 24) + lo);
        }
        __syncthreads();
        // (no job has more than 2^23 chunks)
        const int least = static_cast<int>(min(max((cost + a.target - 1) / a.target, 1ull), 1ull << 23));
        const auto raised = [](int m) { return m + m / 16 + 1; };
        // two waves a size
        const int step = wave % kSteps;
        int size = least;
        for (int i = 0; i < step; ++i) size = raised(size);
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            if (several) look(b0);
            unsigned sum = 0;
            each_job(b0, tid / (kWave * kSteps) * kWave + lane, kThreads / kSteps, [&](int n, int tiles) {
                const Cut c(n, size);
                if (2 * c.each > size) sum += static_cast<unsigned>(c.parts * tiles);
            });
            sum = wave_add(sum);
            if (lane == 0 && sum) atomicAdd(&large[step], sum);
        }
        __syncthreads();
        most = least;
        for (int i = 0; i < kSteps && large[i] > static_cast<unsigned>(a.target); ++i) most = raised(most);
    }
    const int finest = (most + kClasses - 1) / kClasses;
    const auto class_of = [&](int each) { return max(kClasses - 1 - each / finest, 0); };
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        if (several) look(b0);
        each_job(b0, tid, kThreads, [&](int n, int tiles) {
            const Cut c(n, most);
            atomicAdd(&place[class_of(c.each)], c.parts * tiles);
        });
    }
    __syncthreads();
    if (wave == 0) {
        static_assert(kClasses == kWave, "a class a lane");
        const int n = place[lane], upto = static_cast<int>(wave_inclusive(static_cast<unsigned>(n)));
        place[lane] = upto - n;
        if (lane == kWave - 1) {
            a.p.head[0] = upto;
            a.p.head[1] = a.B;
            a.p.head[2] = a.N;
            a.p.head[3] = a.M;
            a.p.head[4] = a.shape;
            a.p.head[5] = a.width << a.page_log2;
        }
    }
    __syncthreads();

    unsigned parts = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        if (several) look(b0);
        const int b = b0 + tid;
        if (a.prefix_row) {
            Run r{};
            if (tid < runs) r = run[tid];
            const Cut c(chunks(r.shared), most);
            unsigned total;
            const unsigned p = block_exclusive(static_cast<unsigned>(r.tiles * c.parts * r.tile), total, sh);
            if (r.tiles) {
                run[tid].part = static_cast<int>(parts + p);
                run[tid].unit = atomicAdd(&place[class_of(c.each)], c.parts * r.tiles);
            }
            parts += total;
            __syncthreads();
            for (int k = wave; k < runs; k += kWaves) {
                const Run r = run[k];
                if (!r.tiles) continue;
                const Cut c(chunks(r.shared), most);
                const int step = c.each * kPgChunk;
                for (int i = lane; i < c.parts * r.tiles; i += kWave) {
                    const int s = i / r.tiles, tile = i - s * r.tiles;
                    PagedUnit w{};
                    w.b0 = r.b0;
                    w.row0 = tile * r.tile;
                    w.rows = r.rows;
                    w.table = r.prefix;
                    w.k0 = s * step;
                    w.k1 = s == c.parts - 1 ? r.shared : w.k0 + step;
                    w.pre = r.shared;
                    w.part = r.part + i * r.tile;
                    w.wide = r.tile == kPgWide;
                    write_unit(a.p.unit + r.unit + i, w);
                }
            }
        }
        if (b < a.B) {
            PagedShared sd = {0, 0, 0, rows[tid].cnt};
            if (a.prefix_row && run[mine].tiles) {
                const Run& r = run[mine];
                sd.first = r.part + (b - r.b0) * a.M;
                sd.step = r.tiles * r.tile;
                sd.count = Cut(chunks(r.shared), most).parts;
            }
            a.p.shared[b] = sd;
        }
        const int n = items(b0);
        for (int j0 = 0; j0 < n; j0 += kThreads) {
            const int j = j0 + tid, row = a.own_tiles == 1 ? j : j / a.own_tiles, i = j - row * a.own_tiles;
            Row r = {0, 0, -1, 0};
            int limit = 0;
            if (j < n) {
                r = rows[row];
                limit = own_limit(a, r, i);
            }
            const Cut c(chunks(limit), most);
            const int step = c.each * kPgChunk;
            const bool joined = j < n && (c.parts > 1 || r.run() >= 0);
            unsigned total;
            const unsigned p = parts + block_exclusive(joined ? static_cast<unsigned>(c.parts * a.own_rows) : 0u, total, sh);
            parts += total;
            if (j >= n) continue;
            a.p.own[static_cast<long long>(b0) * a.own_tiles + j] = PagedOwn{static_cast<int>(p), joined ? c.parts : 0};
            const int u = atomicAdd(&place[class_of(c.each)], c.parts);
            for (int s = 0; s < c.parts; ++s) {
                PagedUnit w{};
                w.b0 = b0 + row;
                w.row0 = i * a.own_rows;
                w.rows = a.M;
                w.table = b0 + row;
                w.k0 = s * step;
                w.k1 = s == c.parts - 1 ? limit : w.k0 + step;
                w.pre = r.pre;
                w.cnt = r.cnt;
                w.part = joined ? static_cast<int>(p) + s * a.own_rows : -1;
                w.wide = a.own_rows == kPgWide;
                write_unit(a.p.unit + u + s, w);
            }
        }
    }
}

}  // namespace

// The key axes are split into about as many workgroups as run at once, two a compute unit, or one where a tile of D = 256 takes
// most of its LDS (44 rows of 7 tokens behind 800 keys, D = 256: 36 us in 512 of them, 32 in 256). A batch whose own rows alone
// are as many is not split, unless there are prefixes: no workspace, a plan of 6-9 us and not 9-13, units in no order of length.
// For rows much alike that is as good (8 heads, D = 128, 8 queries a head, one token: 64 rows of 4096 keys 174 us, 177 split; 256 of
// 512..2048 233 and 225; 1024 of 256..1024 481 and 485); one much longer than the rest is not (131072 keys among 63 rows of 500: 1358 us,
// 123 split), and a caller who has such gives prefix rows of -1.
void paged_plan_sizes(PagedPlanArgs& a) {
    a.own_rows = a.M <= kPgNarrow ? kPgNarrow : kPgWide;
    a.own_tiles = (a.M + a.own_rows - 1) / a.own_rows;
    const long long own = static_cast<long long>(a.B) * a.own_tiles;
    const int workgroups = a.D == 256 ? 256 : 512;
    const long long target = (workgroups + a.heads - 1) / a.heads;
    a.shape = 4 * a.heads + 2 * (a.D == 256) + (a.prefix_row ? 1 : 0);
    a.target = a.prefix_row || own < target ? static_cast<int>(target) : 0;
    // Every job is a unit, and the split makes fewer than `target` more. The tiles of a run are no more than those of its batch rows by
    // themselves; their query rows, filled up, are the most for runs of one batch row, or of the fewest that need 128.
    const bool all_narrow = static_cast<long long>(a.B) * a.M <= kPgNarrow;
    const long long fewest = a.M <= kPgNarrow ? kPgNarrow / a.M + 1 : 1;
    long long shared = 0, tile = a.own_rows;
    if (a.prefix_row) {
        shared = a.M > kPgNarrow || all_narrow ? own * a.own_rows
                                               : std::max(own * kPgNarrow, (a.B * static_cast<long long>(kPgWide) + fewest - 1) / fewest);
        if (!all_narrow) tile = kPgWide;
    }
    a.max_units = own + (a.prefix_row ? own : 0) + a.target;
    a.max_parts = a.target ? own * a.own_rows + shared + a.target * tile : 0;
}

hipError_t launch_paged_plan(const PagedPlanArgs& a, hipStream_t s, Timing t) {
    launch_timed(t, paged_plan_kernel, dim3(1), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace sv
