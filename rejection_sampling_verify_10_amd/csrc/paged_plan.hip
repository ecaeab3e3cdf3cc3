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

#include "paged.hpp"

namespace sv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kClasses = kWave;         // of length, the longest first
constexpr int kSteps = 8;               // sizes of a unit that are tried, each a sixteenth above the one before

// Sum over the block's threads below this one, and over all.
__device__ __forceinline__ long long block_exclusive(long long v, long long& total, long long (&sh)[kWaves]) {
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    long long i = v;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const long long t = __shfl_up(i, o, kWave);
        if (lane >= o) i += t;
    }
    __syncthreads();
    if (lane == kWave - 1) sh[wave] = i;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += sh[w];
        total += sh[w];
    }
    return before + i - v;
}

struct Row {
    int pre, cnt, prefix, shared;   // own committed slots, new tokens, table row and slots of its prefix
    bool ok;
};
__device__ __forceinline__ Row read_row(const PagedPlanArgs& a, int b) {
    Row r;
    const long long capacity = static_cast<long long>(a.width) << a.page_log2;
    r.pre = a.lengths[b];
    r.cnt = a.counts ? a.counts[b] : a.N;
    r.prefix = a.prefix_row ? a.prefix_row[b] : -1;
    r.ok = r.pre >= 0 && r.cnt >= 0 && r.cnt <= a.N && static_cast<long long>(r.pre) + r.cnt <= capacity && r.prefix < a.T;
    r.shared = 0;
    if (r.prefix >= 0 && r.prefix < a.T) {
        r.shared = a.lengths[r.prefix];
        r.ok = r.ok && r.shared >= 0 && r.shared <= capacity;
    }
    if (!r.ok) r.pre = r.cnt = r.shared = 0;
    return r;
}
// Slots of its own that the i-th tile of a batch row's query rows looks at (windows that may have a mask: all of them).
__device__ __forceinline__ int own_limit(const PagedPlanArgs& a, const Row& r, int i) {
    const int first = i * a.own_rows / a.G, last = (min((i + 1) * a.own_rows, a.M) - 1) / a.G;     // tokens
    if (!r.ok || first >= r.cnt) return 0;
    return r.pre + (a.N <= kPgMaskN ? r.cnt : min(last + 1, r.cnt));
}
__device__ __forceinline__ int chunks(int slots) { return (slots + kPgChunk - 1) / kPgChunk; }

// A job of `n` chunks for units of at most `most`: its parts, and the chunks of each but the last. (Whether 128 query rows meet
// them or 32: the few take as long, waiting for memory.)
struct Cut {
    int parts, each;
    __device__ __forceinline__ Cut(int n, int most) {
        parts = max((n + most - 1) / most, 1);
        each = max((n + parts - 1) / parts, 1);
        parts = max((n + each - 1) / each, 1);
    }
};

struct Run {
    int b0, rows, prefix, shared, tile, tiles;  // tile: query rows of a unit
};

__global__ __launch_bounds__(kThreads) void paged_plan_kernel(PagedPlanArgs a) {
    __shared__ long long sh[kWaves];
    __shared__ int lead[kThreads + 1];
    __shared__ Run run[kThreads];
    __shared__ long long run_part[kThreads];
    __shared__ int place[kClasses];                     // where the next unit of a class goes
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    const long long items = static_cast<long long>(a.B) * a.own_tiles;

    // The runs among batch rows b0 .. b0 + 1023 (a run ends there too): thread t has the t-th; their number.
    const auto runs = [&](int b0, Run& mine) {
        const int b = b0 + tid;
        Row r{};
        if (b < a.B) r = read_row(a, b);
        const int here = r.ok && r.shared > 0 && r.cnt > 0 ? r.prefix : -1;
        int before = __shfl_up(here, 1, kWave);
        __syncthreads();
        if (lane == kWave - 1) sh[wave] = here;
        __syncthreads();
        if (lane == 0) before = wave > 0 ? static_cast<int>(sh[wave - 1]) : -2;
        const bool first = b < a.B && here != before;
        long long count;
        const int rank = static_cast<int>(block_exclusive(first ? 1 : 0, count, sh));
        if (first) {
            lead[rank] = b;
            run[rank].prefix = here;
            run[rank].shared = r.shared;
        }
        if (tid == 0) lead[count] = min(a.B, b0 + kThreads);
        __syncthreads();
        mine = Run{};
        if (tid < count) {
            mine.b0 = lead[tid];
            mine.prefix = run[tid].prefix;
            mine.shared = mine.prefix >= 0 ? run[tid].shared : 0;
            mine.rows = (lead[tid + 1] - lead[tid]) * a.M;
            mine.tile = mine.rows <= kPgNarrow ? kPgNarrow : kPgWide;
            mine.tiles = mine.shared > 0 ? (mine.rows + mine.tile - 1) / mine.tile : 0;
        }
        __syncthreads();
        return static_cast<int>(count);
    };

    // f(chunks, tiles) for each job (or all tiles of a run at once)
    const auto each_job = [&](const auto& f) {
        for (int b0 = 0; a.prefix_row && b0 < a.B; b0 += kThreads) {
            Run r;
            runs(b0, r);
            if (r.tiles) f(chunks(r.shared), r.tiles);
        }
        for (long long j = tid; j < items; j += kThreads)
            f(chunks(own_limit(a, read_row(a, static_cast<int>(j / a.own_tiles)), static_cast<int>(j % a.own_tiles))), 1);
    };
    // the chunks that no unit passes
    int most = 1 << 29;
    if (a.target > 0) {
        long long cost = 0;
        each_job([&](int n, int tiles) { cost += static_cast<long long>(n) * tiles; });
        long long total;
        block_exclusive(cost, total, sh);
        most = static_cast<int>(max((total + a.target - 1) / a.target, 1ll));
        for (int step = 0; step < kSteps; ++step) {
            long long large = 0;
            each_job([&](int n, int tiles) {
                const Cut c(n, most);
                if (2 * c.each > most) large += static_cast<long long>(c.parts) * tiles;
            });
            block_exclusive(large, total, sh);
            if (total <= a.target) break;
            most += most / 16 + 1;
        }
    }
    const int finest = (most + kClasses - 1) / kClasses;
    const auto class_of = [&](int each) { return max(kClasses - 1 - each / finest, 0); };
    if (tid < kClasses) place[tid] = 0;
    __syncthreads();
    each_job([&](int n, int tiles) {
        const Cut c(n, most);
        atomicAdd(&place[class_of(c.each)], c.parts * tiles);
    });
    __syncthreads();
    if (wave == 0) {
        static_assert(kClasses == kWave, "a class a lane");
        const int n = place[lane];
        int before = n;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const int t = __shfl_up(before, o, kWave);
            if (lane >= o) before += t;
        }
        place[lane] = before - n;
        if (lane == kWave - 1) {
            a.p.head[0] = before;
            a.p.head[1] = a.B;
            a.p.head[2] = a.N;
            a.p.head[3] = a.M;
            a.p.head[4] = a.prefix_row != nullptr;
            a.p.head[5] = a.width << a.page_log2;
            a.p.head[6] = a.heads;
        }
    }
    __syncthreads();

    long long parts = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        if (b < a.B) {
            const Row r = read_row(a, b);
            a.p.shared[b] = PagedShared{0, 0, 0, r.ok ? r.cnt : 0};
        }
        if (!a.prefix_row) continue;
        Run mine;
        const int count = runs(b0, mine);
        const Cut cut(chunks(mine.shared), most);
        long long part_total;
        const long long p = block_exclusive(static_cast<long long>(mine.tiles) * cut.parts * mine.tile, part_total, sh);
        if (tid < count) run[tid] = mine, run_part[tid] = parts + p;
        __syncthreads();
        for (int k = wave; k < count; k += kWaves) {
            const Run r = run[k];
            if (!r.tiles) continue;
            const Cut c(chunks(r.shared), most);
            const int n = c.parts, step = c.each * kPgChunk;
            int u = 0;
            if (lane == 0) u = atomicAdd(&place[class_of(c.each)], n * r.tiles);
            u = __builtin_amdgcn_readfirstlane(u);
            for (int i = lane; i < n * r.tiles; i += kWave) {
                const int s = i / r.tiles, tile = i % r.tiles;
                PagedUnit w{};
                w.b0 = r.b0;
                w.row0 = tile * r.tile;
                w.rows = r.rows;
                w.table = r.prefix;
                w.k0 = s * step;
                w.k1 = s == n - 1 ? r.shared : w.k0 + step;
                w.pre = r.shared;
                w.part = static_cast<int>(run_part[k] + static_cast<long long>(i) * r.tile);
                w.wide = r.tile == kPgWide;
                a.p.unit[u + i] = w;
            }
            for (int row = lane; row < r.rows / a.M; row += kWave) {
                PagedShared* at = a.p.shared + r.b0 + row;
                at->first = static_cast<int>(run_part[k]) + row * a.M;
                at->step = r.tiles * r.tile;
                at->count = n;
            }
        }
        parts += part_total;
        __syncthreads();
    }
    for (long long j0 = 0; j0 < items; j0 += kThreads) {
        const long long j = j0 + tid;
        const int b = static_cast<int>(j / a.own_tiles), i = static_cast<int>(j % a.own_tiles);
        Row r{};
        int limit = 0;
        if (j < items) {
            r = read_row(a, b);
            limit = own_limit(a, r, i);
        }
        const Cut c(chunks(limit), most);
        const int n = c.parts, step = c.each * kPgChunk;
        const bool joined = j < items && (n > 1 || (r.shared > 0 && r.cnt > 0));
        long long part_total;
        const long long p = parts + block_exclusive(joined ? static_cast<long long>(n) * a.own_rows : 0, part_total, sh);
        if (j < items) {
            a.p.own[j] = PagedOwn{static_cast<int>(p), joined ? n : 0};
            const int u = atomicAdd(&place[class_of(c.each)], n);
            for (int s = 0; s < n; ++s) {
                PagedUnit w{};
                w.b0 = b;
                w.row0 = i * a.own_rows;
                w.rows = a.M;
                w.table = b;
                w.k0 = n > 1 ? s * step : 0;
                w.k1 = s == n - 1 ? limit : w.k0 + step;
                w.pre = r.pre;
                w.cnt = r.cnt;
                w.part = joined ? static_cast<int>(p) + s * a.own_rows : -1;
                w.wide = a.own_rows == kPgWide;
                a.p.unit[u + s] = w;
            }
        }
        parts += part_total;
    }
}

}  // namespace

// The key axes are split into about 512 workgroups (two a compute unit); a batch whose own rows alone are as many is not
// split, unless there are prefixes.
void paged_plan_sizes(PagedPlanArgs& a) {
    a.own_rows = a.M <= kPgNarrow ? kPgNarrow : kPgWide;
    a.own_tiles = (a.M + a.own_rows - 1) / a.own_rows;
    const long long own = static_cast<long long>(a.B) * a.own_tiles;
    const long long target = (512 + a.heads - 1) / a.heads;
    a.target = a.prefix_row || own < target ? static_cast<int>(target) : 0;
    // a unit more than the split for each job; a run's rows come to one tile more than fit
    const long long rows = static_cast<long long>(a.B) * a.M;
    const long long shared = a.prefix_row ? rows / kPgWide + a.B : 0;
    a.max_units = own + shared + a.target;
    a.max_parts = a.target ? (own + a.target) * a.own_rows + (a.prefix_row ? (shared + a.target) * kPgWide : 0) : 0;
}

hipError_t launch_paged_plan(const PagedPlanArgs& a, hipStream_t s, Timing t) {
    launch_timed(t, paged_plan_kernel, dim3(1), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace sv
