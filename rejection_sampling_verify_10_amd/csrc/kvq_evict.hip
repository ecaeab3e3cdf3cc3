// Eviction from the four-bit cache: each head keeps its `keep` best rows.
//
// Selection: one workgroup a (batch row, head) finds the keep-th largest 32-bit
// key (a protected slot has the largest one, then the scores in order, NaN last)
// by a radix select of 11, 11 and 10 bits -- the first digit holds the exponent
// and two bits more, so that scores of one magnitude already spread over several
// counters -- and takes ties in slot order.  Up to 4096 slots a head keep their
// keys in the LDS of four waves, up to 36864 in that of sixteen; longer heads read
// them again every pass, from L2 (32768 slots of 64 heads: 52 us so, 31 kept).  In
// LDS and not in registers, because a loop over registers is unrolled, and code
// that runs once waits for its own instructions (36 us).
//
// The selection of 64 heads has 64 compute units busy, each with what a CU takes:
// of 31 us at 32768 slots, 11 read scores and positions and count first digits
// (LDS counters of one address take turns), 4 the second digits, 4 find what
// stays, 5 write the plan.
//
// The plan moves as little as there is to move: kept rows below slot `keep` stay,
// and the i-th kept row above fills the i-th gap below.  No slot is both read and
// written, so the rows move in one parallel pass with no order between them; a
// handful is moved by the selecting workgroup itself.  Rows of 64 bytes here and
// there, half a memory line each: 6148 rows of each of 64 heads, 107 MB, are 183
// MB of whole lines (by the byte counters) and take 37 us, 4.9 TB/s, the rate of
// a large copy.

#include <type_traits>

#include "kvq.hpp"

namespace sv {

namespace {

constexpr int kMoveThreads = 256;
constexpr int kBins = 2048;

// Order key of a score: larger first, NaN (0) after every number.
__device__ __forceinline__ uint32_t evict_key(float score, int pos, int sink, long from) {
    return pos < sink || pos >= from ? 0xffffffffu : order_key(score);
}

// Sum of a wave-uniform count over the waves before this one; `total` gets the sum over all.
template <int WAVES, typename N>
__device__ __forceinline__ N waves_before(N v, N* sh, N& total) {
    const int wave = wave_id();
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == 0) sh[wave] = v;
    __syncthreads();
    N below = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const N s = sh[w];
        below += w < wave ? s : 0;
        total += s;
    }
    return below;
}
__device__ __forceinline__ int lanes_before(unsigned long long m) {
    return __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(m >> 32),
                                     __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(m), 0));
}

// Whether the lane's bit of a wave-uniform mask is set.
__device__ __forceinline__ bool in_ballot(unsigned long long m) {
#if SV_KVQ_DEVICE
    return __builtin_amdgcn_inverse_ballot_w64(m);
#else
    return false;
#endif
}

// A head's plan carried out: D/32 lanes a row of K and as many of V, 16 bytes of codes each; one of them moves the
// scales, another the row's score, position and source.
template <int D, int TURNS>
__device__ __forceinline__ void move_rows(const KvqEvictArgs& a, int bh, int moves, int thread, int threads) {
    constexpr int kParts = D / 32;
    using Scales = std::conditional_t<D == 64, uint16_t, std::conditional_t<D == 128, uint32_t, u32x2>>;
    const int h = bh % a.c.H, b = bh / a.c.H;
    const int part = thread % kParts;
    const bool is_v = (thread / kParts) & 1;
    uint8_t* codes = (is_v ? a.c.vc : a.c.kc) + b * a.c.cb + h * a.c.ch + part * 16;
    uint8_t* scales = (is_v ? a.c.vs : a.c.ks) + b * a.c.sb + h * a.c.sh;
    const int32_t* plan = a.plan + static_cast<long>(bh) * a.gap_stride * 2;
    const long at = static_cast<long>(bh) * a.c.capacity;
    const int step = threads / (2 * kParts);
    for (int i = thread / (2 * kParts); i < moves; i += TURNS * step) {
        long to[TURNS], from[TURNS];
        u32x4 row[TURNS];
        Scales scale[TURNS];
        float score[TURNS];
        int32_t position[TURNS];
#pragma unroll
        for (int u = 0; u < TURNS; ++u) {
            const int j = min(i + u * step, moves - 1);
            to[u] = plan[2 * j], from[u] = plan[2 * j + 1];
        }
#pragma unroll
        for (int u = 0; u < TURNS; ++u) row[u] = *reinterpret_cast<const u32x4*>(codes + from[u] * a.c.cp);
        if (part == 0) {
#pragma unroll
            for (int u = 0; u < TURNS; ++u) scale[u] = *reinterpret_cast<const Scales*>(scales + from[u] * a.c.sp);
        }
        if (part == 1 && !is_v) {
#pragma unroll
            for (int u = 0; u < TURNS; ++u) {
                score[u] = a.scores[at + from[u]];
                position[u] = a.positions[at + from[u]];
            }
        }
#pragma unroll
        for (int u = 0; u < TURNS; ++u) {
            if (i + u * step >= moves) break;
            *reinterpret_cast<u32x4*>(codes + to[u] * a.c.cp) = row[u];
            if (part == 0) *reinterpret_cast<Scales*>(scales + to[u] * a.c.sp) = scale[u];
            if (part == 1 && !is_v) {
                a.out_source[static_cast<long>(bh) * a.keep + to[u]] = static_cast<int32_t>(from[u]);
                a.out_scores[at + to[u]] = score[u];
                a.out_positions[at + to[u]] = position[u];
            }
        }
    }
}

// T threads; K: slots a thread holds at most (0: any number, read again every time).
template <int D, int T, int K, bool MOVE>
__global__ __launch_bounds__(T) void kvq_select_kernel(KvqEvictArgs a) {
    const int bh = blockIdx.x, b = bh / a.c.H;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    constexpr int kWaves = T / kWave;
    const int len = a.lengths[b], seen = a.seen[b];
    __shared__ int hist[kBins];
    if (K > 0) {
        for (int i = tid; i < kBins; i += T) hist[i] = 0;
    }
    int32_t* source = a.out_source + static_cast<long>(bh) * a.keep;
    const bool ok = len >= 0 && len <= a.c.capacity;
    const int kept = ok ? min(len, a.keep) : 0;
    if (bh % a.c.H == 0 && tid == 0) a.out_len[b] = ok ? kept : -1;
    if (!MOVE && tid == 0) a.moves[bh] = 0;
    for (int j = kept + tid; j < a.keep; j += T) source[j] = -1;
    if (kept == 0) return;
    const long at = static_cast<long>(bh) * a.c.capacity;
    const float* sc = a.scores + at;
    const int32_t* pos = a.positions + at;
    float* osc = a.out_scores + at;
    int32_t* opos = a.out_positions + at;
    // every kept slot as if nothing moved (the gaps are written over at the end): here, or as the keys are read
    const bool apart = osc != sc || opos != pos;
    for (int j0 = K == 0 || len == kept ? tid : kept; j0 < kept; j0 += 4 * T) {
        float x[4];
        int p[4];
        if (apart) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = min(j0 + u * T, kept - 1);
                x[u] = sc[j];
                p[u] = pos[j];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + u * T;
            if (j >= kept) break;
            source[j] = j;
            if (apart) {
                osc[j] = x[u];
                opos[j] = p[u];
            }
        }
    }
    if (len == kept) return;                            // nothing to evict
    const long from = static_cast<long>(seen) - a.recent;
    int32_t* plan = a.plan + static_cast<long>(bh) * a.gap_stride * 2;

    __shared__ int sh[kWaves];
    __shared__ long sh_both[kWaves];
    __shared__ int sh_bin, sh_need, sh_count;

    // a wave's slots lie together: slot s0 + 64*e + lane, e < ne
    const int ne = (len + T - 1) / T;
    const int w0 = wave * ne * kWave, s0 = w0 + lane;
    // eight slots side by side (the last slot's again past the end)
    constexpr int kBatch = 8;
    const auto fetch = [&](int e0, float (&x)[kBatch], int32_t (&p)[kBatch]) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int s = min(s0 + (e0 + u) * kWave, len - 1);
            x[u] = sc[s];
            p[u] = pos[s];
        }
    };
    const int left = len - s0;                          // slot s0 + 64*e is one if 64*e < left
    // f(e, x, p, keys) for the thread's slots from e = `first`, eight at a time, the next eight under way
    const auto stream = [&](int first, int last, auto&& f) {
        float x[2][kBatch];
        int32_t p[2][kBatch];
        uint32_t k[kBatch];
        fetch(first, x[0], p[0]);
        for (int e0 = first; e0 < last; e0 += 2 * kBatch) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = e0 + h * kBatch;
                fetch(at + kBatch, x[h ^ 1], p[h ^ 1]);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) k[u] = evict_key(x[h][u], p[h][u], a.sink, from);
                f(at, x[h], p[h], k);
            }
        }
    };
    static_assert(K % 4 == 0 && K <= kWave, "held slots are read four at a time, and what stays of them is a lane's row each");
    __shared__ uint32_t held[K > 0 ? K * T : 1];
    if (K > 0) {                                        // their first digits are counted as they come
        __syncthreads();
        stream(0, ne, [&](int at, const float (&x)[kBatch], const int32_t (&p)[kBatch], const uint32_t (&k)[kBatch]) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int s = s0 + (at + u) * kWave;
                if (s >= len || at + u >= ne) break;
                held[s] = k[u];
                atomicAdd(&hist[k[u] >> 21], 1);
                if (s >= kept) continue;
                source[s] = s;
                if (apart) {
                    osc[s] = x[u];
                    opos[s] = p[u];
                }
            }
        });
    }
    // f(e, key) for the thread's slots from `first` to before `last`, in order
    const auto each = [&](int first, int last, auto&& f) {
        if (K > 0) {
            for (int e0 = first; e0 < last; e0 += 4) {
                uint32_t k[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) k[u] = held[s0 + (e0 + u) * kWave];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (e0 + u < last) f(e0 + u, k[u]);
            }
        } else {
            stream(first, last, [&](int at, const float (&)[kBatch], const int32_t (&)[kBatch], const uint32_t (&k)[kBatch]) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (at + u < last) f(at + u, k[u]);
            });
        }
    };

    // digits of the keep-th largest key, until all slots that share them are kept (or all its digits are known)
    uint32_t edge = 0;
    int need = kept, equal = len, low = 32;             // slots of those digits that are kept, that there are; bits left
    while (need < equal && low > 0) {
        const int bits = low == 10 ? 10 : 11, shift = low - bits;
        if (K == 0 || low < 32) {
            for (int i = tid; i < kBins; i += T) hist[i] = 0;
            __syncthreads();
            each(0, ne, [&](int e, uint32_t k) {
                const bool in = e * kWave < left && (low == 32 || (k >> low) == edge);
                if (in) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
            });
        }
        __syncthreads();
        // some counters a thread, from the largest digit down
        constexpr int kMine = kBins / T;
        const int first = kBins - 1 - kMine * tid;
        int n[kMine], mine = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) mine += n[i] = hist[first - i];
        const int x = wave_scan_int(mine);
        int total;
        int above = waves_before<kWaves>(bcast(x, kWave - 1), sh, total) + x - mine;
        if (above < need && need <= above + mine) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                if (above < need && need <= above + n[i]) {
                    sh_bin = first - i;
                    sh_need = need - above;
                    sh_count = n[i];
                }
                above += n[i];
            }
        }
        __syncthreads();
        edge = (edge << bits) | static_cast<uint32_t>(sh_bin);
        need = sh_need;
        equal = sh_count;
        low = shift;
    }

    // ties in slot order, where not all of them stay
    int tied = 0, total;
    if (need < equal) {
        int n = 0;
        each(0, ne, [&](int e, uint32_t k) { n += __popcll(__ballot(e * kWave < left && k >> low == edge)); });
        tied = waves_before<kWaves>(n, sh, total);
    }
    // which of 64 rows of the wave's slots stay: lane i gets row e0 + i's, bit l for lane l's slot
    const uint32_t least = edge << low;
    const auto staying = [&](int e0, int& t) {
        unsigned long long mine = 0;
        const auto put = [&](int e, unsigned long long m) { mine = lane == e - e0 ? m : mine; };
        const int last = min(ne, e0 + kWave);
        if (need == equal) {
            each(e0, last, [&](int e, uint32_t k) { put(e, __ballot(e * kWave < left) & __ballot(k >= least)); });
        } else {
            each(e0, last, [&](int e, uint32_t k) {
                const unsigned long long in = __ballot(e * kWave < left), tie = in & __ballot(k >> low == edge);
                put(e, (in & __ballot(k >= least)) & ~(tie & __ballot(t + lanes_before(tie) >= need)));
                t += __popcll(tie);
            });
        }
        return mine;
    };
    // of those, what does not stay below slot `kept` leaves a gap, and what stays above it moves
    const auto split = [&](int e0, unsigned long long m, unsigned long long& gap, unsigned long long& mover) {
        const int n = kept - (w0 + (e0 + lane) * kWave);
        const unsigned long long below = n >= kWave ? ~0ull : n > 0 ? (1ull << n) - 1 : 0;
        gap = e0 + lane < ne ? ~m & below : 0;
        mover = m & ~below;
    };
    unsigned long long mine, gap, mover;
    int gaps = 0, movers = 0, t = tied;
    for (int e0 = 0; e0 < ne; e0 += kWave) {            // one turn where the keys are held
        mine = staying(e0, t);
        split(e0, mine, gap, mover);
        gaps += __popcll(gap);
        movers += __popcll(mover);
    }
    // as many gaps as movers
    const long both = static_cast<long>(bcast(wave_scan_int(movers), kWave - 1)) << 32 | bcast(wave_scan_int(gaps), kWave - 1);
    long sum;
    const long before = waves_before<kWaves>(both, sh_both, sum);
    gaps = static_cast<int>(before);
    movers = static_cast<int>(before >> 32);
    const int moves = static_cast<int>(sum);
    t = tied;
    for (int e0 = 0; e0 < ne; e0 += kWave) {
        if (K == 0) {
            mine = staying(e0, t);
            split(e0, mine, gap, mover);
        }
        const int mine_gaps = __popcll(gap), mine_movers = __popcll(mover);
        const int gap_at = gaps + wave_scan_int(mine_gaps), mover_at = movers + wave_scan_int(mine_movers);
        // its 64 rows' slots one row after the other, in slot order
        const auto write = [&](unsigned long long m, int from_at, int field) {
            for (int i = 0; i < min(ne - e0, kWave); ++i) {
                const unsigned long long row = static_cast<unsigned>(bcast(static_cast<int>(m), i)) |
                                               static_cast<unsigned long long>(bcast(static_cast<int>(m >> 32), i)) << 32;
                if (row == 0) continue;
                if (in_ballot(row))
                    plan[2u * (bcast(from_at, i) + lanes_before(row)) + field] = w0 + (e0 + i) * kWave + lane;
            }
        };
        write(gap, gap_at - mine_gaps, 0);
        write(mover, mover_at - mine_movers, 1);
        gaps = bcast(gap_at, kWave - 1);
        movers = bcast(mover_at, kWave - 1);
    }
    if (!MOVE) {
        if (tid == 0) a.moves[bh] = moves;
        return;
    }
    __syncthreads();
    move_rows<D, 1>(a, bh, moves, tid, T);
}

template <int D>
__global__ __launch_bounds__(kMoveThreads) void kvq_move_kernel(KvqEvictArgs a, int wgs) {
    const int bh = blockIdx.x / wgs, part = blockIdx.x % wgs;
    move_rows<D, 4>(a, bh, a.moves[bh], part * kMoveThreads + threadIdx.x, wgs * kMoveThreads);
}

template <int D> void evict(const KvqEvictArgs& a, hipStream_t s, Timing t) {
    const dim3 grid(a.c.B * a.c.H);
    // few moves (a step's rows against a budget) are not worth a second launch (2048 slots kept of 128 heads: 2304 of
    // them 15 us in one, 12 + 5 in two; 2560 of them 20, 13 + 5)
    const bool fused = a.gap_stride <= 256;
    // four waves a head where they hold its slots: 2054 of 512 heads 13 us, with sixteen 24.  By the capacity, as the host
    // knows no lengths: those 2054 rows are 19 us in a cache of 4096 slots (a second launch), 30 in 8192 to 32768, 55 in
    // 65536
    const auto select = [&](auto small, auto large, auto any) {
        if (a.c.capacity <= 256 * 16) launch_timed(t, small, grid, dim3(256), 0, s, a);
        else if (a.c.capacity <= 1024 * 36) launch_timed(t, large, grid, dim3(1024), 0, s, a);
        else launch_timed(t, any, grid, dim3(1024), 0, s, a);
    };
    if (fused) {
        select(kvq_select_kernel<D, 256, 16, true>, kvq_select_kernel<D, 1024, 36, true>,
               kvq_select_kernel<D, 1024, 0, true>);
        return;
    }
    select(kvq_select_kernel<64, 256, 16, false>, kvq_select_kernel<64, 1024, 36, false>,
           kvq_select_kernel<64, 1024, 0, false>);
    constexpr int rows = kMoveThreads / (2 * (D / 32));
    int wgs = (a.gap_stride + rows - 1) / rows;         // rows of a head side by side, four turns a thread at most
    wgs = (wgs + 3) / 4;
    kvq_move_kernel<D><<<dim3(static_cast<unsigned>(wgs) * a.c.B * a.c.H), kMoveThreads, 0, s>>>(a, wgs);
}

}  // namespace

hipError_t launch_kvq_evict(const KvqEvictArgs& a, hipStream_t s, Timing t) {
    if (a.c.D == 64) evict<64>(a, s, t);
    else if (a.c.D == 128) evict<128>(a, s, t);
    else evict<256>(a, s, t);
    return hipGetLastError();
}

}  // namespace sv
