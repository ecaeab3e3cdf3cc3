// Eviction from the four-bit cache: each head keeps its `keep` best rows.
//
// Selection: one workgroup a (batch row, head) finds the keep-th largest 32-bit
// key (a protected slot has the largest one, then the scores in order, NaN last)
// by a radix select of 11, 11 and 10 bits -- the first digit holds the exponent
// and two bits more, so that scores of one magnitude already spread over several
// counters -- and takes ties in slot order.  Up to 4096 slots a head keep their
// keys in the registers of four waves, up to 49152 in those of sixteen; longer
// heads read them again every pass (from L2).
//
// The plan moves as little as there is to move: kept rows below slot `keep` stay,
// and the i-th kept row above fills the i-th gap below.  No slot is both read and
// written, so the rows move in one parallel pass with no order between them; a
// handful is moved by the selecting workgroup itself.

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
template <int WAVES>
__device__ __forceinline__ int waves_before(int v, int* sh, int& total) {
    const int wave = wave_id();
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == 0) sh[wave] = v;
    __syncthreads();
    int below = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const int s = sh[w];
        below += w < wave ? s : 0;
        total += s;
    }
    return below;
}
__device__ __forceinline__ int lanes_before(unsigned long long m) {
    return __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(m >> 32),
                                     __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(m), 0));
}

// A head's plan carried out: D/32 lanes a row of K and as many of V, 16 bytes of codes each; one of them moves the
// scales, another the row's score, position and source.
template <int D>
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
    for (int i = thread / (2 * kParts); i < moves; i += threads / (2 * kParts)) {
        const long to = plan[2 * i], from = plan[2 * i + 1];
        *reinterpret_cast<u32x4*>(codes + to * a.c.cp) = *reinterpret_cast<const u32x4*>(codes + from * a.c.cp);
        if (part == 0)
            *reinterpret_cast<Scales*>(scales + to * a.c.sp) = *reinterpret_cast<const Scales*>(scales + from * a.c.sp);
        if (part == 1 && !is_v) {
            a.out_source[static_cast<long>(bh) * a.keep + to] = static_cast<int32_t>(from);
            a.out_scores[at + to] = a.scores[at + from];
            a.out_positions[at + to] = a.positions[at + from];
        }
    }
}

// T threads; K: slots a thread holds at most (0: any number, read again every time).
template <int D, int T, int K, bool MOVE>
__global__ __launch_bounds__(T) void kvq_select_kernel(KvqEvictArgs a) {
    const int bh = blockIdx.x, b = bh / a.c.H;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    constexpr int kWaves = T / kWave;
    const int len = a.lengths[b];
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
    // every kept slot as if nothing moved; the gaps are written over at the end
    const bool apart = osc != sc || opos != pos;
    for (int j0 = tid; j0 < kept; j0 += 4 * T) {
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
    const long from = static_cast<long>(a.seen[b]) - a.recent;
    int32_t* plan = a.plan + static_cast<long>(bh) * a.gap_stride * 2;

    __shared__ int hist[kBins];
    __shared__ int sh[kWaves], sh2[kWaves];
    __shared__ int sh_bin, sh_need, sh_count;

    // a wave's slots lie together: slot s0 + 64*e + lane, e < ne
    const int ne = (len + T - 1) / T;
    const int s0 = wave * ne * kWave + lane;
    // eight slots' keys, their loads side by side (the last slot's again past the end)
    constexpr int kBatch = 8;
    const auto load = [&](int e0, uint32_t (&k)[kBatch]) {
        float x[kBatch];
        int p[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int s = min(s0 + (e0 + u) * kWave, len - 1);
            x[u] = sc[s];
            p[u] = pos[s];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) k[u] = evict_key(x[u], p[u], a.sink, from);
    };
    uint32_t held[K > 0 ? K / kBatch : 1][kBatch];
    if (K > 0) {
#pragma unroll
        for (int e0 = 0; e0 < K; e0 += kBatch)
            if (e0 < ne) load(e0, held[e0 / kBatch]);
    }
    const auto each = [&](auto&& f) {                   // f(e, key) for the thread's slots, in order
        if (K > 0) {
#pragma unroll
            for (int e = 0; e < (K > 0 ? K : 1); ++e)
                if (e < ne) f(e, held[e / kBatch][e % kBatch]);
        } else {
            uint32_t k[2][kBatch];
            load(0, k[0]);
            for (int e0 = 0; e0 < ne; e0 += 2 * kBatch) {
                load(e0 + kBatch, k[1]);
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (e0 + u < ne) f(e0 + u, k[0][u]);
                load(e0 + 2 * kBatch, k[0]);
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (e0 + kBatch + u < ne) f(e0 + kBatch + u, k[1][u]);
            }
        }
    };

    // digits of the keep-th largest key, until all slots that share them are kept (or all its digits are known)
    uint32_t edge = 0;
    int need = kept, equal = len, low = 32;             // slots of those digits that are kept, that there are; bits left
    while (need < equal && low > 0) {
        const int bits = low == 10 ? 10 : 11, shift = low - bits;
        for (int i = tid; i < kBins; i += T) hist[i] = 0;
        __syncthreads();
        each([&](int e, uint32_t k) {
            const bool in = s0 + e * kWave < len && (low == 32 || (k >> low) == edge);
            if (in) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
        });
        __syncthreads();
        // some counters a thread, from the largest digit down
        constexpr int kMine = kBins / T;
        const int first = kBins - 1 - kMine * tid;
        int n[kMine], mine = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) mine += n[i] = hist[first - i];
        int x = mine;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const int y = __shfl_up(x, o, kWave);
            if (lane >= o) x += y;
        }
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
        each([&](int e, uint32_t k) { n += __popcll(__ballot(s0 + e * kWave < len && k >> low == edge)); });
        tied = waves_before<kWaves>(n, sh, total);
    }
    const auto stays = [&](int s, uint32_t k, int& t) {
        if (need == equal) return s < len && k >> low >= edge;
        const bool tie = s < len && k >> low == edge;
        const unsigned long long m = __ballot(tie);
        const bool take = s < len && (k >> low > edge || (tie && t + lanes_before(m) < need));
        t += __popcll(m);
        return take;
    };
    // a wave's slots are all below `kept`, where what does not stay leaves a gap, or all above, where what stays moves
    // (the wave across it looks for both)
    const int w0 = wave * ne * kWave;
    const bool low_side = w0 < kept, high_side = w0 + ne * kWave > kept;
    int gaps = 0, movers = 0, t = tied;
    each([&](int e, uint32_t k) {
        const int s = s0 + e * kWave;
        const bool take = stays(s, k, t);
        if (low_side) gaps += __popcll(__ballot(s < kept && !take));
        if (high_side) movers += __popcll(__ballot(s >= kept && take));
    });
    int moves;
    gaps = waves_before<kWaves>(gaps, sh, moves);       // as many as there are movers
    movers = waves_before<kWaves>(movers, sh2, total);
    t = tied;
    each([&](int e, uint32_t k) {
        const int s = s0 + e * kWave;
        const bool take = stays(s, k, t);
        if (low_side) {
            const unsigned long long m = __ballot(s < kept && !take);
            if (s < kept && !take) plan[2 * (gaps + lanes_before(m))] = s;
            gaps += __popcll(m);
        }
        if (high_side) {
            const unsigned long long m = __ballot(s >= kept && take);
            if (s >= kept && take) plan[2 * (movers + lanes_before(m)) + 1] = s;
            movers += __popcll(m);
        }
    });
    if (!MOVE) {
        if (tid == 0) a.moves[bh] = moves;
        return;
    }
    __syncthreads();
    move_rows<D>(a, bh, moves, tid, T);
}

template <int D>
__global__ __launch_bounds__(kMoveThreads) void kvq_move_kernel(KvqEvictArgs a, int wgs) {
    const int bh = blockIdx.x / wgs, part = blockIdx.x % wgs;
    move_rows<D>(a, bh, a.moves[bh], part * kMoveThreads + threadIdx.x, wgs * kMoveThreads);
}

template <int D> void evict(const KvqEvictArgs& a, hipStream_t s, Timing t) {
    const dim3 grid(a.c.B * a.c.H);
    // few moves (a step's rows against a budget) are not worth a second launch
    const bool fused = a.gap_stride <= 256;
    const auto select = [&](auto small, auto large, auto any) {
        if (a.c.capacity <= 256 * 16) launch_timed(t, small, grid, dim3(256), 0, s, a);
        else if (a.c.capacity <= 1024 * 48) launch_timed(t, large, grid, dim3(1024), 0, s, a);
        else launch_timed(t, any, grid, dim3(1024), 0, s, a);
    };
    if (fused) {
        select(kvq_select_kernel<D, 256, 16, true>, kvq_select_kernel<D, 1024, 48, true>,
               kvq_select_kernel<D, 1024, 0, true>);
        return;
    }
    select(kvq_select_kernel<64, 256, 16, false>, kvq_select_kernel<64, 1024, 48, false>,
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
