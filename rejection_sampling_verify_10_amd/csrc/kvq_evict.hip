// Eviction from the four-bit cache: each head keeps its `keep` best rows.
//
// Selection: one workgroup a (batch row, head) finds the keep-th largest 32-bit
// key (a protected slot has the largest one, then the scores in order, NaN last)
// by a radix select of 11, 11 and 10 bits -- the first digit holds the exponent
// and two bits more, so that scores of one magnitude already spread over several
// counters -- and takes ties in slot order.  Up to 32 slots a thread keep their
// keys in registers; longer heads read them again every pass (from L2).
//
// The plan moves as little as there is to move: kept rows below slot `keep` stay,
// and the i-th kept row above fills the i-th gap below.  No slot is both read and
// written, so the rows move in one parallel pass with no order between them; a
// handful is moved by the selecting workgroup itself.

#include "kvq.hpp"

namespace sv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kMoveThreads = 256;
constexpr int kBins = 2048;

// Order key of a score: larger first, NaN (0) after every number.
__device__ __forceinline__ uint32_t evict_key(float score, int pos, int sink, long from) {
    return pos < sink || pos >= from ? 0xffffffffu : order_key(score);
}

// Sum of a wave-uniform count over the waves before this one; `total` gets the sum over all.
__device__ __forceinline__ int waves_before(int v, int* sh, int& total) {
    const int wave = wave_id();
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == 0) sh[wave] = v;
    __syncthreads();
    int below = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
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

// Rows i0, i0 + step, .. of a head's plan: D/32 lanes a row of K and as many of V, 16 bytes of codes and one scale
// byte each.
template <int D>
__device__ __forceinline__ void move_rows(const KvqEvictArgs& a, int bh, int moves, int thread, int threads) {
    constexpr int kParts = D / 32;
    const int h = bh % a.c.H, b = bh / a.c.H;
    const int part = thread % kParts;
    const bool is_v = (thread / kParts) & 1;
    uint8_t* codes = (is_v ? a.c.vc : a.c.kc) + b * a.c.cb + h * a.c.ch + part * 16;
    uint8_t* scales = (is_v ? a.c.vs : a.c.ks) + b * a.c.sb + h * a.c.sh + part;
    const int32_t* plan = a.plan + static_cast<long>(bh) * a.gap_stride * 2;
    for (int i = thread / (2 * kParts); i < moves; i += threads / (2 * kParts)) {
        const long to = plan[2 * i], from = plan[2 * i + 1];
        const u32x4 w = *reinterpret_cast<const u32x4*>(codes + from * a.c.cp);
        const uint8_t s = scales[from * a.c.sp];
        *reinterpret_cast<u32x4*>(codes + to * a.c.cp) = w;
        scales[to * a.c.sp] = s;
    }
}

// K: slots a thread holds at most (0: any number, read again every time).
template <int D, int K, bool MOVE>
__global__ __launch_bounds__(kThreads) void kvq_select_kernel(KvqEvictArgs a) {
    const int bh = blockIdx.x, b = bh / a.c.H;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    const int len = a.lengths[b];
    int32_t* source = a.out_source + static_cast<long>(bh) * a.keep;
    const bool ok = len >= 0 && len <= a.c.capacity;
    const int kept = ok ? min(len, a.keep) : 0;
    if (bh % a.c.H == 0 && tid == 0) a.out_len[b] = ok ? kept : -1;
    if (!MOVE && tid == 0) a.moves[bh] = 0;
    for (int j = kept + tid; j < a.keep; j += kThreads) source[j] = -1;
    if (kept == 0) return;
    const long at = static_cast<long>(bh) * a.c.capacity;
    const float* sc = a.scores + at;
    const int32_t* pos = a.positions + at;
    float* osc = a.out_scores + at;
    int32_t* opos = a.out_positions + at;
    if (len == kept) {                                  // nothing to evict
        for (int s = tid; s < len; s += kThreads) {
            source[s] = s;
            if (osc != sc) {
                osc[s] = sc[s];
                opos[s] = pos[s];
            }
        }
        return;
    }
    const long from = static_cast<long>(a.seen[b]) - a.recent;
    int32_t* plan = a.plan + static_cast<long>(bh) * a.gap_stride * 2;

    __shared__ int hist[kBins];
    __shared__ int sh[kWaves], sh2[kWaves];
    __shared__ int sh_bin, sh_need, sh_count;

    // a wave's slots lie together: slot s0 + 64*e + lane, e < ne
    const int ne = (len + kThreads - 1) / kThreads;
    const int s0 = wave * ne * kWave + lane;
    const auto load = [&](int e) {
        const int s = s0 + e * kWave;
        return s < len ? evict_key(sc[s], pos[s], a.sink, from) : 0u;
    };
    uint32_t held[K > 0 ? K : 1];
    if (K > 0) {
#pragma unroll
        for (int e = 0; e < K; ++e) held[e] = e < ne ? load(e) : 0u;
    }
    const auto each = [&](auto&& f) {                   // f(e, key) for the thread's slots, in order
        if (K > 0) {
#pragma unroll
            for (int e = 0; e < (K > 0 ? K : 1); ++e)
                if (e < ne) f(e, held[e]);
        } else {
            for (int e = 0; e < ne; ++e) f(e, load(e));
        }
    };

    uint32_t edge = 0;                                  // the keep-th largest key
    int need = kept, equal = 0;                         // how many slots of that key are kept, and how many there are
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
        each([&](int e, uint32_t k) {
            const bool in = s0 + e * kWave < len && (pass == 0 || (k >> (shift + bits)) == edge);
            if (in) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
        });
        __syncthreads();
        // two counters a thread, from the largest digit down
        const int hi = kBins - 1 - 2 * tid, nh = hist[hi], nl = hist[hi - 1];
        int x = nh + nl;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const int y = __shfl_up(x, o, kWave);
            if (lane >= o) x += y;
        }
        int total;
        const int above = waves_before(bcast(x, kWave - 1), sh, total) + x - nh - nl;
        if (above < need && need <= above + nh + nl) {
            const bool low = need > above + nh;
            sh_bin = low ? hi - 1 : hi;
            sh_need = need - above - (low ? nh : 0);
            sh_count = low ? nl : nh;
        }
        __syncthreads();
        edge = (edge << bits) | static_cast<uint32_t>(sh_bin);
        need = sh_need;
        equal = sh_count;
    }

    // ties in slot order, where not all of them stay
    int tied = 0, total;
    if (need < equal) {
        int n = 0;
        each([&](int e, uint32_t k) { n += __popcll(__ballot(s0 + e * kWave < len && k == edge)); });
        tied = waves_before(n, sh, total);
    }
    const auto stays = [&](int s, uint32_t k, int& t) {
        const bool tie = s < len && k == edge;
        const unsigned long long m = __ballot(tie);
        const bool take = s < len && (k > edge || (tie && (need == equal || t + lanes_before(m) < need)));
        t += __popcll(m);
        return take;
    };
    int gaps = 0, movers = 0, t = tied;
    each([&](int e, uint32_t k) {
        const int s = s0 + e * kWave;
        const bool take = stays(s, k, t);
        gaps += __popcll(__ballot(s < kept && !take));
        movers += __popcll(__ballot(s >= kept && take));
    });
    int moves;
    gaps = waves_before(gaps, sh, moves);               // as many as there are movers
    movers = waves_before(movers, sh2, total);
    t = tied;
    each([&](int e, uint32_t k) {
        const int s = s0 + e * kWave;
        const bool take = stays(s, k, t);
        const bool gap = s < kept && !take, mover = s >= kept && take;
        const unsigned long long mg = __ballot(gap), mm = __ballot(mover);
        if (gap) plan[2 * (gaps + lanes_before(mg))] = s;
        if (mover) plan[2 * (movers + lanes_before(mm)) + 1] = s;
        gaps += __popcll(mg);
        movers += __popcll(mm);
        if (take && s < kept) {
            source[s] = s;
            if (osc != sc) {
                osc[s] = sc[s];
                opos[s] = pos[s];
            }
        }
    });
    __syncthreads();
    for (int i = tid; i < moves; i += kThreads) {
        const int to = plan[2 * i], s = plan[2 * i + 1];
        source[to] = s;
        osc[to] = sc[s];
        opos[to] = pos[s];
    }
    if (MOVE) move_rows<D>(a, bh, moves, tid, kThreads);
    else if (tid == 0) a.moves[bh] = moves;
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
    const int per = (a.c.capacity + kThreads - 1) / kThreads;
    if (fused) {
        if (per <= 4) launch_timed(t, kvq_select_kernel<D, 4, true>, grid, dim3(kThreads), 0, s, a);
        else if (per <= 32) launch_timed(t, kvq_select_kernel<D, 32, true>, grid, dim3(kThreads), 0, s, a);
        else launch_timed(t, kvq_select_kernel<D, 0, true>, grid, dim3(kThreads), 0, s, a);
        return;
    }
    if (per <= 4) launch_timed(t, kvq_select_kernel<64, 4, false>, grid, dim3(kThreads), 0, s, a);
    else if (per <= 32) launch_timed(t, kvq_select_kernel<64, 32, false>, grid, dim3(kThreads), 0, s, a);
    else launch_timed(t, kvq_select_kernel<64, 0, false>, grid, dim3(kThreads), 0, s, a);
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
