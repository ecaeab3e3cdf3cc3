// Eviction from the four-bit cache: each head keeps its `keep` best rows.
//
// Selection: one workgroup a (batch row, head) finds the keep-th largest 32-bit
// key (a protected slot has the largest one, then the scores in order, NaN last)
// by a radix select, eight bits a pass, and takes ties in slot order.  The plan
// moves as little as there is to move: kept rows below slot `keep` stay, and the
// i-th kept row above fills the i-th gap below.  No slot is both read and
// written, so the rows move in one parallel pass with no order between them.

#include "kvq.hpp"

namespace sv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kMoveThreads = 256;

// Order key of a score: larger first, NaN (0) after every number.
__device__ __forceinline__ uint32_t evict_key(float score, int pos, int sink, long from) {
    return pos < sink || pos >= from ? 0xffffffffu : order_key(score);
}

// Exclusive prefix of a count over the workgroup; `total` gets the sum.
__device__ __forceinline__ int block_prefix(int v, int* sh, int& total) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    int x = v;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int y = __shfl_up(x, o, kWave);
        if (lane >= o) x += y;
    }
    if (lane == kWave - 1) sh[wave] = x;
    __syncthreads();
    int below = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int s = sh[w];
        below += w < wave ? s : 0;
        total += s;
    }
    __syncthreads();
    return below + x - v;
}

__global__ __launch_bounds__(kThreads) void kvq_select_kernel(KvqEvictArgs a) {
    const int bh = blockIdx.x, b = bh / a.c.H;
    const int tid = threadIdx.x;
    const int len = a.lengths[b];
    int32_t* source = a.out_source + static_cast<long>(bh) * a.keep;
    const bool ok = len >= 0 && len <= a.c.capacity;
    const int kept = ok ? min(len, a.keep) : 0;
    if (bh % a.c.H == 0 && tid == 0) a.out_len[b] = ok ? kept : -1;
    for (int j = kept + tid; j < a.keep; j += kThreads) source[j] = -1;
    if (kept == 0) return;
    const long at = static_cast<long>(bh) * a.c.capacity;
    const float* sc = a.scores + at;
    const int32_t* pos = a.positions + at;
    float* osc = a.out_scores + at;
    int32_t* opos = a.out_positions + at;
    int32_t* gaps = a.gaps + static_cast<long>(bh) * a.gap_stride;
    const long from = static_cast<long>(a.seen[b]) - a.recent;

    __shared__ int hist[256];
    __shared__ int sh[kWaves];
    __shared__ uint32_t sh_prefix;
    __shared__ int sh_need;
    uint32_t edge = 0;                                  // the keep-th largest key
    int ties = 0;                                       // how many slots of that key are kept
    if (len > kept) {
        uint32_t prefix = 0;
        int need = kept;
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int s = tid; s < len; s += kThreads) {
                const uint32_t k = evict_key(sc[s], pos[s], a.sink, from);
                if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int left = need, v = 255;
                while (left > hist[v]) left -= hist[v--];
                sh_prefix = (prefix << 8) | static_cast<uint32_t>(v);
                sh_need = left;
            }
            __syncthreads();
            prefix = sh_prefix;
            need = sh_need;
        }
        edge = prefix;
        ties = need;
    }
    // slots in order: gaps below `kept` are listed, then filled by the kept slots above
    int tied = 0, gap = 0, moved = 0;                   // so far
    for (int s0 = 0; s0 < len; s0 += kThreads) {
        const int s = s0 + tid;
        const bool in = s < len;
        uint32_t k = 0;
        float score = 0.f;
        int p = 0;
        if (in) {
            score = sc[s];
            p = pos[s];
            k = evict_key(score, p, a.sink, from);
        }
        bool take = in && len > kept ? k > edge : in;
        int total;
        if (len > kept) {
            const int rank = block_prefix(in && k == edge ? 1 : 0, sh, total);
            if (in && k == edge && tied + rank < ties) take = true;
            tied += total;
        }
        const bool hole = in && s < kept && !take;
        const int hr = block_prefix(hole ? 1 : 0, sh, total);
        if (hole) gaps[gap + hr] = s;
        gap += total;
        const bool mover = take && s >= kept;
        const int mr = block_prefix(mover ? 1 : 0, sh, total);   // its barriers order the gaps before their readers
        if (mover) {
            const int to = gaps[moved + mr];
            source[to] = s;
            osc[to] = score;
            opos[to] = p;
        }
        moved += total;
        if (take && s < kept) {
            source[s] = s;
            if (osc != sc) {
                osc[s] = score;
                opos[s] = p;
            }
        }
    }
}

// Moves the rows of the plan: D/32 lanes a row of K and as many of V, 16 bytes of codes and one scale byte each.
template <int D>
__global__ __launch_bounds__(kMoveThreads) void kvq_move_kernel(KvqEvictArgs a) {
    constexpr int kParts = D / 32;
    const long i = static_cast<long>(blockIdx.x) * kMoveThreads + threadIdx.x;
    const int part = static_cast<int>(i % kParts);
    const bool is_v = (i / kParts) & 1;
    const long row = i / (2 * kParts);
    if (row >= static_cast<long>(a.c.B) * a.c.H * a.keep) return;
    const int to = static_cast<int>(row % a.keep);
    const int from = a.out_source[row];
    if (from < 0 || from == to) return;
    const int bh = static_cast<int>(row / a.keep), h = bh % a.c.H, b = bh / a.c.H;
    uint8_t* codes = (is_v ? a.c.vc : a.c.kc) + b * a.c.cb + h * a.c.ch + part * 16;
    uint8_t* scales = (is_v ? a.c.vs : a.c.ks) + b * a.c.sb + h * a.c.sh + part;
    const u32x4 w = *reinterpret_cast<const u32x4*>(codes + from * a.c.cp);
    const uint8_t s = scales[from * a.c.sp];
    *reinterpret_cast<u32x4*>(codes + to * a.c.cp) = w;
    scales[to * a.c.sp] = s;
}

template <int D> void move(const KvqEvictArgs& a, hipStream_t s) {
    const long lanes = static_cast<long>(a.c.B) * a.c.H * a.keep * (2 * (D / 32));
    kvq_move_kernel<D><<<dim3(static_cast<unsigned>((lanes + kMoveThreads - 1) / kMoveThreads)), kMoveThreads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_kvq_evict(const KvqEvictArgs& a, hipStream_t s, Timing t) {
    launch_timed(t, kvq_select_kernel, dim3(a.c.B * a.c.H), dim3(kThreads), 0, s, a);
    if (a.c.D == 64) move<64>(a, s);
    else if (a.c.D == 128) move<128>(a, s);
    else move<256>(a, s);
    return hipGetLastError();
}

}  // namespace sv
