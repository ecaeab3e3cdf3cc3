// Accumulated attention weight of the cached rows (what an eviction goes by).
//
// w_s = sum over the accepted queries and the G query heads of a cache head of
// exp2(c * (q . K_s) - lse * log2(e)), c = scale * log2(e): the softmax's
// statistics are known, so one product with the K codes gives the weights, half
// of attention's reads.  Every slot's sum is one workgroup's, in a fixed order, so
// no atomics and the same bits every time.  Operands are laid out as in attention
// (16x16x32 bf16 MFMAs, lane (c, g) with c = lane % 16, g = lane / 16).
//
// A wave streams keys, S = Q K^T, 32 a step, against query rows 16 a tile: lane
// (c, g) gets rows 4g + i against key c, so a key's sum is over registers and two
// exchanges.  A tree's path has a handful of rows, kept in registers: bound by the
// K codes.  More rows are kept in LDS, a lot of them at a time, for the eight
// waves of a workgroup.  A prompt has thousands, bound by the exponentials, and
// too few keys to fill the GPU: there the rows are split over workgroups as well,
// whose sums meet in the workspace.
//
// 32 batch rows of 8 heads at ragged lengths to 4096 (27-node trees, paths of up
// to 6 nodes): 17.5-18 us a call for 52 MB, 2.9 TB/s; a workgroup's few steps hardly
// cover the latency of its first loads.  2048 tokens x 4 heads against their own
// 2048 keys, 8 heads: 46 us for 17 GFLOP, 374 TFLOP/s: the vector units are busy
// 32% of the cycles and the matrix units 15%, the rest waits between short steps
// that each need the one before (LDS, product, exponential).

#include "kvq.hpp"

namespace sv {

namespace {

// Eight float32 values as NQ bf16 operands whose sum they are.
template <int NQ, typename F> __device__ __forceinline__ void bf16_parts(float (&x)[8], F&& put) {
#pragma unroll
    for (int p = 0; p < NQ; ++p) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
            x[2 * e] -= bf16_lo(w[e]);
            x[2 * e + 1] -= bf16_hi(w[e]);
        }
        put(p, w);
    }
}

constexpr int kKeyWaves = 4;                            // waves of a workgroup that streams keys

// The weight of a slot: added to a committed one's score, the score of one this step added.
__device__ __forceinline__ void put_weight(const KvqScoreArgs& a, int b, int h, int pre, int slot, float x, float old) {
    const long at = (static_cast<long>(b) * a.c.H + h) * a.c.capacity + slot;
    a.scores[at] = slot >= pre ? x : old + x;
    if (slot >= pre) a.positions[at] = a.seen[b] + (slot - pre);
}

// What a wave that streams keys works with: two tiles of 16 keys a step, read ahead through buffer descriptors that
// end at the last slot, and the scores its lanes add to.
template <int D> struct KeyStream {
    const uint8_t *kc, *ks;
    float* scores;
    long cp, sp;
    uint32_t ko, kso;
    int all, mine;                                      // slots; this lane's slot of a step's 32 (lanes of g < 2 write)
    uint32_t k[2][D / 32], s[2];
    float old;
    __device__ __forceinline__ KeyStream(const KvqScoreArgs& a, int b, int h, int all, int lane) : all(all) {
        const int c = lane & 15, g = lane >> 4;
        kc = a.c.kc + b * a.c.cb + h * a.c.ch;
        ks = a.c.ks + b * a.c.sb + h * a.c.sh;
        scores = a.scores + (static_cast<long>(b) * a.c.H + h) * a.c.capacity;
        cp = a.c.cp;
        sp = a.c.sp;
        ko = k_offset(D, c, g, static_cast<int>(cp));
        kso = k_scale_offset(D, c, g, static_cast<int>(sp));
        mine = (g & 1) * 16 + c;
    }
    __device__ __forceinline__ void load(int kb) {
        old = scores[min(kb + mine, all - 1)];
        load_k_step<D>(kc, ks, cp, sp, kb, all, ko, kso, k, s);
    }
    __device__ __forceinline__ u32x4 operand(int t, int x) const {
        const float sc = scale_value(D == 256 && x >= 4 ? s[t] >> 8 : s[t]);
        const uint32_t w = k[t][x];
        return u32x4{fp4_pair<0>(w, sc), fp4_pair<1>(w, sc), fp4_pair<2>(w, sc), fp4_pair<3>(w, sc)};
    }
};

// The accepted tokens of a batch row.
struct Accepted {
    int pre, d, all, node;                              // node: lane t holds path[t] of a tree
    __device__ __forceinline__ bool read(const KvqScoreArgs& a, int b) {
        const int lane = threadIdx.x & (kWave - 1);
        pre = a.prefix[b];
        d = a.accept_len[b];
        all = pre + d + 1;                              // slots after the commit
        return !(d < 0 || d >= a.N || d >= a.path_stride || pre < 0 || static_cast<long>(pre) + d + 1 > a.c.capacity) &&
               (node = lane, true);
    }
    __device__ __forceinline__ bool read_path(const KvqScoreArgs& a, int b) {
        if (!a.path) return true;
        const int lane = threadIdx.x & (kWave - 1);
        node = lane < a.path_stride ? a.path[static_cast<long>(b) * a.path_stride + lane] : 0;
        const int before = __shfl_up(node, 1, kWave);
        return __ballot(lane <= d && (lane == 0 ? node != 0 : (node <= before || node >= a.N))) == 0ull;
    }
};

// One query row as loaded for an operand (elements 32g' .. of its lane's quarter) with its lse in base 2 and token.
template <int D, int DT, int NQ>
__device__ __forceinline__ void load_row(const KvqScoreArgs& a, const Accepted& ac, int b, int h, int row, int rows,
                                         int g, u32x4 (&q)[NQ][D / 32], float& lse, int& tok) {
    const int r = row < rows ? row : 0;
    const int t = r / a.G;
    const int tk = a.path ? __shfl(ac.node, t, kWave) : t;
    const int hq = h * a.G + (r - t * a.G);
    const char* p = static_cast<const char*>(a.q.data) +
                    (b * a.q.batch + tk * a.q.pos + hq * a.q.head + g * (D / 4)) * (DT == 1 ? 2 : 4);
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        if (DT == 1) {
            q[0][s] = reinterpret_cast<const u32x4*>(p)[s];
        } else {
            const f32x4 lo = reinterpret_cast<const f32x4*>(p)[2 * s], hi = reinterpret_cast<const f32x4*>(p)[2 * s + 1];
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = lo[e], x[4 + e] = hi[e];
            bf16_parts<NQ>(x, [&](int part, const u32x4& w) { q[part][s] = w; });
        }
    }
    const float lse2 = a.lse[(static_cast<long>(b) * a.N + tk) * a.Hq + hq] * 1.44269504089f;
    // a query that saw nothing, or a row past the last, weighs nothing
    lse = row < rows && lse2 != -INFINITY ? lse2 : INFINITY;
    tok = row < rows ? t : -1;
}

// Few rows: the queries stay in registers, the keys stream.
template <int D, int DT, int QT>
__global__ __launch_bounds__(kKeyWaves* kWave) void kvq_score_kernel(KvqScoreArgs a) {
    constexpr int NQ = DT == 1 ? 1 : 3;
    const int h = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & (kWave - 1), c = lane & 15, g = lane >> 4;
    Accepted ac;
    if (!ac.read(a, b)) return;
    const int pre = ac.pre, all = ac.all;
    const int stride = static_cast<int>(gridDim.x) * kKeyWaves * 32;
    int kb = (static_cast<int>(blockIdx.x) * kKeyWaves + wave_id()) * 32;
    if (kb >= all) return;
    KeyStream<D> cur(a, b, h, all, lane);
    cur.load(kb);
    if (!ac.read_path(a, b)) return;
    const int rows = (ac.d + 1) * a.G;
    u32x4 Q[QT][NQ][D / 32];
    float lse[QT][4];
    int tok[QT][4];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        // lane (c, g) loads a quarter of row 16*qt + c, and keeps the lse and tokens of rows 16*qt + 4g + i
        float l;
        int t;
        load_row<D, DT, NQ>(a, ac, b, h, 16 * qt + c, rows, g, Q[qt], l, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lse[qt][i] = lane_gather(l, 4 * g + i);
            tok[qt][i] = static_cast<int>(lane_gather(static_cast<uint32_t>(t), 4 * g + i));
        }
    }
    for (; kb < all; kb += stride) {
        f32x4 S[2][QT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) S[t][qt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const u32x4 K = cur.operand(t, s);
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int p = 0; p < NQ; ++p) S[t][qt] = mfma(Q[qt][p][s], K, S[t][qt]);
            }
        }
        const float old = cur.old;
        cur.load(kb + stride);
        const bool part = kb + 31 > pre;                // some key is newer than the first token
        float x[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int key = kb + 16 * t + c - pre;
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p = __builtin_amdgcn_exp2f(fmaf(S[t][qt][i], a.cexp, -lse[qt][i]));
                    if (part) p = key <= tok[qt][i] ? p : 0.f;
                    x[t] += p;
                }
            }
            x[t] += xshfl(x[t], 16);
            x[t] += xshfl(x[t], 32);
        }
        const int slot = kb + cur.mine;
        if (g < 2 && slot < all) put_weight(a, b, h, pre, slot, g ? x[1] : x[0], old);
    }
}

// More rows: they stay in LDS, a lot of kRows at a time, and the keys stream once for each lot.
// (2048 tokens x 4 heads: 44 us; lots of half the rows 48, four or sixteen waves 50 and 45, 64 keys a wave and step 70.)
constexpr int kLdsWaves = 8;
constexpr int lds_rows(int D, int DT) { return 65536 / (2 * D * (DT == 1 ? 1 : 3)) / 16 * 16; }

template <int D, int DT>
__global__ __launch_bounds__(kLdsWaves* kWave) void kvq_score_lds_kernel(KvqScoreArgs a) {
    constexpr int NQ = DT == 1 ? 1 : 3, kRows = lds_rows(D, DT), kTiles = kRows / 16;
    __shared__ u32x4 sh_q[kTiles][NQ * (D / 32)][kWave];
    __shared__ f32x4 sh_lse[kRows / 4];
    __shared__ int sh_tok[kRows];
    // heads side by side in the grid, so that one XCD (every eighth workgroup) has one head's queries in its L2
    const int bhs = a.c.B * a.c.H, bh = blockIdx.x % bhs, turn = blockIdx.x / bhs;
    const int seg = turn / a.key_wgs, block = turn % a.key_wgs;
    const int h = bh % a.c.H, b = bh / a.c.H;
    const int lane = threadIdx.x & (kWave - 1), c = lane & 15, g = lane >> 4, wave = wave_id();
    Accepted ac;
    if (!ac.read(a, b)) return;
    const int pre = ac.pre, all = ac.all;
    const int stride = a.key_wgs * kLdsWaves * 32, first = block * kLdsWaves * 32;
    if (first >= all || !ac.read_path(a, b)) return;
    const int rows = (ac.d + 1) * a.G;
    // this segment's lots, as many for each segment as the row count needs
    const int lots = (rows + kRows - 1) / kRows, per = (lots + a.segs - 1) / a.segs;
    const int row0 = seg * per * kRows, row1 = min(row0 + per * kRows, rows);
    float* const part = a.part ? a.part + (static_cast<long>(seg) * bhs + bh) * a.c.capacity : nullptr;
    KeyStream<D> cur(a, b, h, all, lane);
    bool again = false;                                 // the keys' sums of an earlier lot are there already
    for (int lot = row0; lot < row1; lot += kRows) {
        if (first - pre > (min(lot + kRows, row1) - 1) / a.G) continue;     // all its tokens are older than the keys
        const int tiles = (min(row1 - lot, kRows) + 15) / 16;
        __syncthreads();
        for (int i = wave; i < tiles; i += kLdsWaves) {
            u32x4 q[NQ][D / 32];
            float l;
            int t;
            load_row<D, DT, NQ>(a, ac, b, h, lot + 16 * i + c, rows, g, q, l, t);
#pragma unroll
            for (int p = 0; p < NQ; ++p)
#pragma unroll
                for (int s = 0; s < D / 32; ++s) sh_q[i][p * (D / 32) + s][lane] = q[p][s];
            if (g == 0) {
                reinterpret_cast<float*>(sh_lse)[16 * i + c] = l;
                sh_tok[16 * i + c] = t;
            }
        }
        __syncthreads();
        int kb = first + wave * 32;
        if (kb < all) cur.load(kb);
        for (; kb < all; kb += stride) {
            u32x4 K[2][D / 32];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int s = 0; s < D / 32; ++s) K[t][s] = cur.operand(t, s);
            const int slot = kb + cur.mine;
            float old = cur.old;
            if (part) old = again && slot < all ? part[slot] : 0.f;
            cur.load(kb + stride);
            float x[2] = {0.f, 0.f};
            // from the first tile of the lot whose tokens see the keys
            const int from = kb > pre ? max(((kb - pre) * a.G - lot) / 16, 0) : 0;
            for (int i = from; i < tiles; ++i) {
                f32x4 S[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int s = 0; s < D / 32; ++s)
#pragma unroll
                    for (int p = 0; p < NQ; ++p) {
                        const u32x4 q = sh_q[i][p * (D / 32) + s][lane];
#pragma unroll
                        for (int t = 0; t < 2; ++t) S[t] = mfma(q, K[t][s], S[t]);
                    }
                const f32x4 lse = sh_lse[4 * i + g];
                // whether some key is newer than the tile's first token
                const bool edge = kb + 31 - pre > __builtin_amdgcn_readfirstlane(sh_tok[16 * i]);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int key = kb + 16 * t + c - pre;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float p = __builtin_amdgcn_exp2f(fmaf(S[t][e], a.cexp, -lse[e]));
                        if (edge) p = key <= sh_tok[16 * i + 4 * g + e] ? p : 0.f;
                        x[t] += p;
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                x[t] += xshfl(x[t], 16);
                x[t] += xshfl(x[t], 32);
            }
            if (g < 2 && slot < all) {
                const float w = g ? x[1] : x[0];
                if (part) part[slot] = old + w;
                else if (again) cur.scores[slot] = old + w;
                else put_weight(a, b, h, pre, slot, w, old);
            }
        }
        again = true;
    }
    if (!part || again) return;
    for (int kb = first; kb < all; kb += stride)        // every lot was older
        for (int slot = kb + static_cast<int>(threadIdx.x); slot < min(kb + kLdsWaves * 32, all); slot += kLdsWaves * kWave)
            part[slot] = 0.f;
}

// Adds up the segments' sums, in their order.
__global__ __launch_bounds__(256) void kvq_score_sum_kernel(KvqScoreArgs a, int lot_rows) {
    const int blocks = (a.c.capacity + 255) / 256;
    const int slot = static_cast<int>(blockIdx.x % blocks) * 256 + threadIdx.x, bh = blockIdx.x / blocks;
    const int h = bh % a.c.H, b = bh / a.c.H;
    Accepted ac;
    if (!ac.read(a, b) || !ac.read_path(a, b) || slot >= ac.all) return;
    const int lots = ((ac.d + 1) * a.G + lot_rows - 1) / lot_rows, per = (lots + a.segs - 1) / a.segs;
    const int used = (lots + per - 1) / per;            // segments that hold rows
    const long bhs = static_cast<long>(a.c.B) * a.c.H;
    float x = 0.f;
    for (int s = 0; s < used; ++s) x += a.part[(s * bhs + bh) * a.c.capacity + slot];
    put_weight(a, b, h, ac.pre, slot, x, a.scores[bh * static_cast<long>(a.c.capacity) + slot]);
}

template <int D, int DT, int QT> void stream_keys(const KvqScoreArgs& a, hipStream_t s, Timing t) {
    launch_timed(t, kvq_score_kernel<D, DT, QT>, dim3(a.key_wgs, a.c.H, a.c.B), dim3(kKeyWaves * kWave), 0, s, a);
}
template <int D, int DT> void score(const KvqScoreArgs& a, hipStream_t s, Timing t) {
    if (a.q_tiles == 1) {
        stream_keys<D, DT, 1>(a, s, t);
    } else if (a.q_tiles == 2) {
        stream_keys<D, DT, 2>(a, s, t);
    } else {
        const unsigned bhs = static_cast<unsigned>(a.c.B) * a.c.H;
        launch_timed(t, kvq_score_lds_kernel<D, DT>, dim3(bhs * a.key_wgs * a.segs), dim3(kLdsWaves * kWave), 0, s, a);
        if (a.segs > 1)
            kvq_score_sum_kernel<<<dim3(bhs * ((a.c.capacity + 255) / 256)), 256, 0, s>>>(a, lds_rows(D, DT));
    }
}

}  // namespace

// Workgroups: four a compute unit for rows in registers (27-node trees, 32 batch rows at 4096 keys: half as many take 1.3
// times as long, twice as many 1.15), two where the rows fill LDS (32 tokens x 4 heads, 8 batch rows at 30000 keys: 74 us;
// half as many 92), and with the rows split as well four (2048 tokens x 4 heads on their own 2048 keys: kernels of 45 + 6
// us; two 65 + 5, eight 49 + 7).  The keys' share goes by the capacity, the host knowing no lengths: that prompt is 50 us
// in a cache of 2053 slots, 56 in 4096, 96 in 8192 and 143 from 32768 on, where most key blocks hold nothing.
void kvq_score_plan(KvqScoreArgs& a) {
    // the most rows there can be (the host knows no lengths)
    const long rows = static_cast<long>(a.path && a.path_stride < a.N ? a.path_stride : a.N) * a.G;
    const long bhs = static_cast<long>(a.c.B) * a.c.H;
    a.q_tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 0;
    a.segs = 1;
    const auto wgs = [&](int waves, long target) {      // workgroups along the keys, each with one step a wave at least
        const long blocks = (static_cast<long>(a.c.capacity) + 32 * waves - 1) / (32 * waves);
        const long most = (target + bhs - 1) / bhs;
        return static_cast<int>(blocks < most ? blocks : most);
    };
    if (a.q_tiles) {
        a.key_wgs = wgs(kKeyWaves, 1024);
        return;
    }
    a.key_wgs = wgs(kLdsWaves, 512);
    const int lot = lds_rows(a.c.D, a.dtype);
    const long lots = (rows + lot - 1) / lot, most = 1024 / (bhs * a.key_wgs);
    if (most > 1 && lots > 1) a.segs = static_cast<int>(lots < most ? lots : most);
}

hipError_t launch_kvq_score(const KvqScoreArgs& a, hipStream_t s, Timing t) {
    if (a.dtype == 1) {
        if (a.c.D == 64) score<64, 1>(a, s, t);
        else if (a.c.D == 128) score<128, 1>(a, s, t);
        else score<256, 1>(a, s, t);
    } else {
        if (a.c.D == 64) score<64, 0>(a, s, t);
        else if (a.c.D == 128) score<128, 0>(a, s, t);
        else score<256, 0>(a, s, t);
    }
    return hipGetLastError();
}

}  // namespace sv
