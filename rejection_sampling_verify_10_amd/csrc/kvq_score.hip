// Accumulated attention weight of the cached rows (what an eviction goes by).
//
// w_s = sum over the accepted queries and the G query heads of a cache head of
// exp2(c * (q . K_s) - lse * log2(e)), c = scale * log2(e): the softmax's
// statistics are known, so one product with the K codes gives the weights, half
// of attention's reads.  Every slot's sum is one workgroup's, in a fixed order, so
// no atomics and the same bits every time.  A wave holds 16*KT keys, converted
// once, and walks the query rows 16 at a time.  Operand layouts as in attention
// (S^T = K Q^T on 16x16x32 bf16 MFMAs): lane (c, g) adds up query c of each tile
// for keys 4g + i, and the 16 lanes of a g-group are summed at the end.
//
// A tree's path has a handful of rows: bound by the K codes, every wave has keys
// of its own.  A prompt has thousands: bound by the exponentials, all waves of a
// workgroup have the same keys and every WAVES-th tile of rows, summed through LDS.

#include "kvq.hpp"

namespace sv {

namespace {

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 p = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
#if SV_KVQ_DEVICE
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
#else
    return c;
#endif
}

// 16 query rows as loaded: lane (c, g) has elements g*D/4 .. of row c, and its lse in base 2.
template <int D, int DT> struct RowTile {
    u32x4 w[D / 32 * (DT == 1 ? 1 : 2)];
    float lse;
    int tok;                                            // which accepted token; -1: no row
};

template <int D, int DT, int KT, int WAVES, bool ROWS>
__global__ __launch_bounds__(WAVES* kWave) void kvq_score_kernel(KvqScoreArgs a) {
    constexpr int NQ = DT == 1 ? 1 : 3;
    constexpr int kKeys = 16 * KT * (ROWS ? 1 : WAVES);             // keys of a workgroup
    const int h = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int pre = a.prefix[b], d = a.accept_len[b];
    if (d < 0 || d >= a.N || d >= a.path_stride || pre < 0 || static_cast<long>(pre) + d + 1 > a.c.capacity) return;
    const int all = pre + d + 1;                        // slots after the commit
    // later keys have fewer rows: every other head takes them from the other end
    const int blk = ROWS && (h & 1) ? static_cast<int>(gridDim.x - 1 - blockIdx.x) : static_cast<int>(blockIdx.x);
    const int kb = blk * kKeys + (ROWS ? 0 : wave * (16 * KT));
    if (kb >= all) return;

    // K rows of the wave's keys
    uint32_t raw[KT][D / 32];
    uint32_t rs[KT][D == 256 ? 2 : 1];
    const uint8_t* kc = a.c.kc + b * a.c.cb + h * a.c.ch;
    const uint8_t* ks = a.c.ks + b * a.c.sb + h * a.c.sh;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const long key = min(kb + 16 * t + c, all - 1);
        const uint8_t* p = kc + key * a.c.cp + g * (D / 8);
        const uint8_t* sp = ks + key * a.c.sp + g * D / 128;
        if (D == 64) {
            const u32x2 w = *reinterpret_cast<const u32x2*>(p);
            raw[t][0] = w[0], raw[t][1] = w[1];
        } else {
#pragma unroll
            for (int x = 0; x < D / 128; ++x) {
                const u32x4 w = reinterpret_cast<const u32x4*>(p)[x];
#pragma unroll
                for (int e = 0; e < 4; ++e) raw[t][(4 * x + e) % (D / 32)] = w[e];
            }
        }
        rs[t][0] = sp[0];
        if (D == 256) rs[t][D == 256 ? 1 : 0] = sp[1];
    }

    int node = lane;                                    // lane t holds path[t] of a tree
    if (a.path) {
        node = lane < a.path_stride ? a.path[static_cast<long>(b) * a.path_stride + lane] : 0;
        const int before = __shfl_up(node, 1, kWave);
        if (__ballot(lane <= d && (lane == 0 ? node != 0 : (node <= before || node >= a.N))) != 0ull) return;
    }
    const int rows = (d + 1) * a.G;
    const auto load = [&](RowTile<D, DT>& r, int r0) {
        const int row = r0 + c;
        const bool live = row < rows;
        const unsigned at = live ? row : 0;
        const int t = a.G == 1 ? at : a.magic ? __umulhi(at, a.magic) : at / a.G;
        const int tk = a.path ? __shfl(node, t, kWave) : t;
        const int hq = h * a.G + (static_cast<int>(at) - t * a.G);
        const long off = b * a.q.batch + tk * a.q.pos + hq * a.q.head + g * (D / 4);
        const float lse = a.lse[(static_cast<long>(b) * a.N + tk) * a.Hq + hq] * 1.44269504089f;
        // a query that saw nothing, or a row past the last, weighs nothing
        r.lse = live && lse != -INFINITY ? lse : INFINITY;
        r.tok = live ? t : -1;
#pragma unroll
        for (int x = 0; x < D / 32 * (DT == 1 ? 1 : 2); ++x)
            r.w[x] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q.data) + off * (DT == 1 ? 2 : 4) + 16 * x);
    };

    const int step = ROWS ? 16 * WAVES : 16;
    // the first tile whose tokens see the keys
    int r0 = kb > pre ? (kb - pre) * a.G / 16 * 16 : 0;
    if (ROWS) r0 += 16 * wave;
    RowTile<D, DT> cur;
    if (r0 < rows) load(cur, r0);

    u32x4 A[KT][D / 32];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            const float sc = scale_value(rs[t][D == 256 ? s / 4 : 0]);
            const uint32_t w = raw[t][s];
            A[t][s] = u32x4{fp4_pair<0>(w, sc), fp4_pair<1>(w, sc), fp4_pair<2>(w, sc), fp4_pair<3>(w, sc)};
        }

    float w[KT][4];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[t][i] = 0.f;

    for (; r0 < rows; r0 += step) {
        RowTile<D, DT> nxt;
        load(nxt, r0 + step);                           // (past the last row: row 0 again, weighing nothing)
        f32x4 S[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) S[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            u32x4 q[NQ];
            if (DT == 1) {
                q[0] = cur.w[s];
            } else {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = __uint_as_float(cur.w[(2 * s + e / 4) % (D / 32 * (DT == 1 ? 1 : 2))][e % 4]);
#pragma unroll
                for (int p = 0; p < NQ; ++p) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        q[p][e] = pack_bf16(x[2 * e], x[2 * e + 1]);
                        x[2 * e] -= bf16_lo(q[p][e]);
                        x[2 * e + 1] -= bf16_hi(q[p][e]);
                    }
                }
            }
#pragma unroll
            for (int p = 0; p < NQ; ++p)
#pragma unroll
                for (int k = 0; k < KT; ++k) S[k] = mfma(A[k][s], q[p], S[k]);
        }
        const bool part = kb + 16 * KT - 1 - pre > r0 / a.G;    // some key is newer than the tile's first token
        const int node0 = kb - pre + 4 * g;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float p = __builtin_amdgcn_exp2f(fmaf(S[k][i], a.cexp, -cur.lse));
                if (part) p = node0 + 16 * k + i <= cur.tok ? p : 0.f;
                w[k][i] += p;
            }
        }
        cur = nxt;
    }

#pragma unroll
    for (int k = 0; k < KT; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = w[k][i];
            x += xshfl(x, 1);
            x += xshfl(x, 2);
            x += xshfl(x, 4);
            x += xshfl(x, 8);
            w[k][i] = x;
        }
    }
    const auto add = [&](int slot, float x) {
        if (slot >= all) return;
        const long at = (static_cast<long>(b) * a.c.H + h) * a.c.capacity + slot;
        if (slot >= pre) {
            a.scores[at] = x;
            a.positions[at] = a.seen[b] + (slot - pre);
        } else {
            a.scores[at] += x;
        }
    };
    if (!ROWS) {
        // lane (c, g) with c < 4*KT keeps key 16*(c/4) + 4g + c%4
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) x = c == 4 * k + i ? w[k][i] : x;
        if (c < 4 * KT) add(kb + 16 * (c / 4) + 4 * g + c % 4, x);
    } else {
        __shared__ float sh[WAVES][16 * KT];
        if (c == 0) {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) sh[wave][16 * k + 4 * g + i] = w[k][i];
        }
        __syncthreads();
        if (threadIdx.x < 16 * KT) {
            float x = 0.f;
#pragma unroll
            for (int v = 0; v < WAVES; ++v) x += sh[v][threadIdx.x];
            add(kb + threadIdx.x, x);
        }
    }
}

template <int D, int DT> void score(const KvqScoreArgs& a, hipStream_t s, Timing t) {
    constexpr int KT = D == 256 ? 2 : 4, W = 8;
    const int tokens = a.path ? (a.path_stride < a.N ? a.path_stride : a.N) : a.N;
    if (static_cast<long>(tokens) * a.G > 512) {        // (the most rows there can be; the host knows no lengths)
        const dim3 grid((a.c.capacity + 16 * KT - 1) / (16 * KT), a.c.H, a.c.B);
        launch_timed(t, kvq_score_kernel<D, DT, KT, W, true>, grid, dim3(W * kWave), 0, s, a);
    } else {
        constexpr int keys = 16 * KT * 4;
        const dim3 grid((a.c.capacity + keys - 1) / keys, a.c.H, a.c.B);
        launch_timed(t, kvq_score_kernel<D, DT, KT, 4, false>, grid, dim3(4 * kWave), 0, s, a);
    }
}

}  // namespace

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
