// Accumulated attention weight of the cached rows (what an eviction goes by).
//
// w_s = sum over the accepted queries and the G query heads of a cache head of
// exp2(c * (q . K_s) - lse * log2(e)), c = scale * log2(e): the softmax's
// statistics are known, so one product with the K codes gives the weights, half
// of attention's reads.  A workgroup owns 16*KT keys a wave and walks the query
// rows 16 at a time; every slot's sum is one workgroup's, in a fixed order, so
// no atomics and the same bits every time.  Operand layouts as in attention
// (S^T = K Q^T on 16x16x32 bf16 MFMAs, K converted once and kept in registers):
// lane (c, g) adds up query c of each tile for keys 4g + i, and the 16 lanes of a
// g-group are summed at the end.

#include "kvq.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

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

template <int D, int DT, int KT>
__global__ __launch_bounds__(kThreads) void kvq_score_kernel(KvqScoreArgs a) {
    constexpr int NQ = DT == 1 ? 1 : 3;
    constexpr int kKeys = 16 * KT * kWaves;             // keys of a workgroup
    const int h = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int pre = a.prefix[b], d = a.accept_len[b];
    if (d < 0 || d >= a.N || d >= a.path_stride || pre < 0 || static_cast<long>(pre) + d + 1 > a.c.capacity) return;
    int node = lane;                                    // lane t holds path[t] of a tree
    if (a.path) {
        node = lane < a.path_stride ? a.path[static_cast<long>(b) * a.path_stride + lane] : 0;
        const int before = __shfl_up(node, 1, kWave);
        if (__ballot(lane <= d && (lane == 0 ? node != 0 : (node <= before || node >= a.N))) != 0ull) return;
    }
    const long all = static_cast<long>(pre) + d + 1;    // slots after the commit
    const long wg0 = static_cast<long>(blockIdx.x) * kKeys;
    const long kb = wg0 + wave * (16 * KT);
    if (kb >= all) return;

    // K rows of the wave's keys as A operands
    u32x4 A[KT][D / 32];
    const uint8_t* kc = a.c.kc + b * a.c.cb + h * a.c.ch;
    const uint8_t* ks = a.c.ks + b * a.c.sb + h * a.c.sh;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const long key = min(kb + 16 * t + c, all - 1);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(kc + key * a.c.cp + g * (D / 8));
        const uint8_t* sp = ks + key * a.c.sp + g * D / 128;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            const float sc = scale_value(sp[D == 256 ? s / 4 : 0]);
            const uint32_t w = p[s];
            A[t][s] = u32x4{fp4_pair<0>(w, sc), fp4_pair<1>(w, sc), fp4_pair<2>(w, sc), fp4_pair<3>(w, sc)};
        }
    }

    float w[KT][4];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[t][i] = 0.f;

    const long rows = static_cast<long>(d + 1) * a.G;
    // the first token that sees the wave's keys
    const long first = kb > pre ? (kb - pre) * a.G / 16 * 16 : 0;
    for (long r0 = first; r0 < rows; r0 += 16) {
        const long r = r0 + c;
        const bool live = r < rows;
        const int t = live ? static_cast<int>(r / a.G) : 0, hq = h * a.G + static_cast<int>(r % a.G);
        const int tk = a.path ? __shfl(node, t, kWave) : t;
        const long qoff = b * a.q.batch + tk * a.q.pos + hq * a.q.head;
        float lse = INFINITY;
        if (live) lse = a.lse[(static_cast<long>(b) * a.N + tk) * a.Hq + hq] * 1.44269504089f;
        if (lse == -INFINITY) lse = INFINITY;           // a query that saw nothing
        f32x4 S[KT];
#pragma unroll
        for (int k = 0; k < KT; ++k) S[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            const long i = qoff + g * (D / 4) + 8 * s;
            u32x4 q[NQ];
            if (DT == 1) {
                q[0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q.data) + i);
            } else {
                const f32x4 lo = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.q.data) + i);
                const f32x4 hi = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.q.data) + i + 4);
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = lo[e], x[4 + e] = hi[e];
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
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int p = 0; p < NQ; ++p) S[k] = mfma(A[k][s], q[p], S[k]);
        }
#pragma unroll
        for (int k = 0; k < KT; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = __builtin_amdgcn_exp2f(fmaf(S[k][i], a.cexp, -lse));
                const bool sees = live && kb + 16 * k + 4 * g + i - pre <= t;
                w[k][i] += sees ? p : 0.f;
            }
        }
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
            const long slot = kb + 16 * k + 4 * g + i;
            if (c == i && slot < all) {
                const long at = (static_cast<long>(b) * a.c.H + h) * a.c.capacity + slot;
                if (slot >= pre) {
                    a.scores[at] = x;
                    a.positions[at] = a.seen[b] + static_cast<int>(slot - pre);
                } else {
                    a.scores[at] += x;
                }
            }
        }
    }
}

template <int D, int DT> void score(const KvqScoreArgs& a, hipStream_t s, Timing t) {
    constexpr int KT = D == 256 ? 1 : 2;
    const int keys = 16 * KT * kWaves;
    const dim3 grid((a.c.capacity + keys - 1) / keys, a.c.H, a.c.B);
    launch_timed(t, kvq_score_kernel<D, DT, KT>, grid, dim3(kThreads), 0, s, a);
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
