// Accumulated attention weight of the cached rows (what an eviction goes by).
//
// w_s = sum over the accepted queries and the G query heads of a cache head of
// exp2(c * (q . K_s) - lse * log2(e)), c = scale * log2(e): the softmax's
// statistics are known, so one product with the K codes gives the weights, half
// of attention's reads.  Every slot's sum is one workgroup's, in a fixed order, so
// no atomics and the same bits every time.  Operands are laid out as in attention
// (16x16x32 bf16 MFMAs, lane (c, g) with c = lane % 16, g = lane / 16).
//
// A tree's path has a handful of rows: bound by the K codes.  A wave keeps all the
// queries (16*QT rows) and streams keys, S = Q K^T, 32 a step: lane (c, g) gets
// rows 4g + i against key c, so a key's sum is over registers and two exchanges.
//
// A prompt has thousands: bound by the exponentials.  The waves of a workgroup
// hold the same 16*KT keys, converted once, and walk every WAVES-th tile of 16
// rows, S^T = K Q^T: lane (c, g) adds up query c for keys 4g + i, and lanes and
// waves are summed at the end.

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

#if SV_KVQ_DEVICE
// A buffer descriptor: loads past `bytes` give zeros and touch nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, bytes, 0x00020000);
}
#endif

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

// 16 query rows as loaded: lane (c, g) has elements 32s + 8g .. of row c, and its lse in base 2.
template <int D, int DT> struct RowTile {
    static constexpr int kVecs = D / 32 * (DT == 1 ? 1 : 2);
    u32x4 w[kVecs];
    float lse;
    int tok;                                            // which accepted token; -1: no row
};

template <int D, int DT, int KT, int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void kvq_score_rows_kernel(KvqScoreArgs a) {
    constexpr int NQ = DT == 1 ? 1 : 3;
    constexpr int kKeys = 16 * KT, kVecs = RowTile<D, DT>::kVecs;
    // heads side by side in the grid, so that one XCD (every eighth workgroup) has one head's queries in its L2
    const int bhs = a.c.B * a.c.H, blocks = static_cast<int>(gridDim.x) / bhs;
    const int bh = blockIdx.x % bhs, turn = blockIdx.x / bhs;
    const int h = bh % a.c.H, b = bh / a.c.H;
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int pre = a.prefix[b], d = a.accept_len[b];
    if (d < 0 || d >= a.N || d >= a.path_stride || pre < 0 || static_cast<long>(pre) + d + 1 > a.c.capacity) return;
    const int all = pre + d + 1;                        // slots after the commit
    // later keys have fewer rows: every other eight heads take them from the other end
    const int blk = (bh / 8) & 1 ? blocks - 1 - turn : turn;
    const int kb = blk * kKeys;
    if (kb >= all) return;

    // K rows of the wave's keys.  Elements are numbered 32s + 8g + j here, not 32g + 8s + j: a load of query rows, of
    // which there are many, then takes 64 bytes of each row instead of every fourth 16
    uint32_t raw[KT][D / 32], rs[KT][D == 256 ? 2 : 1];
    const uint8_t* kc = a.c.kc + b * a.c.cb + h * a.c.ch;
    const uint8_t* ks = a.c.ks + b * a.c.sb + h * a.c.sh;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const long key = min(kb + 16 * t + c, all - 1);
        const uint8_t* sp = ks + key * a.c.sp;
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
            raw[t][s] = *reinterpret_cast<const uint32_t*>(kc + key * a.c.cp + 16 * s + 4 * g);
        if (D == 64) rs[t][0] = *reinterpret_cast<const uint16_t*>(sp);
        else rs[t][0] = *reinterpret_cast<const uint32_t*>(sp);
        if (D == 256) rs[t][D == 256 ? 1 : 0] = *reinterpret_cast<const uint32_t*>(sp + 4);
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
        const long off = b * a.q.batch + tk * a.q.pos + hq * a.q.head + 8 * g;
        const float lse = a.lse[(static_cast<long>(b) * a.N + tk) * a.Hq + hq] * 1.44269504089f;
        // a query that saw nothing, or a row past the last, weighs nothing
        r.lse = live && lse != -INFINITY ? lse : INFINITY;
        r.tok = live ? t : -1;
        const char* q = static_cast<const char*>(a.q.data) + off * (DT == 1 ? 2 : 4);
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            if (DT == 1) {
                r.w[s] = *reinterpret_cast<const u32x4*>(q + 64 * s);
            } else {
                r.w[(2 * s) % kVecs] = *reinterpret_cast<const u32x4*>(q + 128 * s);
                r.w[(2 * s + 1) % kVecs] = *reinterpret_cast<const u32x4*>(q + 128 * s + 16);
            }
        }
    };

    constexpr int step = 16 * WAVES;
    // the first tile whose tokens see the keys
    int r0 = (kb > pre ? (kb - pre) * a.G / 16 * 16 : 0) + 16 * wave;
    RowTile<D, DT> ta, tb;
    load(ta, r0);                                       // (past the last row: row 0, weighing nothing)

    u32x4 A[KT][D / 32];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            const float sc = scale_value(rs[t][D == 256 ? s / 4 : 0] >> (8 * (s % 4)) & 255u);
            const uint32_t w = raw[t][s];
            A[t][s] = u32x4{fp4_pair<0>(w, sc), fp4_pair<1>(w, sc), fp4_pair<2>(w, sc), fp4_pair<3>(w, sc)};
        }

    float w[KT][4];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[t][i] = 0.f;

    const auto weigh = [&](const RowTile<D, DT>& cur, int r0) {
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
                    x[e] = __uint_as_float(cur.w[(2 * s + e / 4) % kVecs][e % 4]);
                bf16_parts<NQ>(x, [&](int p, const u32x4& w) { q[p] = w; });
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
    };
    // two tiles in turn: one is on its way while the other is weighed
    for (; r0 < rows; r0 += 2 * step) {
        load(tb, r0 + step);
        weigh(ta, r0);
        load(ta, r0 + 2 * step);
        if (r0 + step < rows) weigh(tb, r0 + step);
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
    __shared__ float sh[WAVES][kKeys];
    if (c == 0) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) sh[wave][16 * k + 4 * g + i] = w[k][i];
    }
    __syncthreads();
    if (threadIdx.x < kKeys && kb + static_cast<int>(threadIdx.x) < all) {
        float x = 0.f;
#pragma unroll
        for (int v = 0; v < WAVES; ++v) x += sh[v][threadIdx.x];
        const int slot = kb + threadIdx.x;
        const float old = a.scores[(static_cast<long>(b) * a.c.H + h) * a.c.capacity + slot];
        put_weight(a, b, h, pre, slot, x, old);
    }
}

// Few rows: the queries stay, the keys stream.
template <int D, int DT, int QT>
__global__ __launch_bounds__(kKeyWaves* kWave) void kvq_score_kernel(KvqScoreArgs a) {
    constexpr int NQ = DT == 1 ? 1 : 3;
    const int h = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int pre = a.prefix[b], d = a.accept_len[b];
    if (d < 0 || d >= a.N || d >= a.path_stride || pre < 0 || static_cast<long>(pre) + d + 1 > a.c.capacity) return;
    const int all = pre + d + 1;                        // slots after the commit
    const int stride = static_cast<int>(gridDim.x) * kKeyWaves * 32;
    int kb = (static_cast<int>(blockIdx.x) * kKeyWaves + wave) * 32;
    if (kb >= all) return;

    // two tiles of 16 keys: codes and scales; past the last slot zeros
    struct Raw {
        uint32_t k[2][D / 32], s[2];
        float old;                                      // the score this lane adds to
    };
    float* const scores = a.scores + (static_cast<long>(b) * a.c.H + h) * a.c.capacity;
    const int mine = (g & 1) * 16 + c;                  // its slot of a step's 32 (lanes of g < 2 write)
    [[maybe_unused]] const uint8_t* kc = a.c.kc + b * a.c.cb + h * a.c.ch;
    [[maybe_unused]] const uint8_t* ks = a.c.ks + b * a.c.sb + h * a.c.sh;
    [[maybe_unused]] const uint32_t ko = static_cast<uint32_t>(c * a.c.cp) + g * (D / 8);
    [[maybe_unused]] const uint32_t kso = static_cast<uint32_t>(c * a.c.sp) + g * D / 128;
    const auto load_k = [&](Raw& r, int kb) {
#if SV_KVQ_DEVICE
        r.old = scores[min(kb + mine, all - 1)];
        const int n = max(min(all - kb, 32), 0), cp32 = static_cast<int>(a.c.cp), sp32 = static_cast<int>(a.c.sp);
        const auto rk = rsrc(kc + kb * a.c.cp, n * cp32), rks = rsrc(ks + kb * a.c.sp, n * sp32);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (D == 64) {
                const auto w = __builtin_amdgcn_raw_buffer_load_b64(rk, ko, 16 * t * cp32, 0);
                r.k[t][0] = w[0], r.k[t][1] = w[1];
            } else {
#pragma unroll
                for (int x = 0; x < D / 128; ++x) {
                    const auto w = __builtin_amdgcn_raw_buffer_load_b128(rk, ko + 16 * x, 16 * t * cp32, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) r.k[t][(4 * x + e) % (D / 32)] = w[e];
                }
            }
            r.s[t] = D == 256 ? __builtin_amdgcn_raw_buffer_load_b16(rks, kso, 16 * t * sp32, 0)
                              : __builtin_amdgcn_raw_buffer_load_b8(rks, kso, 16 * t * sp32, 0);
        }
#endif
    };
    Raw cur;
    load_k(cur, kb);

    int node = lane;                                    // lane t holds path[t] of a tree
    if (a.path) {
        node = lane < a.path_stride ? a.path[static_cast<long>(b) * a.path_stride + lane] : 0;
        const int before = __shfl_up(node, 1, kWave);
        if (__ballot(lane <= d && (lane == 0 ? node != 0 : (node <= before || node >= a.N))) != 0ull) return;
    }
    const int rows = (d + 1) * a.G;
    u32x4 Q[QT][NQ][D / 32];
    float lse[QT][4];
    int tok[QT][4];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        // lane (c, g) loads a quarter of row 16*qt + c, and keeps the lse and tokens of rows 16*qt + 4g + i
        const int row = 16 * qt + c < rows ? 16 * qt + c : 0;
        const int t = row / a.G;
        const int tk = a.path ? __shfl(node, t, kWave) : t;
        const int hq = h * a.G + (row - t * a.G);
        const char* q = static_cast<const char*>(a.q.data) +
                        (b * a.q.batch + tk * a.q.pos + hq * a.q.head + g * (D / 4)) * (DT == 1 ? 2 : 4);
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            if (DT == 1) {
                Q[qt][0][s] = reinterpret_cast<const u32x4*>(q)[s];
            } else {
                const f32x4 lo = reinterpret_cast<const f32x4*>(q)[2 * s], hi = reinterpret_cast<const f32x4*>(q)[2 * s + 1];
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = lo[e], x[4 + e] = hi[e];
                bf16_parts<NQ>(x, [&](int p, const u32x4& w) { Q[qt][p][s] = w; });
            }
        }
        const float lse2 = a.lse[(static_cast<long>(b) * a.N + tk) * a.Hq + hq] * 1.44269504089f;
        // a query that saw nothing, or a row past the last, weighs nothing
        const float l = 16 * qt + c < rows && lse2 != -INFINITY ? lse2 : INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lse[qt][i] = lane_gather(l, 4 * g + i);
            tok[qt][i] = 16 * qt + 4 * g + i < rows ? static_cast<int>(lane_gather(static_cast<uint32_t>(t), 4 * g + i)) : -1;
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
                const float sc = scale_value(D == 256 && s >= 4 ? cur.s[t] >> 8 : cur.s[t]);
                const uint32_t w = cur.k[t][s];
                const u32x4 K = {fp4_pair<0>(w, sc), fp4_pair<1>(w, sc), fp4_pair<2>(w, sc), fp4_pair<3>(w, sc)};
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int p = 0; p < NQ; ++p) S[t][qt] = mfma(Q[qt][p][s], K, S[t][qt]);
            }
        }
        const float old = cur.old;
        load_k(cur, kb + stride);
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
        const int slot = kb + mine;
        if (g < 2 && slot < all) put_weight(a, b, h, pre, slot, g ? x[1] : x[0], old);
    }
}

#ifndef SKT
#define SKT 4
#define SW 8
#endif
#ifndef SCORE_WGS
#define SCORE_WGS 1024
#endif
template <int D, int DT, int QT> void stream_keys(const KvqScoreArgs& a, hipStream_t s, Timing t) {
    const int keys = kKeyWaves * 32, bh = a.c.B * a.c.H;
    const int blocks = (a.c.capacity + keys - 1) / keys, most = (SCORE_WGS + bh - 1) / bh;
    launch_timed(t, kvq_score_kernel<D, DT, QT>, dim3(blocks < most ? blocks : most, a.c.H, a.c.B),
                 dim3(kKeyWaves * kWave), 0, s, a);
}
template <int D, int DT> void score(const KvqScoreArgs& a, hipStream_t s, Timing t) {
    // the most rows there can be (the host knows no lengths)
    const long rows = static_cast<long>(a.path && a.path_stride < a.N ? a.path_stride : a.N) * a.G;
    if (rows <= 16) {
        stream_keys<D, DT, 1>(a, s, t);
    } else if (rows <= 32) {
        stream_keys<D, DT, 2>(a, s, t);
    } else if (DT == 1 && D <= 128 && rows <= 64) {
        stream_keys<DT == 1 && D <= 128 ? D : 64, DT, DT == 1 && D <= 128 ? 4 : 1>(a, s, t);
    } else {
        constexpr int KT = SKT, W = SW;
        const unsigned blocks = (a.c.capacity + 16 * KT - 1) / (16 * KT);
        launch_timed(t, kvq_score_rows_kernel<D, DT, KT, W>, dim3(blocks * a.c.H * a.c.B), dim3(W * kWave), 0, s, a);
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
