// Softmax attention of a step's queries over the four-bit cache.
//
// For a cache head, the M = N*G query rows (N tokens, G query heads sharing the
// head) meet keys s in one pass with a running maximum and sum: S = q . K_s,
// P = exp2(c*(S - m)), O += P V_s, where c = scale*log2(e) and m is the largest
// S so far.  Workgroups split the key axis; their (m, l, O) join at the end.
//
// A wave takes 32 keys a step and 16*QT query rows, on 16x16x32 bf16 MFMAs in the
// transposed form, S^T = K Q^T and O^T = V^T P^T, so that nothing crosses lanes
// but the row maximum: lane (c, g), c = lane%16, g = lane/16, ends up with the
// scores of query c against keys 16t + 4g + i (t < 2, i < 4), and those eight
// values, rounded to bf16, ARE the second product's operand when its
// contraction index is numbered 8g + 4t + i.  The order of a contraction is free,
// so the cache is read in whole runs and the queries are laid out to match:
//   K: lane (c, g) loads the g-th quarter of key 16t + c (D/8 bytes);
//   V: lane (c, g) loads bytes c*D/32 .. of keys 16t + 4g + i, D/16 elements each.
// Codes become bf16 by the conversion that multiplies by the block's scale, two a
// instruction, exactly (E2M1 times a power of two).  V pairs two elements of one
// key where the product wants two keys of one element: one byte permute each.
//
// float32 queries enter as three bf16 parts (exact) and P as two.

#include "kvq.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kStep = 32;                               // keys a wave takes at a time
constexpr int kRound = kStep * kWaves;                  // keys a workgroup takes at a time

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
#if SV_KVQ_DEVICE
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
#else
    return c;
#endif
}
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 p = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, p);
}

// The lane's codes and scales of one step, as loaded.
template <int D> struct Raw {
    static constexpr int kKW = D / 32;                  // words of a quarter K row
    static constexpr int kVW = D <= 128 ? 1 : 2;        // words of a lane's V elements
    uint32_t k[2][kKW], ks[2];
    uint32_t v[8][kVW], vs[8];
};

template <int D> struct Loader {
    const uint8_t *kc, *ks, *vc, *vs;                   // of the (b, h)
    long cp, sp;
    int c, g;
    // keys kb .. kb+31, those at or past `lim` replaced by key lim - 1
    __device__ __forceinline__ void load(Raw<D>& r, long kb, long lim) const {
        const int last = static_cast<int>(min(lim - kb, 32l)) - 1;
        const uint8_t* kcb = kc + kb * cp;
        const uint8_t* ksb = ks + kb * sp;
        const uint8_t* vcb = vc + kb * cp;
        const uint8_t* vsb = vs + kb * sp;
        const uint32_t cp32 = static_cast<uint32_t>(cp), sp32 = static_cast<uint32_t>(sp);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t key = min(16 * t + c, last);
            const uint8_t* p = kcb + (key * cp32 + static_cast<uint32_t>(g * (D / 8)));
            if (D == 64) {
                const u32x2 w = *reinterpret_cast<const u32x2*>(p);
                r.k[t][0] = w[0], r.k[t][1] = w[1];
            } else {
#pragma unroll
                for (int x = 0; x < D / 128; ++x) {
                    const u32x4 w = reinterpret_cast<const u32x4*>(p)[x];
#pragma unroll
                    for (int e = 0; e < 4; ++e) r.k[t][(4 * x + e) % Raw<D>::kKW] = w[e];
                }
            }
            const uint8_t* s = ksb + (key * sp32 + static_cast<uint32_t>(g * D / 128));
            r.ks[t] = D == 256 ? *reinterpret_cast<const uint16_t*>(s) : *s;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t key = min(16 * (j / 4) + 4 * g + j % 4, last);
            const uint8_t* p = vcb + (key * cp32 + static_cast<uint32_t>(c * (D / 32)));
            if (D == 64) r.v[j][0] = *reinterpret_cast<const uint16_t*>(p);
            else if (D == 128) r.v[j][0] = *reinterpret_cast<const uint32_t*>(p);
            else {
                const u32x2 w = *reinterpret_cast<const u32x2*>(p);
                r.v[j][0] = w[0], r.v[j][Raw<D>::kVW - 1] = w[1];
            }
            r.vs[j] = vsb[key * sp32 + static_cast<uint32_t>(c * (D / 16) / kQBlock)];
        }
    }
};

// Query rows as the B operand of S^T: lane (c, g) holds elements g*D/4 .. of row c.  bf16 rows are one part, float32
// rows three whose sum is the value.
template <int D, int NQ, int DT>
__device__ __forceinline__ void load_query(const KvqRows& q, long off, bool live, int g, u32x4 (&out)[NQ][D / 32]) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        const long i = off + g * (D / 4) + 8 * s;
        if (DT == 1) {
            const u32x4 z = {0, 0, 0, 0};
            out[0][s] = live ? *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(q.data) + i) : z;
        } else {
            float x[8] = {};
            if (live) {
                const f32x4 a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(q.data) + i);
                const f32x4 b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(q.data) + i + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = a[e], x[4 + e] = b[e];
            }
#pragma unroll
            for (int p = 0; p < NQ; ++p) {
                u32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
                    x[2 * e] -= bf16_lo(w[e]);
                    x[2 * e + 1] -= bf16_hi(w[e]);
                }
                out[p][s] = w;
            }
        }
    }
}

template <int D, int DT, int QT>
__global__ __launch_bounds__(kThreads) void kvq_attention_kernel(KvqAttnArgs a) {
    constexpr int NQ = DT == 1 ? 1 : 3, NP = DT == 1 ? 1 : 2;
    constexpr int kNT = D / 16;                         // 16-row tiles of O^T
    constexpr int kRows = 16 * QT;
    // units (b, h, split) of one residue mod 8 with all their row tiles: neighbours in time on one XCD, whose L2 serves
    // the row tiles that read the same keys
    const int RT = a.row_tiles;
    const int x = blockIdx.x % 8, y = blockIdx.x / 8;
    const int rt = y % RT, unit = (y / RT) * 8 + x;
    const int split = unit % a.splits, bh = unit / a.splits;
    if (bh >= a.c.B * a.c.H) return;
    const int h = bh % a.c.H, b = bh / a.c.H;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    const int c = lane & 15, g = lane >> 4;

    const int pre = a.prefix[b], cnt = a.counts ? a.counts[b] : a.N;
    const bool ok = kvq_row_ok(pre, cnt, a.N, a.c.capacity);
    const int row0 = rt * kRows;
    // tokens of this tile that exist, and the slots any of them may see
    const int tok_end = ok ? min(cnt, (min(row0 + kRows, a.M) - 1) / a.G + 1) : 0;
    const bool any = ok && row0 / a.G < tok_end;
    const long lim = any ? static_cast<long>(pre) + (a.mask ? cnt : tok_end) : 0;
    const long all = ok ? static_cast<long>(pre) + cnt : 0;
    // equal chunks of whole rounds over the row's own slots
    const long rounds = (all + kRound - 1) / kRound;
    const long chunk = (rounds + a.splits - 1) / a.splits * kRound;
    const long k0 = split * chunk, k1 = min(k0 + chunk, lim);

    // this lane's query (one a tile): its row, token, and whether it exists
    u32x4 Q[QT][NQ][D / 32];
    int tok[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const int r = row0 + qt * 16 + c;
        tok[qt] = r / a.G;
        const bool live = r < a.M && tok[qt] < (ok ? cnt : 0);
        const int hq = h * a.G + r % a.G;
        load_query<D, NQ, DT>(a.q, b * a.q.batch + tok[qt] * a.q.pos + hq * a.q.head, live, g, Q[qt]);
        if (!live) tok[qt] = -1;
    }

    f32x4 O[QT][kNT];
    float m[QT], l[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        m[qt] = -INFINITY;
        l[qt] = 0.f;
#pragma unroll
        for (int n = 0; n < kNT; ++n) O[qt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    Loader<D> ld;
    ld.kc = a.c.kc + b * a.c.cb + h * a.c.ch;
    ld.vc = a.c.vc + b * a.c.cb + h * a.c.ch;
    ld.ks = a.c.ks + b * a.c.sb + h * a.c.sh;
    ld.vs = a.c.vs + b * a.c.sb + h * a.c.sh;
    ld.cp = a.c.cp;
    ld.sp = a.c.sp;
    ld.c = c;
    ld.g = g;

    Raw<D> cur, nxt;
    long kb = k0 + kStep * wave;
    if (kb < k1) ld.load(cur, kb, lim);
    for (; kb < k1; kb += kRound) {
        if (kb + kRound < k1) ld.load(nxt, kb + kRound, lim);

        // S^T = K Q^T
        f32x4 S[QT][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) S[qt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < D / 32; ++s) {
                const float sc = scale_value(D == 256 && s >= 4 ? cur.ks[t] >> 8 : cur.ks[t] & 255u);
                const uint32_t w = cur.k[t][s];
                const u32x4 A = {fp4_pair<0>(w, sc), fp4_pair<1>(w, sc), fp4_pair<2>(w, sc), fp4_pair<3>(w, sc)};
#pragma unroll
                for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                    for (int p = 0; p < NQ; ++p) S[qt][t] = mfma(A, Q[qt][p][s], S[qt][t]);
            }
        }
        const bool edge = kb + kStep > pre;             // some of the 32 slots are new ones, or past the end
        if (edge) {
            // selects, not branches: a lane's eight slots may fall on either side of every limit
            const int node0 = static_cast<int>(kb - pre) + 4 * g;
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                const uint8_t* mrow = a.mask + b * a.mask_batch + static_cast<long>(max(tok[qt], 0)) * a.N;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int node = node0 + 16 * (j / 4) + j % 4;
                    int sees = a.mask ? mrow[min(max(node, 0), a.N - 1)] : node <= tok[qt];
                    sees = (sees != 0) & (node < cnt);
                    const float x = S[qt][j / 4][j % 4];
                    S[qt][j / 4][j % 4] = (node < 0) | sees ? x : -INFINITY;
                }
            }
        }

        // running maximum and sum; P rounded to bf16 parts
        u32x4 P[QT][NP];
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            float mx = S[qt][0][0];
#pragma unroll
            for (int j = 1; j < 8; ++j) mx = fmaxf(mx, S[qt][j / 4][j % 4]);
            mx = fmaxf(mx, xshfl(mx, 16));
            mx = fmaxf(mx, xshfl(mx, 32));
            const float mn = fmaxf(m[qt], mx);
            if (__ballot(mn > m[qt]) != 0ull) {
                const float al = m[qt] == -INFINITY ? 0.f : exp2_fast((m[qt] - mn) * a.cexp);
                l[qt] *= al;
#pragma unroll
                for (int n = 0; n < kNT; ++n) O[qt][n] *= al;
                m[qt] = mn;
            }
            const float mc = m[qt] == -INFINITY ? 0.f : m[qt] * a.cexp;
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] = exp2_fast(fmaf(S[qt][j / 4][j % 4], a.cexp, -mc));
                l[qt] += p[j];
            }
#pragma unroll
            for (int x = 0; x < NP; ++x) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    P[qt][x][e] = pack_bf16(p[2 * e], p[2 * e + 1]);
                    p[2 * e] -= bf16_lo(P[qt][x][e]);
                    p[2 * e + 1] -= bf16_hi(P[qt][x][e]);
                }
            }
        }

        // O^T += V^T P^T
        float vsc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // a slot past the end holds anything; its P is 0, its V has to be finite
            const bool past = kb + 16 * (j / 4) + 4 * g + j % 4 >= lim;
            vsc[j] = past ? 0.f : scale_value(min(cur.vs[j], 254u));
#pragma unroll
            for (int x = 0; x < Raw<D>::kVW; ++x) cur.v[j][x] = past ? 0u : cur.v[j][x];
        }
#pragma unroll
        for (int pr = 0; pr < kNT / 2; ++pr) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = fp4_pair(cur.v[j][pr / 4], vsc[j], pr % 4);
            u32x4 lo, hi;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo[e] = __builtin_amdgcn_perm(w[2 * e + 1], w[2 * e], 0x05040100u);
                hi[e] = __builtin_amdgcn_perm(w[2 * e + 1], w[2 * e], 0x07060302u);
            }
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
#pragma unroll
                for (int x = 0; x < NP; ++x) {
                    O[qt][2 * pr] = mfma(lo, P[qt][x], O[qt][2 * pr]);
                    O[qt][2 * pr + 1] = mfma(hi, P[qt][x], O[qt][2 * pr + 1]);
                }
            }
        }
        cur = nxt;
    }

    // join the waves: the sums of a lane's four g-groups, then the four waves, two at a time through LDS
    __shared__ float sh_o[2][kRows * D];
    __shared__ float sh_ml[2][kRows][2];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        l[qt] += xshfl(l[qt], 16);
        l[qt] += xshfl(l[qt], 32);
        if (tok[qt] < 0) {                              // no query here (a padded token, or the tile's end)
            m[qt] = -INFINITY;
            l[qt] = 0.f;
#pragma unroll
            for (int n = 0; n < kNT; ++n) O[qt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
        __syncthreads();
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                // element (row, d) of O^T in the lane's own order: one 16-byte run per (qt, n)
#pragma unroll
                for (int n = 0; n < kNT; ++n)
                    *reinterpret_cast<f32x4*>(&sh_o[wave - half][((qt * kNT + n) * kWave + lane) * 4]) = O[qt][n];
                if (g == 0) {
                    sh_ml[wave - half][qt * 16 + c][0] = m[qt];
                    sh_ml[wave - half][qt * 16 + c][1] = l[qt];
                }
            }
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                const float om = sh_ml[wave][qt * 16 + c][0], ol = sh_ml[wave][qt * 16 + c][1];
                const float mn = fmaxf(m[qt], om);
                const float wa = m[qt] == -INFINITY ? 0.f : exp2_fast((m[qt] - mn) * a.cexp);
                const float wb = om == -INFINITY ? 0.f : exp2_fast((om - mn) * a.cexp);
                m[qt] = mn;
                // a sum that is NaN stays NaN whatever its maximum
                l[qt] = l[qt] * wa + ol * wb;
#pragma unroll
                for (int n = 0; n < kNT; ++n)
                    O[qt][n] = O[qt][n] * wa +
                               *reinterpret_cast<const f32x4*>(&sh_o[wave][((qt * kNT + n) * kWave + lane) * 4]) * wb;
            }
        }
    }
    if (wave != 0) return;

    // O^T tile n, register i is element (D/16)*(4g + i) + n of query c
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const int r = row0 + qt * 16 + c;
        if (r >= a.M) continue;
        if (a.splits > 1) {
            const long at = (static_cast<long>(bh) * a.splits + split) * a.M + r;
            if (g == 0) {
                a.part_ml[2 * at] = m[qt];
                a.part_ml[2 * at + 1] = l[qt];
            }
            float* o = a.part_o + at * D + (D / 4) * g;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < kNT; n += 4)
                    *reinterpret_cast<f32x4*>(o + (D / 16) * i + n) =
                        f32x4{O[qt][n][i], O[qt][n + 1][i], O[qt][n + 2][i], O[qt][n + 3][i]};
        } else {
            const int tk = r / a.G, hq = h * a.G + r % a.G;
            const long at = (static_cast<long>(b) * a.N + tk) * a.Hq + hq;
            const bool empty = l[qt] == 0.f;
            const float inv = empty ? 0.f : 1.f / l[qt];
            if (g == 0 && a.out_lse)
                a.out_lse[at] = empty ? -INFINITY : (m[qt] * a.cexp + __builtin_amdgcn_logf(l[qt])) * 0.69314718056f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long d = at * D + (D / 4) * g + (D / 16) * i;
#pragma unroll
                for (int n = 0; n < kNT; n += 4) {
                    const float o0 = O[qt][n][i] * inv, o1 = O[qt][n + 1][i] * inv, o2 = O[qt][n + 2][i] * inv,
                                o3 = O[qt][n + 3][i] * inv;
                    if (DT == 1)
                        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + d + n) =
                            u32x2{pack_bf16(o0, o1), pack_bf16(o2, o3)};
                    else
                        *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + d + n) = f32x4{o0, o1, o2, o3};
                }
            }
        }
    }
}

// Joins the splits: four elements a thread, D/4 neighbouring threads a row.
template <int D, int DT>
__global__ __launch_bounds__(kThreads) void kvq_join_kernel(KvqAttnArgs a) {
    const long row = (static_cast<long>(blockIdx.x) * kThreads + threadIdx.x) / (D / 4);
    const int d = static_cast<int>(threadIdx.x % (D / 4)) * 4;
    if (row >= static_cast<long>(a.c.B) * a.c.H * a.M) return;
    const int r = static_cast<int>(row % a.M), bh = static_cast<int>(row / a.M);
    const int h = bh % a.c.H, b = bh / a.c.H;
    const int pre = a.prefix[b], cnt = a.counts ? a.counts[b] : a.N;
    const long all = kvq_row_ok(pre, cnt, a.N, a.c.capacity) ? static_cast<long>(pre) + cnt : 0;
    const long rounds = (all + kRound - 1) / kRound;
    const long per = (rounds + a.splits - 1) / a.splits;
    const int used = per ? static_cast<int>((rounds + per - 1) / per) : 0;   // splits that hold keys
    const long at0 = static_cast<long>(bh) * a.splits * a.M + r;
    float m = -INFINITY;
    for (int s = 0; s < used; ++s) m = fmaxf(m, a.part_ml[2 * (at0 + static_cast<long>(s) * a.M)]);
    float l = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < used; ++s) {
        const long at = at0 + static_cast<long>(s) * a.M;
        const float ms = a.part_ml[2 * at], ls = a.part_ml[2 * at + 1];
        const float w = ms == -INFINITY ? 0.f : exp2_fast((ms - m) * a.cexp);
        l += ls * w;
        o += *reinterpret_cast<const f32x4*>(a.part_o + at * D + d) * w;
    }
    const bool empty = l == 0.f;
    const float inv = empty ? 0.f : 1.f / l;
    const long at = (static_cast<long>(b) * a.N + r / a.G) * a.Hq + h * a.G + r % a.G;
    if (d == 0 && a.out_lse)
        a.out_lse[at] = empty ? -INFINITY : (m * a.cexp + __builtin_amdgcn_logf(l)) * 0.69314718056f;
    o *= inv;
    if (DT == 1)
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at * D + d) =
            u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    else
        *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at * D + d) = o;
}

int query_tiles(int D, int dtype, int M) {
    const int most = (D == 256 || dtype == 0) ? 2 : 4;
    const int t = (M + 15) / 16;
    return t >= most ? most : (t == 3 ? 4 : t);
}

template <int D, int DT, int QT> void attend(const KvqAttnArgs& a, hipStream_t s, Timing t) {
    const long units = static_cast<long>(a.c.B) * a.c.H * a.splits;
    const dim3 grid(static_cast<unsigned>((units + 7) / 8 * 8 * a.row_tiles));
    launch_timed(t, kvq_attention_kernel<D, DT, QT>, grid, dim3(kThreads), 0, s, a);
}
template <int D, int DT> void attend(const KvqAttnArgs& a, hipStream_t s, Timing t) {
    switch (query_tiles(D, DT, a.M)) {
        case 1: attend<D, DT, 1>(a, s, t); break;
        case 2: attend<D, DT, 2>(a, s, t); break;
        default:
            if constexpr (D != 256 && DT == 1) attend<D, DT, 4>(a, s, t);
    }
    if (a.splits > 1) {
        const long threads = static_cast<long>(a.c.B) * a.c.H * a.M * (D / 4);
        kvq_join_kernel<D, DT><<<dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads)), kThreads, 0, s>>>(a);
    }
}

}  // namespace

void kvq_attention_plan(KvqAttnArgs& a) {
    const int rows = 16 * query_tiles(a.c.D, a.dtype, a.M);
    a.row_tiles = (a.M + rows - 1) / rows;
    const long items = static_cast<long>(a.c.B) * a.c.H * a.row_tiles;
    const long most = (static_cast<long>(a.c.capacity) + kRound - 1) / kRound;
    long n = (1024 + items - 1) / items;
    a.splits = static_cast<int>(n < most ? n : most);
}

hipError_t launch_kvq_attention(const KvqAttnArgs& a, hipStream_t s, Timing t) {
    if (a.dtype == 1) {
        if (a.c.D == 64) attend<64, 1>(a, s, t);
        else if (a.c.D == 128) attend<128, 1>(a, s, t);
        else attend<256, 1>(a, s, t);
    } else {
        if (a.c.D == 64) attend<64, 0>(a, s, t);
        else if (a.c.D == 128) attend<128, 0>(a, s, t);
        else attend<256, 0>(a, s, t);
    }
    return hipGetLastError();
}

}  // namespace sv
