// Softmax attention of a step's queries over the four-bit cache.
//
// For a cache head, the M = N*G query rows (N tokens, G query heads sharing the
// head) meet keys s in one pass with a running maximum and sum: S = q . K_s,
// P = exp2(c*(S - m)), O += P V_s, where c = scale*log2(e) and m follows the
// largest S so far.  Parts of the key axis join at the end.
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
// float32 queries enter as three bf16 parts, and so does P: exact both.  With bf16
// queries P is the one bf16 of it: at most 2^-8 relative a key, of either sign,
// which is the output's own rounding; the sum l, and so the lse, is of the
// unrounded values.  Against 64 bits whole cases' outputs are off by 0.0022 of
// their size, where float32 probabilities leave 0.0017 (the output's rounding);
// two parts more would triple the second product.
//
// Where the rows are few the cache's bytes bound it, so the key axis is what is
// spread: the waves of a workgroup take 32 keys each in turn and join through
// LDS, and workgroups take units of the batch's whole key axis, alike whatever
// the lengths, which a second kernel joins.
//
// Measured (8 cache heads, D = 128, bf16, whole calls): 64 sequences of one token
// and 8 query heads a cache head, ragged lengths to 8192: 75-78 us for 359 MB, 4.7
// TB/s, short of the 5.7 and more that kernels reach which only read: a lane has
// one step of narrow loads (V: eight of 4 bytes and eight of 1) under way.  8
// tokens x 4 heads at 131071 keys: 42 us for 143 MB, the join 5 of them,
// conversions and bytes alike.  27-node trees x 4 heads, 32 sequences to 4096:
// 64 us for 36 GFLOP, 570 TFLOP/s: of the cycles, the vector units are busy 58%
// (the conversions of K and V, half rate, are nearly half of that) and the matrix
// units 25%, and a wave does one or the other, in turn.  A prompt of 2 x 1023
// tokens: 58-63 us for 39 GFLOP, the same.  One token in a cache of 1000 slots:
// 9-10 us, the chain of load, product, exponential, product, join.

#include "kvq.hpp"

namespace sv {

namespace {

constexpr int kChunk = 128;                             // units of the key axis' split

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A call's split of the key axis.  Batch rows hold pre + cnt slots each, in whole
// chunks; a unit is `per` chunks of one batch row, and the units are numbered
// through the batch, so that a long row gets many and a short one few and all
// of them cost the same.  Every workgroup finds its own from the lengths (the
// host does not know them): row b has ceil(chunks(b) / per) units.
__device__ __forceinline__ int kvq_chunks(const KvqAttnArgs& a, int pre, int cnt) {
    return kvq_row_ok(pre, cnt, a.N, a.c.capacity) ? static_cast<int>((static_cast<long>(pre) + cnt + kChunk - 1) / kChunk)
                                                   : 0;
}
// The batch's chunks, 64 batch rows at a time: lane i has rows i, i + 64, ..; the first 64 are read once.
struct Lengths {
    const KvqAttnArgs& a;
    int lane, pre, cnt, own;
    __device__ __forceinline__ explicit Lengths(const KvqAttnArgs& a) : a(a), lane(threadIdx.x & (kWave - 1)) {
        const int b = min(lane, a.c.B - 1);
        pre = a.prefix[b];
        cnt = a.counts ? a.counts[b] : a.N;
        own = lane < a.c.B ? kvq_chunks(a, pre, cnt) : 0;
    }
    __device__ __forceinline__ int chunks(int b0) const {
        if (b0 == 0) return own;
        const int b = b0 + lane;
        return b < a.c.B ? kvq_chunks(a, a.prefix[b], a.counts ? a.counts[b] : a.N) : 0;
    }
    // Committed and new slots of batch row b.
    __device__ __forceinline__ void row(int b, int& p, int& n) const {
        const bool read = b < kWave;
        p = read ? bcast(pre, b) : a.prefix[b];
        n = read ? bcast(cnt, b) : a.counts ? a.counts[b] : a.N;
    }
    __device__ __forceinline__ int units(int b0, int per) const { return (chunks(b0) + per - 1) / per; }
    // Chunks a unit holds: the fewest for which the batch has no more than a.units units.  (The same in every lane, and
    // kept in scalar registers, as everything derived from it.)
    __device__ __forceinline__ int per() const {
        int most = 1;
        for (int b0 = 0; b0 < a.c.B; b0 += kWave) most = max(most, chunks(b0));
        int lo = a.min_per, hi = max(__builtin_amdgcn_readfirstlane(wave_max_int(most)), lo);
        while (lo < hi) {                               // one a batch row, at hi = the longest, always fits
            const int mid = (lo + hi) / 2;
            int n = 0;
            for (int b0 = 0; b0 < a.c.B; b0 += kWave) n += __builtin_amdgcn_readfirstlane(wave_sum(units(b0, mid)));
            if (n <= a.units) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    }
    // Batch row and place in it of unit u, and how many units the row has; false past the last unit.
    __device__ __forceinline__ bool find(int u, int per, int& b, int& split, int& mine) const {
        int base = 0;
        for (int b0 = 0; b0 < a.c.B; b0 += kWave) {
            const int n = units(b0, per), incl = wave_scan_int(n);
            const unsigned long long past = __ballot(base + incl > u);
            if (past) {
                const int l = __builtin_amdgcn_readfirstlane(__ffsll(static_cast<long long>(past)) - 1);
                b = b0 + l;
                mine = bcast(n, l);
                split = u - base - (bcast(incl, l) - mine);
                return true;
            }
            base += bcast(incl, kWave - 1);
        }
        return false;
    }
    // The units' first numbers by batch row (and their count at the end), for the kernel that joins them.
    __device__ __forceinline__ void note(int per) const {
        int base = 0;
        for (int b0 = 0; b0 < a.c.B; b0 += kWave) {
            const int n = units(b0, per), incl = wave_scan_int(n);
            if (b0 + lane < a.c.B) a.first_unit[b0 + lane] = base + incl - n;
            base += bcast(incl, kWave - 1);
        }
        if (lane == 0) a.first_unit[a.c.B] = base;
    }
    // The batch row with the turn-th most slots (a batch of at most 64): long rows start first, so that the short ones
    // fill the end of the launch.
    __device__ __forceinline__ int by_length(int turn) const {
        const int mine = lane < a.c.B ? own : -1;
        int before = 0;                                 // rows that come before this lane's
        for (int r = 0; r < a.c.B; ++r) {
            const int n = bcast(mine, r);
            before += n > mine || (n == mine && r < lane) ? 1 : 0;
        }
        return __builtin_amdgcn_readfirstlane(__ffsll(static_cast<long long>(__ballot(before == turn))) - 1);
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

// The queries of a wave: row, token (-1: no query here) and, for a tree, the new
// tokens each sees as bits (the four lanes of a query read 16 mask bytes each).
template <int QT> struct Queries {
    int tok[QT];
    unsigned long long tree[QT];
    __device__ __forceinline__ void place(const KvqAttnArgs& a, int row0, int cnt, int c) {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            const int r = row0 + qt * 16 + c;
            tok[qt] = r < a.M && r / a.G < cnt ? r / a.G : -1;
        }
    }
    // Whether some of slots first .. first+31 are hidden from some query of rows row0 .. (or lie past the end).
    __device__ static __forceinline__ bool edge(const KvqAttnArgs& a, long first, long pre, int row0) {
        return first + kStep > pre + (a.mask ? 0 : row0 / a.G + 1);
    }
    __device__ __forceinline__ void read_mask(const KvqAttnArgs& a, int b, int cnt, int g) {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            const uint8_t* row = a.mask + b * a.mask_batch + static_cast<long>(max(tok[qt], 0)) * a.N;
            unsigned bits = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int node = 16 * g + e;
                bits |= static_cast<unsigned>((row[min(node, a.N - 1)] != 0) & (node < cnt)) << e;
            }
            const unsigned half = bits << (16 * (g & 1));
            unsigned w0 = g < 2 ? half : 0u, w1 = g < 2 ? 0u : half;
            w0 |= xshfl(w0, 16);
            w0 |= xshfl(w0, 32);
            w1 |= xshfl(w1, 16);
            w1 |= xshfl(w1, 32);
            tree[qt] = (static_cast<unsigned long long>(w1) << 32) | w0;
        }
    }
    // Scores of slots the query does not see become -inf; node0: the new token that the lane's first slot holds
    // (negative: a committed slot, which every query sees).  Selects, not branches: a lane's eight slots may fall on
    // either side of every limit.
    __device__ __forceinline__ void hide(f32x4 (&S)[QT][2], int node0, bool masked) const {
        if (masked) {
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int node = node0 + 16 * (j / 4) + j % 4;
                    const bool sees = (node < 0) | ((node < 64) & static_cast<int>((tree[qt] >> (node & 63)) & 1u));
                    S[qt][j / 4][j % 4] = sees ? S[qt][j / 4][j % 4] : -INFINITY;
                }
            }
        } else {
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    S[qt][j / 4][j % 4] = node0 + 16 * (j / 4) + j % 4 <= tok[qt] ? S[qt][j / 4][j % 4] : -INFINITY;
        }
    }
};

// Running maximum, sum and output of a wave's queries.  m follows the true
// maximum within a factor of 2^8 of the probabilities (slack): sums stay as exact
// in float32, a bf16 keeps its eight bits at any size, and a step whose scores
// stay below needs no exchange between the lanes and no rescaling.
template <int D, int QT, int NP> struct Softmax {
    static constexpr int kNT = D / 16;                  // 16-row tiles of O^T
    f32x4 O[QT][kNT];
    float m[QT], l[QT];
    __device__ __forceinline__ Softmax() {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            m[qt] = -INFINITY;
            l[qt] = 0.f;
#pragma unroll
            for (int n = 0; n < kNT; ++n) O[qt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
    __device__ static __forceinline__ float slack(float cexp) { return fminf(8.f / cexp, 1e30f); }
    __device__ __forceinline__ void weigh(const f32x4 (&S)[QT][2], u32x4 (&P)[QT][NP], float cexp, float slack) {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            float mx = S[qt][0][0];
#pragma unroll
            for (int j = 1; j < 8; ++j) mx = fmaxf(mx, S[qt][j / 4][j % 4]);
            if (__ballot(mx > m[qt] + slack) != 0ull) {
                mx = fmaxf(mx, xshfl(mx, 16));
                mx = fmaxf(mx, xshfl(mx, 32));
                const float mn = fmaxf(m[qt], mx);
                const float al = m[qt] == -INFINITY ? 0.f : exp2_fast((m[qt] - mn) * cexp);
                l[qt] *= al;
#pragma unroll
                for (int n = 0; n < kNT; ++n) O[qt][n] *= al;
                m[qt] = mn;
            }
            const float mc = m[qt] == -INFINITY ? 0.f : m[qt] * cexp;
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] = exp2_fast(fmaf(S[qt][j / 4][j % 4], cexp, -mc));
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
    }
    // The sums over the keys of all four g-groups; queries that are not there give nothing.
    __device__ __forceinline__ void finish(const int (&tok)[QT]) {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            l[qt] += xshfl(l[qt], 16);
            l[qt] += xshfl(l[qt], 32);
            if (tok[qt] < 0) {
                m[qt] = -INFINITY;
                l[qt] = 0.f;
#pragma unroll
                for (int n = 0; n < kNT; ++n) O[qt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
        }
    }
    // Rows row0 .. of (unit, h) `uh` as a part to be joined, or as the call's output.  O^T tile n, register i is
    // element (D/16)*(4g + i) + n of query c.
    template <int DT>
    __device__ __forceinline__ void write(const KvqAttnArgs& a, int row0, int b, int h, long uh, bool part, int c,
                                          int g) const {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            const int r = row0 + qt * 16 + c;
            if (r >= a.M) continue;
            if (part) {
                const long at = uh * a.M + r;
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
                const long at = (static_cast<long>(b) * a.N + r / a.G) * a.Hq + h * a.G + r % a.G;
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
};

// What a workgroup works on: batch row, head and a part of its key axis.
struct Place {
    int b, h, cnt;
    long uh;                // (unit, head) index of its part
    bool ok, part;          // the batch row is valid; its units are to be joined
    long pre, k0, k1;       // committed slots; first key and the end of the unit (the row's slots may end before)
};
__device__ __forceinline__ bool kvq_place(const KvqAttnArgs& a, int uh, Place& p) {
    p.uh = uh;
    p.h = uh % a.c.H;
    const int unit = uh / a.c.H;
    int b = unit, split = 0, per = 0, mine = 1, pre;
    if (a.units) {
        const Lengths len(a);
        per = len.per();
        if (blockIdx.x == 0 && wave_id() == 0) len.note(per);
        if (!len.find(unit, per, b, split, mine)) return false;
        len.row(b, pre, p.cnt);
    } else if (b >= a.c.B) {
        return false;
    } else if (a.c.B > 1 && a.c.B <= kWave) {
        const Lengths len(a);
        b = len.by_length(b);
        len.row(b, pre, p.cnt);
    } else {
        pre = a.prefix[b];
        p.cnt = a.counts ? a.counts[b] : a.N;
    }
    p.b = b;
    p.part = mine > 1;
    p.pre = pre;
    p.ok = kvq_row_ok(static_cast<int>(p.pre), p.cnt, a.N, a.c.capacity);
    p.k0 = static_cast<long>(split) * per * kChunk;
    p.k1 = a.units ? p.k0 + static_cast<long>(per) * kChunk : a.c.capacity;
    if (!p.ok) p.pre = p.cnt = 0;
    return true;
}
// End of the slots that rows row0 .. row0 + rows - 1 see (0: no query there).
__device__ __forceinline__ long kvq_limit(const KvqAttnArgs& a, const Place& p, int row0, int rows) {
    const int end = min(p.cnt, (min(row0 + rows, a.M) - 1) / a.G + 1);
    return row0 < a.M && row0 / a.G < end ? p.pre + (a.mask ? p.cnt : end) : 0;
}

constexpr int kJoinThreads = 256;

// The lane's codes and scales of one step, as loaded.
template <int D> struct Raw {
    static constexpr int kKW = D / 32;                  // words of a quarter K row
    static constexpr int kVW = D <= 128 ? 1 : 2;        // words of a lane's V elements
    uint32_t k[2][kKW], ks[2];
    uint32_t v[8][kVW], vs[8];
};

// Reads keys through buffer descriptors that end at the last visible slot: what
// lies past it comes back as zeros (code 0, scale 0) and costs no traffic, so
// every step, the last and the one prefetched past the end too, is the same
// straight run of loads and the wait for a step never includes the next one's.
// A descriptor is one tile of 16 slots, and the loads' offsets are vector offsets
// (kvq_window.hpp says why).
template <int D> struct Loader {
    const uint8_t *kc, *ks, *vc, *vs;                   // of the (b, h)
    long cp, sp;
    uint32_t ko, kso, vo, vso;                          // the lane's offsets
    __device__ __forceinline__ Loader(const KvqCache& c, int b, int h, int lane) {
        const int col = lane & 15, g = lane >> 4;
        kc = c.kc + b * c.cb + h * c.ch;
        vc = c.vc + b * c.cb + h * c.ch;
        ks = c.ks + b * c.sb + h * c.sh;
        vs = c.vs + b * c.sb + h * c.sh;
        cp = c.cp;
        sp = c.sp;
        ko = k_offset(D, col, g, static_cast<int>(cp));
        kso = k_scale_offset(D, col, g, static_cast<int>(sp));
        vo = v_offset(D, col, g, static_cast<int>(cp));
        vso = v_scale_offset(D, col, g, static_cast<int>(sp));
    }
    // keys kb .. kb+31 of those below lim
    __device__ __forceinline__ void load_k(Raw<D>& r, int kb, int lim) const {
        load_k_step<D>(kc, ks, cp, sp, kb, lim, ko, kso, r.k, r.ks);
    }
    __device__ __forceinline__ void load_v(Raw<D>& r, int kb, int lim) const {
#if SV_KVQ_DEVICE
        const int cp32 = static_cast<int>(cp), sp32 = static_cast<int>(sp);
        const uint8_t *p = vc + kb * cp, *ps = vs + kb * sp;
        uint32_t o = vo, so = vso;
        asm volatile("" : "+v"(o), "+v"(so));           // the four offsets are formed every step, not kept
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int n = scalar_slots(kb + kTile * t, lim);
            const auto rv = tile_rsrc(p, t, cp32, n), rvs = tile_rsrc(ps, t, sp32, n);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t at = o + i * cp32, sat = so + i * sp32;
                uint32_t(&w)[Raw<D>::kVW] = r.v[4 * t + i];
                if (D == 64) w[0] = __builtin_amdgcn_raw_buffer_load_b16(rv, at, 0, 0);
                else if (D == 128) w[0] = __builtin_amdgcn_raw_buffer_load_b32(rv, at, 0, 0);
                else {
                    const auto x = __builtin_amdgcn_raw_buffer_load_b64(rv, at, 0, 0);
                    w[0] = x[0], w[Raw<D>::kVW - 1] = x[1];
                }
                r.vs[4 * t + i] = __builtin_amdgcn_raw_buffer_load_b8(rvs, sat, 0, 0);
            }
        }
#endif
    }
};

// Waves a SIMD to fit the registers of one variant to.
constexpr int attend_occupancy(int D, int DT, int QT) {
    const int size = (D / 64) * QT * (DT == 1 ? 2 : 3);     // of the sums and the queries
    return size <= 4 || (D == 128 && DT == 1) ? 3 : 2;
}
// 32 bf16 queries of D = 128 and 256 are read from LDS every step: their registers make room for a third wave a SIMD
// (prompts of 1023 tokens x 4 heads 74 -> 69 us), and for a second (27 nodes x 4 heads, 16 batch rows at 4096 keys,
// D = 256: 94 -> 68 us).
constexpr bool queries_in_lds(int D, int DT, int QT) { return D >= 128 && DT == 1 && QT == 2; }
template <bool ON> __device__ __forceinline__ void fence() {        // keeps operands from being formed early
#if SV_KVQ_DEVICE
    if (ON) __builtin_amdgcn_sched_barrier(0);
#endif
}
constexpr int larger(int a, int b) { return a > b ? a : b; }

template <int D, int DT, int QT, int WAVES>
__global__ __launch_bounds__(WAVES* kWave, attend_occupancy(D, DT, QT)) void kvq_attention_kernel(KvqAttnArgs a) {
    constexpr int NQ = DT == 1 ? 1 : 3, NP = NQ;
    constexpr int kNT = D / 16, kRows = 16 * QT;
    constexpr int kRound = kStep * WAVES;               // keys a workgroup takes at a time
    // (unit, head) pairs of one residue mod 8 with all their row tiles: neighbours in time on one XCD, whose L2 serves
    // the row tiles that read the same keys
    const int x = blockIdx.x % 8, y = blockIdx.x / 8;
    const int row0 = (a.row_tiles - 1 - y % a.row_tiles) * kRows;      // a prompt's last rows see the most keys
    Place pl;
    if (!kvq_place(a, y / a.row_tiles * 8 + x, pl)) return;
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const long lim = kvq_limit(a, pl, row0, kRows);
    const long k0 = pl.k0, k1 = min(pl.k1, lim);

    Queries<QT> qs;
    qs.place(a, row0, pl.cnt, c);
    // LDS: the queries during the loop (if they are there), the waves' sums after it
    constexpr bool kQL = queries_in_lds(D, DT, QT);
    constexpr int kQOps = kQL ? QT * NQ * (D / 32) : 0, kSumOps = WAVES / 2 * QT * kNT;
    __shared__ u32x4 shared[larger(kQOps, kSumOps)][kWave];
    __shared__ float sh_ml[WAVES / 2][kRows][2];
    u32x4 Q[kQL ? 1 : QT][NQ][D / 32];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        if (kQL && qt % WAVES != wave) continue;
        const int r = row0 + qt * 16 + c;
        const long off = pl.b * a.q.batch + max(qs.tok[qt], 0) * a.q.pos + (pl.h * a.G + r % a.G) * a.q.head;
        load_query<D, NQ, DT>(a.q, off, qs.tok[qt] >= 0, g, Q[kQL ? 0 : qt]);
        if (kQL) {
#pragma unroll
            for (int p = 0; p < NQ; ++p)
#pragma unroll
                for (int s = 0; s < D / 32; ++s) shared[(qt * NQ + p) * (D / 32) + s][lane] = Q[0][p][s];
        }
    }
    if (kQL) __syncthreads();
    if (a.mask && k1 > pl.pre) qs.read_mask(a, pl.b, pl.cnt, g);

    const Loader<D> ld(a.c, pl.b, pl.h, lane);
    Softmax<D, QT, NP> sm;
    const float slack = sm.slack(a.cexp);
    Raw<D> cur;
    long kb = k0 + kStep * wave;
    if (kb < k1) {
        ld.load_k(cur, kb, k1);
        ld.load_v(cur, kb, k1);
    }
    for (; kb < k1; kb += kRound) {
        // S^T = K Q^T
        f32x4 S[QT][2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) S[qt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (kQL) asm volatile("" ::: "memory");         // read again every step, not kept
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            u32x4 A[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float sc = scale_value(D == 256 && s >= 4 ? cur.ks[t] >> 8 : cur.ks[t]);
                const uint32_t w = cur.k[t][s];
                A[t] = u32x4{fp4_pair<0>(w, sc), fp4_pair<1>(w, sc), fp4_pair<2>(w, sc), fp4_pair<3>(w, sc)};
            }
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
#pragma unroll
                for (int p = 0; p < NQ; ++p) {
                    const u32x4 q = kQL ? shared[(qt * NQ + p) * (D / 32) + s][lane] : Q[kQL ? 0 : qt][p][s];
#pragma unroll
                    for (int t = 0; t < 2; ++t) S[qt][t] = mfma(A[t], q, S[qt][t]);
                }
            }
            fence<D == 256>();
        }
        ld.load_k(cur, kb + kRound, k1);
        if (qs.edge(a, kb, pl.pre, row0)) qs.hide(S, static_cast<int>(kb - pl.pre) + 4 * g, a.mask != nullptr);
        u32x4 P[QT][NP];
        sm.weigh(S, P, a.cexp, slack);

        // O^T += V^T P^T
        float vsc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // a block stored as NaN has zero codes: its V is finite, and its K row says NaN.  Nor may bytes that append
            // does not write give an infinity, which would reach queries that give the slot no weight.
            vsc[j] = scale_value(min(cur.vs[j], static_cast<uint32_t>(kQScaleMax)));
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
                for (int p = 0; p < NP; ++p) {
                    sm.O[qt][2 * pr] = mfma(lo, P[qt][p], sm.O[qt][2 * pr]);
                    sm.O[qt][2 * pr + 1] = mfma(hi, P[qt][p], sm.O[qt][2 * pr + 1]);
                }
            }
            fence<D == 256>();
        }
        ld.load_v(cur, kb + kRound, k1);
    }

    // join the waves, half of them at a time through LDS
    f32x4(*const sh_o)[kWave] = reinterpret_cast<f32x4(*)[kWave]>(shared);
    sm.finish(qs.tok);
#pragma unroll
    for (int half = WAVES / 2; half >= 1; half >>= 1) {
        __syncthreads();
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
#pragma unroll
                for (int n = 0; n < kNT; ++n) sh_o[((wave - half) * QT + qt) * kNT + n][lane] = sm.O[qt][n];
                if (g == 0) {
                    sh_ml[wave - half][qt * 16 + c][0] = sm.m[qt];
                    sh_ml[wave - half][qt * 16 + c][1] = sm.l[qt];
                }
            }
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                const float om = sh_ml[wave][qt * 16 + c][0], ol = sh_ml[wave][qt * 16 + c][1];
                const float mn = fmaxf(sm.m[qt], om);
                const float wa = sm.m[qt] == -INFINITY ? 0.f : exp2_fast((sm.m[qt] - mn) * a.cexp);
                const float wb = om == -INFINITY ? 0.f : exp2_fast((om - mn) * a.cexp);
                sm.m[qt] = mn;
                // a sum that is NaN stays NaN whatever its maximum
                sm.l[qt] = sm.l[qt] * wa + ol * wb;
#pragma unroll
                for (int n = 0; n < kNT; ++n) sm.O[qt][n] = sm.O[qt][n] * wa + sh_o[(wave * QT + qt) * kNT + n][lane] * wb;
            }
        }
    }
    if (wave == 0) sm.template write<DT>(a, row0, pl.b, pl.h, pl.uh, pl.part, c, g);
}

// Joins the units of each query row: D/4 neighbouring threads a row, four elements each, and S such groups that
// share the row's units and add up through LDS.
template <int D, int DT, int S>
__global__ __launch_bounds__(kJoinThreads) void kvq_join_kernel(KvqAttnArgs a) {
    constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes, kRowsWg = kGroups / S;
    const int d = static_cast<int>(threadIdx.x % kLanes) * 4;
    const int grp = threadIdx.x / kLanes, sub = grp % S, rw = grp / S;
    // rows of one (b, h) a workgroup, so that the units are found once
    const int tiles = (a.M + kRowsWg - 1) / kRowsWg;
    const int r = static_cast<int>(blockIdx.x % tiles) * kRowsWg + rw, bh = blockIdx.x / tiles;
    const int h = bh % a.c.H, b = bh / a.c.H;
    const int first = a.first_unit[b], used = a.first_unit[b + 1] - first;
    if (used == 1) return;                              // written by its one unit
    const bool live = r < a.M;
    const long step = static_cast<long>(a.c.H) * a.M;
    const long at0 = (static_cast<long>(first) * a.c.H + h) * a.M + (live ? r : 0);
    float m = -INFINITY, l = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = sub; s0 < used; s0 += 4 * S) {
        // four units at a time: their loads are independent
        float ms[4], ls[4];
        f32x4 os[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int s = min(s0 + e * S, used - 1);
            const long at = at0 + s * step;
            ms[e] = a.part_ml[2 * at];
            ls[e] = a.part_ml[2 * at + 1];
            os[e] = *reinterpret_cast<const f32x4*>(a.part_o + at * D + d);
        }
        float mn = m;
#pragma unroll
        for (int e = 0; e < 4; ++e) mn = fmaxf(mn, ms[e]);
        const float w = m == -INFINITY ? 0.f : exp2_fast((m - mn) * a.cexp);
        l *= w;
        o *= w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float we = ms[e] == -INFINITY || s0 + e * S >= used ? 0.f : exp2_fast((ms[e] - mn) * a.cexp);
            l += s0 + e * S < used ? ls[e] * we : 0.f;
            o += os[e] * we;
        }
        m = mn;
    }
    if (S > 1) {
        __shared__ float sh[kGroups][kLanes][4];
        __shared__ float sml[kGroups][2];
        *reinterpret_cast<f32x4*>(sh[grp][threadIdx.x % kLanes]) = o;
        if (d == 0) sml[grp][0] = m, sml[grp][1] = l;
        __syncthreads();
        if (sub != 0) return;
        float mn = m;
#pragma unroll
        for (int e = 1; e < S; ++e) mn = fmaxf(mn, sml[grp + e][0]);
        const float w = m == -INFINITY ? 0.f : exp2_fast((m - mn) * a.cexp);
        l *= w;
        o *= w;
#pragma unroll
        for (int e = 1; e < S; ++e) {
            const float me = sml[grp + e][0];
            const float we = me == -INFINITY ? 0.f : exp2_fast((me - mn) * a.cexp);
            l += sml[grp + e][1] * we;
            o += *reinterpret_cast<const f32x4*>(sh[grp + e][threadIdx.x % kLanes]) * we;
        }
        m = mn;
    }
    if (!live) return;
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

template <int D, int DT, int S> void join(const KvqAttnArgs& a, hipStream_t s) {
    constexpr int rows = kJoinThreads / (D / 4) / S;
    const unsigned grid = static_cast<unsigned>(a.c.B) * a.c.H * ((a.M + rows - 1) / rows);
    kvq_join_kernel<D, DT, S><<<dim3(grid), kJoinThreads, 0, s>>>(a);
}

template <int D, int DT, int QT, int WAVES> void attend(const KvqAttnArgs& a, hipStream_t s, Timing t) {
    const long uh = static_cast<long>(a.units ? a.units : a.c.B) * a.c.H;
    const dim3 grid(static_cast<unsigned>((uh + 7) / 8 * 8 * a.row_tiles));
    launch_timed(t, kvq_attention_kernel<D, DT, QT, WAVES>, grid, dim3(WAVES * kWave), 0, s, a);
}
// 16-row tiles of a workgroup's queries: two share each key's conversion where the registers allow two waves a SIMD
// (float32 at D = 128 and 256 does not: 27 nodes x 4 heads, 16 batch rows at 4096 keys, 69 us against 61 with one).
constexpr int most_tiles(int D, int DT) { return DT == 1 || D == 64 ? 2 : 1; }

template <int D, int DT> void attend(const KvqAttnArgs& a, hipStream_t s, Timing t) {
    if (a.q_tiles == 2) {
        if constexpr (most_tiles(D, DT) == 2) attend<D, DT, 2, 4>(a, s, t);
    } else if (a.waves == 8) {
        attend<D, DT, 1, 8>(a, s, t);
    } else {
        attend<D, DT, 1, 4>(a, s, t);
    }
    if (!a.units) return;
    if (a.units >= 4 * a.c.B) join<D, DT, 4>(a, s);     // many units a row
    else join<D, DT, 1>(a, s);
}

}  // namespace

// The key axis is split so that a launch has about 512 workgroups (two a compute unit: 131071 keys, 8 heads, 32 rows
// each: 39 + 5 us; 1024 workgroups 51 + 12, 256 41 + 5), into units of 256 keys at least.  A cache of up to 1024 slots
// is not: its one launch beats two (one token of 8 heads at 1000 keys: 9.8 us in a cache of 1024 slots, 12.3 in one of
// 1025), with eight waves where the rows fit one tile.  Nor are batches whose row tiles alone are 512 workgroups, whatever
// their lengths (the host knows none): one sequence of 131071 keys among 63 of 1000, 8 heads, is 720 us, and 370 among 62,
// where it gets two units.
void kvq_attention_plan(KvqAttnArgs& a) {
    a.q_tiles = a.M > 16 ? most_tiles(a.c.D, a.dtype) : 1;
    const int rows = 16 * a.q_tiles;
    a.row_tiles = (a.M + rows - 1) / rows;
    const long target = 512, items = static_cast<long>(a.c.B) * a.c.H * a.row_tiles;
    a.units = 0;
    a.min_per = 2;
    a.waves = 4;
    if (items >= target) return;
    if (a.c.capacity > 1024) {
        const long units = target / (static_cast<long>(a.c.H) * a.row_tiles);
        const long chunks = (static_cast<long>(a.c.capacity) + kChunk - 1) / kChunk * a.c.B;
        a.units = static_cast<int>(units < chunks ? units : chunks);
    } else if (a.q_tiles == 1) {
        a.waves = 8;
    }
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
