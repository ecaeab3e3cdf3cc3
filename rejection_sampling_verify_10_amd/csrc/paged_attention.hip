// Softmax attention over a paged cache: a prefix that many batch rows share, each
// row's own slots and the visible new ones.
//
// One pass over the keys with a running maximum and sum: S = q . K_s,
// P = exp2(c*(S - m)), O += P V_s, c = scale*log2(e); units of a plan
// (paged_plan.hip) that belong together join at the end.
//
// K and V come to LDS in tiles of 32 keys, by loads that go there directly.  A unit
// of up to 128 query rows: its four waves have 32 rows each and share the tiles,
// which are brought four ahead.  One of up to 32: its waves have the same rows and
// every fourth tile each, all by themselves, and join at the end.  On 32x32x16 bf16
// MFMAs in the transposed form, S^T = K Q^T and O^T = V^T P^T, a lane has one query:
// lane (c, h), c = lane%32, h = lane/32, ends up with scores of query c against keys
// 8a + 4h + i (a, i < 4), and those, rounded to bf16, ARE the second product's
// operand when its contraction runs over keys in that order.  V's operand wants
// four keys of one element: the transposing LDS read gives them.  LDS rows are
// permuted in 16-byte chunks so that neither read has bank conflicts.
//
// float32 queries enter as three bf16 parts, and so does P: exact both.  With bf16
// queries P has two parts in units of up to 32 query rows, 2^-17 of it off, which wait
// for memory (64 sequences of 4096 keys 125.9 us, 126.4 with two; four of 600 12.8 and
// 13.3).  In those of up to 128 it rounds to one bf16: beside the output's own rounding,
// a third more error (0.0022 of the outputs off the 64-bit ones, 0.0017 with the latter
// alone).  A second part takes 21-35% longer there (64 sequences behind 32768 keys 109
// -> 139 us, 32 chains of eight 81 -> 98); who wants it passes the queries widened to
// float32.
//
// The sum is float32, a tile's added together first, with what it rounds off kept
// beside it.  An output's is the matrix instruction's: eight keys' products at a time.
//
// What bounds it (D = 128, 8 heads, bf16): many query rows, the tiles' way through LDS
// (a wave reads all of a tile for 32 rows: 600 of some 1400 clocks a tile) beside the
// products (64 rows of 8 tokens x 4 heads behind 65536 keys in common: 872-885 TFLOP/s,
// matrix units busy half of the time; a library product of 8192^3 1089); few, HBM (one sequence of 131072 keys:
// 99 us, 5.4 TB/s; the read probe 7.0); in between both (64 sequences of one token
// behind 32768 keys, ragged tails to 1024: 102-125 us by the clock, 304 MB, 70 GFLOP);
// short ones, a chain of latencies (4 sequences of one token, 600 keys: 7.4 + 3.5 us).

#include <stddef.h>

#include <type_traits>

#include "kvq.hpp"
#include "paged.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTileKeys = 32;                           // keys of a tile
constexpr int kWindow = kWave;                          // 16-key groups whose pages a wave holds, one a lane
constexpr int kBatch = 8;                               // parts under way in the join
constexpr float kSlack = 8.f;                           // powers of two a score may pass the running maximum by
constexpr float kFar = 1024.f;                          // of a maximum in base two: half a step of it is 2^-15 and more from here on

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ f32x16 mfma32(const u32x4& a, const u32x4& b, const f32x16& c) {
#if SV_KVQ_DEVICE
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
#else
    return c;
#endif
}
// The same with the sums in AGPRs, for good: left to itself the compiler takes them to VGPRs and back in every tile, for the few
// tiles that rescale them, and spills others (float32 chains of eight behind 16384 keys, D = 256: 318 us, 206 so). It sees no
// matrix instruction here, so the waits are ours: two states after a VALU write of an operand, four after one of exec; sums_done
// before anything else reads or writes the sums, sums_set after it has. Products that follow each other on the same sums
// need none.
__device__ __forceinline__ void mfma32_sums(const u32x4& a, const u32x4& b, f32x16& c) {
#if SV_KVQ_DEVICE
    asm("s_nop 3\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
#endif
}
__device__ __forceinline__ void sums_done(f32x16& c) {
#if SV_KVQ_DEVICE
    asm volatile("s_nop 15\n\ts_nop 15" : "+a"(c));
#endif
}
__device__ __forceinline__ void sums_set(f32x16& c) {
#if SV_KVQ_DEVICE
    asm volatile("s_nop 3" : "+a"(c));
#endif
}
// Four 16-bit elements down a column of the 4 x 16 tile that sixteen lanes point at, four elements each.
__device__ __forceinline__ u32x2 read_transposed(const unsigned char* p) {
#if SV_KVQ_DEVICE
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p)));
#else
    return u32x2{0u, 0u};
#endif
}

// LDS rows of D elements in 16-byte chunks.  K: sixteen keys' same chunk falls on sixteen different ones of 256 bytes; V: four
// keys' same pair of chunks on four different pairs.
template <int D> __device__ __forceinline__ constexpr int k_turn(int key) { return D == 64 ? (key >> 1) & 7 : key & 15; }
template <int D> __device__ __forceinline__ constexpr int v_turn(int key) { return D == 64 ? 2 * ((key >> 1) & 3) : 2 * (key & 7); }
template <int D> __device__ __forceinline__ constexpr int k_at(int key, int chunk) { return key * 2 * D + ((chunk ^ k_turn<D>(key)) << 4); }
template <int D> __device__ __forceinline__ constexpr int v_at(int key, int chunk) { return key * 2 * D + ((chunk ^ v_turn<D>(key)) << 4); }

constexpr int kStages = 4;                              // tiles under way; a power of two, at most half a window
template <int D> struct Lds {
    unsigned char k[kStages][kTileKeys * 2 * D];
    unsigned char v[kStages][kTileKeys * 2 * D];
    int32_t page[kWaves][kWindow];
    float ml[kWaves][2][kWave];
};

// Query row r of a unit's job: its batch row, token and head.
struct QueryRow {
    int b, n, g;
};
__device__ __forceinline__ QueryRow query_row(const PagedAttnArgs& a, int b0, int r) {
    QueryRow q;
    const int row = r / a.M, in = r - row * a.M;
    q.b = b0 + row;
    q.n = in / a.G;
    q.g = in - q.n * a.G;
    return q;
}

#if SV_KVQ_DEVICE
// 16 (or 4) bytes a lane from base + offset to LDS at `to` + 16 (4) * lane.  As assembly, so that the compiler does not wait for
// them at every read of LDS; the loads write no register.  ONCE: what no other workgroup reads is not kept in the caches
// (one sequence of 131072 keys: 111 -> 99 us).
template <bool ONCE> __device__ __forceinline__ void load_lds16(unsigned to, unsigned offset, unsigned long long base) {
    if (ONCE) asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(to), "v"(offset), "s"(base) : "memory");
    else asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void load_lds4(unsigned to, unsigned offset, unsigned long long base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory");
}
template <int N> __device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ unsigned lds_address(const void* p) {
    return static_cast<unsigned>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)(p)));
}
#else
template <bool ONCE> __device__ __forceinline__ void load_lds16(unsigned, unsigned, unsigned long long) {}
__device__ __forceinline__ void load_lds4(unsigned, unsigned, unsigned long long) {}
template <int N> __device__ __forceinline__ void wait_loads() {}
__device__ __forceinline__ void wait_lds() {}
__device__ __forceinline__ void barrier() {}
__device__ __forceinline__ unsigned lds_address(const void*) { return 0; }
#endif

// Brings tiles of a unit's keys to LDS. A load of a wave is 1 KiB: kKeys keys. Four waves share a tile's loads (each has some of
// one of its two 16-key groups), or a wave makes them all (ALONE), to the buffer of its number. Groups past the end repeat
// the last one. The pages of 64 groups, a window, are held one a lane.
template <int D, bool ALONE> struct Loader {
    static constexpr int kRow = D / 8, kKeys = kWave / kRow;
    static constexpr int kN = ALONE ? 16 / kKeys : kTileKeys / kKeys / kWaves;      // loads of a group
    static constexpr int kLoads = 2 * kN;               // of K and V, a tile (not ALONE)
    const PagedAttnArgs& a;
    const int32_t* table;
    Lds<D>& lds;
    int h, k0, end;
    unsigned ko[kN], vo[kN];                            // the lane's offsets from its group's first row, bytes
    unsigned to;                                        // LDS address of the wave's loads in the first buffer of K (ALONE: in its own)
    long long first;                                    // lane i: where group i of this window begins, bytes
    unsigned long long bad;                             // groups of the window that have no page

    __device__ __forceinline__ Loader(const PagedAttnArgs& a, const PagedUnit& u, int h, Lds<D>& lds)
        : a(a), table(a.tables + u.table * a.table_stride), lds(lds), h(h), k0(u.k0), end(u.k1) {
        const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
        to = ALONE ? lds_address(lds.k[wave]) : lds_address(lds.k[0]) + wave * kN * 1024;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int key = ((ALONE ? 0 : wave * kN) + i) * kKeys + lane / kRow, chunk = lane % kRow;
            const unsigned row = static_cast<unsigned>(key & 15) * static_cast<unsigned>(a.c.slot_stride) * 2u;
            ko[i] = row + ((chunk ^ k_turn<D>(key)) << 4);
            vo[i] = row + ((chunk ^ v_turn<D>(key)) << 4);
        }
    }
    __device__ __forceinline__ int last_group() const { return (end - 1) & ~15; }
    // First key of the lane's group of window w.
    __device__ __forceinline__ int group_key(int w) const {
        return min(k0 + 16 * (w * kWindow + static_cast<int>(threadIdx.x & (kWave - 1))), last_group());
    }
    __device__ __forceinline__ void take(int w, int page) {
        const bool none = page < 0 || page >= a.c.pages;
        bad = __ballot(none);
        first = 2 * ((none ? 0 : page) * a.c.page_stride + (group_key(w) & ((1 << a.c.page_log2) - 1)) * a.c.slot_stride +
                     h * a.c.head_stride);
    }
    __device__ __forceinline__ void first_window() { take(0, table[group_key(0) >> a.c.page_log2]); }
    __device__ __forceinline__ int32_t* slot(int w) const { return lds.page[ALONE ? wave_id() : w & 1]; }
    __device__ __forceinline__ void next_window(int w) { take(w, slot(w)[threadIdx.x & (kWave - 1)]); }
    __device__ __forceinline__ void fetch_window(int w) const {         // one load of the wave's (or of the first one's)
        if (ALONE || wave_id() == 0)
            load_lds4(lds_address(slot(w)), static_cast<unsigned>(group_key(w) >> a.c.page_log2) * 4u,
                      reinterpret_cast<unsigned long long>(table));
    }
    // Where a group of the window at hand begins in the pages, bytes.
    __device__ __forceinline__ unsigned long long where(int group) const {
        return (static_cast<unsigned long long>(bcast(static_cast<int>(first >> 32), group & (kWindow - 1))) << 32) |
               static_cast<unsigned>(bcast(static_cast<int>(first), group & (kWindow - 1)));
    }
    __device__ __forceinline__ void load_group(const uint16_t* pages, unsigned long long off, unsigned at, const unsigned (&o)[kN]) const {
        const unsigned long long base = reinterpret_cast<unsigned long long>(pages) + off;
#pragma unroll
        for (int i = 0; i < kN; ++i) load_lds16<ALONE>(at + 1024 * i, o[i], base);
    }
    static constexpr unsigned kV = kStages * kTileKeys * 2 * D;         // from K's buffers to V's
    // Tile t, whose groups are in the window at hand, to buffer `buf` (not ALONE).
    __device__ __forceinline__ void load(int t, int buf) const {
        const unsigned long long off = where(2 * t + (wave_id() >= kWaves / 2 ? 1 : 0));
        load_group(a.c.k, off, to + buf * (kTileKeys * 2 * D), ko);
        load_group(a.c.v, off, to + buf * (kTileKeys * 2 * D) + kV, vo);
    }
    // ALONE: K's half of it and V's.
    __device__ __forceinline__ void load_k(int t) const {
#pragma unroll
        for (int g = 0; g < 2; ++g) load_group(a.c.k, where(2 * t + g), to + g * 1024 * kN, ko);
    }
    __device__ __forceinline__ void load_v(int t) const {
#pragma unroll
        for (int g = 0; g < 2; ++g) load_group(a.c.v, where(2 * t + g), to + kV + g * 1024 * kN, vo);
    }
};

template <int D, int NQ, int DT>
__device__ __forceinline__ void load_query(const PagedRows& q, long long off, bool live, int h2, u32x4 (&out)[NQ][D / 16]) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        const long long i = off + 16 * s + 8 * h2;
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

// A wave's 32 queries: Q, and the running maximum, sum and output (NT tiles of 32 elements of O^T).
template <int D, int DT> struct Wave {
    static constexpr int NT = D / 32;
    static constexpr int NQ = DT == 1 ? 1 : 3;
    static constexpr int kWideP = NQ, kNarrowP = DT == 1 ? 2 : 3;       // parts of P, in a wide unit and in a narrow one
    static constexpr bool kSums = D == 256;             // O is in AGPRs
    // V's operands are read before the scores' products where there are registers to hold them.
    static constexpr bool kEarlyV = D == 64 || (D == 128 && DT == 1);
    // K's before the tile's turn, likewise: in a wide unit (bf16 chains of eight, D = 128: 85 us with, 82 without, D = 256: 128 and
    // 139; float32 ones behind 16384 keys, D = 256: 573 and 324, much of it spilled registers) and in a narrow one, whose buffer
    // is free sooner with them (64 sequences of one bf16 token: 120 us, 135 without).
    static constexpr bool kWideK = D == 64 || (D == 256 && DT == 1), kNarrowK = D == 64 || DT == 1;
    u32x4 Q[NQ][D / 16];
    f32x16 O[NT];
    float m, l, low;                                    // the sum is l + low
    bool far;                                           // a maximum of the wave's passes kFar
    u32x4 K[D / 16];                                    // of the tile to come
    u32x4 V[kEarlyV ? 2 : 1][NT];
    unsigned ka, va;                                    // the lane's LDS offsets in a buffer of K and V
    __device__ __forceinline__ Wave() : m(-INFINITY), l(0.f), low(0.f), far(false) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) O[t][i] = 0.f;
        if (kSums) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sums_set(O[t]);
        }
        const int lane = threadIdx.x & (kWave - 1), c = lane & 31, h2 = lane >> 5;
        ka = k_at<D>(c, h2);
        va = v_at<D>(4 * h2 + (lane & 15) / 4, 2 * ((lane >> 4) & 1) + (lane & 3) / 2) + 8 * (lane & 1);
    }
    // Chunks are turned by an exclusive or, so that of another chunk is one away: k_at(c, 2s + h2) = ka ^ 32s, and v_at with
    // chunks 4t more is va ^ 64t. Eight keys on is the same turn.
    __device__ __forceinline__ u32x4 read_k(const Lds<D>& lds, int buf, int s) const {
        return *reinterpret_cast<const u32x4*>(lds.k[buf] + (ka ^ (32 * s)));
    }
    __device__ __forceinline__ void read_k(const Lds<D>& lds, int buf) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) K[s] = read_k(lds, buf, s);
    }
    __device__ __forceinline__ void read_v(const Lds<D>& lds, int buf, int s, u32x4 (&out)[NT]) const {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const unsigned char* p = lds.v[buf] + (va ^ (64 * t)) + 16 * s * 2 * D;
            const u32x2 lo = read_transposed(p), hi = read_transposed(p + 8 * 2 * D);
            out[t] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
    }

    __device__ __forceinline__ void read_v(const Lds<D>& lds, int buf) {
#pragma unroll
        for (int s = 0; s < 2; ++s) read_v(lds, buf, s, V[kEarlyV ? s : 0]);
    }
    template <bool READ> __device__ __forceinline__ f32x16 scores(const Lds<D>& lds, int buf) const {     // READ: K's operands are
        f32x16 s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const u32x4 k = READ ? K[i] : read_k(lds, buf, i);
#pragma unroll
            for (int p = 0; p < NQ; ++p) s = mfma32(k, Q[p][i], s);
        }
        return s;
    }
    // V's elements that are no numbers would reach queries that give their key no weight: they become zeros in an operand,
    // and the keys they belong to come back as bits.
    __device__ __forceinline__ static unsigned clean(u32x4& w) {
        unsigned odd = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool lo = (w[e] & 0x7f80u) == 0x7f80u, hi = (w[e] & 0x7f800000u) == 0x7f800000u;
            odd |= (lo ? 1u : 0u) << (2 * e) | (hi ? 2u : 0u) << (2 * e);
            w[e] = (lo ? 0u : w[e] & 0xffffu) | (hi ? 0u : w[e] & 0xffff0000u);
        }
        return odd;
    }
    // Nonzero where an element's exponent is all ones: a half's exponent and one more make its top bit, and no carry.
    __device__ __forceinline__ static unsigned not_finite(const u32x4& w) {
        unsigned any = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) any |= (w[e] & 0x7f807f80u) + 0x00800080u;
        return any & 0x80008000u;
    }
    // The keys of the lane's scores, as bits, that are no numbers: V's elements of them (cleaned, where they are held), and
    // those of groups without a page. Seldom any: the tile is looked over first.
    __device__ __forceinline__ unsigned odd_keys(const Lds<D>& lds, int buf, unsigned none) {
        const int h2 = (threadIdx.x & (kWave - 1)) >> 5;
        unsigned odd = (none & 1 ? 0xffu : 0u) | (none & 2 ? 0xff00u : 0u);
        unsigned some = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (!kEarlyV) read_v(lds, buf, s, V[0]);
#pragma unroll
            for (int t = 0; t < NT; ++t) some |= not_finite(V[kEarlyV ? s : 0][t]);
        }
        if (__ballot(some != 0) == 0ull) return odd;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (!kEarlyV) read_v(lds, buf, s, V[0]);
            unsigned any = 0;
#pragma unroll
            for (int t = 0; t < NT; ++t) any |= clean(V[kEarlyV ? s : 0][t]);
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                const unsigned long long all = __ballot((any >> j) & 1u);
                odd |= (static_cast<unsigned>(h2 ? all >> 32 : all) ? 1u : 0u) << (8 * s + j);
            }
        }
        return odd;
    }
    // P of a tile's scores (which may be gone then), and the maximum and sums.
    template <int NP> __device__ __forceinline__ void weigh(f32x16& S, float cexp, float slack, u32x4 (&P)[NP][2]) {
        float mx = S[0];                                // NaN propagates, and moves no maximum
#pragma unroll
        for (int i = 1; i < 15; i += 2) mx = maximum3(mx, S[i], S[i + 1]);
        mx = __builtin_elementwise_maximum(mx, S[15]);
        if (__ballot(mx > m + slack) != 0ull) {
            // each query by itself: what one sees moves no other's maximum
            mx = __builtin_elementwise_maximum(mx, xshfl(mx, 32));
            const float mn = mx > m + slack ? mx : m;
            const float al = m == -INFINITY ? 0.f : exp2_fast((m - mn) * cexp);
            l *= al;
            low *= al;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (kSums) sums_done(O[t]);
                O[t] *= al;
                if (kSums) sums_set(O[t]);
            }
            m = mn;
            far = __ballot(fabsf(m) * cexp >= kFar && m > -INFINITY) != 0ull;
        }
        const float mr = m == -INFINITY ? 0.f : m;
        float mc = mr * cexp;
        if (__builtin_expect(far, 0)) {                                      // its rounding would be in every exponent; each query by itself, again
            const bool mine = fabsf(mr) * cexp >= kFar;
            mc = mine ? 0.f : mc;
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] -= mine ? mr : 0.f;
        }
        float sum[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = exp2_fast(__builtin_fmaf(S[8 * s + i], cexp, -mc));
            sum[s] = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
            for (int x = 0; x < NP; ++x) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    P[x][s][e] = pack_bf16(p[2 * e], p[2 * e + 1]);
                    p[2 * e] -= bf16_lo(P[x][s][e]);
                    p[2 * e + 1] -= bf16_hi(P[x][s][e]);
                }
            }
        }
        // Behind a key of weight 1 what a tile adds may be less than l's last place: low has what l leaves behind (one key and 16384 of
        // 2^-25 behind it: lse off by 2.4e-4 with a key at a time added to l; 1% of the time).
        const float t = sum[0] + sum[1], to = l + t, back = to - l;
        low += (l - (to - back)) + (t - back);
        l = to;
    }
    // After the last tile: the sum over both halves of the lanes' keys.
    __device__ __forceinline__ void finish() {
        l += low;
        l += xshfl(l, 32);
        if (kSums) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sums_done(O[t]);
        }
    }
    // O += V P. V's operands are in registers, or still in the buffer (and perhaps to be cleaned).
    template <int NP> __device__ __forceinline__ void add(const Lds<D>& lds, int buf, const u32x4 (&P)[NP][2], bool edge) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (!kEarlyV) {
                read_v(lds, buf, s, V[0]);
                if (edge) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) clean(V[0][t]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < NP; ++x) {
                    if (kSums) mfma32_sums(V[kEarlyV ? s : 0][t], P[x][s], O[t]);
                    else O[t] = mfma32(V[kEarlyV ? s : 0][t], P[x][s], O[t]);
                }
        }
    }
};

// The new tokens that a query of a masked call sees, as bits.
__device__ __forceinline__ unsigned long long read_mask(const PagedAttnArgs& a, int b, int tok, int cnt) {
    const int h2 = (threadIdx.x & (kWave - 1)) >> 5;
    const uint8_t* row = a.mask + b * a.mask_batch + static_cast<long long>(max(tok, 0)) * a.N;
    unsigned bits = 0;
    for (int e = 0; e < 32; ++e) {
        const int node = 32 * h2 + e;
        bits |= static_cast<unsigned>((row[min(node, a.N - 1)] != 0) & (node < cnt)) << e;
    }
    const unsigned other = xshfl(bits, 32);
    const unsigned lo = h2 ? other : bits, hi = h2 ? bits : other;
    return (static_cast<unsigned long long>(hi) << 32) | lo;
}

// Rows of O^T tile t0 + t, register i: element 32*(t0 + t) + 8*(i/4) + 4*h2 + i%4 of query c, to the call's output or a part.
template <int D, int DT, int NT>
__device__ __forceinline__ void write_rows(const PagedAttnArgs& a, const PagedUnit& u, int h, int r, int t0, bool first,
                                           const f32x16 (&O)[NT], float m, float l, bool live) {
    const int h2 = (threadIdx.x & (kWave - 1)) >> 5;
    if (r >= u.rows) return;
    if (u.part >= 0) {
        const long long at = (static_cast<long long>(u.part) + (r - u.row0)) * a.c.H + h;
        if (h2 == 0 && first) {
            a.part_ml[2 * at] = m;
            a.part_ml[2 * at + 1] = l;
        }
        float* o = a.part_o + at * D + 4 * h2;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f32x4*>(o + 32 * (t0 + t) + 8 * i) =
                    f32x4{O[t][4 * i], O[t][4 * i + 1], O[t][4 * i + 2], O[t][4 * i + 3]};
        return;
    }
    const QueryRow q = query_row(a, u.b0, r);
    const long long at = (static_cast<long long>(q.b) * a.N + q.n) * a.Hq + h * a.G + q.g;
    const bool empty = !live || l == 0.f;
    const float inv = empty ? 0.f : 1.f / l;
    if (h2 == 0 && first && a.out_lse)
        a.out_lse[at] = empty ? -INFINITY : (m * a.cexp + __builtin_amdgcn_logf(l)) * 0.69314718056f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long d = at * D + 32 * (t0 + t) + 8 * i + 4 * h2;
            float o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = empty ? 0.f : O[t][4 * i + e] * inv;
            if (DT == 1)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + d) = u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
            else
                *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + d) = f32x4{o[0], o[1], o[2], o[3]};
        }
}

// What the query of a lane sees: its token (-1: none there) and, in a tree, the new tokens as bits.
struct Sight {
    const PagedAttnArgs& a;
    const PagedUnit& u;
    int tok, seen;                  // slots below `seen` are seen by every query of the unit
    bool shared;
    unsigned long long tree;
    __device__ __forceinline__ Sight(const PagedAttnArgs& a, const PagedUnit& u, const QueryRow& q, bool there) : a(a), u(u) {
        shared = u.table != u.b0 || u.cnt == 0;
        tok = there && (shared || q.n < u.cnt) ? q.n : -1;
        seen = shared ? u.k1 : min(u.k1, a.mask ? u.pre : u.pre + u.row0 / a.G + 1);
        tree = !shared && a.mask && u.k1 > u.pre ? read_mask(a, q.b, tok, u.cnt) : 0;
    }
    // The keys of the tile that begins at `first` that the query sees, as bits.
    __device__ __forceinline__ unsigned sees(int first) const {
        const auto below = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; };
        const int node = first - u.pre;                 // the new token that the tile's first key is (negative: a committed slot)
        unsigned bits;
        if (a.mask) {
            const unsigned long long nodes = node >= 64 ? 0ull : node >= 0 ? tree >> node : node > -32 ? tree << -node : 0ull;
            bits = static_cast<unsigned>(nodes) | below(-node);
        } else {
            bits = below(tok + 1 - node);
        }
        return bits & below(u.k1 - first);
    }
    // Scores of that tile: -inf where the query does not see the key, NaN where the key is none.
    __device__ __forceinline__ void hide(f32x16& S, int first, unsigned odd) const {
        const unsigned bits = sees(first) >> (4 * ((threadIdx.x & (kWave - 1)) >> 5));
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = (bits >> (8 * (i / 4) + i % 4)) & 1u ? S[i] : -INFINITY;
        if (__ballot(odd != 0) != 0ull) {
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] = ((bits >> (8 * (i / 4) + i % 4)) & (odd >> i)) & 1u ? __builtin_nanf("") : S[i];
        }
    }
};

template <int D, int DT> __device__ __forceinline__ void load_queries(const PagedAttnArgs& a, const QueryRow& q, int h, bool there, Wave<D, DT>& w) {
    using W = Wave<D, DT>;
    const int h2 = (threadIdx.x & (kWave - 1)) >> 5;
    load_query<D, W::NQ, DT>(a.q, q.b * a.q.batch + q.n * a.q.pos + (static_cast<long long>(h) * a.G + q.g) * a.q.head, there, h2, w.Q);
}
// They are there: the compiler places no wait for them, which would be one for the tiles too, in the loop.
template <int D, int DT> __device__ __forceinline__ void queries_loaded(Wave<D, DT>& w) {
#pragma unroll
    for (int p = 0; p < Wave<D, DT>::NQ; ++p)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) asm volatile("" : "+v"(w.Q[p][i]));
}

constexpr int kPer = kWindow / 2;                       // tiles of a window of pages

// A unit of up to 128 query rows: wave w has rows 32w .. of it.
//
// An iteration: V's operands of its tile are read and the scores formed from K's, read before; then the next tile has
// arrived, this one's buffer takes the tile four further on, K's operands of the next are read, and the output follows. (Where
// there are no registers to hold K's or V's operands, they are read as the products need them.)
template <int D, int DT> __device__ __forceinline__ void attend_wide(const PagedAttnArgs& a, const PagedUnit& u, int h, Lds<D>& lds) {
    using W = Wave<D, DT>;
    using L = Loader<D, false>;
    const int r = u.row0 + 32 * wave_id() + static_cast<int>(threadIdx.x & 31);
    const bool there = r < u.rows;
    const QueryRow q = query_row(a, u.b0, there ? r : u.row0);
    const int tiles = (u.k1 - u.k0 + kTileKeys - 1) / kTileKeys;

    L ld(a, u, h, lds);
    if (tiles > 0) ld.first_window();
    W w;
    load_queries(a, q, h, there, w);
    const bool working = u.row0 + 32 * wave_id() < u.rows;
    const Sight sight(a, u, q, there);
    const float slack = fminf(kSlack / a.cexp, 1e30f);
    // The window of pages is that of the tile to be loaded; the tile worked on may lie in the one before.
    unsigned long long bad = tiles > 0 ? ld.bad : 0, bad_before = 0;

    for (int t = 0; t < min(kStages, tiles); ++t) ld.load(t, t);
    if (tiles > kPer) ld.fetch_window(1);
    queries_loaded(w);
    wait_loads<0>();
    barrier();
    if (W::kWideK && tiles > 0 && working) w.read_k(lds, 0);

    const auto iterate = [&](auto buffer, int t, bool edge, unsigned none) {
        const int buf = buffer;
        u32x4 P[W::kWideP][2];
        if (working) {
            if (W::kEarlyV) w.read_v(lds, buf);
            f32x16 S = w.template scores<W::kWideK>(lds, buf);
            if (edge) sight.hide(S, u.k0 + t * kTileKeys, w.odd_keys(lds, buf, none));
            w.weigh(S, a.cexp, slack, P);
            if (!W::kEarlyV) w.add(lds, buf, P, edge);
        }
        if (t + kStages <= tiles) wait_loads<(kStages - 2) * L::kLoads>();
        else wait_loads<0>();
        wait_lds();                                     // this wave has read all it wants of the buffer
        barrier();
        const int next = t + kStages;
        if (next < tiles) {
            if (next % kPer == 0) {
                ld.next_window(next / kPer);
                bad_before = bad;
                bad = ld.bad;
            }
            ld.load(next, buf);
            // the next window's pages, long before they are wanted
            if (next % kPer == 1 && next > kPer && next + kPer - 1 < tiles) ld.fetch_window(next / kPer + 1);
        }
        if (working) {
            if (W::kWideK && t + 1 < tiles) w.read_k(lds, (buf + 1) % kStages);
            if (W::kEarlyV) w.add(lds, buf, P, edge);
        }
    };
    int t = 0;
    // four at a time, their buffers known, while every query sees every key
    const int whole = max(0, sight.seen - u.k0) / kTileKeys;
    for (; t + kStages <= whole && (bad | bad_before) == 0; t += kStages) {
        iterate(std::integral_constant<int, 0>(), t, false, 0u);
        iterate(std::integral_constant<int, 1>(), t + 1, false, 0u);
        iterate(std::integral_constant<int, 2>(), t + 2, false, 0u);
        iterate(std::integral_constant<int, 3>(), t + 3, false, 0u);
    }
    for (; t < tiles; ++t) {
        const bool same = t / kPer == min(t + kStages - 1, tiles - 1) / kPer;     // the last tile loaded is in the window at hand
        const unsigned none = static_cast<unsigned>((same ? bad : bad_before) >> (2 * t & (kWindow - 1))) & 3u;
        iterate(t % kStages, t, t >= whole || none != 0, none);
    }
    w.finish();
    if (working) write_rows<D, DT, W::NT>(a, u, h, r, 0, true, w.O, w.m, w.l, sight.tok >= 0);
}

// A unit of up to 32 query rows: wave w has tiles w, w + 4, .. of its keys. Nothing passes between the waves before the end: a
// wave's operands are in registers when its next tile is brought over the one they came from.
template <int D, int DT> __device__ __forceinline__ void attend_narrow(const PagedAttnArgs& a, const PagedUnit& u, int h, Lds<D>& lds) {
    using W = Wave<D, DT>;
    const int wave = wave_id(), lane = threadIdx.x & (kWave - 1);
    const int r = u.row0 + (lane & 31);
    const bool there = r < u.rows;
    const QueryRow q = query_row(a, u.b0, there ? r : u.row0);
    const int tiles = (u.k1 - u.k0 + kTileKeys - 1) / kTileKeys;

    Loader<D, true> ld(a, u, h, lds);
    if (tiles > 0) ld.first_window();
    if (wave < tiles) {
        ld.load_k(wave);
        ld.load_v(wave);
        if (tiles > kPer) ld.fetch_window(1);
    }
    W w;
    load_queries(a, q, h, there, w);
    const Sight sight(a, u, q, there);
    const float slack = fminf(kSlack / a.cexp, 1e30f);
    queries_loaded(w);
    for (int t = wave; t < tiles; t += kWaves) {
        const unsigned none = static_cast<unsigned>(ld.bad >> (2 * t & (kWindow - 1))) & 3u;
        const int first = u.k0 + t * kTileKeys, next = t + kWaves;
        const bool edge = first + kTileKeys > sight.seen || none != 0;
        wait_loads<0>();
        if (W::kNarrowK) w.read_k(lds, wave);
        if (W::kEarlyV) w.read_v(lds, wave);
        wait_lds();
        if (next < tiles) {
            if (next / kPer != t / kPer) {
                ld.next_window(next / kPer);
                if ((next / kPer + 1) * kPer < tiles) {
                    wait_lds();                         // the window's pages are read before the next ones take their place
                    ld.fetch_window(next / kPer + 1);
                }
            }
            if (W::kNarrowK) ld.load_k(next);
            if (W::kEarlyV) ld.load_v(next);
        }
        f32x16 S = w.template scores<W::kNarrowK>(lds, wave);
        if (!W::kNarrowK && next < tiles) {
            wait_lds();
            ld.load_k(next);
        }
        u32x4 P[W::kNarrowP][2];
        if (edge) sight.hide(S, first, w.odd_keys(lds, wave, none));
        w.weigh(S, a.cexp, slack, P);
        w.add(lds, wave, P, edge);
        if (!W::kEarlyV && next < tiles) {
            wait_lds();
            ld.load_v(next);
        }
    }
    // join the waves: each leaves its sums, and takes a quarter of the elements (D = 64: two waves a half)
    w.finish();
    f32x16(*const sh)[W::NT][kWave] = reinterpret_cast<f32x16(*)[W::NT][kWave]>(&lds);
    static_assert(sizeof(f32x16) * kWaves * W::NT * kWave == offsetof(Lds<D>, page), "the sums take the buffers' place");
    wait_lds();
    barrier();
#pragma unroll
    for (int t = 0; t < W::NT; ++t) sh[wave][t][lane] = w.O[t];
    lds.ml[wave][0][lane] = w.m;
    lds.ml[wave][1][lane] = w.l;
    wait_lds();
    barrier();
    constexpr int kOwn = W::NT < kWaves ? 1 : W::NT / kWaves;
    if (wave * kOwn >= W::NT) return;
    float m = lds.ml[0][0][lane], l = 0.f;
#pragma unroll
    for (int i = 1; i < kWaves; ++i) m = fmaxf(m, lds.ml[i][0][lane]);
    f32x16 O[kOwn];
#pragma unroll
    for (int t = 0; t < kOwn; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) O[t][e] = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const float mi = lds.ml[i][0][lane], f = mi == -INFINITY ? 0.f : exp2_fast((mi - m) * a.cexp);
        l += lds.ml[i][1][lane] * f;                    // a sum that is NaN stays NaN whatever its maximum
#pragma unroll
        for (int t = 0; t < kOwn; ++t) O[t] += sh[i][wave * kOwn + t][lane] * f;
    }
    write_rows<D, DT, kOwn>(a, u, h, r, wave * kOwn, wave == 0, O, m, l, sight.tok >= 0);
}

// Whether the plan was made for a call of these sizes (one that was not names rows that are not there).
__device__ __forceinline__ bool plan_fits(const PagedAttnArgs& a) {
    const int32_t* h = a.p.head;
    return h[1] == a.B && h[2] == a.N && h[3] == a.M && h[4] == a.shape && h[5] == a.capacity;
}

constexpr int occupancy(int D, int DT) { return D == 256 ? 1 : 2; }

template <int D, int DT>
__global__ __launch_bounds__(kThreads, occupancy(D, DT)) void paged_attention_kernel(PagedAttnArgs a) {
    __shared__ __attribute__((aligned(256))) Lds<D> lds;
    const int unit = blockIdx.x / a.c.H, h = blockIdx.x % a.c.H;
    const PagedUnit u = a.p.unit[unit];                 // there is room for it, whether or not the plan has one
    if (!plan_fits(a) || unit >= a.p.head[0]) return;
    if (u.wide) attend_wide<D, DT>(a, u, h, lds);
    else attend_narrow<D, DT>(a, u, h, lds);
}

// Joins the parts of each query row: D/4 neighbouring lanes a row, four elements each. The lanes first weigh the row's parts, one
// each, so that the parts' loads wait for nothing.
template <int D, int DT>
__global__ __launch_bounds__(kThreads) void paged_join_kernel(PagedAttnArgs a, unsigned rows) {
    constexpr int kLanes = D / 4, kRows = kThreads / kLanes;
    const int sub = static_cast<int>(threadIdx.x) % kLanes, d = 4 * sub;
    const unsigned at = blockIdx.x * kRows + threadIdx.x / kLanes;      // (b, n, query head): fewer than 2^31 of them
    if (at >= rows) return;                             // kLanes lanes at a time
    const unsigned bn = at / a.Hq, hq = at - bn * a.Hq, h = hq / a.G;
    const int b = static_cast<int>(bn / a.N), n = static_cast<int>(bn - static_cast<unsigned>(b) * a.N);
    const int r = n * a.G + static_cast<int>(hq - h * a.G);
    const PagedOwn own = a.p.own[static_cast<long long>(b) * a.own_tiles + r / a.own_rows];
    const PagedShared sh = a.p.shared[b];
    if (!plan_fits(a) || own.count == 0) return;        // written by its one unit
    const int count = n < sh.live ? sh.count + own.count : 0;
    const auto part = [&](int i) {                      // the prefix's parts, then the row's own
        const long long p = i < sh.count ? sh.first + static_cast<long long>(i) * sh.step + r
                                         : own.first + static_cast<long long>(i - sh.count) * a.own_rows + r % a.own_rows;
        return p * a.c.H + h;
    };
    float m = -INFINITY, l = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < count; i0 += kLanes) {
        float mi = -INFINITY, li = 0.f;
        if (i0 + sub < count) {
            const long long p = part(i0 + sub);
            mi = a.part_ml[2 * p];
            li = a.part_ml[2 * p + 1];
        }
        float mn = fmaxf(m, mi);
#pragma unroll
        for (int x = 1; x < kLanes; x <<= 1) mn = fmaxf(mn, __shfl_xor(mn, x, kLanes));
        const float before = m == -INFINITY ? 0.f : exp2_fast((m - mn) * a.cexp);
        const float w = mi == -INFINITY ? 0.f : exp2_fast((mi - mn) * a.cexp);
        float lw = li * w;                              // a sum that is NaN stays NaN whatever its maximum
#pragma unroll
        for (int x = 1; x < kLanes; x <<= 1) lw += __shfl_xor(lw, x, kLanes);
        l = l * before + lw;
        o *= before;
        m = mn;
        const int here = min(kLanes, count - i0);
        for (int i = 0; i < here; i += kBatch) {
            f32x4 os[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e) os[e] = *reinterpret_cast<const f32x4*>(a.part_o + part(i0 + min(i + e, here - 1)) * D + d);
#pragma unroll
            for (int e = 0; e < kBatch; ++e) o += os[e] * (i + e < here ? __shfl(w, i + e, kLanes) : 0.f);
        }
    }
    const bool empty = l == 0.f;
    const float inv = empty ? 0.f : 1.f / l;
    if (d == 0 && a.out_lse) a.out_lse[at] = empty ? -INFINITY : (m * a.cexp + __builtin_amdgcn_logf(l)) * 0.69314718056f;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = empty ? 0.f : o[e] * inv;
    const long long to = static_cast<long long>(at) * D + d;
    if (DT == 1)
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + to) = u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    else
        *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + to) = o;
}

template <int D, int DT> void attend(const PagedAttnArgs& a, hipStream_t s, Timing t) {
    const dim3 grid(static_cast<unsigned>(a.max_units * a.c.H));
    launch_timed(t, paged_attention_kernel<D, DT>, grid, dim3(kThreads), 0, s, a);
    if (!a.part_o) return;
    constexpr int rows_wg = kThreads / (D / 4);
    const long long rows = static_cast<long long>(a.B) * a.N * a.Hq;
    paged_join_kernel<D, DT><<<dim3(static_cast<unsigned>((rows + rows_wg - 1) / rows_wg)), kThreads, 0, s>>>(a, static_cast<unsigned>(rows));
}

}  // namespace

hipError_t launch_paged_attention(const PagedAttnArgs& a, hipStream_t s, Timing t) {
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
