// Log probabilities of given tokens under logit rows, with the rows' entropy and
// most likely tokens; and the gradient of the two for the logits.
//
// With x_i = log2(e)/T * (z_i - m), m the row's largest logit, S = sum 2^x_i and
// W = sum 2^x_i x_i:  log p(t) = ln2 * (x_t - log2 S),  H = ln2 * (log2 S - W/S).
// x is never above 0 but for its rounding (of m*log2(e)/T, which is in every x alike).
//
// Forward: a workgroup streams a row, or a slice of one where the rows are few.  Each
// wave takes its vectors as they arrive, against a running reference, a logit that
// moves only where one passes it by 2^2, so that exponentials overlap the loads.
// (What is added meanwhile is below 4, and the largest element's exponent so small
// that its rounding is lost in the sum's: with 2^40 a confident token's log
// probability was off by 2.4e-6 and the entropy by 9.9e-6, 5e-7 both so. Some 1% of
// the time.)
// Of the likeliest: the first eight vectors a thread stay in registers until their
// threads' maxima say what the rest is measured by.  The n-th largest of them bounds
// the row's n-th largest element from below, and few elements reach it: the
// vectors that hold some go to LDS, those of the rest of the row as they come, and
// each element's place among them is counted.  (Where the first
// vectors tell too little, the row is looked through again with the bound of all.)
// The workgroups of a row leave (m, S, W, list) in the workspace, and the last of
// them joins.
//
// What bounds it: 1024 rows of 128256 bf16 logits and more, HBM (2048 rows, no list:
// 88-92 us, 5.8 TB/s); 512 rows of which 288 are read, with the 20 likeliest: 28 us,
// 2.7 TB/s, 22 of them without the list, and 15 by the bytes at a large copy's rate
// (4.9 TB/s): a workgroup's row is a chain of first loads, 31 vectors a thread, the
// list; when it took 26, it was still 20 with one exponential in eight, and 27 and 29
// with more vectors under way (12, 16), which cost occupancy.  Rows with -inf, half of
// their logits: 33 us, 2048 of them 107.  8 rows of 32000: 9 us, latency.  The gradient is one read and one write of each row at
// 6.1 TB/s (2048 rows of 128256: 170 us), more than a large copy reaches (4.9).

#include <float.h>

#include "logprob.hpp"

namespace sv {

namespace {

constexpr int kWaves = kLpThreads / kWave;
constexpr int kLpVecs = 8, kFewVecs = 4;                // 16-byte vectors of a thread under way; of a small slice, all of them
constexpr int kLpWorkgroups = 256;
constexpr int kStage = kWave, kCand = kLpThreads;       // vectors of a wave, and elements, that may reach the threshold

typedef u32x4 __attribute__((aligned(4))) u32x4_a4;
typedef u32x4 __attribute__((aligned(2))) u32x4_a2;

// 16 bytes at any element's address.
template <int DT> __device__ __forceinline__ u32x4 load_vec(const void* row, long i) {
    if (DT == 1) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(static_cast<const uint16_t*>(row) + i));
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(row) + i));
}
template <int DT> __device__ __forceinline__ void store_vec(void* row, long i, const u32x4& v) {
    if (DT == 1) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2*>(static_cast<uint16_t*>(row) + i));
    else __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a4*>(static_cast<float*>(row) + i));
}
template <int DT> __device__ __forceinline__ float vec_max(const u32x4& v) {
    if (DT == 1) {
        float a = maximum3(bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]));
        float b = maximum3(bf16_hi(v[1]), bf16_lo(v[2]), bf16_hi(v[2]));
        return maximum3(maximum3(a, b, bf16_lo(v[3])), bf16_hi(v[3]), a);
    }
    const float a = maximum3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
    return __builtin_elementwise_maximum(a, __uint_as_float(v[3]));
}
// This wave's stores have been acknowledged.  Words stored at agent scope are then past the XCD's L2, so that a ticket taken
// after it promises them to a reader at agent scope; a fence would write back all that the L2 holds (the gradient of 2048 rows
// took ten times as long with one).
__device__ __forceinline__ void stores_done() {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#endif
}
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
constexpr float kSlack = 2.f;                           // powers of two
constexpr float kLowest = -1e30f;                       // 0 * kLowest is 0, 0 * -inf is not a number
constexpr double kLn2 = 0.69314718055994530942;

// x of a logit, mc = m * c, whose rounding is in every x alike.  Where it may pass a power of two (a small temperature, a row of
// the type's lowest values: 2^x would overflow, or be 0 for all) or mc is infinite, the difference is taken first.
__device__ __forceinline__ float exponent(float z, float c, float mc) { return fmaxf(__builtin_fmaf(z, c, -mc), kLowest); }
__device__ __forceinline__ float exponent_wide(float z, float c, float m) { return fmaxf((z - m) * c, kLowest); }
__device__ __forceinline__ bool is_wide(float m, float c) { return !(fabsf(m * c) <= 16777216.f); }

// What exponents are relative to: m*c as it was used.
__device__ __forceinline__ double product(float m, float c, bool wide) {
    return wide ? static_cast<double>(m) * static_cast<double>(c) : static_cast<double>(m * c);
}
__device__ __forceinline__ double reference(float m, float c) { return product(m, c, is_wide(m, c)); }

struct Smem {
    float red[kWaves];
    double sums[kWaves][3];         // S, W, and what they are relative to
    uint32_t lists[2][kWaves][kWave];
    u32x4 stage[kWaves][kStage];
    int32_t stage_i[kWaves][kStage];
    pkey_t cand[kCand];
    int count, full;                // full: a wave had more vectors than its part of the stage holds
    pkey_t best[kWave];
};

__device__ __forceinline__ float wave_maximum(float v) {    // NaN wins
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = __builtin_elementwise_maximum(v, xshfl(v, o));
    return v;
}

// A row is asked for unless it has tokens and all are negative; bad: a token past the vocabulary.
__device__ __forceinline__ bool row_used(const int32_t* tokens, int M, int V, int& tok, bool& bad) {
    const int lane = threadIdx.x & (kWave - 1);
    tok = lane < M ? tokens[lane] : -1;
    bad = __ballot(tok >= V) != 0ull;
    return M == 0 || __ballot(tok >= 0) != 0ull;
}

// What a row is told by: r = log2(e)/T * m, S and W over the elements relative to it.
struct Sums {
    double r;               // NaN: a NaN or +inf among the logits
    double S, W;
};

// No probability is above 1, whatever the sum's rounding.
__device__ __forceinline__ float log_prob(double base_two) { return static_cast<float>(fmin(base_two, 0.0) * kLn2); }

// The row's results, by one wave: lane l holds the l-th best element (key), the row's sums are the same in every lane.
__device__ __forceinline__ void finish_row(const LogprobArgs& a, long r, const Sums& s, float m, pkey_t key, int tok,
                                           float z_tok, bool bad) {
    const int lane = threadIdx.x & (kWave - 1);
    const double lS = log2(s.S);
    const bool ok = !bad && s.S > 0.0 && s.S < INFINITY;    // neither NaN, nor +inf, nor all -inf
    const float nan = __builtin_nanf("");
    if (lane < a.M) {
        const double x = static_cast<double>(z_tok) * static_cast<double>(a.c) - s.r;
        a.out_lp[r * a.M + lane] = tok < 0 && !bad ? 0.f : ok ? log_prob(x - lS) : nan;
    }
    if (lane == 0) {
        const float h = ok ? static_cast<float>(fmax(0.0, (lS - s.W / s.S) * kLn2)) : nan;
        if (a.out_entropy) a.out_entropy[r] = h;
        if (a.out_stats) {
            a.out_stats[kLpStats * r] = ok ? m : nan;
            a.out_stats[kLpStats * r + 1] = ok ? static_cast<float>(lS) : nan;
            a.out_stats[kLpStats * r + 2] = h;
        }
    }
    if (lane < a.top_n) {
        const bool have = ok && key > empty_key();
        const double x = static_cast<double>(key_val(key)) * static_cast<double>(a.c) - s.r;
        a.out_top[r * a.top_n + lane] = have ? key_idx(key) : -1;
        a.out_top_lp[r * a.top_n + lane] = have ? log_prob(x - lS) : ok ? -INFINITY : nan;
    }
}

template <int DT, int NV, bool TOP>
__global__ __launch_bounds__(kLpThreads, 4) void logprobs_kernel(LogprobArgs a) {
    using E = Elem<DT>;
    constexpr int PV = E::kPerVec;
    __shared__ Smem sm;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    const long r = blockIdx.x / a.slices;
    const int slice = blockIdx.x % a.slices;
    const char* row = static_cast<const char*>(a.logits) + r * a.stride * E::kBytes;
    int tok;
    bool bad;
    if (!row_used(a.tokens + r * a.M, a.M, a.V, tok, bad)) {
        if (slice == 0 && wave == 0) {
            if (lane < a.M) a.out_lp[r * a.M + lane] = 0.f;
            if (lane == 0 && a.out_entropy) a.out_entropy[r] = 0.f;
            if (lane < kLpStats && a.out_stats) a.out_stats[kLpStats * r + lane] = 0.f;
            if (lane < a.top_n) {
                a.out_top[r * a.top_n + lane] = -1;
                a.out_top_lp[r * a.top_n + lane] = -INFINITY;
            }
        }
        return;
    }

    // the slice: vectors first .. last - 1 of the row, and the row's last few elements with its last slice
    const int vecs = a.V / PV, first = slice * a.per, last = min(vecs, first + a.per);
    const auto fetch = [&](int i) {
        const uint32_t none = DT == 1 ? 0xff80ff80u : 0xff800000u;     // -inf
        u32x4 w = {none, none, none, none};
        if (i < last) w = load_vec<DT>(row, static_cast<long>(i) * PV);
        return w;
    };
    u32x4 v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = fetch(first + j * kLpThreads + tid);
    const int rest = vecs * PV + tid;
    const bool has_rest = slice == a.slices - 1 && rest < a.V;
    const float z_rest = has_rest ? E::scalar(row, rest) : -INFINITY;
    const float z_tok = tok >= 0 && !bad ? E::scalar(row, tok) : 0.f;

    constexpr int kGroup = 4;                           // vectors between two looks at the reference
    // sums relative to ref = mz*c, or (wide) by the differences from mz; the three are the same in a wave's lanes
    float tm = -INFINITY, mz = -FLT_MAX, ref = mz * a.c, S = 0.f, W = 0.f;
    bool wide = true, masked = false;                   // masked: a -inf has been met
    const auto add_to = [](float& S, float& W, float x) {
        const float p = exp2_fast(x);
        S += p;
        W = __builtin_fmaf(p, x, W);
    };
    const auto move = [&](float to, bool to_wide) {
        const float d = static_cast<float>(product(mz, a.c, wide) - product(to, a.c, to_wide)), w = exp2_fast(d);
        W = w > 0.f ? w * __builtin_fmaf(S, d, W) : 0.f;
        S = w > 0.f ? S * w : 0.f;
        mz = to;
        ref = to * a.c;
        wide = to_wide;
    };
    const auto look = [&](float mx) {
        tm = __builtin_elementwise_maximum(tm, mx);
        if (__ballot((mx - mz) * a.c > kSlack) != 0ull) {
            const float to = bcast(fmaxf(mz, wave_max(mx)), 0);
            move(to, masked || is_wide(to, a.c));
        }
    };
    // A group of vectors, the first of them number `at` of the row, by two sums of its own (with 250 additions one after the other
    // the entropies of 128256 logits were off by 9e-7 of them, by 3e-7 with one a group; peaked rows 7e-7, 5e-7 with two). -inf makes a NaN of w (0 * -inf): that group
    // and the wave's later ones are taken by differences, held above that (half of 2048 rows of 128256 masked: 107 us, 90 with none, 151 with
    // such groups taken twice); what stands for vectors past the end is -inf too, and left out.
    const auto sum = [&](const u32x4* v, int at) {
        float s[2] = {}, w[2] = {};
        if (!wide) {
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                const float before = w[e / 2];
#pragma unroll
                for (int i = 0; i < PV; ++i) add_to(s[e / 2], w[e / 2], __builtin_fmaf(E::get(v[e], i), a.c, -ref));
                w[e / 2] = at + e * kLpThreads < last ? w[e / 2] : before;
            }
            const float any = w[0] + w[1];
            if (__ballot(any != any) != 0ull) {
                masked = true;
                move(mz, true);
            }
        }
        if (wide) {
            s[0] = s[1] = w[0] = w[1] = 0.f;
            if (__ballot(tm > -INFINITY) != 0ull) {     // (the wave has met something else)
#pragma unroll
                for (int e = 0; e < kGroup; ++e)
#pragma unroll
                    for (int i = 0; i < PV; ++i) add_to(s[e / 2], w[e / 2], exponent_wide(E::get(v[e], i), a.c, mz));
            }
        }
        S += s[0] + s[1];
        W += w[0] + w[1];
    };
    // Vectors with an element that reaches tau, to the wave's part of the stage (past its end they are only counted).
    float tau = INFINITY;
    int staged = 0;                                     // the same in a wave's lanes
    const auto offer = [&](const u32x4& w, float mx, int i) {
        const unsigned long long hits = __ballot(mx >= tau);
        if (hits == 0ull) return;
        const int at = staged + __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(hits >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(hits), 0));
        if (mx >= tau && at < kStage) {
            sm.stage[wave][at] = w;
            sm.stage_i[wave][at] = i * PV;
        }
        staged += __popcll(hits);
    };
    // A lower bound of the n-th largest of the elements that the threads' maxima are of: the n-th largest of those (the waves'
    // sorted lists, merged two by two).
    const auto bound = [&](float top) {
        uint32_t k = wave_sort_desc(order_key(top));
        if (tid == 0) sm.count = sm.full = 0;
        staged = 0;
#pragma unroll
        for (int w = 1; w < kWaves; w <<= 1) {
            uint32_t(&list)[kWaves][kWave] = sm.lists[w == 2 ? 1 : 0];
            if (w == 4) __syncthreads();                // the first lists have been read
            list[wave][lane] = k;
            __syncthreads();
            k = wave_bitonic_clean(max(k, list[wave ^ w][kWave - 1 - lane]), true);
        }
        return fmaxf(order_value(lane_gather(k, a.top_n - 1)), -FLT_MAX);       // -inf is in no list
    };

#pragma unroll
    for (int j = 0; j < NV; j += kGroup) {
        float mx = vec_max<DT>(v[j]);
#pragma unroll
        for (int e = 1; e < kGroup; ++e) mx = __builtin_elementwise_maximum(mx, vec_max<DT>(v[j + e]));
        look(mx);
        sum(v + j, first + j * kLpThreads + tid);
#pragma unroll
        for (int e = 0; e < kGroup; ++e) asm volatile("" : "+v"(v[j + e]));     // widened again later, not kept
    }
    u32x4 ahead[kGroup];                                // under way while the bound is found
#pragma unroll
    for (int j = 0; j < kGroup; ++j) ahead[j] = fetch(first + (NV + j) * kLpThreads + tid);
    if (TOP) tau = bound(tm);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = first + j * kLpThreads + tid;
        if (TOP) offer(v[j], vec_max<DT>(v[j]), i);
        v[j] = j < kGroup ? ahead[j] : fetch(i + NV * kLpThreads);
    }
    // the rest of the slice, each register's next vector under way as soon as it is free
#pragma unroll 1
    for (int base = first + NV * kLpThreads; base < last; base += NV * kLpThreads) {
#pragma unroll
        for (int j = 0; j < NV; j += kGroup) {
            float own[kGroup], mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                own[e] = vec_max<DT>(v[j + e]);
                mx = __builtin_elementwise_maximum(mx, own[e]);
            }
            look(mx);
            sum(v + j, base + j * kLpThreads + tid);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
                const int i = base + (j + e) * kLpThreads + tid;
                if (TOP) offer(v[j + e], own[e], i);
                v[j + e] = fetch(i + NV * kLpThreads);
            }
        }
    }
    if (slice == a.slices - 1) {
        look(z_rest);
        if (has_rest) {
            float s = 0.f, w = 0.f;
            add_to(s, w, wide ? exponent_wide(z_rest, a.c, mz) : exponent(z_rest, a.c, ref));
            S += s;
            W += w;
        }
    }
    {
        const float w = wave_maximum(tm);
        if (lane == 0) sm.red[wave] = w;
        if (TOP && staged > kStage) sm.full = 1;
    }
    __syncthreads();
    float m = sm.red[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = __builtin_elementwise_maximum(m, sm.red[w]);
    const bool some = m > -INFINITY && m < INFINITY;
    const double Sw = wave_sum(static_cast<double>(S)), Ww = wave_sum(static_cast<double>(W));
    if (lane == 0) sm.sums[wave][0] = Sw, sm.sums[wave][1] = Ww, sm.sums[wave][2] = product(mz, a.c, wide);

    pkey_t key = empty_key();
    if (TOP && some) {
        if (sm.full) {                                  // the same in every thread
            __syncthreads();
            tau = bound(tm);
#pragma unroll 1
            for (int base = first; base < last; base += kLpThreads) {
                const u32x4 w = fetch(base + tid);
                offer(w, vec_max<DT>(w), base + tid);
            }
            if (staged > kStage) sm.full = 1;
            __syncthreads();
        }
        // a staged vector a lane: its elements that reach tau go behind those of the lanes, and the waves, before
        const bool one = lane < min(staged, kStage);
        const u32x4 w = sm.stage[wave][lane];
        const int at0 = sm.stage_i[wave][lane];
        int hits = 0;
#pragma unroll
        for (int e = 0; e < PV; ++e) hits += one && E::get(w, e) >= tau ? 1 : 0;
        hits += has_rest && z_rest >= tau ? 1 : 0;
        int upto = hits;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const int t = __shfl_up(upto, o, kWave);
            if (lane >= o) upto += t;
        }
        int at = 0;
        if (lane == kWave - 1) at = atomicAdd(&sm.count, upto);
        at = bcast(at, kWave - 1) + upto - hits;
#pragma unroll
        for (int e = 0; e < PV; ++e) {
            const float z = E::get(w, e);
            if (one && z >= tau) {
                if (at < kCand) sm.cand[at] = pair_key(z, at0 + e);
                ++at;
            }
        }
        if (has_rest && z_rest >= tau && at < kCand) sm.cand[at] = pair_key(z_rest, rest);
        __syncthreads();
        const int count = sm.count;
        if (!sm.full && count <= kCand) {
            // kShare neighbouring threads an element (all of them at once, or in turns): as many are better as its place says
            if (tid < kWave) sm.best[tid] = empty_key();
            __syncthreads();
            constexpr int kShare = 4;
            for (int base = 0; base < count; base += kLpThreads / kShare) {
                const int mine = base + tid / kShare;
                const pkey_t k = mine < count ? sm.cand[mine] : 0;
                int place = 0;
#pragma unroll 4
                for (int i = tid % kShare; i < count; i += kShare) place += sm.cand[i] > k;
                place += xshfl(place, 1);
                place += xshfl(place, 2);
                if (mine < count && place < a.top_n) sm.best[place] = k;
            }
            __syncthreads();
            key = sm.best[lane];
        } else {
            // many equal elements: the best one below the last found, n times
            const int end = slice == a.slices - 1 ? a.V : last * PV;
            pkey_t found = ~0ull;
            for (int n = 0; n < a.top_n; ++n) {
                pkey_t best = 0;
#pragma unroll 1
                for (int i = first * PV + tid; i < end; i += kLpThreads) {
                    const pkey_t k = pair_key(E::scalar(row, i), i);
                    if (k < found && k > best) best = k;
                }
#pragma unroll
                for (int o = 32; o > 0; o >>= 1) {
                    const pkey_t other = xshfl(best, o);
                    best = other > best ? other : best;
                }
                __syncthreads();
                if (lane == 0) sm.best[wave] = best;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kWaves; ++w) best = sm.best[w] > best ? sm.best[w] : best;
                if (best == 0 || key_val(best) == -INFINITY) break;
                if (lane == n) key = best;
                found = best;
            }
        }
    } else {
        __syncthreads();
    }
    if (wave != 0) return;
    // the waves' sums, relative to the row's (or slice's) largest
    const bool odd = !(m < INFINITY);                   // NaN or +inf; a slice of -inf alone has no sum
    Sums s = {0.0, 0.0, 0.0};
    if (some) {
        const int w = lane % kWaves;
        const double d = sm.sums[w][2] - reference(m, a.c);
        const double f = lane < kWaves ? exp2(d) : 0.0, Sw = sm.sums[w][0];
        s.S = wave_sum(Sw * f);
        s.W = wave_sum(f > 0.0 ? f * (Sw * d + sm.sums[w][1]) : 0.0);
    }
    if (odd) s.S = __builtin_nan("");
    s.r = reference(m, a.c);
    if (a.slices == 1) {
        finish_row(a, r, s, m, key, tok, z_tok, bad);
        return;
    }

    // leave the slice's record; the last workgroup of the row joins them
    const int per = kLpHead + a.top_n;
    unsigned long long* rec = a.words + (r * a.slices + slice) * per;
    if (lane == 0) {
        st_agent64(rec, (static_cast<unsigned long long>(__float_as_uint(odd ? __builtin_nanf("") : m)) << 32));
        st_agent64(rec + 1, static_cast<unsigned long long>(__double_as_longlong(s.S)));
        st_agent64(rec + 2, static_cast<unsigned long long>(__double_as_longlong(s.W)));
    }
    if (TOP && lane < a.top_n) st_agent64(rec + kLpHead + lane, key);
    stores_done();
    unsigned ticket = 0;
    if (lane == 0) ticket = __hip_atomic_fetch_add(a.done + r, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    ticket = __builtin_amdgcn_readfirstlane(ticket);
    asm volatile("" ::: "memory");
    if (ticket != static_cast<unsigned>(a.slices) - 1) return;
    if (lane == 0) __hip_atomic_store(a.done + r, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // lane l has slice l (at most 64 of them)
    unsigned long long* base = a.words + r * a.slices * per;
    float ms = -INFINITY;
    double Ss = 0.0, Ws = 0.0;
    if (lane < a.slices) {
        const unsigned long long w0 = ld_agent64(base + lane * per), w1 = ld_agent64(base + lane * per + 1),
                                 w2 = ld_agent64(base + lane * per + 2);
        ms = __uint_as_float(static_cast<uint32_t>(w0 >> 32));
        Ss = __longlong_as_double(static_cast<long long>(w1));
        Ws = __longlong_as_double(static_cast<long long>(w2));
    }
    if (TOP) {
        // all lists as one: 64 keys at a time, four loads under way
        const int total = a.slices * a.top_n;
        const auto entry = [&](int i) {
            const int l = i / a.top_n;
            return ld_agent64(base + l * per + kLpHead + (i - l * a.top_n));
        };
        for (int b = 0; b < total; b += 4 * kWave) {
            pkey_t k[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) k[e] = b + e * kWave + lane < total ? entry(b + e * kWave + lane) : empty_key();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (b + e * kWave >= total) break;
                wave_sort_keys(k[e]);
                if (b + e == 0) key = k[0];
                else wave_merge_keys(key, k[e]);
            }
        }
    }
    for (int i = lane; i < a.slices * per; i += kWave) st_agent64(base + i, 0ull);      // left zero for the next call
    const float mr = wave_maximum(ms);
    const double rs = reference(ms, a.c);
    s.r = reference(mr, a.c);
    const double d = ms > -INFINITY ? rs - s.r : 0.0;
    const double w = ms > -INFINITY ? exp2(d) : 0.0;
    s.S = wave_sum(Ss * w);
    s.W = wave_sum(w > 0.0 ? w * (Ws + Ss * d) : 0.0);
    if (!(mr < INFINITY)) s.S = __builtin_nan("");
    finish_row(a, r, s, mr, key, tok, z_tok, bad);
}

// Gradient: dz_i = p_i (A + B x'_i) + (1/T) sum_m g_m [i = t_m], x' = log2 p_i, A = -(G + h H)/T, B = -h ln2 / T,
// G = sum g_m.  One pass; the elements of given tokens are written once more, after the row's own pass.
constexpr int kGradVecs = 4, kGradThreads = 256;

template <int DT, bool ENT>
__global__ __launch_bounds__(kGradThreads) void logprobs_grad_kernel(LogprobGradArgs a) {
    using E = Elem<DT>;
    constexpr int PV = E::kPerVec;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const long r = blockIdx.x / a.slices;
    const int slice = blockIdx.x % a.slices;
    const char* row = static_cast<const char*>(a.logits) + r * a.stride * E::kBytes;
    char* out = static_cast<char*>(a.grad) + r * a.grad_stride * E::kBytes;
    const int vecs = a.V / PV, first = slice * (kGradVecs * kGradThreads);
    int tok;
    bool bad;
    const bool used = row_used(a.tokens + r * a.M, a.M, a.V, tok, bad);
    const int rest = vecs * PV + tid;
    const bool has_rest = slice == a.slices - 1 && rest < a.V;
    const auto put = [&](long i, float g) {
        if (DT == 1) reinterpret_cast<__bf16*>(out)[i] = static_cast<__bf16>(g);
        else reinterpret_cast<float*>(out)[i] = g;
    };
    if (!used) {
        const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < kGradVecs; ++j) {
            const int i = first + j * kGradThreads + tid;
            if (i < vecs) store_vec<DT>(out, static_cast<long>(i) * PV, zero);
        }
        if (has_rest) put(rest, 0.f);
        return;
    }
    u32x4 v[kGradVecs];
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
        const int i = first + j * kGradThreads + tid;
        if (i < vecs) v[j] = load_vec<DT>(row, static_cast<long>(i) * PV);
    }
    const float z_rest = has_rest ? E::scalar(row, rest) : 0.f;
    // the given tokens of this slice (lane m has token m, in every wave)
    const bool last = slice == a.slices - 1;
    const bool mine = !bad && tok >= first * PV && (last || tok < (first + kGradVecs * kGradThreads) * PV);
    const float z_tok = mine ? E::scalar(row, tok) : 0.f;
    const float g = tok >= 0 && lane < a.M ? a.g_lp[r * a.M + lane] : 0.f;
    const float m = a.stats[kLpStats * r], l = bad ? __builtin_nanf("") : a.stats[kLpStats * r + 1];
    const float h = ENT ? a.g_entropy[r] : 0.f, H = ENT ? a.stats[kLpStats * r + 2] : 0.f;
    const float G = wave_sum(g);
    const float A = -a.invT * __builtin_fmaf(h, H, G), B = -a.invT * h * static_cast<float>(kLn2);
    float same = 0.f;                                   // gradients of all mentions of this lane's token
    for (int j = 0; j < a.M; ++j) same += bcast(tok, j) == tok ? bcast(g, j) : 0.f;
    const bool wide = is_wide(m, a.c);
    const float mc = m * a.c;
    const auto at = [&](float z) {
        const float x = (wide ? exponent_wide(z, a.c, m) : exponent(z, a.c, mc)) - l;
        const float p = exp2_fast(x);
        return p == 0.f ? 0.f : p * (ENT ? __builtin_fmaf(B, x, A) : A);      // its factor may be infinite there
    };
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("" ::"v"(z_tok));                      // the gradient may take the logits' place: z_tok has arrived
#endif
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
        const int i = first + j * kGradThreads + tid;
        if (i >= vecs) continue;
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (DT == 1) {
                typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                const bf16x2 pr = {static_cast<__bf16>(at(bf16_lo(v[j][e]))), static_cast<__bf16>(at(bf16_hi(v[j][e])))};
                o[e] = __builtin_bit_cast(uint32_t, pr);
            } else {
                o[e] = __float_as_uint(at(__uint_as_float(v[j][e])));
            }
        }
        store_vec<DT>(out, static_cast<long>(i) * PV, o);
    }
    if (has_rest) put(rest, at(z_rest));
    if (__ballot(mine) == 0ull) return;                 // the same in every wave
    stores_done();                                      // the row's own pass is in place before the tokens' elements follow
    __syncthreads();
    if (tid < kWave && mine) put(tok, __builtin_fmaf(a.invT, same, at(z_tok)));
}

template <int DT, int NV> void logprobs(const LogprobArgs& a, hipStream_t s, Timing t) {
    const dim3 grid(static_cast<unsigned>(static_cast<long>(a.R) * a.slices));
    if (a.top_n > 0) launch_timed(t, logprobs_kernel<DT, NV, true>, grid, dim3(kLpThreads), 0, s, a);
    else launch_timed(t, logprobs_kernel<DT, NV, false>, grid, dim3(kLpThreads), 0, s, a);
}
template <int DT> void logprobs(const LogprobArgs& a, hipStream_t s, Timing t) {
    if (a.per <= kFewVecs * kLpThreads) logprobs<DT, kFewVecs>(a, s, t);
    else logprobs<DT, kLpVecs>(a, s, t);
}

}  // namespace

// A workgroup a row where there is a row for each compute unit (512 rows of 128256 bf16 logits: 28 us, two workgroups a row 38);
// fewer rows are cut up, so that their loads spread over the compute units, into slices of four vectors a thread at least.
void logprob_plan(LogprobArgs& a) {
    const int vecs = a.V / (a.dtype == 1 ? 8 : 4), least = kFewVecs * kLpThreads;
    const int wanted = a.R < kLpWorkgroups ? (kLpWorkgroups + a.R - 1) / a.R : 1;
    int per = (vecs + wanted - 1) / wanted;
    per = (per + kLpThreads - 1) / kLpThreads * kLpThreads;
    if (per < least) per = least;
    a.slices = (vecs + per - 1) / per;
    if (a.slices > kWave) {                             // joined one a lane
        per = ((vecs + kWave - 1) / kWave + kLpThreads - 1) / kLpThreads * kLpThreads;
        a.slices = (vecs + per - 1) / per;
    }
    if (a.slices < 1) a.slices = 1;
    a.per = per;
}

hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s, Timing t) {
    if (a.dtype == 1) logprobs<1>(a, s, t);
    else logprobs<0>(a, s, t);
    return hipGetLastError();
}

int logprob_grad_slices(int dtype, int V) {
    const int elems = kGradVecs * kGradThreads * (dtype == 1 ? 8 : 4), n = (V + elems - 1) / elems;
    return n < 1 ? 1 : n;
}

hipError_t launch_logprobs_grad(const LogprobGradArgs& a, hipStream_t s, Timing t) {
    const dim3 grid(static_cast<unsigned>(static_cast<long>(a.R) * a.slices));
    if (a.dtype == 1) {
        if (a.g_entropy) launch_timed(t, logprobs_grad_kernel<1, true>, grid, dim3(kGradThreads), 0, s, a);
        else launch_timed(t, logprobs_grad_kernel<1, false>, grid, dim3(kGradThreads), 0, s, a);
    } else {
        if (a.g_entropy) launch_timed(t, logprobs_grad_kernel<0, true>, grid, dim3(kGradThreads), 0, s, a);
        else launch_timed(t, logprobs_grad_kernel<0, false>, grid, dim3(kGradThreads), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace sv
