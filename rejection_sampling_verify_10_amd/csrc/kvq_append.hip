// Rows into and out of the four-bit cache (the layout is stated in kvq.hpp).
//
// A block of 32 elements gets the scale 2^e with the smallest e for which
// max|x| <= 7 * 2^e: then x / 2^e rounds to a code whose value is off by at
// most half a step (1 above 4, .5 above 2, .25 below), the largest element
// among them, since 7 lies half a step past the largest code, 6.  The division
// is exact (a power of two) and the rounding is the conversion instruction's
// (nearest, ties to the even code), so the codes depend on the inputs alone.
//
// Both kernels are bound by the wide side's bytes: eight elements a lane (one or
// two 16-byte vectors), D/8 neighbouring lanes a row, four of them a block, so
// the block's maximum is two lane exchanges and the row's codes leave as one
// run of D/2 bytes.  A prompt's 4 x 2047 float32 rows of 8 heads: 13.6 us for
// 76 MB, 5.6 TB/s (and 9.2 us to read 8.4 million values of each back as bf16);
// a tree's 32 x 27 rows are a launch and one load's latency, 4 us each way.  A lane handles the same elements of K and of V, because a
// value that is not finite in either poisons the slot's K row.

#include "kvq.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;

template <int DT> __device__ __forceinline__ void load8(const void* base, long i, float x[8]) {
    if (DT == 1) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + i);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = Elem<1>::get(v, e);
    } else {
        const f32x4 a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + i);
        const f32x4 b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + i + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = a[e], x[4 + e] = b[e];
    }
}

// Scale byte of the block the lane's group of four holds; x holds only finite values.
__device__ __forceinline__ uint32_t block_scale(const float x[8]) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
    top = fmaxf(top, xshfl(top, 1));
    top = fmaxf(top, xshfl(top, 2));
    // 7 * 2^e = 1.75 * 2^(e+2): a mantissa above 1.75 takes the next exponent
    const int byte = static_cast<int>((__float_as_uint(top) + 0x1fffffu) >> 23) - 2;
    return top == 0.f ? 0u : static_cast<uint32_t>(min(max(byte, kQScaleMin), kQScaleMax));
}

__device__ __forceinline__ uint32_t pack8(float x[8], uint32_t byte) {
    uint32_t w = 0;
    if (byte == kQScaleMax) {                           // past 7 * 2^125 a block has no larger scale to go to
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fminf(fmaxf(x[e], -0x1.8p127f), 0x1.8p127f);
    }
#if SV_KVQ_DEVICE
    const float s = scale_value(byte == 0 ? 127u : byte);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
#endif
    return w;
}

// Zeroes the lane's values if one of them, or of its block's, is not finite.
__device__ __forceinline__ bool take_bad(float x[8]) {
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) bad = bad || !(fabsf(x[e]) <= 3.402823466e+38f);
    int any = bad ? 1 : 0;
    any |= xshfl(any, 1);
    any |= xshfl(any, 2);
    if (any) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
    return any != 0;
}

template <int D, int DT>
__global__ __launch_bounds__(kThreads) void kvq_append_kernel(KvqAppendArgs a) {
    constexpr int kLanes = D / 8;                       // lanes of a row
    const long row = (static_cast<long>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    const int part = threadIdx.x % kLanes, lane = threadIdx.x & (kWave - 1);
    const long rows = static_cast<long>(a.c.B) * a.N * a.c.H;
    const long r = row < rows ? row : rows - 1;         // every lane stays for the exchanges
    const int h = static_cast<int>(r % a.c.H);
    const long bn = r / a.c.H;
    const int n = static_cast<int>(bn % a.N), b = static_cast<int>(bn / a.N);
    const int pre = a.prefix[b], cnt = a.counts ? a.counts[b] : a.N;
    const bool live = row < rows && kvq_row_ok(pre, cnt, a.N, a.c.capacity) && n < cnt;
    float k[8] = {}, v[8] = {};
    if (live) {
        load8<DT>(a.k.data, b * a.k.batch + n * a.k.pos + h * a.k.head + part * 8, k);
        load8<DT>(a.v.data, b * a.v.batch + n * a.v.pos + h * a.v.head + part * 8, v);
    }
    const bool kbad = take_bad(k), vbad = take_bad(v);
    const unsigned long long mine = (kLanes == 64 ? ~0ull : ((1ull << kLanes) - 1)) << (lane & ~(kLanes - 1));
    const bool poisoned = (__ballot(kbad || vbad) & mine) != 0;
    uint32_t ks = block_scale(k), vs = block_scale(v);
    const uint32_t kw = pack8(k, ks), vw = pack8(v, vs);
    if (kbad || (poisoned && part < 4)) ks = kQScaleNaN;
    if (vbad) vs = kQScaleNaN;
    if (!live) return;
    const long slot = pre + static_cast<long>(n);
    const long at = b * a.c.cb + h * a.c.ch + slot * a.c.cp + part * 4;
    *reinterpret_cast<uint32_t*>(a.c.kc + at) = kw;
    *reinterpret_cast<uint32_t*>(a.c.vc + at) = vw;
    if (part % 4 == 0) {
        const long st = b * a.c.sb + h * a.c.sh + slot * a.c.sp + part / 4;
        a.c.ks[st] = static_cast<uint8_t>(ks);
        a.c.vs[st] = static_cast<uint8_t>(vs);
    }
}

template <int DT> __device__ __forceinline__ void store8(void* out, long i, uint32_t w, uint32_t byte) {
    const float s = scale_value(byte);
    const u32x4 p = {fp4_pair<0>(w, s), fp4_pair<1>(w, s), fp4_pair<2>(w, s), fp4_pair<3>(w, s)};
    if (DT == 1) {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + i) = p;
    } else {
        const f32x4 lo = {bf16_lo(p[0]), bf16_hi(p[0]), bf16_lo(p[1]), bf16_hi(p[1])};
        const f32x4 hi = {bf16_lo(p[2]), bf16_hi(p[2]), bf16_lo(p[3]), bf16_hi(p[3])};
        *reinterpret_cast<f32x4*>(static_cast<float*>(out) + i) = lo;
        *reinterpret_cast<f32x4*>(static_cast<float*>(out) + i + 4) = hi;
    }
}

template <int D, int DT>
__global__ __launch_bounds__(kThreads) void kvq_read_kernel(KvqReadArgs a) {
    constexpr int kLanes = D / 8;
    const long row = (static_cast<long>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    const int part = threadIdx.x % kLanes;
    if (row >= static_cast<long>(a.c.B) * a.N * a.c.H) return;
    const int h = static_cast<int>(row % a.c.H);
    const long bn = row / a.c.H;
    const int n = static_cast<int>(bn % a.N), b = static_cast<int>(bn / a.N);
    const int pre = a.prefix[b], cnt = a.counts ? a.counts[b] : a.N;
    uint32_t kw = 0, vw = 0, ks = 0, vs = 0;            // zeros where no row is read
    if (kvq_row_ok(pre, cnt, a.N, a.c.capacity) && n < cnt) {
        const long slot = pre + static_cast<long>(n);
        const long at = b * a.c.cb + h * a.c.ch + slot * a.c.cp + part * 4;
        const long st = b * a.c.sb + h * a.c.sh + slot * a.c.sp + part / 4;
        kw = *reinterpret_cast<const uint32_t*>(a.c.kc + at);
        vw = *reinterpret_cast<const uint32_t*>(a.c.vc + at);
        ks = a.c.ks[st];
        vs = a.c.vs[st];
    }
    store8<DT>(a.out_k, row * D + part * 8, kw, ks);
    store8<DT>(a.out_v, row * D + part * 8, vw, vs);
}

template <int D> dim3 row_grid(int B, int N, int H) {
    const long lanes = static_cast<long>(B) * N * H * (D / 8);
    return dim3(static_cast<unsigned>((lanes + kThreads - 1) / kThreads));
}

template <int D> void append(const KvqAppendArgs& a, hipStream_t s, Timing t) {
    const dim3 grid = row_grid<D>(a.c.B, a.N, a.c.H);
    if (a.dtype == 1) launch_timed(t, kvq_append_kernel<D, 1>, grid, dim3(kThreads), 0, s, a);
    else launch_timed(t, kvq_append_kernel<D, 0>, grid, dim3(kThreads), 0, s, a);
}
template <int D> void read(const KvqReadArgs& a, hipStream_t s, Timing t) {
    const dim3 grid = row_grid<D>(a.c.B, a.N, a.c.H);
    if (a.dtype == 1) launch_timed(t, kvq_read_kernel<D, 1>, grid, dim3(kThreads), 0, s, a);
    else launch_timed(t, kvq_read_kernel<D, 0>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

hipError_t launch_kvq_append(const KvqAppendArgs& a, hipStream_t s, Timing t) {
    if (a.c.D == 64) append<64>(a, s, t);
    else if (a.c.D == 128) append<128>(a, s, t);
    else append<256>(a, s, t);
    return hipGetLastError();
}

hipError_t launch_kvq_read(const KvqReadArgs& a, hipStream_t s, Timing t) {
    if (a.c.D == 64) read<64>(a, s, t);
    else if (a.c.D == 128) read<128>(a, s, t);
    else read<256>(a, s, t);
    return hipGetLastError();
}

}  // namespace sv
