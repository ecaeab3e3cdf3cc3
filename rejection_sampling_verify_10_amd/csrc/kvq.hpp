// The four-bit key/value cache: argument blocks of its kernels, the rows' layout
// and the conversions between E2M1 codes and bfloat16 (gfx950 has both as
// instructions that take the block's scale).
#pragma once

#include "common.hpp"
#include "internal.hpp"
#include "kvq_window.hpp"

namespace sv {

constexpr int kQBlock = 32;            // elements that share a scale byte
constexpr int kQScaleMin = -96 + 127;  // smallest scale byte of a block that is not all zero
constexpr int kQScaleMax = 125 + 127;  // largest: 6 * 2^125 is the largest value that is a float32
constexpr int kQScaleNaN = 255;

// Row (b, h, slot) of the codes at kc/vc + b*cb + h*ch + slot*cp, of the scales at ks/vs + b*sb + h*sh + slot*sp.
struct KvqCache {
    uint8_t *kc, *ks, *vc, *vs;
    long long cb, ch, cp, sb, sh, sp;
    int B, H, capacity, D;
};
// Rows (b, n, head) of D elements, strides in elements.
struct KvqRows {
    const void* data;
    long long batch, pos, head;
};

struct KvqAppendArgs {
    KvqCache c;
    KvqRows k, v;
    int dtype, N;
    const int32_t* prefix;
    const int32_t* counts;
};
struct KvqReadArgs {
    KvqCache c;
    int dtype, N;
    const int32_t* prefix;
    const int32_t* counts;
    void *out_k, *out_v;
};
struct KvqAttnArgs {
    KvqCache c;
    KvqRows q;
    int dtype, Hq, G, N, M;             // G query heads a cache head, M = N*G rows of a (b, h)
    const int32_t* prefix;
    const int32_t* counts;
    const uint8_t* mask;
    long long mask_batch;
    float cexp;                         // scale * log2(e): scores in base 2
    void* out;
    float* out_lse;
    int q_tiles, row_tiles, waves;      // 16-row tiles of a wave's queries, workgroups a unit, waves a workgroup
    int units, min_per;                 // parts of the batch's key axis and their least chunks; 0: one a batch row
    float* part_o;                      // [units][H][M][D] (units > 0)
    float* part_ml;                     // [units][H][M][2]
    int32_t* first_unit;                // [B + 1]
};
struct KvqScoreArgs {
    KvqCache c;
    KvqRows q;
    int dtype, Hq, G, N;
    const float* lse;
    const int32_t* prefix;
    const int32_t* path;
    int path_stride;
    const int32_t* accept_len;
    float cexp;
    float* scores;
    int32_t* positions;
    const int32_t* seen;
    int q_tiles;                        // 16-row tiles kept in registers; 0: rows in LDS
    int key_wgs, segs;                  // workgroups along the keys of a head, and along its rows
    float* part;                        // [segs][B*H][capacity] (segs > 1)
};
struct KvqEvictArgs {
    KvqCache c;
    const float* scores;
    const int32_t* positions;
    const int32_t* lengths;
    const int32_t* seen;
    int keep, sink, recent;
    float* out_scores;
    int32_t* out_positions;
    int32_t* out_len;
    int32_t* out_source;
    int32_t* plan;                      // [B*H][gap_stride][2]: the slot to fill, and the one it is filled from
    int32_t* moves;                     // [B*H] entries of the plan
    int gap_stride;                     // min(keep, capacity - keep), the most moves there can be
};

hipError_t launch_kvq_append(const KvqAppendArgs& a, hipStream_t s, Timing t = {});
hipError_t launch_kvq_read(const KvqReadArgs& a, hipStream_t s, Timing t = {});
// How an attention call is cut up: fills a.q_tiles .. a.min_per.
void kvq_attention_plan(KvqAttnArgs& a);
hipError_t launch_kvq_attention(const KvqAttnArgs& a, hipStream_t s, Timing t = {});
void kvq_score_plan(KvqScoreArgs& a);    // fills q_tiles, key_wgs and segs
hipError_t launch_kvq_score(const KvqScoreArgs& a, hipStream_t s, Timing t = {});
hipError_t launch_kvq_evict(const KvqEvictArgs& a, hipStream_t s, Timing t = {});

#ifdef __HIP_DEVICE_COMPILE__
#define SV_KVQ_DEVICE 1
#else
#define SV_KVQ_DEVICE 0
#endif

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// Byte `sel` of w (two E2M1 codes, the lower element first) times scale, as a pair of bfloat16: exact.
template <int SEL> __device__ __forceinline__ uint32_t fp4_pair(uint32_t w, float scale) {
#if SV_KVQ_DEVICE
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
#else
    return 0;
#endif
}
__device__ __forceinline__ uint32_t fp4_pair(uint32_t w, float scale, int sel) {
    return sel == 0 ? fp4_pair<0>(w, scale) : sel == 1 ? fp4_pair<1>(w, scale) : sel == 2 ? fp4_pair<2>(w, scale)
                                                                                          : fp4_pair<3>(w, scale);
}

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
#if SV_KVQ_DEVICE
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
#else
    return c;
#endif
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 p = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, p);
}

#if SV_KVQ_DEVICE
// A buffer descriptor: loads whose vector offset is not below `bytes` give zeros and touch nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, bytes, 0x00020000);
}
// That of tile t of a step whose slots start at p, `pos` bytes apart, with `slots` of the tile's there.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(const uint8_t* p, int t, int pos, int slots) {
    return rsrc(p + kTile * t * pos, slots * pos);
}
// tile_slots(slots_left(..)), in two: the compiler makes one clamp of both, on the vector unit, and a descriptor's
// registers are scalar ones.
__device__ __forceinline__ int scalar_slots(int first, int end) {
    int left = slots_left(first, end);
    asm("" : "+s"(left));
    return tile_slots(left);
}
#endif
// Codes and scales of slots first .. first+31 of those below `end`, as the lane of offsets ko, kso holds them; zeros for the
// others.
template <int D>
__device__ __forceinline__ void load_k_step(const uint8_t* codes, const uint8_t* scales, long cp, long sp, int first, int end,
                                            uint32_t ko, uint32_t kso, uint32_t (&k)[2][D / 32], uint32_t (&ks)[2]) {
#if SV_KVQ_DEVICE
    const uint8_t *c = codes + first * cp, *s = scales + first * sp;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int n = scalar_slots(first + kTile * t, end);
        const auto rk = tile_rsrc(c, t, static_cast<int>(cp), n), rks = tile_rsrc(s, t, static_cast<int>(sp), n);
        if (D == 64) {
            const auto w = __builtin_amdgcn_raw_buffer_load_b64(rk, ko, 0, 0);
            k[t][0] = w[0], k[t][1] = w[1];
        } else {
#pragma unroll
            for (int x = 0; x < D / 128; ++x) {
                const auto w = __builtin_amdgcn_raw_buffer_load_b128(rk, ko + 16 * x, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) k[t][(4 * x + e) % (D / 32)] = w[e];
            }
        }
        ks[t] = D == 256 ? __builtin_amdgcn_raw_buffer_load_b16(rks, kso, 0, 0) : __builtin_amdgcn_raw_buffer_load_b8(rks, kso, 0, 0);
    }
#endif
}

__device__ __forceinline__ int wave_scan_int(int v) {   // sum over the lanes up to this one
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int t = __shfl_up(v, o, kWave);
        if (lane >= o) v += t;
    }
    return v;
}

// Slots of a batch row: committed ones and new ones; false for an error row.
__device__ __forceinline__ bool kvq_row_ok(int pre, int cnt, int N, int capacity) {
    return pre >= 0 && cnt >= 0 && cnt <= N && static_cast<long>(pre) + cnt <= capacity;
}

}  // namespace sv
