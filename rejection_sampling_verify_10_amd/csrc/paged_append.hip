// New K and V rows into the pages their slots name.  A copy: eight elements a
// thread, rounded to bfloat16 where they are float32, so that a row of 128 is
// written in two full lines.  Bound by HBM for prompts (4 x 4095 float32 rows of 8
// heads of 128: 37.6 us, 5.4 TB/s), by latency for a step (32 x 27 bf16 rows: 3.2 us).

#include "kvq.hpp"
#include "paged.hpp"

namespace sv {

namespace {

constexpr int kThreads = 256;

template <int DT, int D>
__global__ __launch_bounds__(kThreads) void paged_append_kernel(PagedAppendArgs a) {
    constexpr unsigned kPer = D / 8;                    // threads a row
    const unsigned i = blockIdx.x * kThreads + threadIdx.x;     // a call has fewer than 2^32 threads
    const int e = static_cast<int>(i % kPer) * 8;
    const unsigned row = i / kPer, bn = row / a.c.H;    // (b, n, head)
    const int h = static_cast<int>(row - bn * a.c.H);
    const int b = static_cast<int>(bn / a.N), n = static_cast<int>(bn - static_cast<unsigned>(b) * a.N);
    if (b >= a.B) return;
    int from = n;
    if (a.path) {
        const int acc = a.accept_len[b];
        if (acc < 0 || acc >= a.N || n > acc) return;
        from = a.path[static_cast<long long>(b) * a.path_stride + n];
        if (from < 0 || from >= a.source_n) return;
    }
    const long long slot = a.slots[b * a.slots_stride + n];
    if (slot < 0 || slot >= static_cast<long long>(a.c.pages) << a.c.page_log2) return;
    const long long to = (slot >> a.c.page_log2) * a.c.page_stride +
                         (slot & ((1 << a.c.page_log2) - 1)) * a.c.slot_stride + h * a.c.head_stride + e;
    const auto copy = [&](const PagedRows& r, uint16_t* pages) {
        const long long at = b * r.batch + from * r.pos + h * r.head + e;
        u32x4 w;
        if (DT == 1) {
            w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(r.data) + at);
        } else {
            const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(r.data) + at);
            const f32x4 lo = p[0], hi = p[1];
            w = u32x4{pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]), pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3])};
        }
        *reinterpret_cast<u32x4*>(pages + to) = w;
    };
    copy(a.k, a.c.k);
    copy(a.v, a.c.v);
}

template <int DT, int D> void append(const PagedAppendArgs& a, hipStream_t s, Timing t) {
    const long long threads = static_cast<long long>(a.B) * a.N * a.c.H * (D / 8);
    const dim3 grid(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
    launch_timed(t, paged_append_kernel<DT, D>, grid, dim3(kThreads), 0, s, a);
}
template <int DT> void append(const PagedAppendArgs& a, hipStream_t s, Timing t) {
    if (a.c.D == 64) append<DT, 64>(a, s, t);
    else if (a.c.D == 128) append<DT, 128>(a, s, t);
    else append<DT, 256>(a, s, t);
}

}  // namespace

hipError_t launch_paged_append(const PagedAppendArgs& a, hipStream_t s, Timing t) {
    if (a.dtype == 1) append<1>(a, s, t);
    else append<0>(a, s, t);
    return hipGetLastError();
}

}  // namespace sv
