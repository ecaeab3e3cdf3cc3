// The paged key/value cache: pages handed out, rows written, attention over a
// shared prefix and each row's own pages.  Argument blocks of its kernels.
#pragma once

#include "common.hpp"
#include "internal.hpp"

namespace sv {

// Pages and slots of a step (paged_step.hip).
struct PageStepArgs {
    int32_t* tables;                // [T][width]
    long long table_stride;
    int T, width, pages, page_log2, N;
    const int32_t* held;            // [T]
    const int32_t* state;           // [2]: head of the ring, free pages
    int32_t* ring;                  // [pages]
    const int32_t* lengths;         // [T]
    const int32_t* counts;          // [T] or null: N
    int32_t* out_held;              // [T], may be held
    int32_t* out_state;             // [2], may be state
    int32_t* out_granted;           // [T]
    int32_t* out_slots;             // [T][N]
    int apart;                      // out_held and out_state are other arrays than held and state
    unsigned* done;                 // workgroups that have read their inputs; zero before and after a call (unless apart)
};
hipError_t launch_page_step(const PageStepArgs& a, hipStream_t s, Timing t = {});

// K and V pages: row (page, slot of it, head) at k/v + page*page_stride + slot*slot_stride + head*head_stride elements, bf16.
struct PagedCache {
    uint16_t *k, *v;
    long long page_stride, slot_stride, head_stride;
    int pages, page_log2, H, D;
};
// Rows (b, n, head) of D elements, strides in elements.
struct PagedRows {
    const void* data;
    long long batch, pos, head;
};
struct PagedAppendArgs {
    PagedCache c;
    PagedRows k, v;
    int dtype, B, N, source_n;      // rows a batch row: N slots, source_n tokens of k and v
    const int32_t* slots;           // [B][slots_stride]
    long long slots_stride;
    const int32_t* path;            // [B][path_stride] or null: token n itself
    int path_stride;
    const int32_t* accept_len;      // [B] with a path
};
hipError_t launch_paged_append(const PagedAppendArgs& a, hipStream_t s, Timing t = {});

// ---- attention ----

constexpr int kPgChunk = 128;       // units of the key axes' split
constexpr int kPgMaskN = 64;         // most new tokens of a call with a mask
constexpr int kPgWide = 128, kPgNarrow = 32;    // query rows of a workgroup: 32 a wave, or the same 32 for all four

// One workgroup's work for each head: query rows row0 .. of a job against keys k0 .. k1 - 1 of one table row.
struct PagedUnit {
    int b0;                         // first batch row of the job's query rows
    int row0, rows;                 // first query row of this unit, and one past the job's last
    int table;                      // row of the tables
    int k0, k1;
    int pre;                        // committed slots: later ones are new tokens' (a prefix: none are)
    int cnt;                        // new tokens
    int part;                       // row of the parts it writes to, -1: the call's output itself
    int wide;                       // kPgWide rows, or kPgNarrow
    int pad[2];
};
// What joins into a batch row's outputs: parts of the shared prefix, the i-th of query row r at first + i*step + r.
struct PagedShared {
    int first, step, count;
    int live;                       // tokens that have an output (error rows: 0)
};
// And of one tile of its query rows against its own slots, i*step rows apart; count 0: written directly.
struct PagedOwn {
    int first, count;
};

constexpr int kPgHead = 6;
struct PagedPlan {                  // device memory
    int32_t* head;                  // [kPgHead]: units, and the sizes it was made for
    PagedUnit* unit;                // [max_units]
    PagedShared* shared;            // [B]
    PagedOwn* own;                  // [B][own_tiles]
};
struct PagedPlanArgs {
    int B, N, T, M, heads, D, width, page_log2;
    const int32_t* lengths;         // [T]
    const int32_t* counts;          // [B] or null
    const int32_t* prefix_row;      // [B] or null
    // from the sizes alone (paged_plan_sizes)
    int G, own_rows, own_tiles;     // query rows a unit of own slots, units a batch row
    int target;                     // units the key axes are split into, 0: not at all
    int shape;                      // heads, D and whether there are prefixes, as far as the plan goes by them
    long long max_units, max_parts; // most units, and rows of parts
    PagedPlan p;
};
void paged_plan_sizes(PagedPlanArgs& a);
hipError_t launch_paged_plan(const PagedPlanArgs& a, hipStream_t s, Timing t = {});

struct PagedAttnArgs {
    PagedCache c;
    PagedRows q;
    int dtype, B, N, Hq, G, M;
    const int32_t* tables;
    long long table_stride;
    PagedPlan p;
    int own_rows, own_tiles, shape, capacity;
    long long max_units;
    const uint8_t* mask;
    long long mask_batch;
    float cexp;
    void* out;
    float* out_lse;
    float* part_o;                  // [max_parts][H][D], null: nothing is joined
    float* part_ml;                 // [max_parts][H][2]
};
hipError_t launch_paged_attention(const PagedAttnArgs& a, hipStream_t s, Timing t = {});

}  // namespace sv
