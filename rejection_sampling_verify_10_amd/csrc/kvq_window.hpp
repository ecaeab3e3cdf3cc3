// Where the loads of a tile of 16 cache slots go: offsets and bounds of the buffer
// loads that read K and V, as plain arithmetic (no GPU code, so that a host test
// can try every slot count and lane of it).
//
// A load reads at base + vector offset + scalar offset and answers zeros past the
// descriptor's bytes.  Only the vector offset is sure to count in that comparison:
// the compiler's description of the load leaves the scalar one out of it, and
// where it is taken off the bytes first the difference may fall below zero.  So
// scalar offsets are zero here, and each tile has a descriptor of its own.
#pragma once

#include <cstdint>

namespace sv {

constexpr int kTile = 16;                               // slots of a descriptor
constexpr int kStep = 2 * kTile;                        // slots of one step

// Slots of the tile at `first` that lie below `end`, of the `left` ones from there: the descriptor's bytes end behind them.
// (Slots end at 2^30: 32 bits hold both.)
constexpr int slots_left(int first, int end) { return end > first ? end - first : 0; }
constexpr int tile_slots(int left) { return left < kTile ? left : kTile; }

// K: lane (c, g), c < 16, g < 4, reads the g-th quarter of the tile's slot c, and the scale byte(s) of it.
constexpr int k_slot(int c) { return c; }
constexpr int k_bytes(int D) { return D / 8; }
constexpr int k_scale_bytes(int D) { return D == 256 ? 2 : 1; }
constexpr uint32_t k_offset(int D, int c, int g, int code_pos) {
    return static_cast<uint32_t>(k_slot(c)) * code_pos + g * k_bytes(D);
}
constexpr uint32_t k_scale_offset(int D, int c, int g, int scale_pos) {
    return static_cast<uint32_t>(k_slot(c)) * scale_pos + g * D / 128;
}

// V: lane (c, g) reads elements c*D/16 .. of the tile's slots 4g + i, i < 4, and the scale byte of their block: at the
// offset for i = 0 and i slots more.
constexpr int v_slot(int g, int i) { return 4 * g + i; }
constexpr int v_bytes(int D) { return D / 32; }
constexpr uint32_t v_offset(int D, int c, int g, int code_pos) {
    return static_cast<uint32_t>(v_slot(g, 0)) * code_pos + c * v_bytes(D);
}
constexpr uint32_t v_scale_offset(int D, int c, int g, int scale_pos) {
    return static_cast<uint32_t>(v_slot(g, 0)) * scale_pos + c * (D / 16) / 32;
}

}  // namespace sv
