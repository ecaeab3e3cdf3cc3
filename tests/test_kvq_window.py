"""The four-bit cache's loads stay inside the rows they may read (no GPU needed).

The offsets and bounds of the buffer loads are plain arithmetic in ``csrc/kvq_window.hpp``; it is compiled for the host
and tried for every slot count and lane.  A load's scalar offset need not count in the hardware's comparison with the
descriptor's bytes, so no load may have one."""

import glob
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rejection_sampling_verify_10_amd", "csrc")

DRIVER = r"""
#include <cstdio>
#include <initializer_list>
#include "kvq_window.hpp"
using namespace sv;

// One load of `size` bytes at vector offset `off` of a tile with `slots` slots of `row` bytes, `pos` apart: it is made
// exactly where its slot is there, and then it stays inside that slot's row, at byte `want` of it.
static bool load_ok(long off, int size, int slots, long pos, int row, int slot, int want) {
    const bool made = off < slots * pos, there = slot < slots;
    if (made != there) return false;
    if (made && off + size > (slots - 1) * pos + row) return false;
    return off == slot * pos + want && want + size <= row;
}

int main() {
    long tried = 0;
    for (int D = 64; D <= 256; D *= 2)
        for (long cp : {(long)D / 2, (long)D / 2 + 16, (long)8 * D, 1l << 24})
            for (long sp : {(long)D / 32, (long)D / 4, 1l << 24})
                for (long first : {0l, 32l, 131040l, (1l << 30) - 32})
                    for (int n = -40; n <= 40; ++n)
                        for (int tile = 0; tile < kStep / kTile; ++tile) {
                            const long end = first + n, at = first + kTile * tile;
                            const int slots = tile_slots(slots_left((int)at, (int)end));
                            long there = 0;                 // counted one by one
                            for (int s = 0; s < kTile; ++s) there += at + s < end;
                            bool ok = slots == there && slots * cp < (1l << 31) && slots * sp < (1l << 31);
                            for (int c = 0; c < 16; ++c)
                                for (int g = 0; g < 4; ++g, ++tried) {
                                    ok = ok && load_ok(k_offset(D, c, g, (int)cp), k_bytes(D), slots, cp, D / 2, k_slot(c), g * D / 8);
                                    ok = ok && load_ok(k_scale_offset(D, c, g, (int)sp), k_scale_bytes(D), slots, sp, D / 32,
                                                       k_slot(c), g * (D / 4) / 32);
                                    for (int i = 0; i < 4; ++i) {
                                        ok = ok && load_ok(v_offset(D, c, g, (int)cp) + i * cp, v_bytes(D), slots, cp, D / 2,
                                                           v_slot(g, i), c * D / 32);
                                        ok = ok && load_ok(v_scale_offset(D, c, g, (int)sp) + i * sp, 1, slots, sp, D / 32,
                                                           v_slot(g, i), c * (D / 16) / 32);
                                    }
                                }
                            if (!ok) {
                                std::printf("D %d strides %ld %ld first %ld slots %d tile %d\n", D, cp, sp, first, n, tile);
                                return 1;
                            }
                        }
    std::printf("%ld lanes\n", tried);
    return 0;
}
"""


def test_loads_stay_inside_the_rows_that_are_there(tmp_path):
    (tmp_path / "driver.cpp").write_text(DRIVER)
    exe = str(tmp_path / "driver")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", exe, str(tmp_path / "driver.cpp")])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def scalar_offsets(text):
    """The scalar-offset operand of every buffer load in a source text."""
    found = []
    for m in re.finditer(r"raw_(?:ptr_)?buffer_load_\w+\(", text):
        depth, parts = 1, [""]
        for ch in text[m.end():]:
            depth += (ch == "(") - (ch == ")")
            if depth == 0:
                break
            if ch == "," and depth == 1:
                parts.append("")
            else:
                parts[-1] += ch
        found.append(parts[2].strip())
    return found


def test_no_load_has_a_scalar_offset():
    assert scalar_offsets("x = __builtin_amdgcn_raw_buffer_load_b8(r, f(a, b) + 1, 16 * t, 0);") == ["16 * t"]
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        with open(path) as f:
            offsets = scalar_offsets(f.read())
        assert all(o == "0" for o in offsets), (path, offsets)
        seen += len(offsets)
    assert seen > 0
