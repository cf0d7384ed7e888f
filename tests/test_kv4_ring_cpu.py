"""CPU check of the 4-bit attention's ring of tile slots (csrc/kv4_ring.cuh): the order in which a warp issues copies and
waits for them, run against a model of the barriers, with copies that land late or never."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "kv4_ring.cuh"
using talker_k::Kv4Ring;

// A slot's barrier: a phase completes when the copy that it expects lands. A wait for a parity passes when the phase
// of that parity is complete, that is, when the barrier is in one of the other parity.
struct Slot {
    unsigned phase = 0;
    bool flying = false;
    int tile = -1, next = -1;   // what it holds, what is on its way
    int late = 0;               // waits that run out before it lands (-1: never)
};
struct Model {
    std::vector<Slot> slots;
    int copies = 0, late_copy, late, faults = 0;
    void issue(int s, int tile) {
        if (slots[s].flying) ++faults, printf("copy %d over one in flight\n", copies);
        slots[s].flying = true, slots[s].next = tile, slots[s].late = copies++ == late_copy ? late : 0;
    }
    bool wait(int s, unsigned parity) {
        Slot &x = slots[s];
        if (x.flying && x.late == 0) x.flying = false, x.tile = x.next, x.phase ^= 1;
        const bool ok = (x.phase & 1) != parity;
        if (!ok && x.late > 0) --x.late;
        return ok;
    }
};

// One warp's way through its rows of `pages` pages each, as in the kernel: K and V of a page in two slots, the next
// page's tiles over them. Returns whether all went well; a row is right, or NaN.
static bool walk(int n_slots, const std::vector<int> &rows, int late_copy, int late, bool &lost) {
    Model m;
    m.slots.resize(n_slots);
    m.late_copy = late_copy, m.late = late;
    Kv4Ring state;
    int slot = 0, n_it = 0, waits_out = 0;
    auto after = [&](int s) { return s == n_slots - 1 ? 0 : s + 1; };
    auto tile = [](int row, int page, bool v) { return (row * 100 + page) * 2 + v; };
    auto issue = [&](int to, int t) { state.issued(to), m.issue(to, t); };
    auto wait = [&](int at) {
        const bool ok = m.wait(at, state.parity(at));
        if (ok) state.landed(at);
        else ++waits_out;
        return ok;
    };
    auto open = [&](int row) {
        n_it = state.lost() ? 0 : rows[row];
        if (n_it > 0) issue(slot, tile(row, 0, false)), issue(after(slot), tile(row, 0, true));
        if (n_slots == 3 && n_it > 1) issue(after(after(slot)), tile(row, 1, false));
    };
    open(0);
    for (int row = 0; row < (int)rows.size(); ++row) {
        for (int it = 0; it < n_it; ++it) {
            const int vslot = after(slot);
            if (!wait(slot)) { state.lose(); break; }
            if (m.slots[slot].tile != tile(row, it, false)) ++m.faults, printf("row %d page %d: K of another\n", row, it);
            if (it + 1 < n_it) issue(slot, tile(row, it + 1, n_slots == 3));
            if (!wait(vslot)) { state.lose(); break; }
            if (m.slots[vslot].tile != tile(row, it, true)) ++m.faults, printf("row %d page %d: V of another\n", row, it);
            if (it + (n_slots == 3 ? 2 : 1) < n_it) issue(vslot, tile(row, it + (n_slots == 3 ? 2 : 1), n_slots != 3));
            slot = after(vslot);
        }
        if (n_it > 0 && state.lost())
            for (int i = 0; i < n_slots; ++i)
                if (state.in_flight(i)) wait(i);
        if (row + 1 < (int)rows.size()) open(row + 1);
    }
    lost = state.lost();
    for (int i = 0; i < n_slots; ++i) {   // nothing is left in flight but a copy that two waits have not seen
        if (m.slots[i].flying != state.in_flight(i)) ++m.faults, printf("slot %d: the state is wrong about its copy\n", i);
        if (m.slots[i].flying && waits_out < 2) ++m.faults, printf("slot %d: a copy that nobody waited for\n", i);
    }
    if (waits_out > 2) ++m.faults, printf("%d waits ran out\n", waits_out);   // the first one, and once more for it
    if (lost != (late != 0 && late_copy < m.copies)) ++m.faults, printf("a late copy was not seen, or one seen that was not\n");
    return m.faults == 0;
}

int main() {
    const std::vector<std::vector<int>> work = {{1}, {2}, {3}, {7}, {1, 1, 1}, {0, 2, 0, 3}, {4, 1, 2}, {5, 0, 0, 1, 6}, {2, 2, 2, 2}};
    int bad = 0, runs = 0;
    for (int n_slots = 2; n_slots <= 3; ++n_slots)
        for (const auto &rows : work)
            for (int late : {0, 1, 2, -1})
                for (int copy = 0; copy < 30; ++copy) {
                    bool lost = false;
                    if (!walk(n_slots, rows, copy, late, lost)) ++bad, printf("%d slots, copy %d late %d\n", n_slots, copy, late);
                    ++runs;
                }
    printf("%d of %d\n", bad, runs);
    return bad != 0;
}
"""


def test_late_copies(tmp_path):
    cxx = shutil.which("g++") or pytest.skip("no C++ compiler")
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "kv_cached_qwen3_gb300", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:]
