"""Where the gated delta rule's passes leave the states and gradients between
blocks, checked on the host: a small C++ program takes the kernels' arithmetic
of blocks, parts and places and replays the walks over rows with segments of
every density, in every number of parts.  What the gradients' pass reads has to
have one writer, the block that it belongs to."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_recurrence_sequence_diag_amd",
                    "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <vector>
#include "delta_blocks.hpp"
using namespace lrscan::delta;

long rows = 0, read = 0, wrong = 0, shared = 0;

// A row's blocks, and the blocks that write each place, walked in parts.
void replay(const std::vector<char>& reset, int parts) {
    const int T = (int)reset.size();
    std::vector<int> starts;
    for (int t = 0, from = 0; t < T; ++t) {
        if (reset[t]) from = t;
        if ((t - from) % kC == 0) starts.push_back(t | (reset[t] ? kCut : 0));
    }
    int n = (int)starts.size();
    starts.push_back(T);
    const Blocks blocks{starts.data(), &n, T};
    if (parts > n) return;
    ++rows;
    std::vector<std::vector<int>> enters(state_slots(T)), leaves(state_slots(T));
    for (int part = 0; part < parts; ++part) {
        const int first = part_start(n, part, parts), end = part_start(n, part + 1, parts);
        int start, len;
        bool cut;
        for (int c = first; c < end; ++c) {  // the walk keeps what enters a block
            blocks.at(0, c, start, len, cut);
            if (!cut) enters[entering_slot(start)].push_back(c);
        }
        bool behind = @BEHIND@;  // the walk back, what leaves one
        for (int c = end - 1; c >= first; --c) {
            blocks.at(0, c, start, len, cut);
            if (!behind) leaves[leaving_slot(T, start + len)].push_back(c);
            behind = cut;
        }
    }
    for (int c = 0; c < n; ++c) {  // the gradients' pass
        int start, len;
        bool cut;
        blocks.at(0, c, start, len, cut);
        const auto check = [&](const std::vector<int>& by) {
            ++read;
            if (by.size() != 1) ++shared;
            else if (by[0] != c) ++wrong;
        };
        if (!cut && start > 0) check(enters[entering_slot(start)]);
        if (!blocks.cut_behind(0, c, n)) check(leaves[leaving_slot(T, start + len)]);
    }
}

int main() {
    srand(1);
    for (int T : {1, 63, 64, 65, 200, 1024, 1700, 2048})
        for (int kind = 0; kind < 9; ++kind) {
            std::vector<char> r(T, 0);
            for (int t = 0; t < T; ++t) {
                const bool dense = kind == 1 || (kind == 2 && t >= T - T / 17) || (kind == 3 && t >= 65 && t < 128) ||
                                   (kind == 4 && t % 7 == 3) || (kind == 5 && t / 64 % 3 == 1 && t % 2);
                r[t] = dense || (kind == 6 && rand() % 3 == 0) || (kind == 7 && rand() % 40 == 0) ||
                       (kind == 8 && (rand() % 300 == 0 || (t > T / 2 && t < T / 2 + 60)));
            }
            for (int parts = 1; parts <= 24; ++parts) replay(r, parts);
        }
    printf("%ld %ld %ld %ld\n", rows, read, shared, wrong);
}
"""


def _replay(tmp_path, behind):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "blocks.cpp", tmp_path / "blocks"
    src.write_text(PROGRAM.replace("@BEHIND@", behind))
    subprocess.run([cxx, "-std=c++17", "-O2", "-D__device__=", "-D__host__=", "-D__forceinline__=inline", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    return [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]


def test_what_the_gradients_read_has_one_writer(tmp_path):
    """As the walk back does: whether a segment starts behind a part's last block is the next block's to say."""
    rows, read, shared, wrong = _replay(tmp_path, "blocks.cut_behind(0, end - 1, n)")
    assert rows > 1000 and read > 10 ** 4 and (shared, wrong) == (0, 0)


def test_the_replay_sees_a_place_with_two_writers(tmp_path):
    """A part that leaves what its last block hands on wherever the next segment starts writes into others' places."""
    _, _, shared, _ = _replay(tmp_path, "false")
    assert shared > 0
