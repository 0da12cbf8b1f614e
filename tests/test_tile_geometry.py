"""Where the gated scan's tiles read and write, checked on the host: a small C++
program takes the kernels' geometry, walks every thread of every tile shape
over rows of every length and counts what lies outside a row, and what is left
unwritten."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_recurrence_sequence_diag_amd",
                    "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <stddef.h>
#include <stdint.h>
#include <vector>
@GEOMETRY@
#include "gated_geo.hpp"
using namespace lrscan;

template <int EB_, int TPR_, int NR_>
struct Shape {
    static constexpr int EB = EB_, V = 16 / EB_, TPR = TPR_, NR = NR_, WAVES = 4;
    static constexpr int RG = 64 / TPR, W = TPR * V, CT = WAVES * RG * NR;
};

long outside = 0, lost = 0, threads = 0;

// One batch row of T steps of D channels, tile by tile.
template <class C, int RK, bool REV>
void rows(int D, int T) {
    Dims d;
    d.T = T, d.D = D, d.nW = (D + C::W - 1) / C::W, d.nS = d.nW, d.NK = (T + C::CT - 1) / C::CT;
    const long rowbytes = (long)D * C::EB, end = rowbytes * T;
    std::vector<char> written((size_t)D * T, 0);
    for (int ticket = 0; ticket < d.nS * d.NK; ++ticket)
        for (int wave = 0; wave < C::WAVES; ++wave)
            for (int rg = 0; rg < C::RG; ++rg)
                for (int cg = 0; cg < C::TPR; ++cg) {
                    const Geo g = gated_geo<C, RK, REV>(ticket, d, wave, rg, cg);
                    ++threads;
                    for (int i = 0; i < C::NR; ++i) {
                        const long at = (long)g.tbase + row_off(g, g.row0 + i, T, (uint32_t)rowbytes);
                        // every thread loads 16 bytes of one row, whatever it owns
                        if (at < 0 || at + 16 > end || at / rowbytes != (at + 15) / rowbytes) ++outside;
                        if (i >= g.nrows) continue;
                        const long want = ((long)(g.row0 + i) * D + g.d0) * C::EB;
                        if (at != want || g.nvalid != C::V) ++outside;
                        else
                            for (int j = 0; j < C::V; ++j) written[at / C::EB + j] = 1;
                    }
                }
    for (char w : written) lost += !w;
}

template <class C>
void lengths() {
    for (int D = C::V; D <= 3 * C::W + C::V; ++D)
        for (int T : {1, C::CT - 1, C::CT + 3}) {
            rows<C, kWhole, false>(D, T);
            rows<C, kWhole, true>(D, T);
            if (D % C::V == 0) rows<C, kAligned, false>(D, T);
        }
}

int main() {
    lengths<Shape<4, 16, 2>>(), lengths<Shape<4, 16, 4>>(), lengths<Shape<4, 8, 4>>(), lengths<Shape<4, 8, 8>>();
    lengths<Shape<2, 16, 2>>(), lengths<Shape<2, 16, 4>>(), lengths<Shape<2, 8, 4>>(), lengths<Shape<2, 8, 8>>();
    printf("%ld %ld %ld\n", threads, outside, lost);
}
"""


def test_every_access_lies_in_its_row(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "geometry.cpp", tmp_path / "geometry"
    with open(os.path.join(CSRC, "fused_common.hpp")) as f:
        text = f.read()
    # from the tile's dimensions to the end of the row offsets: plain integer code
    geometry = text[text.index("struct Dims {"):text.index("// Segment-start byte of row i")]
    src.write_text(PROGRAM.replace("@GEOMETRY@", geometry))
    subprocess.run([cxx, "-std=c++17", "-O2", "-D__device__=", "-D__forceinline__=inline", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    threads, outside, lost = map(int, subprocess.run([str(exe)], check=True, capture_output=True,
                                                     text=True).stdout.split())
    assert threads > 10 ** 6 and (outside, lost) == (0, 0)
