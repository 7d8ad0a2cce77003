"""The row tiles of the MXFP4 product (csrc/mx4_tiles.h), compiled for the host: every group's rows are covered once, in
order, by tiles of at most BN rows -- up to the largest group that an int32 counts."""
import subprocess

import pytest

from expert_offload_serving_router_b200 import build as ftbuild

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "mx4_tiles.h"
using namespace ftmoe;
template <int BN> static long check(const std::vector<int>& n, int m_tiles) {
    std::vector<int> off{0}, nt{0};
    for (int v : n) { off.push_back(off.back() + v); nt.push_back(nt.back() + px_row_tiles<BN>(v)); }
    const int G = int(n.size());
    long bad = 0;
    std::vector<long> next(off.begin(), off.end() - 1);
    for (long t = 0; t < long(nt[G]) * m_tiles; ++t) {
        const PxTile x = px_tile<BN>(int(t), nt.data(), off.data(), G, m_tiles);
        if (x.g < 0 || x.g >= G || x.m != t % m_tiles || x.nvalid < 1 || x.nvalid > BN || x.row0 < off[x.g] ||
            long(x.row0) + x.nvalid > off[x.g + 1] || x.row0 != next[x.g]) { ++bad; if (bad > 3) return bad; }
        if (x.m == m_tiles - 1) next[x.g] += x.nvalid;
    }
    for (int g = 0; g < G; ++g) bad += next[g] != off[g + 1];
    return bad;
}
static long all(const std::vector<int>& n, int m) { return check<32>(n, m) + check<96>(n, m) + check<224>(n, m); }
int main() {
    long bad = 0;
    for (int n = 1; n < 3000; ++n) bad += all({n}, 1);
    bad += all({0, 1, 0, 33, 225, 0, 0, 97, 4096, 31}, 3);
    for (int n : {2147483647, 2138000000, 2082408385}) bad += all({n}, 1);
    bad += all({5, 2147483000, 0, 600}, 1);
    std::printf("%ld\n", bad);
}
"""


@pytest.mark.parametrize("flags", [["-O2"], ["-O2", "-fsanitize=undefined", "-fno-sanitize-recover"]])
def test_row_tiles_cover_every_group(tmp_path, flags):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", *flags, "-I", ftbuild.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert int(r.stdout) == 0
