"""How the attention counts the units of a request's tiles, on the CPU: the functions of csrc/hq_attention.cuh, compiled for the
host, against a count of every tile's units.  A block finds its work by these sums alone."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_weight_matvec_hq_gb300", "csrc")
FUNCTIONS = ("floor_sum", "unit_sum", "seen_by", "tiles_of", "units_before", "window_of", "quotient", "first_unit", "block_of")

HARNESS = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#define __device__
#define __forceinline__ inline
using std::max; using std::min;
struct CacheView { long long table_width; int page_shift; };
struct AttnArgs { CacheView c; int tokens, causal, unit_shift, blocks; long long window; };
struct Request { int first, n, length; bool bad; };
%s
// argv: the window of the call, then a request's tokens and length, a tile's tokens, the unit, causal.  Prints the units before
// each tile, and counted tile by tile: from the first position that its first token sees to the last one's last.
// With two arguments, the units and the blocks: that the blocks' ranges follow one another to the end, and which block has a unit.
int main(int argc, char **argv) {
    AttnArgs a;
    if (argc == 3) {
        const long long total = std::atoll(argv[1]);
        a.blocks = std::atoi(argv[2]);
        long long at = 0, wrong = first_unit(a, total, 0) != 0, most = 0, least = total;
        for (int b = 0; b < a.blocks; ++b) {
            const long long x0 = first_unit(a, total, b), end = first_unit(a, total, b + 1);
            wrong += x0 != at || end < x0;
            if (end > x0) {
                wrong += block_of(a, total, x0) != b || block_of(a, total, end - 1) != b || block_of(a, total, (x0 + end) / 2) != b;
                most = max(most, end - x0);
                least = min(least, end - x0);
            }
            at = end;
        }
        std::printf("%%lld\n", wrong + (at != total) + (total > 0 && most - least > 1));
        return 0;
    }
    a.c = {1 << 10, 6};
    a.window = window_of(std::atoll(argv[1]), a.c);
    const Request q = {0, std::atoi(argv[2]), std::atoi(argv[3]), false};
    a.tokens = std::atoi(argv[4]);
    a.unit_shift = std::atoi(argv[5]);
    a.causal = std::atoi(argv[6]);
    const unsigned long long w = std::strtoull(argv[1], nullptr, 10);
    long long count = 0;
    for (int j = 0; j <= tiles_of(a, q); ++j) {
        std::printf("%%lld %%lld\n", units_before(a, q, j), count);
        const long long p0 = (long long)q.length - q.n + (long long)j * a.tokens;           // position of the first token
        const long long p1 = (long long)q.length - q.n + min((long long)(j + 1) * a.tokens, (long long)q.n) - 1;
        const long long lo = w > 0 && p0 >= 0 && w <= (unsigned long long)p0 ? p0 + 1 - (long long)w : 0;
        const long long hi = a.causal ? max(p1 + 1, 0ll) : q.length, size = 1ll << a.unit_shift;
        count += max(1ll, (hi + size - 1) / size - lo / size);
    }
}
"""


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    text = open(os.path.join(CSRC, "hq_attention.cuh")).read()
    parts = [re.search(r"struct Range \{[^\n]*\};", text).group(0)]
    for name in FUNCTIONS:
        m = re.search(r"^(?:__device__ __forceinline__|inline) [\w ]+ \b%s\([^{;]*\) \{" % name, text, flags=re.M)
        assert m, name
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        parts.append(text[m.start():i])
    out = tmp_path_factory.mktemp("units")
    (out / "units.cpp").write_text(HARNESS % "\n".join(parts))
    gxx = shutil.which("g++")
    assert gxx
    subprocess.run([gxx, "-O1", "-fwrapv", "-std=c++17", "-o", str(out / "units"), str(out / "units.cpp")], check=True)
    return str(out / "units")


@pytest.mark.parametrize("window", [0, 1, 2, 31, 64, 65, 1000, 65535, 65536, 65537, 10 ** 9, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 40,
                                    2 ** 62, 2 ** 63 - 20, 2 ** 63 - 1])
def test_units_of_tiles(harness, window):
    for n, length in ((2011, 2011), (2011, 40000), (1, 1), (1, 65536), (64, 64), (333, 1000), (30, 3), (5, 0), (130, 128)):
        for tokens, shift in ((128, 7), (32, 7), (9, 7), (1, 7), (16, 6), (5, 6), (1, 6)):
            for causal in (1, 0) if window == 0 else (1,):
                args = [str(i) for i in (window, n, length, tokens, shift, causal)]
                lines = subprocess.run([harness, *args], check=True, capture_output=True, text=True).stdout.split("\n")[:-1]
                wrong = [i for i in lines if len(set(i.split())) != 1]
                assert not wrong, (args, len(wrong), len(lines), wrong[:2])


@pytest.mark.parametrize("total", [0, 1, 2, 7, 303, 304, 305, 607, 608, 609, 12345, 10 ** 6, 2 ** 31 + 1, 2 ** 40 + 12345])
def test_units_of_blocks(harness, total):
    """Equal contiguous shares, one unit apart at most; a block finds the block of any unit."""
    for blocks in (1, 2, 152, 304, 456, 608):
        assert subprocess.run([harness, str(total), str(blocks)], check=True, capture_output=True, text=True).stdout == "0\n", blocks
