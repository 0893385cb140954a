"""How the cache attention's line of units is cut, on the host (no GPU needed): the arithmetic of kda_attend_line.h under
a plain walk over all workgroups' shares, as the kernels do it, for row starts of any kind.  Each row of units is to be
covered once, its pieces in workgroups that exist; a line that is too long is left alone."""

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MODEL = r"""
#include "kda_attend_line.h"
#include <cstdio>
#include <cstdlib>
#include <vector>
using namespace kda;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

// input: cases of  tokens G Hk block grid at_least room  B  starts[B + 1] contexts[B]; output: accepted, units of each
int main()
{
    int tokens, G, Hk, block, grid, at_least, B;
    long long room;
    while (scanf("%d %d %d %d %d %d %lld %d", &tokens, &G, &Hk, &block, &grid, &at_least, &room, &B) == 8) {
        std::vector<int> start(B + 1), context(B);
        for (int &x : start) if (scanf("%d", &x) != 1) return 2;
        for (int &x : context) if (scanf("%d", &x) != 1) return 2;
        if (!line_fits((room + 63) / 64, (long long)tokens * G, block, B, Hk)) { printf("refused\n"); continue; }
        std::vector<Sequence> seq;
        unsigned units = 0, rows = 0;
        for (int b = 0; b < B; ++b) {
            const Sequence s = sequence_of(start[b], start[b + 1], tokens, context[b], room);
            CHECK(s.first >= 0 && s.queries >= 0 && s.first + s.queries <= tokens && s.context >= 0 && s.context <= room);
            const unsigned r = (unsigned)blocks_of(s, G, block) * Hk;
            CHECK((unsigned long long)r * tiles_of(s) < LINE_LIMIT);
            rows = units_add(rows, r);
            units = units_add(units, r * tiles_of(s));
            seq.push_back(s);
        }
        printf("%u\n", units);
        if (units == 0 || units >= LINE_LIMIT) continue;
        const int share = share_of(units, rows, grid, at_least);
        CHECK(share > 0 && (long long)share * grid >= units);
        // the walk: sequence, unit of it; of the row of units that is open: who began it, who is to end it
        int b = 0, first = 0, last = 0;
        long long u = 0, seen = 0;
        for (int w = 0; w < grid; ++w) {
            long long at = (long long)share * w;
            if (at >= units) break;
            int left = (long long)units - at < share ? (int)(units - at) : share, fronts = 0, others = 0;
            while (left > 0) {
                CHECK(b < B);
                const int tiles = tiles_of(seq[b]);
                if (u >= (long long)tiles * blocks_of(seq[b], G, block) * Hk) { u = 0; ++b; continue; }
                const int from = (int)(u % tiles), to = from + left < tiles ? from + left : tiles, n = to - from;
                if (from == 0) {
                    first = w;
                    last = last_share((unsigned)at, tiles, share);
                    CHECK(last >= first && last < grid);
                    fronts += to < tiles;
                } else {
                    CHECK(w > first && w <= last);
                    ++others;
                }
                CHECK((to == tiles) == (w == last));      // the row's last piece is where it was said to be
                u += n; at += n; left -= n; seen += n;
            }
            CHECK(fronts <= 1 && others <= 1);            // one piece of a kind a workgroup
        }
        CHECK(seen == units);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("g++ or the HIP headers not found")
    d = tmp_path_factory.mktemp("line")
    (d / "model.cpp").write_text(MODEL)
    subprocess.run([gxx, "-O1", "-std=c++17", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
                    os.path.join(ROOT, "gated_delta_rule_101_amd", "csrc"), str(d / "model.cpp"), "-o", str(d / "model")],
                   check=True)

    def run(cases):
        text = "\n".join(" ".join(str(x) for x in (*c[:7], len(c[8]), *c[7], *c[8])) for c in cases)
        r = subprocess.run([str(d / "model")], input=text, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout[-300:]
        out = r.stdout.split()
        assert len(out) == len(cases)
        return out
    return run


def test_lines_are_cut_inside_the_grid(model):
    rng = random.Random(1)
    cases = []
    for _ in range(400):
        B, tokens = rng.choice([1, 2, 3, 7, 64, 65, 300]), rng.choice([1, 5, 64, 700, 5000])
        room = rng.choice([0, 16, 64, 100 * 16, 4096, 40000])
        kind = rng.randrange(3)
        starts = [rng.randint(-9, tokens + 9) for _ in range(B + 1)]
        if kind == 0:
            starts = sorted(starts)
        elif kind == 1:
            starts = [(b & 1) * tokens for b in range(B + 1)]
        contexts = [rng.choice([-3, 0, 1, 63, 64, 65, room, rng.randint(0, room + 1), 2 ** 31 - 1]) for _ in range(B)]
        cases.append((tokens, rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 8]), rng.choice([16, 64, 128]),
                      rng.choice([1, 7, 256, 512, 1024]), rng.choice([1, 4]), room, starts, contexts))
    out = model(cases)
    assert sum(x not in ("refused", "0") for x in out) > 300


def test_lines_that_are_too_long_are_seen_to_be(model):
    """Row starts that alternate count every row of the call for every other sequence: sums past 2^32, whose low bits
    would be a line of any length."""
    cases = []
    for B, tokens, room in ((4096, 4096, 32768), (8192, 8192, 32768), (8192, 8192, 131072), (300, 60000, 60000)):
        for odd in range(3):
            contexts = [room - 64 * ((odd * b) % 97) for b in range(B)]
            cases.append((tokens, 8 if B == 4096 else 4, 8, 16, 512, 4, room, [(b & 1) * tokens for b in range(B + 1)], contexts))
    exact = [sum(-(-n // 64) * -(-c[0] * c[1] // c[3]) * c[2] for n in c[8][::2]) for c in cases]
    assert min(exact) > 2 ** 32 and any(0 < x % 2 ** 32 < 2 ** 31 for x in exact)
    assert model(cases) == [str(2 ** 32 - 1)] * len(cases)
    # and one of nearly the longest that is done
    n = 1200
    assert int(model([(n * 16, 1, 8, 16, 512, 4, 64 * 1000, [(b & 1) * n * 16 for b in range(301)], [64000] * 300)])[0]) == \
        150 * 1000 * n * 8
