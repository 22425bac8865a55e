"""The paged attention's walk over a segment's keys (csrc/paged_walk.cuh), compiled
with the host C++ compiler: every key of a segment is taken by one warp and one
lane, none beyond its end is, and the walk ends, up to rows of the largest size,
where a step beyond the end passes 2^31."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hierarchical_kv_routing_b200", "csrc")

HARNESS = r"""
#include <cstdio>
#include <map>
#include "paged_walk.cuh"
using namespace hga;
// segment [u, u + cnt) of a row of n keys: the number of things that are wrong
static long check(int n, int u, int cnt, int keys, int kw) {
    const int uk = 4 * keys, nu = units_of(n, uk);
    const long long first = (long long)u * uk, last = u + cnt >= nu ? n : (long long)(u + cnt) * uk;
    long bad = nu != ((long long)n + uk - 1) / uk;
    std::map<long long, int> seen;
    for (int ksub = 0; ksub < kw; ++ksub) {
        int tiles = 0;
        for (KeyWalk w = key_walk(u, cnt, nu, n, uk, ksub, kw, keys); w.more(); w.next()) {
            if (++tiles > cnt * 4) return bad + 1;              // does not end
            for (int lane = 0; lane < keys; ++lane) {
                bool live;
                const unsigned k = w.key(lane, live);
                if (!live) continue;
                if ((int)k < first || (int)k >= last) return bad + 1;
                seen[k]++;
            }
        }
    }
    bad += (long)seen.size() != last - first;
    for (auto &s : seen) bad += s.second != 1;
    return bad;
}
int main() {
    long bad = 0;
    const int keys_of[] = {8, 16, 32}, kw_of[] = {4, 2}, top = 0x7fffffff;
    for (int keys : keys_of)
        for (int kw : kw_of) {
            const int uk = 4 * keys;
            for (int n = 1; n < 9 * uk; ++n)
                for (int u = 0; u < units_of(n, uk); ++u)
                    for (int cnt = 1; u + cnt <= units_of(n, uk); ++cnt) bad += check(n, u, cnt, keys, kw);
            for (int less = 0; less < 3 * uk; ++less)
                for (int back = 1; back < 5; ++back)
                    for (int cnt = 1; cnt <= back; ++cnt) {
                        const int n = top - less;
                        bad += check(n, units_of(n, uk) - back, cnt, keys, kw);
                    }
        }
    std::printf("%ld\n", bad);
    return 0;
}
"""


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    d = tmp_path_factory.mktemp("walk")
    src, exe = d / "walk.cpp", d / "walk"
    src.write_text(HARNESS)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover",
                           "-I", CSRC, "-o", str(exe), str(src)])
    return str(exe)


def test_every_key_once_and_none_beyond(harness):
    assert subprocess.check_output([harness], timeout=300).decode().strip() == "0"
