"""Every copy with which a cluster's CTAs bring in G stays inside G, for sizes of every kind (no GPU).

The kernel's own arithmetic (csrc/slab.h) is compiled for the host and every word that it copies is compared with
the tensor's bounds; the staging area's too.  A cluster is a power of two of CTAs, so the last ones may begin past
the last column, and matrices after the first may begin off 16 bytes."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_expert_layer_permute_gb300", "csrc")

HARNESS = r"""
#include <cstdio>
#include <algorithm>
#include "slab.h"
using namespace moe;
// lines "N R C bytes" -> "S idle copies outside", where a tensor begins on a 16-byte boundary
template <int W, int STEP>
static void copies(uintptr_t from, const NsRun& run, int bytes, uintptr_t lo, uintptr_t hi, long long room, long long* n, long long* bad) {
    const NsWords<W> words(from, run.count * bytes);
    for (int t = 0; t < STEP; ++t)
        words.template each<STEP, 1>(t, [&](int w, int held) {
            ++*n;
            const uintptr_t at = words.at + w;
            if (at < lo || at + held > hi || held <= 0 || held > W || run.at + w < 0 || run.at + w + W > room) ++*bad;
        });
}
int main() {
    long long N, R, C, bytes;
    while (std::scanf("%lld %lld %lld %lld", &N, &R, &C, &bytes) == 4) {
        const long long m = std::min(R, C), n = std::max(R, C);
        const bool flip = R > C;
        int mp, S = ns_small_cluster(N, m, n, &mp), log_mp = 0;
        while ((1 << log_mp) < mp) ++log_mp;
        const uintptr_t base = 1 << 20, end = base + (uintptr_t)(N * R * C * bytes);
        const int pitch = kSmallCols * (int)bytes + 4;
        const long long room = 163840;
        long long count = 0, bad = 0, idle = 0;
        for (int rank = 0; rank < S; ++rank) {
            const NsSlab slab{(int)m, (int)n, log_mp, flip, rank * (128 >> log_mp) * kSmallCols};
            idle += slab.cta0 >= n;
            for (long long mat : {0ll, N / 2, N - 1}) {
                const uintptr_t g = base + (uintptr_t)(mat * R * C * bytes);
                for (int warp = 0; warp < (flip ? 1 : kSmallThreads / 32); ++warp)
                    slab.each(pitch, warp, [&](const NsRun& run) {
                        const uintptr_t from = g + (uintptr_t)((long long)run.first * bytes);
                        if (flip) copies<16, kSmallThreads>(from, run, (int)bytes, base, end, room, &count, &bad);
                        else copies<4, 32>(from, run, (int)bytes, base, end, room, &count, &bad);
                    });
            }
        }
        std::printf("%d %lld %lld %lld\n", S, idle, count, bad);
    }
}
"""

SIZES = [(2, 2501, 61), (2, 2051, 127), (5, 2101, 21), (18, 2049, 127), (18, 1025, 127), (2, 1300, 33), (3, 61, 2501), (1, 127, 32768),
         (1, 32767, 127), (7, 9, 17), (2, 128, 129), (2, 129, 128), (3, 257, 9), (3, 33, 1030), (2, 16, 32768)]


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    d = tmp_path_factory.mktemp("copies")
    (d / "copies.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-I", CSRC, str(d / "copies.cpp"), "-o",
                    str(d / "copies")], check=True)
    return str(d / "copies")


def drawn():
    rng = random.Random(1)
    for _ in range(1500):
        a, b = rng.randint(9, 128), int(2 ** rng.uniform(3.2, 15))
        yield (rng.choice([1, 2, 3, 5, 18, 101]), a, b) if rng.random() < 0.4 else (rng.choice([1, 2, 3, 5, 18, 101]), b, a)


def test_copies_stay_inside(harness):
    cases = [(N, R, C, size) for N, R, C in SIZES + list(drawn()) for size in (2, 4)]
    out = subprocess.run([harness], input="".join("%d %d %d %d\n" % c for c in cases), capture_output=True, text=True, check=True).stdout
    rows = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert len(rows) == len(cases)
    assert sum(idle > 0 for _, idle, _, _ in rows) > 100     # clusters with CTAs past the last column are among them
    assert all(copies > 0 for S, _, copies, _ in rows if S)
    assert [c for c, r in zip(cases, rows) if r[3]] == []
