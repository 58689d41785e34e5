"""The norm's launches and the room for their sums (csrc/norm_plan.h), on the host: every block of every launch has its place."""
import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_expert_layer_permute_gb300", "csrc")


def _run(tmp_path, program, text=""):
    (tmp_path / "p.cpp").write_text(program)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "p.cpp"), "-o", str(tmp_path / "p")], check=True)
    return subprocess.run([str(tmp_path / "p")], input=text, capture_output=True, text=True, check=True).stdout


ROOM = r"""
#include <cstdio>
#include "norm_plan.h"
// lines "count n period" -> bytes that the launches' sums end at; tensor i has n values, or none where `period` divides i
int main() {
    long long count, n, period;
    while (std::scanf("%lld %lld %lld", &count, &n, &period) == 3) {
        auto size = [&](long long i) { return period && i % period == 0 ? 0ll : n; };
        for (int sms : {1, 2, 148, 152, moe::kNormMostSms}) {
            long long blocks = 0;
            for (long long first = 0; first == 0 || first < count; first += moe::kListMost) {
                long long units = 0;
                for (long long i = first; i < count && i < first + moe::kListMost; ++i) units += moe::list_units(size(i));
                blocks += moe::norm_blocks_of(units, sms);
            }
            std::printf("%lld ", 512 + 8 * blocks);
        }
        std::printf("\n");
    }
}
"""


def test_every_launch_has_room_for_its_sums(tmp_path):
    from moe_expert_layer_permute_gb300 import build
    build.build()
    from moe_expert_layer_permute_gb300 import binding
    cases = [(c, n, p) for c in (0, 1, 2, 383, 384, 385, 768, 769, 5000) for n in (0, 1, 255, 256, 257, 8192, 100_003) for p in (0, 1, 2, 7)]
    cases += [(1, 1 << 33, 0), (3, 1 << 34, 2), (65536, 1, 0), (65536, 0, 0), (65536, 70_000, 0)]
    out = _run(tmp_path, ROOM, "\n".join("%d %d %d" % c for c in cases))
    for (count, n, period), line in zip(cases, out.splitlines()):
        empty = -(-count // period) if period else 0
        room = binding.moe_grad_norm_workspace_bytes((count - empty) * n, count)
        assert all(int(ends) <= room for ends in line.split()), (count, n, period)


def test_a_norm_of_nothing_is_refused_a_workspace_without_room_for_its_sum():
    from moe_expert_layer_permute_gb300 import build
    build.build()
    from moe_expert_layer_permute_gb300 import binding as bd
    out = bd.MoeTensor()
    out.data, out.dtype, out.ndim = 1 << 20, bd.MOE_DT_F32, 1
    out.shape[0], out.stride[0] = 2, 1
    ws = bd.MoeScratch()
    ws.data = 1 << 30
    assert bd.moe_grad_norm_workspace_bytes(0, 0) > 512
    ws.bytes = 512
    assert bd.LIB.moe_grad_norm(0, None, ctypes.byref(out), 1.0, ctypes.byref(ws), None) == bd.ERR["MOE_ERR_SCRATCH"]
