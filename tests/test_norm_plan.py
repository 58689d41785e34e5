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


LAUNCHES = r"""
#include <cassert>
#include <vector>
#include "norm_plan.h"
int main() {
    using namespace moe;
    for (long long count : {0ll, 1ll, 384ll, 385ll, 2000ll}) {
        const int all = (int)std::max(1ll, (count + kListMost - 1) / kListMost);
        for (int fails = 0; fails <= all; ++fails) {        // the launch that fails (the last of them: none)
            uint64_t state = kWorkspaceZero;
            std::vector<long long> at;
            const int e = norm_launches(count, &state, [&](int64_t first) {
                assert(state == kWorkspaceData);            // nothing else takes it meanwhile
                at.push_back(first);
                return (int)at.size() - 1 == fails ? 7 : 0;
            });
            for (int i = 0; i < (int)at.size(); ++i) assert(at[i] == (long long)i * kListMost);
            assert((int)at.size() == (fails < all ? fails + 1 : all));
            assert(e == (fails < all ? 7 : 0) && state == (fails < all ? kWorkspaceData : kWorkspaceSums));
        }
    }
}
"""


def test_a_norm_that_failed_between_its_launches_leaves_a_workspace_that_is_refused(tmp_path):
    _run(tmp_path, LAUNCHES)
    with open(os.path.join(CSRC, "moe_api.cu")) as f:
        body = f.read().split("int moe_grad_norm(")[1].split("\n}\n")[0]
    assert "norm_launches(count, &workspace->state[0]" in body and body.count("workspace->state[0]") == 2   # by this alone
