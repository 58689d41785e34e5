"""What a launch sets once for each GPU (csrc/per_device.h), on the host: each device has its own, an error is not kept."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_expert_layer_permute_gb300", "csrc")

PROGRAM = r"""
#include <cassert>
#include "per_device.h"
enum Error { kOk = 0, kBad = 7 };
int main() {
    static moe::PerDevice<int> held;
    int made = 0, v = -1;
    bool fail = true;
    auto ask = [&](int device) {
        return held.get(device, &v, [&](int* out) {
            ++made;
            if (fail) return kBad;
            *out = 100 + device;
            return kOk;
        });
    };
    assert(ask(0) == kBad && made == 1);
    fail = false;
    assert(ask(0) == kOk && v == 100 && made == 2);   // tried again
    assert(ask(1) == kOk && v == 101 && made == 3);   // another device's own
    assert(ask(0) == kOk && v == 100 && made == 3);   // held
    assert(ask(1) == kOk && v == 101 && made == 3);
    assert(ask(64) == kOk && v == 164 && made == 4);  // beyond the table: made each time
    assert(ask(64) == kOk && made == 5);
}
"""


def test_each_device_has_its_own_and_errors_are_not_kept(tmp_path):
    (tmp_path / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "p.cpp"), "-o", str(tmp_path / "p")], check=True)
    subprocess.run([str(tmp_path / "p")], check=True)


def test_the_orthogonalisation_keeps_nothing_for_the_process(tmp_path):
    """Its launches hold what they set in such tables alone."""
    with open(os.path.join(CSRC, "orthogonal.cu")) as f:
        source = f.read()
    assert "call_once" not in source and source.count("static PerDevice<") == 2
