"""Which seed a step of 8-bit states gets (no GPU): without one, another for each step."""
import torch

from test_abi_host import bd  # noqa: F401  (bd: the library fixture)


def test_a_step_without_a_seed_has_its_own(bd, monkeypatch):  # noqa: F811
    seen = []

    class Marshal:
        make_list = staticmethod(lambda tensors: None)

        @staticmethod
        def adamw_step(*args):
            seen.append((args[12], args[13]))                    # the step's number (0: on the device), the seed
            return 0

    monkeypatch.setattr(bd, "_MARSHAL", Marshal)
    monkeypatch.setattr(bd, "_marshal", lambda: Marshal)
    on_device = torch.tensor([3], dtype=torch.int32)
    for step in (1, 2, 3, on_device):
        bd.moe_adamw_step([], [], [], [], step, stream=0)
    assert seen == [(1, 1), (2, 2), (3, 3), (0, 0)]              # (the library adds a step on the device)
    seen.clear()
    for seed in (0, 7):
        bd.moe_adamw_step([], [], [], [], 2, seed=seed, stream=0)
        bd.moe_adamw_step([], [], [], [], on_device, seed=seed, stream=0)
    assert seen == [(2, 0), (0, 0), (2, 7), (0, 7)]
