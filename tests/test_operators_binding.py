"""What the binding of the balance loss and the orthogonalisation does with arguments of wrong kinds (no GPU)."""
import numpy as np
import pytest
import torch

from test_abi_host import bd  # noqa: F401  (the library fixture)
from test_operators_host import _Holder


@pytest.mark.parametrize("kw", [{"steps": 4000, "coeffs": (1.0, 1.0, 1.0), "eps": "x"}, {"steps": 17.5, "coeffs": [(1, 1, 1)] * 400},
                                {"steps": 2 ** 70, "coeffs": [(1, 1, 1)] * 400}, {"steps": 5, "coeffs": [("x", 1, 1)] * 5},
                                {"steps": 16, "coeffs": [(1, 1, 1)] * 16, "eps": None}])
def test_coefficients_beside_arguments_of_other_kinds(bd, kw):  # noqa: F811
    """More coefficients than any call takes, and steps or eps that are no numbers: an exception, nothing else."""
    G = torch.zeros(1, 4, 4)
    with pytest.raises((TypeError, OverflowError)):
        bd.moe_orthogonalise(G, G, _Holder(bd), stream=0, **kw)


@pytest.mark.parametrize("steps,code", [(-2 ** 32 + 5, "SHAPE"), (-2 ** 62, "SHAPE"), (0, "SHAPE"), (2 ** 32 + 5, "UNSUPPORTED")])
def test_step_counts_beyond_32_bits(bd, steps, code):  # noqa: F811
    """Refused as what they are, and not taken modulo 2^32."""
    G, O = torch.zeros(1, 4, 4), torch.zeros(1, 4, 4, dtype=torch.bfloat16)
    with pytest.raises(bd.MoeError, match=code):
        bd.moe_orthogonalise(G, O, _Holder(bd), stream=0, steps=steps)


@pytest.mark.parametrize("coeffs", [torch.tensor([3.0, -4.0, 2.0]), torch.tensor([[3.0, -4.0, 2.0]] * 5), [torch.tensor([3.0, -4.0, 2.0])] * 5,
                                    np.array([3.0, -4.0, 2.0]), np.array([[3.0, -4.0, 2.0]] * 5), ((3, -4, 2),) * 5, [3.0, -4.0, 2.0], [torch.tensor(3.0), torch.tensor(-4.0), torch.tensor(2.0)]])
def test_coefficients_in_arrays(bd, coeffs):  # noqa: F811
    """Tensors and arrays of one triple or of one for each step pass as far as the tensors' own check."""
    G, O = torch.zeros(1, 4, 4), torch.zeros(1, 4, 4, dtype=torch.bfloat16)
    with pytest.raises(bd.MoeError, match="NULL"):
        bd.moe_orthogonalise(G, O, _Holder(bd), stream=0, steps=5, coeffs=coeffs)


@pytest.mark.parametrize("coeffs", [(), [], torch.zeros(0), torch.zeros(5, 2), [(1, 1), (1, 1, 1, 1)] + [(1, 1, 1)] * 3, torch.zeros(4, 3)])
def test_coefficients_that_are_no_triples(bd, coeffs):  # noqa: F811
    G, O = torch.zeros(1, 4, 4), torch.zeros(1, 4, 4, dtype=torch.bfloat16)
    with pytest.raises(bd.MoeError, match="SHAPE"):
        bd.moe_orthogonalise(G, O, _Holder(bd), stream=0, steps=5, coeffs=coeffs)
