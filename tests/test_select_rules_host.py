"""Rules of the routing by scores that the binding refuses (no GPU)."""
import pytest

from test_abi_host import bd  # noqa: F401  (bd: the library fixture)


@pytest.mark.parametrize("name", ["groups", "topk_groups", "group_rank"])
@pytest.mark.parametrize("value", [2 ** 32 + 1, 2 ** 31, -2 ** 32 + 1, 2 ** 80])
def test_numbers_that_a_field_cannot_hold(bd, name, value):  # noqa: F811
    """Taken modulo 2^32 they would be other, allowed ones."""
    with pytest.raises(bd.MoeError, match="UNSUPPORTED"):
        bd.RouterRule(**{name: value})


@pytest.mark.parametrize("kw", [{"groups": "4"}, {"topk_groups": 1.5}, {"group_rank": None}, {"scale": "x"}])
def test_other_kinds_of_numbers(bd, kw):  # noqa: F811
    with pytest.raises(TypeError):
        bd.RouterRule(**kw)
