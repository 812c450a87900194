"""A ``KVCache`` describes the tensors that it was made of (no GPU needed): they
can be looked at and not replaced, or calls would go on with the old ones'
memory after it is freed."""
import pytest

torch = pytest.importorskip("torch")

import entropy_coded_weight_canonical_amd as ent  # noqa: E402
from tests.test_attn_devices_host import cache_tensors  # noqa: E402

NAMES = ["k_codes", "v_codes", "k_scales", "v_scales"]


def test_holds_its_tensors():
    t = cache_tensors()
    c = ent.KVCache(*t)
    for name, x, y in zip(NAMES, t, c.tensors):
        assert getattr(c, name) is x and y is x


@pytest.mark.parametrize("name", NAMES + ["desc"])
def test_cannot_be_replaced(name):
    c = ent.KVCache(*cache_tensors())
    was = getattr(c, name)
    other = c.desc + bytes(1) if name == "desc" else cache_tensors()[NAMES.index(name)]
    with pytest.raises(AttributeError):
        setattr(c, name, other)
    with pytest.raises(AttributeError):
        delattr(c, name)
    assert getattr(c, name) is was
    setattr(c, name, was)   # what an operation in place does


def test_same_tensors_as_given_in_order():
    a, b = cache_tensors(), cache_tensors()
    with pytest.raises(AttributeError):
        ent.KVCache(*a).k_codes = b[0]
    assert ent.KVCache(*b).tensors[0] is b[0]
