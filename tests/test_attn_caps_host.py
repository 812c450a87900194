"""``set_max_workgroups`` sets the two caps of the library, and what it returns
sets both back, whatever they were (no GPU needed)."""
import pytest

import entropy_coded_weight_canonical_amd as ent


@pytest.fixture()
def lib():
    lib = ent.load()
    yield lib
    lib.entro_set_max_workgroups(0)
    lib.entro_attn_set_max_workgroups(0)


def caps(lib):
    """Both caps, read by setting them again."""
    out = []
    for fn in (lib.entro_set_max_workgroups, lib.entro_attn_set_max_workgroups):
        now = fn(0)
        fn(now)
        out.append(now)
    return tuple(out)


@pytest.mark.parametrize("before", [(0, 0), (7, 7), (7, 0), (0, 9), (7, 9)])
def test_both_caps_are_set_and_set_back(lib, before):
    lib.entro_set_max_workgroups(before[0])
    lib.entro_attn_set_max_workgroups(before[1])
    old = ent.set_max_workgroups(5)
    assert old == before[0]
    assert caps(lib) == (5, 5)
    inner = ent.set_max_workgroups(3)
    assert inner == 5 and caps(lib) == (3, 3)
    ent.set_max_workgroups(inner)
    assert caps(lib) == (5, 5)
    ent.set_max_workgroups(old)
    assert caps(lib) == before
