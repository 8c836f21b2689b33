"""moe_route_scored refuses arrays that are not aligned to their elements."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from bit_moe_expert_top_amd import _lib

    return _lib.lib


P = 1 << 20  # an aligned address that is never dereferenced


@pytest.mark.parametrize("bad", [dict(lg=P + 2), dict(bias=P + 1), dict(ids=P + 2), dict(w=P + 3)])
def test_route_alignment(lib, bad):
    a = dict(lg=P, bias=P, ids=P, w=P)
    a.update(bad)
    assert lib.moe_route_scored(a["lg"], a["bias"], 4, 32, 4, 1, 1, 1, 1, 0, 1.0, a["ids"], a["w"], None) == -1
