"""moe_linear's out may be its residual where their types are equal; any other overlap of the two is refused on
the host."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from bit_moe_expert_top_amd import _lib

    return _lib.lib


P = 1 << 20  # an aligned address that is never dereferenced
F32, BF16 = 1, 2


def linear(lib, r, rd, out, od, T=4, N=64, act=0):
    return lib.moe_linear(P // 2, None, P // 4, None, BF16, T, N, 64, None, act, r, rd, out, od, None)


@pytest.mark.parametrize("r,rd,out,od", [
    (P, F32, P, BF16), (P, BF16, P, F32),                 # one address, two types
    (P, F32, P + 16, F32), (P + 16, F32, P, F32),         # part of each other
    (P, BF16, P + 4 * 64 * 2 - 2, BF16),                  # the residual's last value
    (P + 4 * 64 * 4 - 2, BF16, P, F32),                   # out's last value
])
def test_out_over_residual(lib, r, rd, out, od):
    assert linear(lib, r, rd, out, od) == -1


def test_gated_columns_count(lib):
    """With SwiGLU the rows are N / 2 values long."""
    assert linear(lib, P, F32, P + 4 * 32 * 4 - 4, F32, act=4) == -1
