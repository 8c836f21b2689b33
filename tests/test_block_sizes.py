"""Sizes that the C ABI's 32-bit integers do not hold are refused by the binding, before anything is
allocated or enqueued (tensors on the meta device have sizes and no memory)."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from bit_moe_expert_top_amd import _lib

    return _lib


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("T", [1 << 31, 1 << 32, (1 << 32) + 5])
def test_rows_past_32_bits(L, T):
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_add_rmsnorm(meta(T, 8), meta(8), 1e-6)
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_linear(meta(T, 8), meta(16, 8))
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_linear(meta(4, 8), meta(T, 8))
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_route_scored(meta(T, 16, dtype=torch.float32), 2)


def test_columns_past_32_bits(L):
    n = (1 << 32) + 64
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_add_rmsnorm(meta(1, n), meta(n), 1e-6)
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_linear(meta(1, n), meta(1, n))
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_route_scored(meta(1, n, dtype=torch.float32), 2)


@pytest.mark.parametrize("bad", [dict(k=(1 << 32) + 2), dict(n_group=(1 << 32) + 4), dict(topk_group=(1 << 32) + 1),
                                 dict(group_top=(1 << 32) + 1), dict(k=-(1 << 32) + 2), dict(n_group=4 - (1 << 32))])
def test_routing_arguments_past_32_bits(L, bad):
    """Their low 32 bits alone would be a call that is allowed."""
    args = dict(k=2, n_group=4, topk_group=1, group_top=1)
    args.update(bad)
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_route_scored(meta(3, 16, dtype=torch.float32), topk_ids=meta(3, 2, dtype=torch.int32),
                           topk_w=meta(3, 2, dtype=torch.float32), **args)
