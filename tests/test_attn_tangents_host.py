"""The attention calls have no derivative in forward mode either: operands that carry a
tangent are refused (no GPU needed) and not taken without it."""
import pytest

torch = pytest.importorskip("torch")

import torch.autograd.forward_ad as fw  # noqa: E402

import entropy_coded_weight_canonical_amd as ent  # noqa: E402
from tests import test_attn_chunk_host as more  # noqa: E402
from tests.test_attn_devices_host import Cache, calls  # noqa: E402


class Dual(torch.Tensor):
    """Stands in for a tensor on a GPU: nothing but its tangent's making touches it."""

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        if func is torch.ops.aten.alias.default:
            return like(args[0])
        if func in (torch.ops.aten.is_same_size.default, torch.ops.aten._has_same_storage_numel.default):
            return True
        raise AssertionError(f"{func} of a tensor that is to be refused")


def like(x):
    return torch.Tensor._make_wrapper_subclass(Dual, x.shape, dtype=x.dtype, device=x.device)


def everything():
    out = {call: (fn, {k: Cache(0) if k == "cache" else v for k, v in x.items()}) for call, (fn, x) in calls().items()}
    out.update({"new " + call: fx for call, fx in more.placed()[4].items()})
    return out


FLOATS = [(call, what) for call, (_, x) in everything().items() for what, t in x.items()
          if isinstance(t, torch.Tensor) and t.is_floating_point()]


@pytest.mark.parametrize("call,what", FLOATS, ids=lambda x: x)
def test_operand_with_a_tangent(call, what):
    fn, x = everything()[call]
    with fw.dual_level():
        x[what] = fw.make_dual(like(x[what]), like(x[what]))
        with pytest.raises(ValueError, match="tangent"):
            fn(x)
        # with no_grad too, which does not end forward mode
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
            fn(x)


def test_plan_with_a_tangent():
    x = torch.Tensor._make_wrapper_subclass(Dual, (32,), dtype=torch.float32, device=torch.device("cuda", 0))
    with fw.dual_level(), pytest.raises(ValueError, match="tangent|freqs"):
        ent.Rotary(fw.make_dual(x, like(x)))
