"""The attention calls have no backward pass: where a gradient would be recorded,
they refuse (no GPU needed) and do not return a result without one."""
import pytest

torch = pytest.importorskip("torch")

import entropy_coded_weight_canonical_amd as ent  # noqa: E402
from tests.test_attn_devices_host import Cache, calls, on  # noqa: E402

FLOATS = [(call, what) for call, (_, x) in calls().items() for what, t in x.items()
          if isinstance(t, torch.Tensor) and t.is_floating_point()]


def case(call, what):
    fn, x = calls()[call]
    x = {k: Cache(0) if k == "cache" else v for k, v in x.items()}
    x[what].requires_grad_()
    return fn, x


@pytest.mark.parametrize("call,what", FLOATS, ids=lambda x: x)
def test_gradient_asked_for(call, what):
    fn, x = case(call, what)
    with pytest.raises(ValueError, match="backward"):
        fn(x)


@pytest.mark.parametrize("call,what", FLOATS, ids=lambda x: x)
def test_no_gradient_recorded(call, what):
    """Under no_grad the call goes on (here: to its next refusal)."""
    fn, x = case(call, what)
    ints = "lens" if call == "cache" else "status"
    x[ints] = on(1, 1, dtype=torch.int32)
    with torch.no_grad(), pytest.raises(ValueError, match="device"):
        fn(x)


def test_scales_of_a_cache():
    codes = on(0, 4, 2, 16, 64, dtype=torch.int8), on(0, 4, 2, 64, 16, dtype=torch.int8)
    scales = [on(0, 4, 2, dtype=torch.float32) for _ in range(2)]
    scales[1].requires_grad_()
    with pytest.raises(ValueError, match="backward"):
        ent.KVCache(*codes, *scales)
