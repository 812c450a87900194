"""``kv_load`` with outputs given and a type named (no GPU needed): the two agree,
or the call is refused."""
import pytest

torch = pytest.importorskip("torch")

import entropy_coded_weight_canonical_amd as ent  # noqa: E402
from tests.test_attn_devices_host import Cache, ints, on  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16


def load(dtype, k, v, status_gpu=0):
    return ent.kv_load(Cache(0), ints(0, 1, 4), ints(0, 1), ints(0, 2), 5, ints(status_gpu, 1), dtype=dtype,
                       out=(on(0, 5, 2, 64, dtype=k), on(0, 5, 2, 64, dtype=v)))


@pytest.mark.parametrize("dtype,k,v", [(F16, BF16, BF16), (BF16, F16, F16), (F16, F16, BF16), (F16, BF16, F16)], ids=str)
def test_another_type_than_the_outputs(dtype, k, v):
    with pytest.raises(ValueError, match="type"):
        load(dtype, k, v)


@pytest.mark.parametrize("dtype,k", [(F16, F16), (BF16, BF16), (None, F16), (None, BF16)], ids=str)
def test_the_outputs_own_type(dtype, k):
    """goes on (here: to the next refusal)."""
    with pytest.raises(ValueError, match="device"):
        load(dtype, k, k, status_gpu=1)
