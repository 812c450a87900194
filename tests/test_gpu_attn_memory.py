"""A call whose results do not fit the GPU raises what torch raises, and the next
call works."""
import pytest

from tests.test_gpu_attn import filled_cache, ints, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_results_that_do_not_fit():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as ent

    say("load: results of 2^31 - 1 rows are refused memory")
    c = filled_cache(ent, 8, 128, 64, 2, 0)
    table, one, status = ints([[0, 1]]), ints([0]), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        ent.kv_load(c, table, one, ints([0, 100]), 2 ** 31 - 1, status)
    k, v = ent.kv_load(c, table, one, ints([0, 100]), 100, status)
    torch.cuda.synchronize()
    assert not status.any() and k.any() and v.any()
