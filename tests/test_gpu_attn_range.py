"""GPU tests of prompts whose bf16 values lie near the ends of the type's range:
sums of weighted values stay finite wherever the result is, for equal weights
(whose sum is largest) and for scores that rise from key to key (so that the
running maximum is behind).  Bounds are those of test_gpu_attn.py."""
import numpy as np
import pytest

from tests.test_gpu_attn import run_prompt, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


LENGTHS = [([1], [1]), ([90, 5], [90, 300]), ([300], [300]), ([5], [1500])]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("heads", [(2, 1, 64), (4, 2, 96), (4, 1, 128)])
@pytest.mark.parametrize("scores", ["equal", "rising", "random"])
def test_largest_values(ent, scores, heads, lengths):
    say(f"prompt: values near the largest, {scores} scores, {heads} {lengths}")

    def edit(q, k, v):
        if scores == "equal":
            q.zero_()
            v.fill_(2.0 ** 127)
            v[..., ::2] = -(2.0 ** 127)
        else:
            v.clamp_(-3.9, 3.9).mul_(2.0 ** 125)
        if scores == "rising":   # by 7 powers of two over the keys
            q.zero_()
            q[..., 0] = 1.0
            k[..., 0] = torch.linspace(0.0, 4.85, k.shape[0], device="cuda")[:, None]

    got = run_prompt(ent, heads, "bf16", *lengths, edit=edit, scale=1.0 if scores == "rising" else None)
    if scores == "equal":
        assert (np.abs(got) >= 2.0 ** 126.9).all()


@pytest.mark.parametrize("power", [-60, -95])
@pytest.mark.parametrize("heads", [(2, 1, 64), (4, 1, 128)])
def test_small_values(ent, heads, power):
    say(f"prompt: values of 2^{power}, {heads}")
    run_prompt(ent, heads, "bf16", [300, 5], [300, 90], edit=lambda q, k, v: v.mul_(2.0 ** power))
    run_prompt(ent, heads, "bf16", [5], [1500], edit=lambda q, k, v: v.mul_(2.0 ** power))
