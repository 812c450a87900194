"""GPU test of the rotary positions' angles where they are many turns: any 32-bit
position, frequencies above one radian a position.

Where the sine is small, float16 results show the angle's error: a result x = sin is
rounded by 2^-11 |x| or, below f16's normal numbers, 2^-25.  The operator states cosine
and sine to 2^-22 + 2^-52 of the angle; of the latter no more is taken here than what the
64-bit product of a frequency and 1 / (2 pi) is off by, since whole turns come out of a
fused product.  The inputs are (1, 0) and the products with them exact.
"""
from fractions import Fraction

import numpy as np
import pytest

from tests.test_gpu_attn import np64, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117068, 10 ** 99)


def sines(positions, freq):
    """sin(position * freq) from whole numbers, in units of 2^-100."""
    turn, step = (2 * PI * 2 ** 100).__floor__(), Fraction(freq) * 2 ** 100
    rests = [(int(p) * step).__floor__() % turn for p in positions]
    return np.sin([(r - turn if 2 * r > turn else r) / 2.0 ** 100 for r in rests])


@pytest.mark.parametrize("base", [0, 1 << 20, (1 << 31) - (1 << 20) - 1, -(1 << 31)])
def test_angles_of_many_turns(ent, base):
    say(f"rope: angles of many turns, positions from {base}")
    freqs = [0.1, 0.7364, 1.0, 1.9, 3.3, 7.77, 100.3, 12345.6]
    at = np.arange(base, base + (1 << 20), dtype=np.int64)
    f = torch.tensor(freqs, dtype=torch.float32, device="cuda")
    rot = ent.Rotary(f)
    worst = 0.0
    for j, freq in enumerate(freqs):
        # positions where the angle is near a whole number of half turns, by a 64-bit guess
        f64 = np.float64(np.float32(freq))
        x = at * f64 / np.pi
        off = float(abs(Fraction(float(f64 * np.float64(1 / (2 * np.pi)))) * 2 * PI / Fraction(float(f64)) - 1))
        assert off <= 2.0 ** -52
        near = np.argsort(np.abs(x - np.rint(x)), kind="stable")[: 2000]
        want = sines(at[near], float(f64))
        assert np.abs(want).max() < 2.0 ** -6      # (the guess is off by up to 2^-8 at angles of 2^44)
        q = torch.zeros(len(near), 1, 64, dtype=torch.float32, device="cuda")
        q[:, 0, j] = 1.0
        pos = torch.from_numpy(at[near].astype(np.int32)).cuda()
        got = np64(ent.rope(rot, q, None, pos, dtype=torch.float16)[0])[:, 0, len(freqs) + j]
        e = 2.0 ** -22 + off * np.abs(at[near] * f64)
        bound = e + 2.0 ** -11 * (np.abs(want) + e) + 2.0 ** -25      # (what is rounded is the sine with its error)
        worst = max(worst, float((np.abs(got - want) / bound).max()))
    assert worst <= 1.0, worst
