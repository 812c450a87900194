"""GPU tests of the attention over the 8-bit cache with scores far from zero, of
either sign, and one token so far ahead that the result is its values: what is
rounded in scores of that size is the same in the product and in the sum, and the
result is as exact as with small ones.

The other tokens' weights are at most 2^-60, n of them change nothing that counts.
The weight itself is rounded to f16 at most (2^-11, and the same number is divided
by before rounding), its exponent's parts (scale, sum's logarithm, at most 2^8)
at 2^-24 each some 8 times, the result to its type.
"""
import math

import pytest

from tests.test_gpu_attn import ROUND, TORCH, ints, make_table, np64, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


def case(ent, dtype, d, page, n, ahead, size, vscale, zeros):
    """A cache whose scores are `size` times the key's first code: 127 for token
    `ahead`, 126 and less for the others.  `zeros`: pages of zero values."""
    pages = -(-n // page)
    c = ent.KVCache.empty(pages + 1, 1, d, page)
    t = make_table([n], page, pages + 1, 1)
    g = torch.Generator(device="cuda").manual_seed(n + d)
    c.k_codes.copy_(torch.randint(-127, 127, c.k_codes.shape, device="cuda", generator=g))
    c.v_codes.copy_(torch.randint(-127, 128, c.v_codes.shape, device="cuda", generator=g))
    c.k_scales.fill_(size)
    c.v_scales.copy_(vscale * (0.5 + torch.rand(c.v_scales.shape, device="cuda", generator=g)))
    for p in zeros:
        if p != ahead // page and p < pages:
            c.v_codes[int(t[0, p])] = 0
            c.v_scales[int(t[0, p])] = 0.0
    at = int(t[0, ahead // page])
    c.k_codes[at, 0, ahead % page, 0] = 127
    q = torch.zeros(1, 4, d, device="cuda", dtype=TORCH[dtype])
    q[:, :, 0] = 1.0
    want = np64(c.v_codes[at, 0, :, ahead % page]) * float(c.v_scales[at, 0])
    return q, c, t, want


@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 14, 2.0 ** 17.3, 2.0 ** 23.1, 2.0 ** 30, 2.0 ** 60], ids=lambda x: f"{math.log2(x):g}")
@pytest.mark.parametrize("n", [100, 1000, 5000])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_token_far_ahead(ent, dtype, n, size):
    say(f"cache attention: scores of 2^{math.log2(size):g} x code, {n} tokens, {dtype}")
    for d, page, sign, vscale in ((64, 16, 1, 0.02), (128, 64, 1, 0.3), (96, 32, -1, 0.004), (128, 128, -1, 0.02)):
        for ahead in (0, 63, n // 2, n - 1):
            for zeros in ((), range(0, 8), range(0, n, 2)):
                q, c, t, want = case(ent, dtype, d, page, n, ahead, size, vscale, zeros)
                if sign < 0:   # all scores negative: the least one is ahead
                    c.k_codes[..., 0].clamp_(min=2)
                    c.k_codes[int(t[0, ahead // page]), 0, ahead % page, 0] = 1
                    q.neg_()
                status = torch.zeros(1, dtype=torch.int32, device="cuda")
                got = np64(ent.attn_cache(q, c, torch.from_numpy(t).cuda(), ints([n]), status, scale=1.0))
                assert not status.any()
                bound = abs(want) * (ROUND[dtype] + 2 * 2.0 ** -11 + 16 * 2.0 ** -24 * 256) + n * 2.0 ** -39 * 127 * 1.5 * vscale + 2.0 ** -25
                err = abs(got[0] - want)
                assert (err <= bound).all(), (d, page, sign, ahead, zeros, float((err / bound).max()))
