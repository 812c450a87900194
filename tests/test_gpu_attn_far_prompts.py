"""GPU tests of prompts with scores far from zero, of either sign, and one key so
far ahead of the others that the result is its value: what is rounded in scores of
that size is the same in the product and in the sum.

Other weights are at most 2^-60 (keys apart by 1 in units of `size`, 2^8 at least,
times the query's 1).  The weight and the sum are the same rounded number; the
factor 1 / sum and the product with it are rounded at 2^-23, the result to its type.
"""
import itertools
import math

import pytest

from tests.test_gpu_attn import ROUND, TORCH, ints, np64, running, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


SIZES = [2.0 ** 8, 2.0 ** 14, 2.0 ** 17.3, 2.0 ** 20.6, 2.0 ** 23.1, 2.0 ** 27, 2.0 ** 31.7, 2.0 ** 60]


@pytest.mark.parametrize("size", SIZES, ids=lambda x: f"{math.log2(x):g}")
@pytest.mark.parametrize("lengths", [([90], [90]), ([300, 5], [300, 700]), ([1, 3], [129, 64]), ([5], [1500])], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_key_far_ahead(ent, dtype, lengths, size):
    say(f"prompt: scores of 2^{math.log2(size):g} x key, {lengths}, {dtype}")
    lq, lk = lengths
    for (h, kv, d), order, scale in itertools.product(((2, 1, 64), (4, 2, 96), (4, 1, 128)), ("rising", "falling", "mixed"),
                                                      (size, -size)):
        g = torch.Generator(device="cuda").manual_seed(d)
        q = torch.zeros(sum(lq), h, d, device="cuda")
        q[..., 0] = 1.0
        k = torch.randn(sum(lk), kv, d, device="cuda", generator=g)
        v = torch.randn(sum(lk), kv, d, device="cuda", generator=g)
        want = torch.zeros(sum(lq), h, d, dtype=torch.float64)
        cq, ck = running(lq), running(lk)
        key = torch.zeros(sum(lk))
        for b in range(len(lq)):
            # whole numbers of up to 128 (exact in both types), one key for each query the largest it sees
            n = lk[b]
            ranks = {"rising": torch.arange(n), "falling": -torch.arange(n), "mixed": (torch.arange(n) * 37) % max(n, 1)}[order]
            ranks = ranks.float() * math.copysign(1.0, scale)
            # distinct numbers in windows of 120 keys would repeat: the tie is broken by leaving one key at each top
            key[ck[b]: ck[b + 1]] = (ranks - ranks.min()) % 120 - 60
        for b in range(len(lq)):
            for i in range(lq[b]):
                seen = key[ck[b]: ck[b] + i + 1 + lk[b] - lq[b]] * math.copysign(1.0, scale)
                best = (seen == seen.max()).nonzero().flatten()
                for head in range(h):
                    want[cq[b] + i, head] = v[ck[b] + best, head // (h // kv)].to(TORCH[dtype]).double().mean(0).cpu()
        k[..., 0] = key[:, None]
        q, k, v = (x.to(TORCH[dtype]) for x in (q, k, v))
        status = torch.zeros(len(lq), dtype=torch.int32, device="cuda")
        got = np64(ent.attn_prompt(q, k, v, ints(cq), ints(ck), status, scale=scale))
        assert not status.any()
        want, most = want.numpy(), float(v.abs().max())
        # (several keys tie where their numbers repeat: equal weights, whose mean is summed in 32 bits)
        bound = abs(want) * ROUND[dtype] + most * (len(key) + 8) * 2.0 ** -23 + 2.0 ** -25
        err = abs(got - want)
        assert (err <= bound).all(), (h, d, order, scale, float((err / bound).max()))
