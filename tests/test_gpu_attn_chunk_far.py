"""GPU tests of the attention of chunks where a sequence's tiles of 64 tokens differ
much from one another: scores far from zero behind near ones, in each of its kernels
(few rows with the wavefronts side by side or in turns, blocks of 128 and of 256 rows).

Keys have one value that is not zero, and so have queries, by powers of two: scores
are exact and equal within a tile.  The bound of an output is that of
test_gpu_attn_chunk.py without what grows with the scores: the result's rounding, the
weights' to f16 (2^-12 of A, the weighted mean of |v|), the logarithms' of the values'
scales and the exponentials', above and below, and the sums' in 32 bits.
"""
import math

import numpy as np
import pytest

from oracle import attention as oa
from tests.test_gpu_attn import ints, np64, running, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TILE = 64

# (new tokens, query heads, key/value heads) and the tiles that one workgroup takes in
# one piece: the work of all blocks is below two shares, or there is one share only
KERNELS = {
    "few": ((20, 2, 1), 4),        # 40 rows: each of four wavefronts has 16 of them and every tile
    "turns": ((4, 512, 512), 12),  # 4 rows: the wavefronts have every fourth tile
    "four": ((30, 2, 1), 4),       # 60 rows, blocks of 128
    "eight": ((80, 2, 1), 4),      # 160 rows, blocks of 256
}


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


def attend(ent, dtype, d, kernel, key_codes, v_scales, scale, codes=None, less=0):
    """One sequence whose tile i has keys of key_codes[i] and values' scale
    v_scales[i], one tile a page, less the last `less` tokens, against the oracle."""
    (new, h, kv), _ = KERNELS[kernel]
    tiles = len(key_codes)
    n = tiles * TILE - less
    g = torch.Generator(device="cuda").manual_seed(tiles)
    c = ent.KVCache.empty(tiles + 1, kv, d, TILE)
    v = torch.randint(-127, 128, c.v_codes.shape, device="cuda", generator=g) if codes is None else torch.full(c.v_codes.shape, codes)
    c.v_codes.copy_(v)
    c.k_scales.fill_(1.0)
    t = torch.randperm(tiles + 1, device="cuda", generator=g)[:tiles].to(torch.int32)
    for i in range(tiles):
        c.k_codes[t[i], :, :, 0] = key_codes[i]
        c.v_scales[t[i]] = v_scales[i]
    q = torch.zeros(new, h, d, dtype=TORCH[dtype], device="cuda")
    q[:, :, 0] = 4.0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ent.attn_chunk(q, c, t[None].contiguous(), ints([n]), ints(running([new])), status, scale=scale)
    assert not status.any()
    again = ent.attn_chunk(q, c, t[None].contiguous(), ints([n]), ints(running([new])), status, scale=scale)
    assert torch.equal(got, again) or torch.isnan(got).any()
    heads = [0, 1] if kv == 1 else [0, 100, kv - 1]
    got = np64(got)[:, heads]
    pages = t.long()
    at = [x // (h // kv) for x in heads]
    k, v = (np64(y).reshape(n + less, len(heads), d)[:n] for y in (
        (c.k_codes[pages].float() * c.k_scales[pages][..., None, None])[:, at].transpose(1, 2),
        (c.v_codes[pages].double() * c.v_scales[pages].double()[..., None, None])[:, at].permute(0, 3, 1, 2)))
    want, mean, _ = oa.chunk(np64(q)[:, heads], [k], [v], [n], [0, new], scale)
    log = max((abs(math.log2(x)) for x in v_scales if x), default=0.0)
    e = 8 * (log + 64) * 2.0 ** -24 + 2.0 ** -20
    b = ROUND[dtype] * np.abs(want) + (2.0 ** -12 + 2 * e + (n / 16 + 4) * 2.0 ** -22) * mean * 1.01
    b += 2.0 ** -25 if dtype == "f16" else 2.0 ** -130
    assert np.isfinite(got).all(), "outputs that are no numbers"
    assert (np.abs(got - want) <= b).all(), float((np.abs(got - want) / b).max())
    return got


def spread(kernel, *parts):
    """A value for each tile of the kernel's piece: equal runs of the given ones."""
    tiles = KERNELS[kernel][1]
    return [parts[i * len(parts) // tiles] for i in range(tiles)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("power", [10, 13, 17, 24, 28, 30])
@pytest.mark.parametrize("kernel", KERNELS)
def test_far_scores_behind_near_ones(ent, kernel, power, dtype):
    """Near scores, then equal far ones, of either sign, in several tiles; and tiles that
    lie far behind or ahead of one another."""
    say(f"chunk: far scores behind near ones, {kernel} {power} {dtype}")
    scale = 2.0 ** (power - 8)          # the score of a key of 64: 2^power
    for d in (64, 128):
        for sign in (1, -1):
            attend(ent, dtype, d, kernel, spread(kernel, 0, 64 * sign, 64 * sign, 64 * sign), spread(kernel, 2.0 ** -7), scale, less=5)
    attend(ent, dtype, 64, kernel, spread(kernel, 0, 64, 64, 32), spread(kernel, 2.0 ** -7), scale)
    attend(ent, dtype, 64, kernel, spread(kernel, 0, 32, 64, 64), spread(kernel, 2.0 ** -7), scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("power", [17, 24, 28, 30])
@pytest.mark.parametrize("kernel", KERNELS)
def test_far_scores_of_small_values(ent, kernel, power, dtype):
    """All scores far and equal; the values' scales so small that the outputs' unit has
    moved to them."""
    say(f"chunk: far scores of small values, {kernel} {power} {dtype}")
    for log in (-13, -20):
        attend(ent, dtype, 96, kernel, spread(kernel, 64), spread(kernel, 2.0 ** log), 2.0 ** (power - 8), less=3)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("power", [10, 13, 14, 17, 24, 28])
@pytest.mark.parametrize("kernel", KERNELS)
def test_far_scores_of_several_scales(ent, kernel, power, dtype):
    """Equal scores, and values' scales for which the outputs' unit moves."""
    say(f"chunk: far scores of several scales, {kernel} {power} {dtype}")
    for logs in ((-7, -4, -7, -4), (-4, -8, -12, -8), (-1, -4, -7, -1)):
        attend(ent, dtype, 64, kernel, spread(kernel, 65), spread(kernel, *(2.0 ** x for x in logs)), 2.0 ** (power - 8))
