"""GPU tests of the attention of chunks where the values' scales move by up to 2^59
from one tile of 64 tokens to the next, each tile's being equal, so that the outputs'
unit would follow them step by step; bounds as in test_gpu_attn_chunk_far.py."""
import random

import pytest

from tests.test_gpu_attn import ints, say
from tests.test_gpu_attn_chunk_far import KERNELS, attend

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


STEPS = {
    "falling": ("bf16", [20, -38, -96]),
    "falling far": ("bf16", [85, 30, -28, -86]),
    "rising": ("bf16", [-90, -31, 28, 87]),
    "rising and falling": ("bf16", [-60, -1, 57, 0, -58, -99]),
    "falling and rising": ("bf16", [40, -18, -76, -30, 25, 40]),
    "there and back": ("bf16", [0, 59, 0, -59, 0]),
    "falling, 16 bits": ("f16", [8, 8, 8, 8, 8, -51, -99]),
    "back again, 16 bits": ("f16", [3, -50, -98, -40, 3]),
}


@pytest.mark.parametrize("name", STEPS)
@pytest.mark.parametrize("kernel", KERNELS)
def test_scales_step_by_step(ent, kernel, name):
    """Equal scores, so that what the largest scales give is the result."""
    dtype, logs = STEPS[name]
    say(f"chunk: scales step by step, {kernel} {name}")
    wide = 4 if kernel == "turns" else 1       # (a wavefront has every fourth tile)
    scales = [2.0 ** x for x in logs for _ in range(wide)]
    for codes in (127, None):
        attend(ent, dtype, 64, kernel, [0] * len(scales), scales, 1.0, codes=codes, less=9)
    attend(ent, dtype, 128, kernel, [0] * len(scales), scales, 1.0, codes=-127)


@pytest.mark.parametrize("kernel", KERNELS)
def test_small_values_of_high_scores(ent, kernel):
    """A first tile of small values whose scores are so far ahead that the others' weights
    are 0: those tiles' scales, however large, change nothing."""
    say(f"chunk: small values of high scores, {kernel}")
    wide = 4 if kernel == "turns" else 1
    for logs in ([-90, -31, 28, 87], [-60, -1, 58, 0], [-20, 39, 98, 39, -20]):
        scales = [2.0 ** x for x in logs for _ in range(wide)]
        attend(ent, "bf16", 64, kernel, [64] * wide + [0] * (len(scales) - wide), scales, 16.0, codes=127)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("behind,log", [(14, 18), (21, 40), (28, 45), (35, 59)])
def test_large_values_of_low_scores(ent, kernel, behind, log):
    """Values so large that they are the result although their weights are some 2^-20 to
    2^-50 of the first tile's: those keep their bits."""
    say(f"chunk: large values of low scores, {kernel} {behind} {log}")
    wide = 4 if kernel == "turns" else 1
    for logs in ([0, log, log, 0], [-30, log - 30, 0, log - 30]):
        scales = [2.0 ** x for x in logs for _ in range(wide)]
        codes = [behind] * wide + [0] * (len(scales) - wide)
        attend(ent, "bf16", 64, kernel, codes, scales, 0.25)
    if kernel != "turns":
        attend(ent, "f16", 64, kernel, [behind, 0, 0, 0], [2.0 ** (x - log) for x in (0, log, log, 0)], 0.25)


@pytest.mark.parametrize("kernel", KERNELS)
def test_scales_and_scores_at_random(ent, kernel):
    """Tiles' scales and scores drawn over wide ranges, apart and together."""
    say(f"chunk: scales and scores at random, {kernel}")
    rng = random.Random(5)
    for i in range(30):
        tiles = KERNELS[kernel][1] + (0 if kernel == "turns" else rng.randint(0, 4))
        wide = rng.choice((3, 12, 40, 90))
        far = rng.choice((0, 1, 8, 60))
        logs = [rng.uniform(-wide, wide) for _ in range(tiles)]
        if rng.random() < 0.3:
            logs = sorted(logs, reverse=rng.random() < 0.5)
        keys = [rng.randint(-far, far) for _ in range(tiles)]
        if rng.random() < 0.3:      # the scores make up for the scales
            keys = [round(max(-127, min(127, far / 16 - x))) for x in logs]
        attend(ent, "bf16", 64, kernel, keys, [2.0 ** x for x in logs], rng.choice((0.25, 0.1733)), less=rng.randint(0, 63))


@pytest.mark.parametrize("kernel", ["few", "four", "eight"])
def test_pieces_at_random(ent, kernel):
    """The same over sequences that are cut into pieces, with scores up to 2^30."""
    say(f"chunk: pieces of scales and scores at random, {kernel}")
    rng = random.Random(6)
    for i in range(16):
        tiles = rng.randint(14, 50)
        wide, far, scale = rng.choice((3, 12, 40, 90)), rng.choice((0, 1, 8, 60)), rng.choice((0.25, 0.1733, 2.0 ** 9, 2.0 ** 22))
        logs = [rng.uniform(-wide, wide) for _ in range(tiles)]
        keys = [rng.randint(-far, far) for _ in range(tiles)]
        attend(ent, "bf16", 64, kernel, keys, [2.0 ** x for x in logs], scale, less=rng.randint(0, 63))


@pytest.mark.parametrize("new,heads", [(20, (2, 1)), (24, (1, 1)), (30, (2, 1)), (80, (2, 1)), (130, (1, 1))], ids=str)
@pytest.mark.parametrize("first,hidden", [(-90, 96), (-90, -31), (0, 59), (0, -59), (60, -90)])
def test_scales_of_a_tile_that_a_row_does_not_see(ent, new, heads, first, hidden):
    """Rows that see the first tile alone give the same results, to the bit, whatever the
    scales of the second are."""
    say(f"chunk: scales of a hidden tile, {new} {heads} {first} {hidden}")
    h, kv = heads
    n = 64 + new // 2
    c = ent.KVCache.empty(3, kv, 64, 64)
    g = torch.Generator(device="cuda").manual_seed(new)
    c.k_codes.copy_(torch.randint(-20, 21, c.k_codes.shape, device="cuda", generator=g))
    c.v_codes.copy_(torch.randint(-127, 128, c.v_codes.shape, device="cuda", generator=g))
    c.k_scales.fill_(1.0 / 16)
    q = torch.randn(new, h, 64, device="cuda", generator=g).to(torch.bfloat16)
    t = ints([[2, 0, 1]])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for log in (first, hidden):
        c.v_scales.fill_(2.0 ** first)
        c.v_scales[0] = 2.0 ** log
        got.append(ent.attn_chunk(q, c, t, ints([n]), ints([0, new]), status))
    rows = 64 - (n - new)            # rows that see the first 64 tokens or fewer
    assert not status.any() and 0 < rows < new
    seen = max(0, new - n)           # the first ones see nothing
    assert torch.equal(got[0][:rows], got[1][:rows])
    assert (got[0][:seen] == 0).all() and (got[0][seen:rows] != 0).any()
    assert torch.isfinite(got[1]).all()
