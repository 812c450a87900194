"""GPU tests of the attention over the 8-bit cache for every scale that a page
can hold: pages of zeros (scale 0, what the store writes for them) as whole
tiles of 64 tokens, scales at both ends of the range and scales far apart.

The bound is that of test_gpu_attn.py (weights in f16 down to 2^-39 of the
largest product of weight and scale) and, for the scales: their logarithms, the
parts' exponents and the parts' logarithms of sums are rounded at their size
some 8 times, 2^-24 (|log2 scale| + |score| / ln 2 + 16) ln 2 each, once in the
weights of the product and once in those of the sum.
"""
import math

import numpy as np
import pytest

from oracle import attention as oa
from tests.test_gpu_attn import TORCH, arrays, bound, filled_cache, ints, make_table, np64, running, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TILE = 64


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


def check(ent, q, c, t, lens, dtype, scale=None):
    """Attention of q over the cache against the oracle; returns the outputs."""
    n, h, d = q.shape
    kv = c.k_codes.shape[1]
    status = torch.zeros(n, dtype=torch.int32, device="cuda")
    got = ent.attn_cache(q, c, torch.from_numpy(t).cuda(), ints(lens), status, scale=scale)
    torch.cuda.synchronize()
    assert not status.any()
    s = 1.0 / math.sqrt(d) if scale is None else scale
    a, out, q64 = arrays(c), np64(got), np64(q)
    assert np.isfinite(out).all()
    for b in range(n):
        k, v = oa.rows_of(*a, t[b], 0, lens[b])
        page = a[0].shape[2]
        vs = a[3][t[b, : -(-lens[b] // page)]]
        log = np.abs(np.log2(vs[vs >= 2.0 ** -126])).max(initial=0.0)
        kmax, vmax = np.abs(k).max(initial=0.0), float(np.abs(v).max(initial=0.0))
        for i in range(h):
            e, mean, top = oa.attend(q64[b, i], k[:, i // (h // kv)], v[:, i // (h // kv)], s)
            bb = bound(e[None, None], mean[None, None], np.array([[top]]), q64[b: b + 1, i: i + 1], kmax, vmax, lens[b], dtype,
                       "cache", s)[0, 0]
            bb = bb + 16 * (log + 1.5 * top + 16) * 2.0 ** -24 * mean
            err = np.abs(out[b, i] - e)
            assert (err <= bb).all(), (b, i, lens[b], float((err / bb).max()), out[b, i][:4], e[:4])
    return got


def setup(ent, heads, dtype, page, lens, seed=0):
    h, kv, d = heads
    pages = sum(-(-n // page) for n in lens) + 2
    c = filled_cache(ent, kv, d, page, pages, seed)
    t = make_table(lens, page, pages, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (1.5 * torch.randn(len(lens), h, d, device="cuda", generator=g)).to(TORCH[dtype])
    return q, c, t


def zero_values(c, t, b, tokens, page):
    """The values of sequence b's pages that hold any of `tokens`: zeros."""
    for p in sorted({x // page for x in tokens}):
        c.v_codes[int(t[b, p])] = 0
        c.v_scales[int(t[b, p])] = 0.0


# Tiles (of 64 tokens) whose values are zero, of `tiles`: a wavefront takes every
# fourth tile of its workgroup's.
PATTERNS = {
    "first": lambda tiles: [0],
    "second": lambda tiles: [1],
    "each_first": lambda tiles: [0, 1, 2, 3],
    "middle": lambda tiles: [tiles // 2],
    "last": lambda tiles: [tiles - 1],
    "first_and_later": lambda tiles: [0, 4, 5],
    "all_but_last": lambda tiles: list(range(tiles - 1)),
    "all_but_first": lambda tiles: list(range(1, tiles)),
    "all": lambda tiles: list(range(tiles)),
}


@pytest.mark.parametrize("pattern", list(PATTERNS))
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("lens", [[100, 164, 1000], [3000, 700]], ids=["whole", "split"])
def test_tiles_of_zero_values(ent, lens, page, pattern):
    say(f"cache attention: tiles of zero values, {lens} page {page} {pattern}")
    for heads, dtype in (((4, 2, 64), "bf16"), ((8, 1, 128), "f16"), ((3, 1, 96), "bf16")):
        q, c, t = setup(ent, heads, dtype, page, lens)
        for b, n in enumerate(lens):
            tiles = -(-n // TILE)
            for tile in PATTERNS[pattern](tiles):
                if tile < tiles:
                    zero_values(c, t, b, range(tile * TILE, min(n, (tile + 1) * TILE)), page)
        got = check(ent, q, c, t, lens, dtype)
        if pattern == "all":
            assert not got.any()


@pytest.mark.parametrize("page", [16, 64, 128])
def test_store_of_zeros_then_attention(ent, page):
    """Values of zero stored by the cache's own store, in front, in between and
    behind others."""
    say(f"cache attention: zeros stored, page {page}")
    kv, d = 2, 128
    lens = [128, 400, 2000]
    c = filled_cache(ent, kv, d, page, sum(-(-n // page) for n in lens) + 2, 3)
    t = make_table(lens, page, c.k_codes.shape[0], 3)
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(sum(lens), kv, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    cu = running(lens)
    for b, (lo, hi) in enumerate([(0, 64), (128, 384), (0, 1900)]):
        v[cu[b] + lo: cu[b] + hi] = 0.0
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    ent.kv_store(c, k, v, torch.from_numpy(t).cuda(), ints([0, 0, 0]), ints(cu), status)
    q = (1.5 * torch.randn(3, 8, d, device="cuda", generator=g)).to(torch.bfloat16)
    got = check(ent, q, c, t, lens, "bf16")
    assert got.any(-1).all()


SCALES = {
    "smallest": lambda i: 2.0 ** -126 + 0.0 * i,
    "tiny": lambda i: 2.0 ** -112 + 0.0 * i,
    "large": lambda i: 2.0 ** 100 + 0.0 * i,
    "largest": lambda i: 2.0 ** 120.5 + 0.0 * i,
    "tiny_and_large": lambda i: np.where(i % 2 == 0, 2.0 ** -112, 2.0 ** 100),
    "smallest_and_one": lambda i: np.where(i % 3 == 0, 1.0, 2.0 ** -126),
    "one_and_zero_last": lambda i: np.where(i % 5 == 0, 0.0, 1.0),
    "falling": lambda i: 2.0 ** (120.0 - 7.0 * (i % 34)),
    "rising": lambda i: 2.0 ** (-120.0 + 7.0 * (i % 34)),
}


@pytest.mark.parametrize("which", list(SCALES))
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("lens", [[70, 300, 1000], [2600, 500]], ids=["whole", "split"])
def test_scales_of_every_size(ent, lens, page, which):
    say(f"cache attention: value scales {which}, {lens} page {page}")
    for heads in ((4, 2, 64), (8, 1, 128)):
        q, c, t = setup(ent, heads, "bf16", page, lens, seed=2)
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                s = float(SCALES[which](np.array(i)))
                c.v_scales[int(t[b, i])] = s
                if s == 0.0:
                    c.v_codes[int(t[b, i])] = 0
        check(ent, q, c, t, lens, "bf16")


@pytest.mark.parametrize("big", [2.0 ** -7, 1.0, 2.0 ** 7, 2.0 ** 100])
@pytest.mark.parametrize("n", [1000, 30000])
def test_many_zero_values_behind_one_high_score(ent, n, big):
    """One token far ahead, all others with values of zero and scores 16 powers
    of two below: together they count in the sum."""
    say(f"cache attention: {n} zero values behind one, scale {big}")
    d, page = 64, 64
    c = ent.KVCache.empty(-(-n // page) + 1, 1, d, page)
    t = make_table([n], page, c.k_codes.shape[0], 0)
    first = int(t[0, 0])
    c.k_scales.fill_(1.0)
    c.k_codes[first, 0, 0, 0] = 127
    c.v_codes[first, 0, :, 0] = torch.arange(d, device="cuda").to(torch.int8) + 40
    c.v_scales[first] = big
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 16 * math.log(2) / 127
    check(ent, q, c, t, [n], "bf16", scale=1.0)


@pytest.mark.parametrize("lens", [[200], [3000]], ids=["whole", "split"])
def test_infinite_and_nan_scales_are_seen(ent, lens):
    """A value scale that is infinite or NaN gives no finite result; so does a
    key scale that is NaN."""
    say(f"cache attention: infinite and NaN scales, {lens}")
    for what, x in (("v_scales", math.inf), ("v_scales", math.nan), ("k_scales", math.nan)):
        for at in (0, 1, -1):
            q, c, t = setup(ent, (4, 2, 64), "bf16", 64, lens)
            getattr(c, what)[int(t[0, : -(-lens[0] // 64)][at]), 1] = x
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = ent.attn_cache(q, c, torch.from_numpy(t).cuda(), ints(lens), status)
            torch.cuda.synchronize()
            assert torch.isfinite(got[0, :2]).all()
            assert not torch.isfinite(got[0, 2:]).any()
