"""GPU tests of the attention of chunks over the 8-bit cache, against the oracle in
64 bits.

The bound of an output o, with A the weighted mean of |v|, u the unit roundoff of
the element type and n the tokens it sees:

* the result's rounding: u |o|
* the weights' rounding to f16: 2^-12 A (f16's own smallest steps below 2^-35 of
  the largest weight: n 2^-35 max |v|)
* scores in 32 bits: the dot product's D roundings, q's own where it is held in f16
  (2^-25 of its row's largest), the scaling's and differences' at the size of the
  score and of the scales' logarithms, 2^-20 for the exponentials: that much
  relative error e in each weight, above and below: 2 e A
* sums in 32 bits and their factors where the maximum rises, in blocks of 16 tokens:
  (n / 16 + 4) 2^-22 A
"""
import math

import numpy as np
import pytest

from oracle import attention as oa
from tests.test_gpu_attn import arrays, filled_cache, ints, make_table, np64, running, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
DTYPES = ["bf16", "f16"]
HEADS = [(4, 4, 64), (6, 2, 96), (8, 2, 128), (7, 1, 64), (3, 3, 128)]


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


def bound(out, mean, top, q, kmax, vmax, n, dtype, scale, log):
    d, scale = q.shape[-1], abs(scale)
    dot = scale * np.abs(q).sum(-1) * kmax * (d + 2) * 2.0 ** -24
    if dtype == "bf16":
        dot = dot + scale * d * np.abs(q).max(-1) * kmax * 2.0 ** -24
    e = dot + 8 * (top + log + 64) * 2.0 ** -24 + 2.0 ** -20
    b = ROUND[dtype] * np.abs(out) + ((2.0 ** -12 + 2 * e + (n / 16 + 4) * 2.0 ** -22)[..., None] * mean) * 1.01
    return b + n[..., None] * 2.0 ** -35 * vmax + (2.0 ** -25 if dtype == "f16" else 2.0 ** -130)


def run(ent, heads, dtype, page, new, lens, seed=0, edit=None, scale=None, spare=1, extra=2, joint=False, check=None, finite=True):
    """Runs chunks (with `extra` rows of no sequence behind them) over a cache of
    random codes and compares with the oracle; returns the outputs."""
    h, kv, d = heads
    pages = sum(-(-n // page) for n in lens) + 2
    c = filled_cache(ent, kv, d, page, pages, seed)
    t = make_table(lens, page, pages, seed, spare)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rows, total = sum(new) + extra, sum(new)
    x = (1.5 * torch.randn(rows, h + (3 if joint else 0), d, device="cuda", generator=g)).to(TORCH[dtype])
    q = x[:, :h]
    if edit:
        edit(q, c, t)
    cu = running(new)
    status = torch.zeros(len(new), dtype=torch.int32, device="cuda")
    place = torch.full((rows, h + (5 if joint else 0), d), 7.0, dtype=TORCH[dtype], device="cuda")
    out = place[:, :h]
    got = ent.attn_chunk(q, c, torch.from_numpy(t).cuda(), ints(lens), ints(cu), status, scale=scale, out=out)
    torch.cuda.synchronize()
    assert got is out and not status.any()
    assert (place[total:] == 7).all() and (place[:, h:] == 7).all(), "rows of no sequence or other places were written"
    s = 1.0 / math.sqrt(d) if scale is None else scale
    a, o = arrays(c), np64(out)
    if finite:
        assert np.isfinite(o).all()
    q64 = np64(q)
    vs = a[3][np.isfinite(a[3]) & (a[3] > 0)]
    log = float(np.abs(np.log2(vs)).max()) if vs.size else 0.0
    worst = 0.0
    for b in range(len(new)) if check is None else check:
        if not new[b]:
            continue
        k, v = (y.astype(np.float64) for y in oa.rows_of(*a, t[b], 0, lens[b]))
        i = slice(cu[b], cu[b + 1])
        e, mean, top = oa.chunk(q64[i], [k], [v], [lens[b]], [0, new[b]], s)
        n = np.maximum(lens[b] - new[b] + 1 + np.arange(new[b]), 0)[:, None] * np.ones((1, h))
        bb = bound(e, mean, top, q64[i], np.abs(k).max(initial=0.0), np.abs(v).max(initial=0.0), n, dtype, s, log)
        err = np.abs(o[i] - e)
        worst = max(worst, float((err / bb).max()))
    assert worst <= 1.0, (heads, dtype, page, new, lens, worst)
    return out[:total]


LENGTHS = [
    ([1], [1]),
    ([5], [90]),
    ([0, 1, 5, 0], [3, 1, 70, 0]),
    ([31, 32, 33, 8], [31, 64, 65, 129]),
    ([3, 40, 1], [70, 45, 200]),
    ([5, 70, 2, 0, 3], [3, 20, 0, 9, 2]),           # more queries than tokens: the first rows see nothing
    ([130, 1, 17], [130, 700, 300]),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("case", range(len(LENGTHS)))
def test_chunk_matches_oracle(ent, heads, dtype, case):
    page = (16, 32, 64, 128)[case % 4]
    say(f"chunk {heads} page {page} {dtype} {LENGTHS[case]}")
    run(ent, heads, dtype, page, *LENGTHS[case], seed=case)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [(16, 1, 64), (17, 1, 128), (40, 1, 64), (32, 2, 96), (5, 1, 96)], ids=str)
def test_chunk_groups_and_pages(ent, heads, page):
    say(f"chunk {heads} page {page}")
    run(ent, heads, "bf16", page, [1, 9, 2, 30], [64, 65, 15, 130])
    run(ent, heads, "f16", page, [3], [17], spare=0)


@pytest.mark.parametrize("heads", [(130, 1, 64), (300, 1, 64), (257, 1, 128), (512, 2, 96)], ids=str)
def test_chunk_groups_wider_than_a_workgroup(ent, heads):
    say(f"chunk {heads}")
    run(ent, heads, "bf16", 32, [1, 3], [70, 40])
    run(ent, heads, "f16", 16, [2], [33])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [(4, 4, 64), (6, 2, 96), (8, 2, 128), (20, 1, 128)], ids=str)
def test_chunk_split(ent, heads, dtype):
    """Long and short sequences together: some blocks are split, some are not."""
    say(f"chunk split {heads} {dtype}")
    run(ent, heads, dtype, 64, [4, 3, 0, 7, 1, 20, 1], [3000, 3, 0, 700, 513, 512, 1])
    run(ent, heads, dtype, 16, [2], [2049])
    run(ent, heads, dtype, 32, [140], [400])


def test_chunk_many_sequences(ent):
    say("chunk: 150 sequences")
    new = [(7 * i) % 4 for i in range(150)]
    lens = [(37 * i) % 300 + n for i, n in enumerate(new)]
    run(ent, (2, 1, 64), "bf16", 32, new, lens, check=range(0, 150, 7))
    for cap in (1, 3, 50):
        old = ent.set_max_workgroups(cap)
        try:
            run(ent, (4, 2, 64), "f16", 64, new[:70], lens[:70], check=range(0, 70, 9))
        finally:
            ent.set_max_workgroups(old)


def test_chunk_long(ent):
    say("chunk: 3 tokens behind 70000")
    run(ent, (4, 1, 128), "bf16", 64, [3], [70003])


def test_chunk_slices(ent):
    say("chunk: slices of wider tensors")
    run(ent, (6, 2, 96), "bf16", 32, [50, 8], [50, 300], joint=True)
    run(ent, (4, 4, 64), "f16", 32, [50, 8], [50, 300], joint=True)


def test_chunk_rows_without_tokens_are_zero(ent):
    say("chunk: rows without tokens")
    got = run(ent, (4, 2, 64), "bf16", 16, [70, 9], [50, 0])
    assert (got[:20] == 0).all() and (got[70:] == 0).all() and (got[20:70] != 0).any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_chunk_hidden_places(ent, dtype):
    """Scales of pages that hold no token, pages that a row does not see, and codes
    behind the last token."""
    say(f"chunk: hidden places, {dtype}")
    new, lens, page = [40, 3, 33], [70, 17, 129], 16
    heads = (4, 2, 64)

    def behind(q, c, t):
        used = {int(p) for b, n in enumerate(lens) for p in t[b, : -(-n // page)]}
        for p in range(c.k_scales.shape[0]):
            if p not in used:
                c.k_scales[p], c.v_scales[p] = math.nan, math.inf
        for b, n in enumerate(lens):
            p, r = int(t[b, n // page]), n % page
            if r:
                c.k_codes[p, :, r:], c.v_codes[p, :, :, r:] = 127, -128

    a = run(ent, heads, dtype, page, new, lens, seed=3)
    assert torch.equal(run(ent, heads, dtype, page, new, lens, seed=3, edit=behind), a)
    # the last pages of the first and the third sequence: tokens 64 on and 112 on
    for k, v in ((math.nan, 1.0), (1.0, math.nan), (math.inf, math.inf), (1.0, math.inf)):

        def seen_late(q, c, t):
            for b, n in ((0, 64), (2, 112)):
                p = int(t[b, n // page])
                c.k_scales[p] *= k
                c.v_scales[p] *= v

        g = raw(ent, heads, dtype, page, new, lens, 3, seen_late)
        first = {0: 40 - (70 - 64), 2: 33 - (129 - 112)}      # the first row of each that sees the page
        clean = torch.ones(76, dtype=torch.bool)
        clean[first[0]: 40] = False
        clean[43 + first[2]: 76] = False
        assert alike(g[clean], a[clean], dtype)
        assert not torch.isfinite(g[~clean]).all(-1).any()


def alike(x, y, dtype, vmax=0.04 * 127):
    """Two results of one row over the cache of filled_cache(), by the operator's
    ways for ordinary and for other tiles: each is off by its own rounding, and by the
    weights' to f16, 2^-12 of a weighted mean of |v| (which is at most vmax; scores
    and sums in 32 bits: within a tenth of that)."""
    x, y = x.double(), y.double()
    return bool(((x - y).abs() <= 2 * ROUND[dtype] * torch.maximum(x.abs(), y.abs()) + 2 * 1.1 * 2.0 ** -12 * vmax).all())


def raw(ent, heads, dtype, page, new, lens, seed, edit, scale=None):
    """The outputs of run()'s inputs, unchecked."""
    h, kv, d = heads
    pages = sum(-(-n // page) for n in lens) + 2
    c = filled_cache(ent, kv, d, page, pages, seed)
    t = make_table(lens, page, pages, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (1.5 * torch.randn(sum(new) + 2, h, d, device="cuda", generator=g)).to(TORCH[dtype])
    edit(q, c, t)
    status = torch.zeros(len(new), dtype=torch.int32, device="cuda")
    out = ent.attn_chunk(q, c, torch.from_numpy(t).cuda(), ints(lens), ints(running(new)), status, scale=scale)
    assert not status.any()
    return out[: sum(new)]


@pytest.mark.parametrize("heads", [(4, 2, 64), (4, 1, 128)], ids=str)
def test_chunk_extremes(ent, heads):
    say(f"chunk: extreme scales and queries, {heads}")

    def wide(q, c, t):     # pages' scales far apart, pages of zeros
        c.v_scales.copy_(2.0 ** torch.arange(-8, c.v_scales.shape[0] - 8, device="cuda")[:, None].expand_as(c.v_scales) / 64)
        c.v_scales[int(t[0, 1])] = 0.0
        c.v_codes[int(t[0, 1])] = 0

    def wider(q, c, t):    # from the type's smallest to near its largest
        n = c.v_scales.shape[0]
        c.v_scales.copy_(2.0 ** torch.linspace(-126, 120, n, device="cuda")[torch.randperm(n, device="cuda")][:, None].expand_as(c.v_scales))

    def zeros(q, c, t):
        c.v_scales.zero_()

    def first(q, c, t):    # no value but in the first and the last page
        c.v_scales[t[0, 1:9].tolist()] = 0.0

    def by(f, scale=1.0):
        return lambda q, c, t: q.mul_(f)

    new, lens = [20, 9, 1], [150, 40, 160]
    for dtype in DTYPES:
        for edit in (wide, zeros, first):
            run(ent, heads, dtype, 16, new, lens, edit=edit)
        run(ent, heads, dtype, 16, new, lens, edit=by(20))
        run(ent, heads, dtype, 16, new, lens, scale=0.0)
        run(ent, heads, dtype, 16, new, lens, scale=-0.2)
    run(ent, heads, "bf16", 16, new, lens, edit=wider)
    run(ent, heads, "bf16", 16, new, lens, edit=by(2.0 ** -60), scale=2.0 ** 55)
    run(ent, heads, "bf16", 16, new, lens, edit=by(2.0 ** 60), scale=2.0 ** -64)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("step", [-1, 1])
def test_chunk_far_scores(ent, dtype, sign, step):
    """All scores far from zero, of either sign, and equal but for one token's, which
    is behind or ahead: its weight follows from the difference alone."""
    say(f"chunk: far scores, {dtype} {sign} {step}")
    kv, d, page, n = 1, 64, 16, 200
    c = ent.KVCache.empty(14, kv, d, page)
    t = torch.arange(13, dtype=torch.int32, device="cuda")[None].contiguous()
    c.k_codes[:, :, :, 0] = (127 if step < 0 else 126) * sign
    c.k_scales.fill_(1.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    c.v_codes.copy_(torch.randint(-127, 128, c.v_codes.shape, device="cuda", generator=g))
    c.v_scales.fill_(2.0 ** -7)
    c.k_codes[3, 0, 7, 0] += step                   # token 55: 2^10 or more behind or ahead
    q = torch.zeros(4, 2, d, dtype=TORCH[dtype], device="cuda")
    q[:, :, 0] = 2.0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for power in (4, 20, 40, 60) if dtype == "bf16" else (4, 12):
        q[:, :, 0] = 2.0 ** power
        scale = 2.0 ** (6 if dtype == "bf16" else 13)
        got = np64(ent.attn_chunk(q, c, t, ints([n]), ints([0, 4]), status, scale=scale))
        v = np64(c.v_codes)[:, 0].transpose(0, 2, 1).reshape(-1, d) * 2.0 ** -7
        for i in range(4):
            m = n - 3 + i
            w = np.full(m, 1.0 if step < 0 else 0.0)
            w[55] = 1.0 - w[55]
            want = w @ v[:m] / w.sum()
            b = ROUND[dtype] * np.abs(want) + (2.0 ** -12 + 40 * 2.0 ** -22) * (w @ np.abs(v[:m]) / w.sum()) + 2.0 ** -20
            assert (np.abs(got[i] - want) <= b).all(), (power, i)
    assert not status.any()


def test_chunk_queries_that_are_no_numbers(ent):
    """An infinity or NaN in a query reaches its own row and head alone."""
    say("chunk: queries that are no numbers")
    new, lens = [40, 3], [70, 300]

    def spoil(q, c, t):
        q[3, 1, 5], q[41, 0, 60] = math.nan, math.inf

    a = run(ent, (4, 2, 64), "bf16", 16, new, lens)
    got = raw(ent, (4, 2, 64), "bf16", 16, new, lens, 0, spoil)
    bad = torch.zeros(43, 4, dtype=torch.bool, device="cuda")
    bad[3, 1] = bad[41, 0] = True
    assert not torch.isfinite(got[bad]).any() and torch.isfinite(got[~bad]).all()
    assert alike(got[~bad], a[~bad], "bf16")
    # over tokens that are split over workgroups
    g2 = raw(ent, (4, 2, 64), "bf16", 16, [4], [3000], 0, lambda q, c, t: q[1, 2].fill_(math.nan))
    assert torch.isnan(g2[1, 2]).all() and torch.isfinite(g2[0]).all() and torch.isfinite(g2[2:]).all()


def test_chunk_flags(ent):
    say("chunk: faults in the data")
    kv, d, page = 2, 64, 16
    t = make_table([40, 40, 40], page, 12, 2, spare=0)
    c = filled_cache(ent, kv, d, page, 12, 7)
    q = torch.randn(30, 4, d, device="cuda").to(torch.bfloat16)
    good = ent.attn_chunk(q, c, torch.from_numpy(t).cuda(), ints([30, 40, 30]), ints([0, 10, 20, 30]),
                          torch.zeros(3, dtype=torch.int32, device="cuda"))
    place = np.arange(9).reshape(3, 3)
    length, page_flag = ent.FLAGS["length"], ent.FLAGS["page"]
    for lens, cu, table, want in (
        ([30, 40, 49], [0, 10, 20, 30], t, [0, 0, length]),
        ([30, -1, 30], [0, 10, 20, 30], t, [0, length, 0]),
        ([30, 40, 30], [0, 10, 20, 31], t, [0, 0, length]),
        ([30, 40, 30], [0, 10, 20, 2 ** 31 - 1], t, [0, 0, length]),
        ([30, 40, 30], [0, 10, -7, 30], t, [0, length, length]),
        ([30, 40, 30], [0, 10, 5, 30], t, [0, length, length]),      # begins before an earlier one's end
        ([30, 40, 30], [0, 10, 20, 30], np.where(place == 7, 12, t), [0, 0, page_flag]),
        ([30, 40, 30], [0, 10, 20, 30], np.where(place == 4, -1, t), [0, page_flag, 0]),
        ([30, 40, 30], [0, 10, 20, 30], np.where(place == 8, 10 ** 9, t), [0, 0, 0]),       # holds no token
    ):
        status = torch.zeros(3, dtype=torch.int32, device="cuda")
        got = ent.attn_chunk(q, c, torch.from_numpy(np.ascontiguousarray(table.astype(np.int32))).cuda(), ints(lens), ints(cu), status)
        assert status.tolist() == want, (lens, cu)
        for b in range(3):
            if not want[b]:
                assert torch.equal(got[10 * b: 10 * b + 10], good[10 * b: 10 * b + 10])


def test_chunk_of_single_tokens_is_the_cache_attention(ent):
    say("chunk: single tokens")
    lens = [1, 40, 700, 3000]
    for heads in ((8, 2, 128), (4, 4, 64)):
        h, kv, d = heads
        c = filled_cache(ent, kv, d, 32, 130, 4)
        t = torch.from_numpy(make_table(lens, 32, 130, 4)).cuda()
        q = torch.randn(4, h, d, device="cuda").to(torch.bfloat16)
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        a = ent.attn_chunk(q, c, t, ints(lens), ints([0, 1, 2, 3, 4]), status)
        b = ent.attn_cache(q, c, t, ints(lens), status)
        v = float(c.v_scales.max()) * 127
        assert ((a.double() - b.double()).abs() <= 2 * 2.0 ** -8 * b.double().abs() + 2 * 2.0 ** -11 * v).all()
        assert not status.any()


def test_chunk_nothing_to_do(ent):
    say("chunk: no sequence, no rows")
    c = filled_cache(ent, 2, 64, 16, 4, 0)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert ent.attn_chunk(q, c, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), none, ints([0]), none).shape == (0, 4, 64)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    t = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    assert ent.attn_chunk(q, c, t, ints([5, 9]), ints([0, 0, 0]), status).shape == (0, 4, 64)
    q = torch.full((3, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7)
    ent.attn_chunk(q, c, t, ints([5, 9]), ints([0, 0, 0]), status, out=out)
    assert (out == 7).all() and not status.any()
    ent.attn_chunk(q, c, t, ints([5, -9]), ints([0, 0, 0]), status, out=out)
    assert status.tolist() == [0, ent.FLAGS["length"]]


def test_chunk_workspace_streams_and_repeats(ent):
    say("chunk: workspace, streams, the same call again")
    h, kv, d, page = 8, 2, 128, 64
    new, lens = [20, 3, 0, 60], [2500, 1900, 4, 333]
    c = filled_cache(ent, kv, d, page, 80, 1)
    t = torch.from_numpy(make_table(lens, page, 80, 1)).cuda()
    q = torch.randn(83, h, d, device="cuda").to(torch.bfloat16)
    cu, ln, status = ints(running(new)), ints(lens), torch.zeros(4, dtype=torch.int32, device="cuda")
    want = ent.attn_chunk(q, c, t, ln, cu, status)
    for _ in range(5):
        assert torch.equal(ent.attn_chunk(q, c, t, ln, cu, status), want)
    size = ent.attn_chunk_work_bytes(4, 83, h, kv, d)
    work = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(ent.attn_chunk(q, c, t, ln, cu, status, work=work), want)
    with pytest.raises(ent.EntroError):
        ent.attn_chunk(q, c, t, ln, cu, status, work=work[:-16])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ent.attn_chunk(q, c, t, ln, cu, status, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    raw_handle = torch.cuda.current_stream().cuda_stream
    out = torch.empty_like(q)
    ent.attn_chunk(q, c, t, ln, cu, status, out=out, work=work, stream=raw_handle)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(ValueError, match="raw stream"):
        ent.attn_chunk(q, c, t, ln, cu, status, stream=raw_handle)
    # two calls at once, a workspace each
    for s in (side, torch.cuda.current_stream()):
        s.wait_stream(torch.cuda.current_stream())
    a = [ent.attn_chunk(q, c, t, ln, cu, status, stream=s) for s in (side, torch.cuda.current_stream()) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in a) and not status.any()


def test_append_and_chunk_in_a_graph(ent):
    """A step (append with rotation, then attention of its chunk) captured once and
    replayed with new inputs and lengths in place, the program's own work between."""
    say("append and chunk: graph replay")
    h, kv, d, page = 8, 2, 128, 64
    new = [5, 1, 40]
    t = torch.from_numpy(make_table([3000, 400, 600], page, 70, 0)).cuda()
    c, e = (filled_cache(ent, kv, d, page, 70, 6) for _ in range(2))
    held, lens, cu = ints([2500, 80, 300]), ints([2505, 81, 340]), ints(running(new))
    x = torch.zeros(46, h + 2 * kv, d, device="cuda")
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    rot = ent.Rotary((10000.0 ** (-torch.arange(64) / 64)).float().cuda())
    rotated, out = (torch.empty(46, h, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    work = torch.empty(ent.attn_chunk_work_bytes(3, 46, h, kv, d), dtype=torch.uint8, device="cuda")

    def step(cache, rotated, out, work):
        q = ent.kv_append(cache, rot, x[:, h: h + kv], x[:, h + kv:], t, held, cu, status, q=x[:, :h], q_out=rotated)
        return ent.attn_chunk(q, cache, t, lens, cu, status, out=out, work=work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(filled_cache(ent, kv, d, page, 70, 6), rotated, out, work)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, rotated, out, work)
    g = torch.Generator(device="cuda").manual_seed(4)
    for i in range(4):
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        graph.replay()
        got = out.clone()
        want = step(e, torch.empty_like(rotated), None, None)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and (got != 0).any()
        for a, b in zip(c.tensors, e.tensors):
            assert torch.equal(a, b)
        step_by = torch.tensor(new, dtype=torch.int32, device="cuda")
        held += step_by
        lens += step_by
    assert not status.any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_in_pieces(ent, dtype):
    """The operators together: a prompt's pieces appended and attended one after
    another over the cache, then drafted tokens, against attention in 64 bits over
    what the cache holds, and near the attention of the rotated rows without one."""
    say(f"append and chunk: a prompt in pieces, {dtype}")
    h, kv, d, page = 8, 2, 64, 32
    g = torch.Generator(device="cuda").manual_seed(9)
    tokens = [150, 64]
    x = [torch.randn(n, h + 2 * kv, d, device="cuda", generator=g) for n in tokens]
    f = (10000.0 ** (-torch.arange(32) / 32)).float().cuda()
    rot = ent.Rotary(f)
    c = ent.KVCache.empty(12, kv, d, page)
    t = make_table(tokens, page, 12, 1)
    tt, status = torch.from_numpy(t).cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
    held = [0, 0]
    for new in ([70, 1], [60, 30], [13, 33], [7, 0]):
        y = torch.cat([x[b][held[b]: held[b] + new[b]] for b in range(2)])
        cu, lens = ints(running(new)), [a + b for a, b in zip(held, new)]
        q = ent.kv_append(c, rot, y[:, h: h + kv], y[:, h + kv:], tt, ints(held), cu, status, q=y[:, :h], dtype=TORCH[dtype])
        out = np64(ent.attn_chunk(q, c, tt, ints(lens), cu, status))
        a, at = arrays(c), running(new)
        for b in range(2):
            if not new[b]:
                continue
            k, v = (z.astype(np.float64) for z in oa.rows_of(*a, t[b], 0, lens[b]))
            i = slice(at[b], at[b + 1])
            e, mean, top = oa.chunk(np64(q)[i], [k], [v], [lens[b]], [0, new[b]], 1 / 8)
            n = (held[b] + 1 + np.arange(new[b]))[:, None] * np.ones((1, h))
            bb = bound(e, mean, top, np64(q)[i], np.abs(k).max(), np.abs(v).max(), n, dtype, 1 / 8, 8.0)
            assert (np.abs(out[i] - e) <= bb).all()
            # without the cache: what differs is its 8 bits, and q's rounding
            whole = np64(x[b])[: lens[b]]
            places = [list(range(lens[b]))]
            qq, kk = (oa.rotate(z, places, f.cpu().numpy())[0] for z in (whole[:, :h], whole[:, h: h + kv]))
            want, _, _ = oa.chunk(qq[held[b]:], [kk], [whole[:, h + kv:]], [lens[b]], [0, new[b]], 1 / 8)
            assert np.linalg.norm(out[i] - want) <= 0.03 * np.linalg.norm(want)
        held = lens
    assert not status.any()


@pytest.mark.parametrize("new,lens", [([3, 1, 0, 16], [400, 70, 5, 16]), ([60, 33], [300, 33]), ([140], [141])], ids=str)
def test_chunk_more_heads_than_workgroups_at_once(ent, new, lens):
    """So many key/value heads that no block is cut: the workspace is nominal."""
    say(f"chunk of 520 key/value heads {new} {lens}")
    assert ent.attn_chunk_work_bytes(len(new), sum(new), 520, 520, 64) == 16
    run(ent, (520, 520, 64), "bf16", 16, new, lens)
