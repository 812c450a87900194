"""GPU tests of the rotary positions and of the append to the 8-bit cache, against
the oracle in 64 bits.

The bound of a rotated element, with S = gain (|x| + |y|) of its pair: cosine and
sine are off by 2^-21 (as the operator states), two products and a sum are rounded
to 24 bits, and the factor gain is: S (2^-21 + 4 * 2^-24).  The result is then
rounded to its type (8 or 11 significant bits, or half of f16's smallest step).  A
code of the cache stands for a value at most half a step of its page's scale away,
and the scale is the largest magnitude over 127 in 32 bits; a code held before is
rounded again where the page's range grows.
"""
import math

import numpy as np
import pytest

from oracle import attention as oa
from tests.test_gpu_attn import arrays, filled_cache, ints, make_table, np64, running, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TURN = 2.0 ** -21 + 4 * 2.0 ** -24
HEADS = [(4, 4, 64), (6, 2, 96), (8, 2, 128), (7, 1, 64), (40, 3, 128)]
TYPES = [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "f16")]


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


def freqs_of(pairs, base=10000.0):
    return (base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()


def near(got, want, size, out, what=""):
    got = np64(got)
    assert np.isfinite(got).all()
    b = ROUND[out] * np.abs(want) + size * TURN * 1.01 + (2.0 ** -25 if out == "f16" else 2.0 ** -130)
    err = np.abs(got - want)
    assert (err <= b).all(), (what, float((err / b).max()))


def run_rope(ent, heads, types, rows, pairs, axes=None, interleaved=False, gain=1.0, seed=0, top=5000, low=0, joint=False, **more):
    h, kv, d = heads
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, h + kv, d, device="cuda", generator=g).to(TORCH[types[0]])
    q, k = x[:, :h], x[:, h:]
    if not joint:
        q, k = q.contiguous(), k.contiguous()
    f = freqs_of(pairs)
    n_axes = 1 if axes is None else max(axes) + 1
    pos = torch.randint(low, top, (n_axes, rows), dtype=torch.int32, device="cuda", generator=g)
    rot = ent.Rotary(f, axes=axes, interleaved=interleaved, gain=gain)
    got = ent.rope(rot, q, k, pos if n_axes > 1 else pos[0], dtype=TORCH[types[1]], **more)
    torch.cuda.synchronize()
    for a, b, what in zip(got, (q, k), "qk"):
        assert a.dtype == TORCH[types[1]] and a.shape == b.shape
        near(a, *oa.rotate(np64(b), pos.cpu().numpy(), f.cpu().numpy(), axes, interleaved, gain), types[1], what)
    return got


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_rope_matches_oracle(ent, heads, types, interleaved):
    say(f"rope {heads} {types} {interleaved}")
    d = heads[2]
    for rows, pairs in ((1, d // 2), (3, 8), (37, d // 4), (300, d // 2)):
        run_rope(ent, heads, types, rows, pairs, interleaved=interleaved, seed=rows)


@pytest.mark.parametrize("rows", [2047, 2048, 4099, 8193])
def test_rope_more_tokens_a_workgroup(ent, rows):
    say(f"rope of {rows} rows")
    run_rope(ent, (3, 1, 96), ("bf16", "bf16"), rows, 48)
    run_rope(ent, (14, 2, 64), ("f32", "f16"), rows, 16, interleaved=True)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_axes(ent, interleaved):
    say("rope on several axes")
    run_rope(ent, (8, 2, 128), ("bf16", "bf16"), 70, 64, axes=[0] * 16 + [1] * 24 + [2] * 24, interleaved=interleaved)
    run_rope(ent, (4, 4, 64), ("f32", "bf16"), 70, 32, axes=[i % 3 for i in range(32)], interleaved=interleaved)
    run_rope(ent, (6, 2, 96), ("f16", "f16"), 70, 24, axes=[3 - i // 6 for i in range(24)], interleaved=interleaved, gain=1.25)
    run_rope(ent, (4, 4, 64), ("f16", "f16"), 5, 8, axes=[1] * 8, gain=-0.5)


def test_rope_far_and_negative_positions(ent):
    """Positions up to the ends of 32 bits: the angle keeps its place in a turn."""
    say("rope: far positions")
    for low, top in ((2 ** 20, 2 ** 20 + 500), (2 ** 31 - 300, 2 ** 31 - 1), (-2 ** 31, -2 ** 31 + 300), (-400, 0)):
        run_rope(ent, (4, 2, 128), ("f32", "f16"), 90, 64, low=low, top=top)


def test_rope_joint_projection_and_one_operand(ent):
    say("rope: slices, one operand, outputs given, in place")
    run_rope(ent, (6, 2, 96), ("f32", "bf16"), 50, 48, joint=True)
    run_rope(ent, (6, 2, 96), ("bf16", "bf16"), 50, 48, joint=True)
    rot, pos = ent.Rotary(freqs_of(32)), ints(list(range(9)))
    x = torch.randn(9, 5, 64, device="cuda").to(torch.bfloat16)
    want = ent.rope(rot, x, x, pos)
    assert torch.equal(want[0], want[1])
    q, k = ent.rope(rot, x, None, pos)
    assert k is None and torch.equal(q, want[0])
    q, k = ent.rope(rot, None, x, pos)
    assert q is None and torch.equal(k, want[0])
    both = torch.full((11, 9, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    both[:9, 2:7] = x
    y = both[:9, 2:7]
    got = ent.rope(rot, y, None, pos, out=(y, None))[0]
    assert got.data_ptr() == y.data_ptr() and torch.equal(y, want[0])
    assert (both[9:] == 3).all() and (both[:9, :2] == 3).all() and (both[:9, 7:] == 3).all()
    for shape in ((0, 5, 64), (9, 0, 64)):
        assert ent.rope(rot, torch.empty(shape, dtype=torch.bfloat16, device="cuda"), None,
                        pos[: shape[0]])[0].shape == shape


def test_rope_special_values(ent):
    """An infinity or NaN reaches its pair alone; elements past the rotated ones stay."""
    say("rope: special values")
    x = torch.randn(3, 2, 64, device="cuda").to(torch.float16)
    x[0, 0, 3], x[1, 1, 20], x[2, 0, 50], x[2, 1, 63] = math.inf, math.nan, math.nan, -math.inf
    got = ent.rope(ent.Rotary(freqs_of(16)), x, None, ints([1, 2, 3]))[0]
    torch.cuda.synchronize()
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[0, 0, 3] = want[0, 0, 19] = want[1, 1, 20] = want[1, 1, 4] = want[2, 0, 50] = want[2, 1, 63] = True
    assert torch.equal(bad, want)
    assert torch.equal(got[:2, :, 32:], x[:2, :, 32:]) and got[2, 1, 63] == -math.inf


def test_rope_far_strides(ent):
    """Rows that lie past 2^32 bytes."""
    say("rope: offsets past 32 bits")
    big = torch.empty((1 << 31) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (5, 2, 64), (1 << 29, 64, 1))
    x.copy_(torch.randn(5, 2, 64, device="cuda"))
    rot, pos = ent.Rotary(freqs_of(32)), ints([5, 6, 7, 8, 9])
    want = ent.rope(rot, x.contiguous(), None, pos)[0]
    assert torch.equal(ent.rope(rot, x, None, pos)[0], want)
    ent.rope(rot, x, None, pos, out=(x, None))
    assert torch.equal(x, want)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def run_append(ent, heads, types, page, held, new, pairs, axes=None, interleaved=False, gain=1.0, seed=0, with_q=True, joint=False):
    """Appends and compares with the oracle: scales, codes old and new, queries."""
    h, kv, d = heads
    lens = [a + b for a, b in zip(held, new)]
    pages = sum(-(-n // page) for n in lens) + 2
    c = filled_cache(ent, kv, d, page, pages, seed)
    t = make_table(lens, page, pages, seed)
    g = torch.Generator(device="cuda").manual_seed(100 + seed)
    rows, total = sum(new) + 2, sum(new)
    x = torch.randn(rows, h + 2 * kv, d, device="cuda", generator=g)
    x[:, h + kv:] *= 3
    x = x.to(TORCH[types[0]])
    q, k, v = x[:, :h], x[:, h: h + kv], x[:, h + kv:]
    if not joint:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    f = freqs_of(pairs)
    rot = ent.Rotary(f, axes=axes, interleaved=interleaved, gain=gain)
    if axes is None:
        pos, places = None, [[p + i for p, n in zip(held, new) for i in range(n)]]
    else:
        pos = torch.randint(0, 3000, (max(axes) + 1, rows), dtype=torch.int32, device="cuda", generator=g)
        places = pos[:, :total].tolist()
    status = torch.zeros(len(held), dtype=torch.int32, device="cuda")
    before = arrays(c)
    q_out = torch.full((rows, h, d), 7.0, dtype=TORCH[types[1]], device="cuda") if with_q else None
    got = ent.kv_append(c, rot, k, v, torch.from_numpy(t).cuda(), ints(held), ints(running(new)), status, positions=pos,
                        q=q if with_q else None, q_out=q_out)
    torch.cuda.synchronize()
    assert not status.any()
    after = arrays(c)
    turn = lambda y: oa.rotate(np64(y)[:total], places, f.cpu().numpy(), axes, interleaved, gain)  # noqa: E731
    if with_q:
        assert got is q_out and (q_out[total:] == 7).all()
        near(got[:total], *turn(q), types[1], "q")
    else:
        assert got is None
    k64, k_size = turn(k)
    sides = ((0, 2, k64, k_size * TURN * 1.01, False), (1, 3, np64(v)[:total], np.zeros((total, kv, d)), True))
    cu = running(new)
    touched = set()
    for codes, scales, want, off, turned in sides:
        rows_of = lambda a, p: (a[p].transpose(0, 2, 1) if turned else a[p]).astype(np.float64)  # noqa: E731, B023
        for b in range(len(held)):
            for lead in range(held[b] // page * page, lens[b] if new[b] else 0, page):
                p, r0 = int(t[b, lead // page]), max(held[b] - lead, 0)
                r1 = min(page, lens[b] - lead)
                touched.add(p)
                i = slice(cu[b] + lead + r0 - held[b], cu[b] + lead + r1 - held[b])
                fresh, slack = want[i].transpose(1, 0, 2), off[i].transpose(1, 0, 2)       # [kv][rows][d]
                s0 = before[scales][p].astype(np.float64) if r0 else np.zeros(kv)
                s1 = after[scales][p].astype(np.float64)
                exp = np.maximum(s0, np.abs(fresh).max((1, 2)) / 127)
                assert (np.abs(s1 - exp) <= slack.max((1, 2)) / 127 + 2.0 ** -22 * exp).all()
                now, was = rows_of(after[codes], p), rows_of(before[codes], p)
                # half a step, in 32 bits (a code of at most 127 times 2^-22), and what the scale is off by
                half = (0.5 + 127 * 2.0 ** -21) * s1[:, None, None]
                err = np.abs(now[:, r0:r1] * s1[:, None, None] - fresh)
                assert (err <= half + slack + 127 * np.abs(s1 - exp)[:, None, None]).all(), ("new codes", turned)
                assert (np.abs(now[:, :r0] * s1[:, None, None] - was[:, :r0] * s0[:, None, None]) <= half).all(), ("codes held", turned)
                assert (now[:, r1:] == was[:, r1:]).all(), "rows behind the last were written"
    rest = [p for p in range(pages) if p not in touched]
    for a, b in zip(after, before):
        assert np.array_equal(a[rest], b[rest]), "other pages were written"


STORES = [
    ([0], [1]),
    ([0, 5, 0], [300, 1, 0]),
    ([15, 16, 17, 63, 64, 65], [1, 1, 1, 1, 1, 1]),
    ([7, 130, 33], [90, 64, 3]),
    ([127, 1, 40], [2, 15, 88]),
]


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [(4, 2, 64), (5, 1, 96), (6, 3, 128)], ids=str)
@pytest.mark.parametrize("case", range(len(STORES)))
def test_append_matches_oracle(ent, types, page, heads, case):
    say(f"append {heads} page {page} {types} {STORES[case]}")
    d = heads[2]
    run_append(ent, heads, types, page, *STORES[case], pairs=d // 2 if case % 2 else d // 4, seed=case, interleaved=case == 3)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_axes_and_slices(ent, interleaved):
    say("append: positions on three axes, slices, no queries")
    held, new = [7, 130, 33], [90, 64, 3]
    axes = [0] * 8 + [1] * 12 + [2] * 12
    run_append(ent, (14, 2, 64), ("bf16", "bf16"), 16, held, new, 32, axes=axes, interleaved=interleaved)
    run_append(ent, (14, 2, 64), ("f32", "f16"), 64, held, new, 32, axes=axes, interleaved=interleaved, joint=True, gain=1.5)
    run_append(ent, (6, 2, 96), ("f32", "bf16"), 32, held, new, 48, interleaved=interleaved, with_q=False)
    run_append(ent, (1, 1, 128), ("bf16", "f16"), 128, held, new, 8, axes=[0, 1] * 4, interleaved=interleaved, joint=True)


def test_append_many(ent):
    """More than 64 sequences, more queries' workgroups than pages, few workgroups."""
    say("append: 130 sequences")
    held, new = [(5 * i) % 70 for i in range(130)], [(3 * i) % 5 for i in range(130)]
    run_append(ent, (64, 1, 64), ("f32", "bf16"), 64, held, new, 32)
    run_append(ent, (8, 1, 128), ("bf16", "bf16"), 128, [0, 60], [2100, 30], 64)
    for cap in (1, 7):
        old = ent.set_max_workgroups(cap)
        try:
            run_append(ent, (8, 2, 64), ("f32", "bf16"), 32, held, new, 32)
            run_rope(ent, (8, 2, 64), ("f32", "bf16"), 100, 32)
        finally:
            ent.set_max_workgroups(old)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_without_a_turn_is_store(ent, dtype, page):
    """Where no pair turns (all angles zero) the codes and scales are the store's bit
    for bit, from 16 or 32 bits, special values of v among them; queries are copied."""
    say(f"append without a turn, {dtype}, pages of {page}")
    kv, d, held, new = 2, 96, [20, 0], [150, 33]
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(183, kv, d, device="cuda", generator=g).to(TORCH[dtype])
    v = (2 * torch.randn(183, kv, d, device="cuda", generator=g)).to(TORCH[dtype])
    v[3, 0, 5], v[44, 1, 6], v[150, 1, 7] = math.inf, -math.inf, math.nan
    v[155:183] *= 0
    q = torch.randn(183, 4, d, device="cuda", generator=g).to(TORCH[dtype])
    rot = ent.Rotary(torch.zeros(48, device="cuda"))
    got = []
    for how in ("store", "append", "append from 32 bits"):
        c = filled_cache(ent, kv, d, page, 16, 5)
        t = torch.from_numpy(make_table([170, 33], page, 16, 5)).cuda()
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        where = (t, ints(held), ints(running(new)), status)
        if how == "store":
            ent.kv_store(c, k, v, *where)
        elif how == "append":
            assert torch.equal(ent.kv_append(c, rot, k, v, *where, q=q), q)
        else:
            assert torch.equal(ent.kv_append(c, rot, k.float(), v.float(), *where, q=q.float(), dtype=TORCH[dtype]), q)
        torch.cuda.synchronize()
        assert not status.any()
        got.append(arrays(c))
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert np.array_equal(a, b)


def test_append_queries_are_rope(ent):
    say("append: queries as by rope, in place")
    q, k = (torch.randn(40, h, 128, device="cuda").to(torch.bfloat16) for h in (8, 2))
    rot = ent.Rotary(freqs_of(64))
    c = ent.KVCache.empty(4, 2, 128, 32)
    t, status = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2), torch.zeros(2, dtype=torch.int32, device="cuda")
    want = ent.rope(rot, q, None, ints([*range(3, 13), *range(30, 60)]))[0]
    got = ent.kv_append(c, rot, k, k, t, ints([3, 30]), ints([0, 10, 40]), status, q=q, q_out=q)
    assert got is q and torch.equal(q, want) and not status.any()


def test_append_flags(ent):
    """Lengths past the table and pages outside the cache are flagged; the other
    sequences are done and nothing else is written."""
    say("append: faults in the data")
    kv, d, page = 1, 64, 16
    t = make_table([40, 40, 40], page, 12, 2, spare=0)
    x = torch.randn(30, kv, d, device="cuda").to(torch.bfloat16)
    rot = ent.Rotary(freqs_of(32))
    place = np.arange(9).reshape(3, 3)
    for held, cu, table, flag, seq in (
        ([20, 20, 39], [0, 10, 20, 30], t, "length", 2),
        ([20, -1, 20], [0, 10, 20, 30], t, "length", 1),
        ([20, 20, 20], [0, 10, 20, 31], t, "length", 2),
        ([20, 20, 20], [0, 10, 5, 30], t, "length", 1),
        ([20, 20, 20], [0, 10, 20, 30], np.where(place == 7, 12, t), "page", 2),
        ([20, 20, 20], [0, 10, 20, 30], np.where(place == 7, -1, t), "page", 2),
    ):
        bad = {seq} | ({2} if cu[2] == 5 else set())      # one that begins before an earlier one's end
        c, e = (filled_cache(ent, kv, d, page, 12, 7) for _ in range(2))
        status = torch.zeros(3, dtype=torch.int32, device="cuda")
        q = torch.full((30, 2, d), 5.0, dtype=torch.bfloat16, device="cuda")
        ent.kv_append(c, rot, x, x, torch.from_numpy(np.ascontiguousarray(table.astype(np.int32))).cuda(), ints(held), ints(cu), status,
                      q=q, q_out=torch.empty_like(q))
        got = status.tolist()
        assert all(bool(got[b]) == (b in bad) for b in range(3)) and got[seq] == ent.FLAGS[flag]
        for b in range(3):
            if b not in bad:
                one = torch.zeros(1, dtype=torch.int32, device="cuda")
                ent.kv_append(e, rot, x[cu[b]: cu[b + 1]], x[cu[b]: cu[b + 1]], torch.from_numpy(t[b: b + 1]).cuda(), ints(held[b: b + 1]),
                              ints([0, cu[b + 1] - cu[b]]), one)
        torch.cuda.synchronize()
        fine = [p for b in range(3) if b not in bad for p in t[b]] + [p for p in range(12) if p not in t]
        for a, w in zip(arrays(c), arrays(e)):
            assert np.array_equal(a[fine], w[fine])


def test_far_cache_and_repeats(ent):
    """Pages whose codes lie past 4 GiB, and the same call again: bit for bit the
    same."""
    say("append: offsets past 32 bits, repeated calls")
    kv, d, page = 8, 128, 128
    pages = (1 << 32) // (kv * d * page) + 40
    c, small = ent.KVCache.empty(pages, kv, d, page), ent.KVCache.empty(3, kv, d, page)
    k, v, q = (torch.randn(300, h, d, device="cuda") for h in (kv, kv, 16))
    rot, status = ent.Rotary(freqs_of(64)), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for cache, first in ((c, pages - 3), (small, 0), (small, 0)):
        t = torch.arange(first, first + 3, dtype=torch.int32, device="cuda")[None]
        r = ent.kv_append(cache, rot, k, v, t, ints([0]), ints([0, 300]), status, q=q)
        got.append((r, *ent.kv_load(cache, t, ints([0]), ints([0, 300]), 300, status)))
    torch.cuda.synchronize()
    assert not status.any()
    for x in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], x))
    assert not c.k_codes[:1000].any() and not c.v_codes[:1000].any()
