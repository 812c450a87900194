"""GPU tests of the attention operators and the 8-bit key/value cache against
the oracle: codes, scales and values read back bit for bit, attention within
an error bound that follows from the roundings the operators state.

The bound of an output o (dim by dim), with A the weighted mean of |v|, u the
unit roundoff of the element type, w that of the weights in the product with
v (the element type for prompts, 2^-12 for the cache):

* the result's rounding: u |o|
* the weights' rounding: w A
* scores in 32 bits: the dot product's D roundings, the scaling's and
  subtraction's at the size of the score, 2^-21 for the exponential; that much
  relative error in each weight, in the sum above and the one below: 2 e A
* f16 weights reach down to 2^-39 of the largest, which the sum below is at
  least: n 2^-39 max |v|; f16 results to 2^-25.
"""
import math
import sys

import numpy as np
import pytest

from oracle import attention as oa

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HEADS = [(4, 4, 64), (6, 2, 96), (8, 2, 128), (7, 1, 64), (3, 3, 128)]
DTYPES = ["bf16", "f16"]
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # 8 and 11 significant bits, to nearest


def say(msg):
    print(f"[gpu-case] {msg}", file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


def np64(t):
    return t.detach().cpu().double().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def running(v):
    return [0] + [int(x) for x in np.cumsum(v)]


def bound(out, mean, top, q, kmax, vmax, n, dtype, weights, scale):
    """Error bound of outputs [rows][heads][dim] (see above); ``top``: the
    largest |score|, ``kmax``, ``vmax``: largest |k|, |v|."""
    d, scale = q.shape[2], abs(scale)
    dot = scale * np.abs(q).sum(2) * kmax * (d + 2) * 2.0 ** -24
    if weights == "cache" and dtype == "bf16":
        dot = dot + scale * d * np.abs(q).max(2) * kmax * 2.0 ** -24    # q in f16, 2^-25 of its row's largest
    e = dot + 8 * (top + 8) * 2.0 ** -24 + 2.0 ** -21
    u = ROUND[dtype]
    w = ROUND["f16"] if weights == "cache" else u
    b = u * np.abs(out) + ((w + 2 * e)[..., None] * mean) * 1.01
    if dtype == "f16" or weights == "cache":
        b = b + n * 2.0 ** -39 * vmax
    return b + (2.0 ** -25 if dtype == "f16" else 2.0 ** -130)


def near(a, b, dtype):
    a, b = np64(a), np64(b)
    assert (np.abs(a - b) <= 2 * ROUND[dtype] * np.abs(b) + 2.0 ** -18).all()


# ---------------------------------------------------------------------------
# prompts
# ---------------------------------------------------------------------------

def run_prompt(ent, heads, dtype, lq, lk, seed=0, edit=None, scale=None, joint=False, extra=3):
    """Runs packed sequences (with `extra` rows of no sequence behind them) and
    compares with the oracle; returns the outputs."""
    h, kv, d = heads
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows_q, rows_k = sum(lq) + extra, sum(lk) + extra
    if joint:   # slices of one joint projection: strided rows, 16-byte aligned
        assert lq == lk
        x = torch.randn(rows_q, h + 2 * kv, d, device="cuda", generator=g).to(TORCH[dtype])
        q, k, v = x[:, :h], x[:, h: h + kv], x[:, h + kv:]
    else:
        q = (1.5 * torch.randn(rows_q, h, d, device="cuda", generator=g)).to(TORCH[dtype])
        k = torch.randn(rows_k, kv, d, device="cuda", generator=g).to(TORCH[dtype])
        v = torch.randn(rows_k, kv, d, device="cuda", generator=g).to(TORCH[dtype])
    if edit:
        edit(q, k, v)
    cu_q, cu_k = running(lq), running(lk)
    status = torch.zeros(len(lq), dtype=torch.int32, device="cuda")
    out = torch.full((rows_q, h, d), 7.0, dtype=TORCH[dtype], device="cuda")
    ent.attn_prompt(q, k, v, ints(cu_q), ints(cu_k), status, scale=scale, out=out)
    torch.cuda.synchronize()
    assert not status.any()
    assert (out[sum(lq):] == 7.0).all(), "rows of no sequence were written"
    s = 1.0 / math.sqrt(d) if scale is None else scale
    exp, mean, top = oa.prompt(np64(q), np64(k), np64(v), cu_q, cu_k, s)
    got = np64(out)
    n = sum(lq)
    k64, v64 = np.abs(np64(k)[: sum(lk)]), np.abs(np64(v)[: sum(lk)])
    kmax = k64[np.isfinite(k64)].max(initial=0.0)
    vmax = v64[np.isfinite(v64)].max(initial=0.0)
    b = bound(exp[:n], mean[:n], top[:n], np64(q)[:n], kmax, vmax, max(lk + [0]), dtype, "prompt", s)
    assert np.isfinite(got[:n]).all()
    err = np.abs(got[:n] - exp[:n])
    assert (err <= b).all(), (heads, dtype, float((err / b).max()))
    return got[:n]


LENGTHS = [
    ([1], [1]),
    ([37], [37]),
    ([0, 1, 5, 0], [0, 1, 5, 0]),
    ([31, 32, 33, 64, 65], [31, 32, 33, 64, 65]),
    ([127, 1, 130], [127, 1, 130]),
    ([3, 40, 1], [70, 45, 200]),              # tokens in front of the queries
    ([5, 70, 2, 0], [3, 20, 0, 9]),           # fewer keys than queries: the first rows see nothing
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda x: "q" + "_".join(map(str, x[0])) + "-k" + "_".join(map(str, x[1])))
def test_prompt_matches_oracle(ent, heads, dtype, lengths):
    say(f"prompt {heads} {dtype} {lengths}")
    run_prompt(ent, heads, dtype, *lengths)


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_long(ent, dtype):
    say(f"prompt of 700 rows, {dtype}")
    run_prompt(ent, (2, 1, 128), dtype, [700], [700])
    run_prompt(ent, (2, 1, 64), dtype, [300, 299], [900, 555])
    run_prompt(ent, (2, 2, 96), dtype, [513], [513])


@pytest.mark.parametrize("heads", HEADS)
def test_prompt_last_tile_seen_whole(ent, heads):
    """One query behind a multiple of two tiles' keys: every tile is seen whole,
    and the outputs go out right behind the last one."""
    say(f"prompt: last tile seen whole, {heads}")
    run_prompt(ent, heads, "bf16", [1] * 40, [128 * (1 + i % 3) for i in range(40)])
    run_prompt(ent, heads, "f16", [1] * 9, [256] * 9)


SPLIT = [
    ([5], [1500]),
    ([1], [4097]),
    ([26, 1, 3], [3506, 1100, 2000]),
    ([3, 2, 7, 4], [5000, 0, 70, 129]),          # parts without tiles, rows without keys
    ([9, 30], [1024, 1024]),
    ([2, 0, 1], [1, 3000, 4000]),
    ([70], [2048]),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lengths", SPLIT, ids=lambda x: "q" + "_".join(map(str, x[0])) + "-k" + "_".join(map(str, x[1])))
def test_prompt_split_keys_match_oracle(ent, heads, dtype, lengths):
    """Few queries with many keys: the keys are split over workgroups."""
    say(f"prompt, keys split: {heads} {dtype} {lengths}")
    lq, lk = lengths
    assert ent.attn_prompt_work_bytes(len(lq), sum(lq) + 3, sum(lk) + 3, *heads) > 0
    run_prompt(ent, heads, dtype, lq, lk)


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_split_keys_hidden_and_given(ent, dtype):
    """Hidden infinities and NaN; workspace given, and none on a raw handle; the
    workgroup cap; another stream."""
    say(f"prompt, keys split: hidden values, workspace, {dtype}")
    h, kv, d = 8, 2, 128
    lq, lk = [20, 3], [2500, 1900]
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn(23, h, d, device="cuda", generator=g).to(TORCH[dtype])
    k, v = (torch.randn(4400, kv, d, device="cuda", generator=g).to(TORCH[dtype]) for _ in range(2))
    cq, ck, status = ints(running(lq)), ints(running(lk)), torch.zeros(2, dtype=torch.int32, device="cuda")
    want = ent.attn_prompt(q, k, v, cq, ck, status)
    size = ent.attn_prompt_work_bytes(2, 23, 4400, h, kv, d)
    assert size > 0
    work = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(ent.attn_prompt(q, k, v, cq, ck, status, work=work), want)
    with pytest.raises(ent.EntroError):
        ent.attn_prompt(q, k, v, cq, ck, status, work=work[:-16])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ent.attn_prompt(q, k, v, cq, ck, status, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    old = ent.set_max_workgroups(5)
    try:
        assert torch.equal(ent.attn_prompt(q, k, v, cq, ck, status), want)
    finally:
        ent.set_max_workgroups(old)
    whole = torch.empty_like(want)
    ent.attn_prompt(q, k, v, cq, ck, status, out=whole, stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    gap = np.abs(np64(whole) - np64(want)).max()
    # on each side the result is rounded, and weights that sum to 1 (scores and
    # sums in 32 bits: within a tenth of that)
    assert gap <= 2 * ROUND[dtype] * (np.abs(np64(want)).max() + 1.1 * np.abs(np64(v)).max())
    # the first sequence's queries 10 on see tokens 2490 on
    k[2490], v[2490], v[2495] = math.nan, math.inf, math.nan
    got = ent.attn_prompt(q, k, v, cq, ck, status)
    torch.cuda.synchronize()
    assert not status.any()
    near(got[:10], want[:10], dtype)
    near(got[20:], want[20:], dtype)
    assert not torch.isfinite(got[10:20]).all(-1).any()


def test_prompt_many_sequences(ent):
    say("prompt: 150 sequences")
    lq = [(7 * i) % 11 for i in range(150)]
    run_prompt(ent, (2, 1, 64), "bf16", lq, [x + (i % 3) for i, x in enumerate(lq)])


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_joint_projection(ent, dtype):
    say("prompt: slices of a joint projection")
    run_prompt(ent, (6, 2, 96), dtype, [50, 81], [50, 81], joint=True)
    run_prompt(ent, (4, 4, 64), dtype, [50, 81], [50, 81], joint=True)


def test_prompt_rows_without_keys_are_zero(ent):
    say("prompt: rows without keys")
    got = run_prompt(ent, (4, 2, 64), "bf16", [70, 9], [50, 0])
    assert (got[:20] == 0).all() and (got[70:] == 0).all() and (got[20:70] != 0).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 96, 128])
def test_prompt_hidden_values_have_no_influence(ent, dtype, d):
    """Infinities and NaN in keys and values that a query does not see: later
    tokens of its own sequence, other sequences, rows of none."""
    say(f"prompt: infinities and NaN in hidden places, {dtype} {d}")
    lens = [40, 100, 33]
    at = {40 + 37: math.inf, 40 + 70: math.nan, 40 + 99: -math.inf}

    def edit(q, k, v):
        k[173:], v[173:] = math.nan, math.inf            # rows of no sequence
        k[140:], v[140:] = math.nan, math.nan            # the whole third sequence
        for r, x in at.items():
            k[r], v[r] = x, x
            v[r, 0, 3] = math.nan

    h = (4, 2, d)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(176, h[0], d, device="cuda", generator=g).to(TORCH[dtype])
    k = torch.randn(176, h[1], d, device="cuda", generator=g).to(TORCH[dtype])
    v = torch.randn(176, h[1], d, device="cuda", generator=g).to(TORCH[dtype])
    cu = ints(running(lens))
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    clean = ent.attn_prompt(q, k, v, cu, cu, status)
    edit(q, k, v)
    got = ent.attn_prompt(q, k, v, cu, cu, status)
    torch.cuda.synchronize()
    assert not status.any()
    assert torch.isfinite(clean[:173]).all()
    # the same but for the order of 32-bit sums (at most one step of the result)
    near(got[:77], clean[:77], dtype)
    # the first query that sees one is no longer finite, nor are those after it
    assert not torch.isfinite(got[77:173]).all(-1).any()


def test_prompt_values_seen_may_be_infinite(ent):
    """An infinite value of token 5 reaches the queries from 5 on, in its own
    dimension only."""
    say("prompt: an infinite value")
    g = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (torch.randn(64, 1, 64, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    cu, status = ints([0, 64]), torch.zeros(1, dtype=torch.int32, device="cuda")
    clean = ent.attn_prompt(q, k, v, cu, cu, status)
    v[5, 0, 17] = math.inf
    got = ent.attn_prompt(q, k, v, cu, cu, status)
    same = torch.ones_like(got, dtype=torch.bool)
    same[5:, 0, 17] = False
    near(got[same], clean[same], "bf16")
    assert (got[5:, 0, 17] == math.inf).all()


def test_prompt_extreme_scores(ent):
    say("prompt: scores far apart")

    def edit(q, k, v):
        q.mul_(30)
        k[7].mul_(40)

    run_prompt(ent, (2, 1, 128), "bf16", [90], [90], edit=edit)
    run_prompt(ent, (2, 1, 128), "f16", [90], [90], edit=edit)
    run_prompt(ent, (2, 1, 64), "bf16", [90], [90], scale=0.0)
    run_prompt(ent, (2, 1, 64), "f16", [90], [90], scale=-0.25)


def test_prompt_small_weights_count_in_f16(ent):
    """One key far ahead of 3000 equal ones, its value zero: the others'
    weights are 2^-20 of it, and the result is theirs alone."""
    say("prompt: small weights, f16")
    n, d = 3001, 64
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.zeros(n, 1, d, device="cuda", dtype=torch.float16)
    k = torch.zeros_like(q)
    v = torch.randn(n, 1, d, device="cuda", generator=g).to(torch.float16)
    q[-1, 0, 0] = 20 * math.log(2)
    k[0, 0, 0] = 1.0
    v[0] = 0.0
    cu, status = ints([0, n]), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ent.attn_prompt(q, k, v, cu, cu, status, scale=1.0)[-1:]
    exp, mean, _ = oa.attend(np64(q)[-1, 0], np64(k)[:, 0], np64(v)[:, 0], 1.0)
    # weights and result 2^-11 each, or half of f16's smallest number
    err = np.abs(np64(got)[0, 0] - exp)
    assert (err <= 2.0 ** -10 * 1.02 * mean + 2.0 ** -25 + 8 * 22 * 2.0 ** -24 * mean).all()


def test_prompt_flags_bad_sums(ent):
    say("prompt: running sums that do not ascend")
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = (torch.randn(60, 2, 64, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    good = ent.attn_prompt(q, k, v, ints([0, 20, 60]), ints([0, 20, 60]), torch.zeros(2, dtype=torch.int32, device="cuda"))
    for cu in ([0, 20, 61], [0, 20, 10], [0, 20, -5], [0, 20, 2 ** 31 - 1]):
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        got = ent.attn_prompt(q, k, v, ints(cu), ints([0, 20, 60]), status)
        assert status.tolist() == [0, ent.FLAGS["length"]]
        assert torch.equal(got[:20], good[:20])
        status.zero_()
        got = ent.attn_prompt(q, k, v, ints([0, 20, 60]), ints(cu), status)
        assert status.tolist() == [0, ent.FLAGS["length"]]
        assert torch.equal(got[:20], good[:20])


# ---------------------------------------------------------------------------
# cache
# ---------------------------------------------------------------------------

PAGES = [16, 32, 64, 128]


def filled_cache(ent, kv, d, page, pages, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = ent.KVCache.empty(pages, kv, d, page)
    c.k_codes.copy_(torch.randint(-127, 128, c.k_codes.shape, device="cuda", generator=g))
    c.v_codes.copy_(torch.randint(-127, 128, c.v_codes.shape, device="cuda", generator=g))
    c.k_scales.copy_(0.01 + 0.03 * torch.rand(c.k_scales.shape, device="cuda", generator=g))
    c.v_scales.copy_(0.01 + 0.03 * torch.rand(c.v_scales.shape, device="cuda", generator=g))
    return c


def arrays(c):
    return [x.cpu().numpy() for x in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]


def make_table(lens, page, pages, seed, spare=1):
    """Pages in no order; entries past a sequence's pages point nowhere."""
    rng = np.random.default_rng(seed)
    ids = list(rng.permutation(pages))
    wide = max([-(-n // page) for n in lens] + [1]) + spare
    t = np.full((len(lens), wide), 2 ** 31 - 1, np.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            t[b, i] = ids.pop()
    return t


STORES = [
    ([0], [1]),
    ([0, 5, 0], [300, 1, 0]),
    ([15, 16, 17, 63, 64, 65], [1, 1, 1, 1, 1, 1]),
    ([7, 130, 33], [90, 64, 3]),
    ([127, 1, 40], [2, 15, 88]),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("heads", [(2, 64), (1, 96), (3, 128)])
@pytest.mark.parametrize("case", range(len(STORES)))
def test_store_matches_oracle(ent, dtype, page, heads, case):
    say(f"store {heads} page {page} {dtype} {STORES[case]}")
    (kv, d), (held, new) = heads, STORES[case]
    lens = [a + b for a, b in zip(held, new)]
    pages = sum(-(-n // page) for n in lens) + 2
    c = filled_cache(ent, kv, d, page, pages, case)
    t = make_table(lens, page, pages, case)
    g = torch.Generator(device="cuda").manual_seed(100 + case)
    rows = sum(new) + 2
    # some sequences grow their page's range, some do not
    k = torch.randn(rows, kv, d, device="cuda", generator=g).to(TORCH[dtype])
    v = (3 * torch.randn(rows, kv, d, device="cuda", generator=g)).to(TORCH[dtype])
    exp = oa.store(*arrays(c), k.float().cpu().numpy(), v.float().cpu().numpy(), t, held, running(new))
    status = torch.zeros(len(held), dtype=torch.int32, device="cuda")
    ent.kv_store(c, k, v, torch.from_numpy(t).cuda(), ints(held), ints(running(new)), status)
    torch.cuda.synchronize()
    assert not status.any()
    for got, want, what in zip(arrays(c), exp, ("key codes", "value codes", "key scales", "value scales")):
        assert np.array_equal(got, want), (what, int((got != want).sum()))
    # and back
    first = [min(h, 3) for h in held]
    count = [n - f for n, f in zip(lens, first)]
    out = [torch.full((sum(count) + 2, kv, d), 7.0, dtype=TORCH[dtype], device="cuda") for _ in range(2)]
    ent.kv_load(c, torch.from_numpy(t).cuda(), ints(first), ints(running(count)), sum(count) + 2, status, out=tuple(out))
    torch.cuda.synchronize()
    assert not status.any()
    want = [oa.rows_of(*exp, t[b], first[b], count[b]) for b in range(len(held))]
    for i in range(2):
        w = torch.from_numpy(np.concatenate([x[i] for x in want])).to(TORCH[dtype])
        assert torch.equal(out[i][: sum(count)].cpu(), w)
        assert (out[i][sum(count):] == 7.0).all(), "rows of no sequence were written"


@pytest.mark.parametrize("dtype", DTYPES)
def test_store_special_values(ent, dtype):
    """Infinities are limited, NaN becomes 0, and neither counts for the scale;
    a page of zeros, of denormals, and of infinities alone."""
    say(f"store: special values, {dtype}")
    d, page = 64, 16
    x = torch.randn(6 * page, 1, d).to(TORCH[dtype])
    x[3, 0, 5], x[4, 0, 6], x[5, 0, 7] = math.inf, -math.inf, math.nan
    x[page: 2 * page] = 0.0
    x[2 * page: 3 * page] = math.inf
    x[3 * page: 4 * page] = math.nan
    x[4 * page: 5 * page] *= 2.0 ** (-130 if dtype == "bf16" else -22)
    x = x.cuda()
    c = filled_cache(ent, 1, d, page, 8, 1)
    t = make_table([6 * page], page, 8, 1)
    xs = x.float().cpu().numpy()
    exp = oa.store(*arrays(c), xs, xs, t, [0], [0, 6 * page])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ent.kv_store(c, x, x, torch.from_numpy(t).cuda(), ints([0]), ints([0, 6 * page]), status)
    torch.cuda.synchronize()
    for got, want in zip(arrays(c), exp):
        assert np.array_equal(got, want)


def test_store_token_by_token(ent):
    """Single tokens one after another: the range grows again and again."""
    say("store: token by token")
    kv, d, page = 2, 128, 32
    c = ent.KVCache.empty(6, kv, d, page)
    t = make_table([70, 70], page, 6, 3)
    tt = torch.from_numpy(t).cuda()
    g = torch.Generator(device="cuda").manual_seed(4)
    exp = arrays(c)
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    for i in range(70):
        x = (torch.randn(2, kv, d, device="cuda", generator=g) * (1 + 0.2 * i)).to(torch.bfloat16)
        y = torch.randn(2, kv, d, device="cuda", generator=g).to(torch.bfloat16)
        exp = oa.store(*exp, x.float().cpu().numpy(), y.float().cpu().numpy(), t, [i, i], [0, 1, 2])
        ent.kv_store(c, x, y, tt, ints([i, i]), ints([0, 1, 2]), status)
    torch.cuda.synchronize()
    assert not status.any()
    for got, want in zip(arrays(c), exp):
        assert np.array_equal(got, want)


def test_store_strided_rows(ent):
    say("store: slices of a joint projection")
    kv, d, page = 2, 96, 64
    x = torch.randn(100, 3 * kv, d, device="cuda").to(torch.bfloat16)
    k, v = x[:, kv: 2 * kv], x[:, 2 * kv:]
    t = make_table([100], page, 4, 0)
    a, b = (filled_cache(ent, kv, d, page, 4, 0) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for c, kk, vv in ((a, k, v), (b, k.contiguous(), v.contiguous())):
        ent.kv_store(c, kk, vv, torch.from_numpy(t).cuda(), ints([0]), ints([0, 100]), status)
    torch.cuda.synchronize()
    for p, q in zip(arrays(a), arrays(b)):
        assert np.array_equal(p, q)


def test_cache_flags(ent):
    """Lengths past the table and pages outside the cache are flagged; the
    other sequences are done and nothing else is written."""
    say("cache: faults in the data")
    kv, d, page = 1, 64, 16
    t = make_table([40, 40, 40], page, 12, 2, spare=0)
    x = torch.randn(30, kv, d, device="cuda").to(torch.bfloat16)
    for held, cu, table, flag, seq in (
        ([20, 20, 39], [0, 10, 20, 30], t, "length", 2),
        ([20, -1, 20], [0, 10, 20, 30], t, "length", 1),
        ([20, 20, 20], [0, 10, 20, 31], t, "length", 2),
        ([20, 20, 20], [0, 10, 20, 30], np.where(np.arange(9).reshape(3, 3) == 7, 12, t), "page", 2),
        ([20, 20, 20], [0, 10, 20, 30], np.where(np.arange(9).reshape(3, 3) == 7, -1, t), "page", 2),
    ):
        c = filled_cache(ent, kv, d, page, 12, 7)
        before = arrays(c)
        status = torch.zeros(3, dtype=torch.int32, device="cuda")
        tt = torch.from_numpy(np.ascontiguousarray(table.astype(np.int32))).cuda()
        ent.kv_store(c, x, x, tt, ints(held), ints(cu), status)
        want = [0, 0, 0]
        want[seq] = ent.FLAGS[flag]
        assert status.tolist() == want
        xs = x.float().cpu().numpy()
        exp = before
        for b in range(3):
            if b != seq:
                exp = oa.store(*exp, xs, xs, t[b: b + 1], held[b: b + 1], [cu[b], cu[b + 1]])
        fine = [p for b in range(3) if b != seq for p in t[b]] + [p for p in range(12) if p not in t]
        for got, w in zip(arrays(c), exp):
            assert np.array_equal(got[fine], w[fine])
        status.zero_()
        ent.kv_load(c, tt, ints(held), ints(cu), 30, status)
        assert status.tolist() == want
        status.zero_()
        q = torch.randn(3, 2, d, device="cuda").to(torch.bfloat16)
        lens = [h + n for h, n in zip(held, np.diff(cu))]
        if flag == "length":
            lens[seq] = -3 if held[seq] < 0 else 49
        ent.attn_cache(q, c, tt, ints(lens), status)
        assert status.tolist() == want


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------

def run_cache(ent, heads, dtype, page, lens, seed=0, edit=None, scale=None, spare=1, check=None):
    h, kv, d = heads
    pages = sum(-(-n // page) for n in lens) + 2
    c = filled_cache(ent, kv, d, page, pages, seed)
    t = make_table(lens, page, pages, seed, spare)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (1.5 * torch.randn(len(lens), h, d, device="cuda", generator=g)).to(TORCH[dtype])
    if edit:
        edit(q, c, t)
    status = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    got = ent.attn_cache(q, c, torch.from_numpy(t).cuda(), ints(lens), status, scale=scale)
    torch.cuda.synchronize()
    assert not status.any()
    s = 1.0 / math.sqrt(d) if scale is None else scale
    a, out = arrays(c), np64(got)
    assert np.isfinite(out).all()
    q64 = np64(q)
    for b in range(len(lens)) if check is None else check:
        k, v = oa.rows_of(*a, t[b], 0, lens[b])
        for i in range(h):
            e, mean, top = oa.attend(q64[b, i], k[:, i // (h // kv)], v[:, i // (h // kv)], s)
            bb = bound(e[None, None], mean[None, None], np.array([[top]]), q64[b: b + 1, i: i + 1], np.abs(k).max(initial=0.0),
                       np.abs(v).max(initial=0.0), lens[b], dtype, "cache", s)[0, 0]
            err = np.abs(out[b, i] - e)
            assert (err <= bb).all(), (heads, dtype, page, lens[b], float((err / bb).max()))
    return got


CACHE_HEADS = HEADS + [(16, 1, 64), (17, 1, 128), (40, 1, 64), (32, 2, 96)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("heads", CACHE_HEADS)
def test_cache_attention_matches_oracle(ent, heads, dtype, page):
    say(f"cache attention {heads} page {page} {dtype}")
    run_cache(ent, heads, dtype, page, [1, 0, 2, 15, 16, 17, 63, 64, 65, 130, 200])
    run_cache(ent, heads, dtype, page, [3], spare=0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [(4, 4, 64), (6, 2, 96), (8, 2, 128), (20, 1, 128)])
def test_cache_attention_split(ent, heads, dtype):
    """Long and short sequences together: some are split, some are not."""
    say(f"cache attention split {heads} {dtype}")
    run_cache(ent, heads, dtype, 64, [5000, 3, 0, 700, 513, 512, 1])
    run_cache(ent, heads, dtype, 16, [2049])


def test_cache_attention_long(ent):
    say("cache attention: 70001 tokens")
    run_cache(ent, (4, 1, 128), "bf16", 64, [70001, 130])


def test_cache_attention_many_sequences(ent):
    say("cache attention: 200 sequences")
    run_cache(ent, (2, 1, 64), "f16", 32, [(37 * i) % 700 for i in range(200)], check=range(0, 200, 9))


@pytest.mark.parametrize("heads", [(2, 1, 64), (6, 3, 96), (8, 2, 128)])
def test_cache_attention_many_sequences_split(ent, heads):
    """More than 64 sequences, one long enough to be split; again with few
    workgroups."""
    say(f"cache attention: 130 sequences, split, {heads}")
    lens = [(53 * i) % 400 for i in range(129)] + [1700]
    run_cache(ent, heads, "bf16", 64, lens, check=[0, 1, 63, 64, 65, 77, 128, 129])
    old = ent.set_max_workgroups(7)
    try:
        run_cache(ent, heads, "f16", 32, lens, check=[0, 1, 63, 64, 65, 77, 128, 129])
    finally:
        ent.set_max_workgroups(old)


def test_cache_attention_split_graph_replays(ent):
    say("cache attention: graph replay of split sequences")
    kv, d, page = 2, 128, 64
    c = filled_cache(ent, kv, d, page, 70, 6)
    t = torch.from_numpy(make_table([3000, 500], page, 70, 0)).cuda()
    lens, status = ints([2900, 480]), torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 8, d, device="cuda", dtype=torch.bfloat16)
    out = torch.empty_like(q)
    work = torch.empty(ent.attn_cache_work_bytes(2, 8, kv, d), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ent.attn_cache(q, c, t, lens, status, out=out, work=work)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ent.attn_cache(q, c, t, lens, status, out=out, work=work)
    g = torch.Generator(device="cuda").manual_seed(4)
    for _ in range(4):
        q.copy_(torch.randn(q.shape, device="cuda", generator=g))
        graph.replay()
        got = out.clone()
        want = ent.attn_cache(q, c, t, lens, status)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        lens += 7
    assert not status.any()


def test_cache_attention_hidden_places(ent):
    """Scales of pages no token lies in, and codes behind the last token."""
    say("cache attention: hidden places")
    lens = [70, 17, 129]
    page = 32

    def spoil(q, c, t):
        used = {int(p) for b, n in enumerate(lens) for p in t[b, : -(-n // page)]}
        for p in range(c.k_scales.shape[0]):
            if p not in used:
                c.k_scales[p], c.v_scales[p] = math.nan, math.inf
        for b, n in enumerate(lens):
            p, r = int(t[b, n // page]), n % page
            if r:
                c.k_codes[p, :, r:], c.v_codes[p, :, :, r:] = 127, -128

    a = run_cache(ent, (4, 2, 64), "bf16", page, lens, seed=3)
    b = run_cache(ent, (4, 2, 64), "bf16", page, lens, seed=3, edit=spoil)
    assert torch.equal(a, b)


def test_cache_attention_extremes(ent):
    say("cache attention: extreme scales and queries")

    def wide(q, c, t):     # pages' scales far apart, one page of zeros
        c.v_scales.copy_(2.0 ** torch.arange(-8, c.v_scales.shape[0] - 8, device="cuda")[:, None].expand_as(c.v_scales) / 64)
        c.v_scales[int(t[0, 1])] = 0.0
        c.v_codes[int(t[0, 1])] = 0

    def big(q, c, t):
        q.mul_(50)

    def tiny(q, c, t):
        q.mul_(2.0 ** -60)

    for heads in ((4, 2, 64), (4, 1, 128)):
        run_cache(ent, heads, "bf16", 16, [150, 40], edit=wide)
        run_cache(ent, heads, "f16", 16, [150, 40], edit=wide)
        run_cache(ent, heads, "bf16", 16, [150, 40], edit=big)
        run_cache(ent, heads, "bf16", 16, [150, 40], edit=tiny, scale=2.0 ** 55)
        run_cache(ent, heads, "f16", 16, [150, 40], scale=0.0)
        run_cache(ent, heads, "f16", 16, [150, 40], scale=-0.2)


def test_cache_offsets_past_32_bits(ent):
    """Pages whose codes lie beyond 4 GiB of the cache's start."""
    say("cache: offsets past 32 bits")
    kv, d, page = 8, 128, 128
    pages = (1 << 32) // (kv * d * page) + 40
    c = ent.KVCache.empty(pages, kv, d, page)
    t = np.arange(pages - 3, pages, dtype=np.int32)[None]
    small = ent.KVCache.empty(3, kv, d, page)
    x = torch.randn(300, kv, d, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, 8, d, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for cache, table in ((c, t), (small, t - (pages - 3))):
        table = torch.from_numpy(np.ascontiguousarray(table)).cuda()
        ent.kv_store(cache, x, x, table, ints([0]), ints([0, 300]), status)
        got.append((*ent.kv_load(cache, table, ints([0]), ints([0, 300]), 300, status),
                    ent.attn_cache(q, cache, table, ints([300]), status)))
    torch.cuda.synchronize()
    assert not status.any()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert not c.k_codes[:1000].any() and not c.v_codes[:1000].any()


# ---------------------------------------------------------------------------
# streams, graphs, workgroup cap, whole path
# ---------------------------------------------------------------------------

def test_same_results_on_another_stream_and_capped(ent):
    say("attention: side stream, workgroup cap")
    g = torch.Generator(device="cuda").manual_seed(11)
    q = torch.randn(300, 8, 128, device="cuda", generator=g).to(torch.bfloat16)
    k, v = (torch.randn(300, 2, 128, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    cu = ints([0, 120, 121, 300])
    t = torch.from_numpy(make_table([600, 1201, 700], 32, 90, 0)).cuda()

    def everything(stream=None):
        c = filled_cache(ent, 2, 128, 32, 90, 5)
        status = torch.zeros(3, dtype=torch.int32, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        o = ent.attn_prompt(q, k, v, cu, cu, status, stream=stream)
        ent.kv_store(c, k, v, t, ints([480, 1200, 521]), cu, status, stream=stream)
        x, y = ent.kv_load(c, t, ints([0, 0, 0]), ints([0, 600, 1801, 2501]), 2501, status, stream=stream)
        r = ent.attn_cache(q[:3], c, t, ints([600, 1201, 700]), status, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        assert not status.any()
        return [o, x, y, r, c.k_codes, c.v_codes, c.k_scales, c.v_scales]

    want = everything()
    for a, b in zip(everything(torch.cuda.Stream()), want):
        assert torch.equal(a, b)
    old = ent.set_max_workgroups(24)
    try:
        got = everything()
    finally:
        ent.set_max_workgroups(old)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_graph_replays(ent):
    """A decode step (store, then attention) captured once and replayed with
    new inputs in place."""
    say("attention: graph replay")
    kv, d, page = 2, 128, 64
    t = torch.from_numpy(make_table([1000, 90], page, 24, 0)).cuda()
    c, e = (filled_cache(ent, kv, d, page, 24, 6) for _ in range(2))
    held, lens, cu = ints([700, 80]), ints([701, 81]), ints([0, 1, 2])
    q = torch.zeros(2, 8, d, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros(2, kv, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    work = torch.empty(ent.attn_cache_work_bytes(2, 8, kv, d), dtype=torch.uint8, device="cuda")

    def step(cache, out):
        ent.kv_store(cache, k, v, t, held, cu, status)
        return ent.attn_cache(q, cache, t, lens, status, out=out, work=work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(filled_cache(ent, kv, d, page, 24, 6), out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, out)
    g = torch.Generator(device="cuda").manual_seed(3)
    for i in range(5):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g) * (1 + i))
        graph.replay()
        got = out.clone()
        want = step(e, torch.empty_like(out))
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for a, b in zip(arrays(c), arrays(e)):
            assert np.array_equal(a, b)
        held += 1
        lens += 1
    assert not status.any()


def test_prompt_piece_by_piece(ent):
    """A prompt in two pieces, the first from the cache, against the whole: the
    same up to the cache's 8 bits."""
    say("attention: a prompt in pieces")
    h, kv, d = 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(12)
    q = torch.randn(200, h, d, device="cuda", generator=g).to(torch.bfloat16)
    k, v = (torch.randn(200, kv, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = ent.KVCache.empty(8, kv, d, 32)
    t = ints([3, 1, 7, 0, 5, 2, 6]).view(1, 7)
    ent.kv_store(c, k[:130], v[:130], t, ints([0]), ints([0, 130]), status)
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    ent.kv_load(c, t, ints([0]), ints([0, 130]), 130, status, out=(kk[:130], vv[:130]))
    kk[130:], vv[130:] = k[130:], v[130:]
    got = ent.attn_prompt(q[130:], kk, vv, ints([0, 70]), ints([0, 200]), status)
    exp, mean, top = oa.prompt(np64(q)[130:], np64(kk), np64(vv), [0, 70], [0, 200], 1 / 8)
    b = bound(exp, mean, top, np64(q)[130:], np64(kk).__abs__().max(), np64(vv).__abs__().max(), 200, "bf16", "prompt", 1 / 8)
    assert (np.abs(np64(got) - exp) <= b).all()
    # and its single tokens over the cache
    ent.kv_store(c, k[130:], v[130:], t, ints([130]), ints([0, 70]), status)
    one = ent.attn_cache(q[199:], c, t, ints([200]), status)
    assert not status.any()
    ks, vs = oa.rows_of(*arrays(c), t.cpu().numpy()[0], 0, 200)
    for i in range(h):
        e, m, tp = oa.attend(np64(q)[199, i], ks[:, i // 2], vs[:, i // 2], 1 / 8)
        bb = bound(e[None, None], m[None, None], np.array([[tp]]), np64(q)[199:, i: i + 1], np.abs(ks).max(), np.abs(vs).max(), 200,
                   "bf16", "cache", 1 / 8)[0, 0]
        assert (np.abs(np64(one)[0, i] - e) <= bb).all()


@pytest.mark.parametrize("shape", [(512, 8, 2, 64), (768, 8, 8, 96), (1024, 8, 2, 128)], ids=str)
def test_attention_block_example(ent, shape):
    """Coded q, k, v, o products around the cache and attention, against the
    float32 block.  A cached value is off by up to half a step of its page's
    range (its largest of 64 x dim values, about 4 sigma, by 127: 1.6% of
    sigma, uniform: 0.9% rms), keys twice rounded at most; bf16 operands add
    0.2% each: within 2% of the norm altogether."""
    say(f"attention block {shape}")
    import importlib.util
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(root, "examples", "attention_block.py"))
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    hidden, heads, kv, dim = shape
    err, _, _ = block.run(hidden, heads, kv, dim, prompt=150, new=9)
    assert err <= 0.02
