"""GPU tests of running sums that name rows twice: a sequence that begins before
an earlier one's end is flagged and left out, the others are done in full."""
import numpy as np
import pytest

from oracle import attention as oa
from tests.test_gpu_attn import arrays, filled_cache, ints, make_table, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


# running sums and the rows there are
SUMS = [
    ([0, 16] * 40, 16),
    ([0, 16] * 12 + [16, 40], 40),             # after them 16 .. 16 (empty) and 16 .. 40
    ([0, 30, 10, 20, 30, 50], 50),             # 10 .. 20 and 20 .. 30 lie within 0 .. 30
    ([0, 10, 99, 10, 20], 20),                 # a sum past the rows counts for its two sequences alone
    ([5, 10, -1, 10, 20], 20),
    ([0] * 70 + [8, 4, 8, 24], 24),            # found by later steps of 64 sequences
]


def sound(cu, total):
    """The sequences that the rule leaves, from its words."""
    ok, end = [], 0
    for b in range(len(cu) - 1):
        lo, hi = cu[b], cu[b + 1]
        if 0 <= lo <= total:
            end = max(end, lo)
        if 0 <= lo <= hi <= total and lo >= end:
            ok.append(b)
    return ok


@pytest.mark.parametrize("case", range(len(SUMS)))
def test_store_and_load_of_rows_named_twice(ent, case):
    cu, total = SUMS[case]
    say(f"store, load: rows named twice {cu[:6]} ...")
    n, page, kv, d = len(cu) - 1, 16, 2, 64
    fine = sound(cu, total)
    lens = [max(0, min(cu[b + 1], total) - max(cu[b], 0)) for b in range(n)]
    pages = sum(-(-x // page) + 1 for x in lens) + 2
    t = make_table([x + 1 for x in lens], page, pages, case)
    c = filled_cache(ent, kv, d, page, pages, case)
    before = arrays(c)
    g = torch.Generator(device="cuda").manual_seed(case)
    x = torch.randn(total, kv, d, device="cuda", generator=g).to(torch.bfloat16)
    tt, status = torch.from_numpy(t).cuda(), torch.zeros(n, dtype=torch.int32, device="cuda")
    zero = ints([0] * n)
    ent.kv_store(c, x, x, tt, zero, ints(cu), status)
    torch.cuda.synchronize()
    want = [0 if b in fine else ent.FLAGS["length"] for b in range(n)]
    assert status.tolist() == want
    exp, xs = before, x.float().cpu().numpy()
    for b in fine:
        exp = oa.store(*exp, xs, xs, t[b: b + 1], [0], [cu[b], cu[b + 1]])
    for got, w in zip(arrays(c), exp):
        assert np.array_equal(got, w)
    status.zero_()
    k, v = (torch.full((total, kv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ent.kv_load(c, tt, zero, ints(cu), total, status, out=(k, v))
    torch.cuda.synchronize()
    assert status.tolist() == want
    for b in fine:
        a, e = oa.rows_of(*exp, t[b], 0, lens[b])
        assert torch.equal(k[cu[b]: cu[b + 1]].cpu(), torch.from_numpy(a).to(torch.bfloat16))
        assert torch.equal(v[cu[b]: cu[b + 1]].cpu(), torch.from_numpy(e).to(torch.bfloat16))


@pytest.mark.parametrize("case", range(len(SUMS)))
def test_prompt_of_rows_named_twice(ent, case):
    """Sound sequences give what they give by themselves."""
    cu, total = SUMS[case]
    say(f"prompt: rows named twice {cu[:6]} ...")
    n = len(cu) - 1
    fine = sound(cu, total)
    g = torch.Generator(device="cuda").manual_seed(case)
    q, k, v = (torch.randn(total, 2, 64, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    lens = [max(0, min(cu[b + 1], total) - max(cu[b], 0)) for b in range(n)]
    # keys: each sequence its own
    ck = [0]
    for x in lens:
        ck.append(ck[-1] + x)
    at = [i for b in range(n) for i in range(max(cu[b], 0), max(cu[b], 0) + lens[b])]
    kk, vv = k[at], v[at]
    status = torch.zeros(n, dtype=torch.int32, device="cuda")
    got = ent.attn_prompt(q, kk, vv, ints(cu), ints(ck), status)
    torch.cuda.synchronize()
    assert status.tolist() == [0 if b in fine else ent.FLAGS["length"] for b in range(n)]
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    for b in fine:
        if lens[b]:
            r = slice(cu[b], cu[b + 1])
            alone = ent.attn_prompt(q[r], k[r], v[r], ints([0, lens[b]]), ints([0, lens[b]]), one)
            assert torch.equal(got[r], alone)
    assert not one.any()
