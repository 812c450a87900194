"""GPU tests on the measured cases of perf/more_operators.py and on draws from their
ranges: rotary positions, the append to the 8-bit cache and the attention of chunks
over it against their definitions in 64 bits, and every call against itself.

The bounds are those of test_gpu_rope.py and test_gpu_attn_chunk.py, with what they
need of a case bounded from above: a pair's size by twice its largest element, a score
by the lengths of its query and the longest key, the weighted mean of |v| from the
definition on |v|.  A cached value whose quotient lies next to the border of two codes
may have either: it is off by one step of its page's scale at most.
"""
import random

import pytest

from tests.test_gpu_attn import say
from tests.test_gpu_rope import ROUND, TURN

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from perf import more_operators as ops  # noqa: E402

MOST = {"bytes": 1e9, "flops": 3e11}   # of a case: some seconds in 64 bits


def cases():
    out = ops.listed()
    rng = random.Random(515)
    while len(out) < 12 + 18:
        c = ops.draw(rng)
        if all(ops.work(c)[k] <= MOST[k] for k in MOST):
            c["name"] = f"drawn{len(out)}"
            out.append(c)
    return [c for c in out if all(ops.work(c)[k] <= MOST[k] for k in MOST)]


CASES = cases()


def of(op):
    return pytest.mark.parametrize("case", [c for c in CASES if c["op"] == op], ids=lambda c: c["name"])


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def run(s):
    ops.own = True
    try:
        return ops.run(s)
    finally:
        ops.own = False


def within(got, want, b, what):
    err = (got.double() - want).abs()
    assert got.shape == want.shape and torch.isfinite(got).all() and (err <= b).all(), (what, float((err / b).max()))


def turned(got, want, x, out, what):
    """Rotated rows; a head's largest element stands for each of its pairs."""
    size = 2 * x.double().abs().amax(-1, keepdim=True)
    tiny = 2.0 ** -25 if out == "f16" else 2.0 ** -130
    within(got, want, ROUND[out] * want.abs() + size * TURN * 1.01 + tiny, what)


@of("rope")
def test_rope_of_measured_cases(case):
    say(f"measured case {case}")
    s = ops.prepare(case, 7)
    got, again, want = run(s), run(s), ops.exact(case, 7)
    for a, b, e, x, what in zip(got, again, want, (s["q"], s["k"]), "qk"):
        assert torch.equal(a, b), "not the same in every call"
        turned(a, e, x, case["out"], what)


@of("append")
def test_append_of_measured_cases(case):
    say(f"measured case {case}")
    a, b = ops.prepare(case, 7), ops.prepare(case, 7)
    k_top, out = 2 * a["k"].double().abs().max() if a["k"].numel() else 0.0, case["out"]
    got, again, want = run(a), run(b), ops.exact(case, 7)
    torch.cuda.synchronize()
    assert not a["status"].any()
    for x, y in zip(got, again):
        assert torch.equal(x, y), "not the same in every call"
    turned(got[0], want[0], a["q"], out, "queries")
    # a scale is its largest magnitude (of a key: rotated) over 127, in 32 bits
    within(got[3], want[3], want[3] * 2.0 ** -22 + k_top * TURN * 1.01 / 127, "key scales")
    within(got[4], want[4], want[4] * 2.0 ** -22, "value scales")
    for i, name in ((1, "keys"), (2, "values")):
        # rows lie page after page of their sequence
        page, first, cu = case["page"], a["first"].tolist(), a["cu_out"].tolist()
        at = torch.cat([a["table"][b, (first[b] + torch.arange(cu[b + 1] - cu[b], device="cuda")) // page]
                        for b in range(len(first))]).long()
        step = want[i + 2][at][..., None]
        within(got[i], want[i], ROUND[out] * want[i].abs() + step * (1.0 + 2.0 ** -7 + ROUND[out]) + 2.0 ** -25, name)
        # ... and few do: most are off by their own rounding and the scale's alone
        off = (got[i].double() - want[i]).abs() > ROUND[out] * want[i].abs() + step * 2.0 ** -7 + 2.0 ** -25
        assert off.double().mean() <= 2.0 ** -8, (name, float(off.double().mean()))


@of("chunk")
def test_chunk_of_measured_cases(case):
    say(f"measured case {case}")
    s = ops.prepare(case, 7)
    got = run(s)
    for _ in range(3):
        assert torch.equal(run(s), got), "not the same in every call"
    assert not s["status"].any()
    want = ops._exact_chunk(s)
    mean = ops._exact_chunk({**s, "v_codes": s["v_codes"].abs()})
    lens, page = s["lens"].tolist(), case["page"]
    used = sorted({int(p) for b, n in enumerate(lens) for p in s["table"][b, : -(-n // page)].tolist()})
    q, scale, d, n = s["q"].double(), s["scale"], s["q"].shape[2], max(lens)
    longest = kmax = vmax = torch.zeros((), dtype=torch.float64, device="cuda")
    for part in torch.tensor(used, device="cuda").split(256):
        k = s["k_codes"][part].double() * s["k_scales"][part].double()[..., None, None]
        v = s["v_codes"][part].double().abs() * s["v_scales"][part].double()[..., None, None]
        longest, kmax, vmax = longest.maximum(k.norm(dim=-1).max()), kmax.maximum(k.abs().max()), vmax.maximum(v.max())
    dot = scale * q.abs().sum(2) * kmax * (d + 2) * 2.0 ** -24
    if case["dtype"] == "bf16":
        dot = dot + scale * d * q.abs().amax(2) * kmax * 2.0 ** -24
    log = s["v_scales"][used].double().log2().abs().max()
    e = dot + 8 * (scale * q.norm(dim=2) * longest + log + 64) * 2.0 ** -24 + 2.0 ** -20
    b = ROUND[case["dtype"]] * want.abs() + (2.0 ** -12 + 2 * e + (n / 16 + 4) * 2.0 ** -22)[..., None] * mean * 1.01
    within(got, want, b + n * 2.0 ** -35 * vmax + (2.0 ** -25 if case["dtype"] == "f16" else 2.0 ** -130), "chunk")
