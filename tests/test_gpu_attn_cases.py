"""GPU tests on the measured cases of perf/operators.py and on draws from their
ranges: attention against its definition in 64 bits, store and load against the
plain form bit for bit (both are defined in 32-bit arithmetic), and every call
against itself.

The bound of an attention's output is that of test_gpu_attn.py, with what it
needs of a case bounded from above: a score by the lengths of its query and the
longest key, the weighted mean of |v| from the definition on |v|.
"""
import random

import pytest

from tests.test_gpu_attn import ROUND, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from perf import operators as ops  # noqa: E402

MOST = {"bytes": 1e9, "flops": 3e11}   # of a case: some seconds in 64 bits


def cases():
    out = ops.listed()
    rng = random.Random(2024)
    while len(out) < 12 + 16:
        c = ops.draw(rng)
        if all(ops.work(c)[k] <= MOST[k] for k in MOST):
            c["name"] = f"drawn{len(out)}"
            out.append(c)
    return [c for c in out if all(ops.work(c)[k] <= MOST[k] for k in MOST)]


CASES = cases()


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def run(s, own):
    ops.own = own
    try:
        return ops.run(s)
    finally:
        ops.own = False


def attention_bound(s, out, mean, k, v, dtype, cache):
    """`k`, `v`: all keys and values of the case, in 64 bits."""
    q, scale, d = s["q"].double(), s["scale"], s["q"].shape[2]
    longest = k.norm(dim=-1).max()
    n = max(s["lens"].tolist()) if cache else s["most_k"]
    top = scale * q.norm(dim=2) * longest
    dot = scale * q.abs().sum(2) * k.abs().max() * (d + 2) * 2.0 ** -24
    if cache and dtype == "bf16":
        dot = dot + scale * d * q.abs().amax(2) * k.abs().max() * 2.0 ** -24
    e = dot + 8 * (top + 8) * 2.0 ** -24 + 2.0 ** -21
    if cache:   # logarithms of scales and sums, see test_gpu_attn_scales.py
        log = s["v_scales"].double().log2().abs().max()
        e = e + 8 * (log + 1.5 * top + 16) * 2.0 ** -24
    w = ROUND["f16"] if cache else ROUND[dtype]
    b = ROUND[dtype] * out.abs() + ((w + 2 * e)[..., None] * mean) * 1.01
    if dtype == "f16" or cache:
        b = b + n * 2.0 ** -39 * v.abs().max()
    return b + (2.0 ** -25 if dtype == "f16" else 2.0 ** -130)


@pytest.mark.parametrize("case", [c for c in CASES if c["op"] in ("prompt", "step")], ids=lambda c: c["name"])
def test_attention_of_measured_cases(case):
    say(f"measured case {case}")
    s = ops.prepare(case, 7)
    got = run(s, True)
    for _ in range(3):
        assert torch.equal(run(s, True), got), "not the same in every call"
    assert not s["status"].any()
    cache = case["op"] == "step"
    if cache:
        exact = ops._exact_step(s)
        used = sorted({int(p) for b, n in enumerate(s["lens"].tolist()) for p in s["table"][b, : -(-n // case["page"])].tolist()})
        k = (s["k_codes"][used].double() * s["k_scales"][used].double()[..., None, None]).flatten(0, 2)
        v = s["v_codes"][used].double() * s["v_scales"][used].double()[..., None, None]
        mean = ops._exact_step({**s, "v_codes": s["v_codes"].abs()})
    else:
        exact = ops._exact_prompt(s)
        k, v = s["k"].double(), s["v"].double()
        mean = ops._exact_prompt({**s, "v": s["v"].abs()})
    b = attention_bound(s, exact, mean, k, v, case["dtype"], cache)
    for what, x in (("kernels", got), ("plain form", run(s, False))):
        err = (x.double() - exact).abs()
        assert torch.isfinite(x).all() and (err <= b).all(), (what, float((err / b).max()))


@pytest.mark.parametrize("case", [c for c in CASES if c["op"] in ("store", "load")], ids=lambda c: c["name"])
def test_cache_of_measured_cases(case):
    say(f"measured case {case}")
    a, b, c = (ops.prepare(case, 7) for _ in range(3))
    got, again, want = run(a, True), run(b, True), run(c, False)
    torch.cuda.synchronize()
    assert not a["status"].any() and len(got) == len(want)
    for x, y, z in zip(got, again, want):
        assert torch.equal(x, z) and torch.equal(x, y)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert torch.equal(a[name], c[name])
