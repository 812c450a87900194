"""Host-side checks of the rotary positions, the append to the cache and the
attention of chunks (no GPU needed): every refusal comes before anything is
enqueued, and the oracle's rotation agrees with its definition."""
import ctypes

import numpy as np
import pytest

import entropy_coded_weight_canonical_amd as ent
from entropy_coded_weight_canonical_amd import attn
from oracle import attention as oa

OK, INVAL, FORMAT, UNSUPPORTED = 0, 1, 3, 4
P = 1 << 20   # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    return ent.load()


def changed(a, change):
    for name, value in change.items():
        setattr(a, name, value)
    return a


def rows(d=P, t=512, h=64):
    return attn.Rows(d, t, h)


def rotary(**change):
    return changed(attn.RotaryArg(P, 32, 1, (ctypes.c_uint32 * 4)(), 0, 1.0), change)


def rope(**change):
    return changed(attn.RopeArgs(rows(), rows(), rows(), rows(), P, 10, 10, 8, 2, 64, 2, 0), change)


def append(**change):
    return changed(attn.AppendArgs(rows(), rows(), rows(), rows(), P, P, P, 10, 10, 8, 2, 0), change)


def chunk(**change):
    return changed(attn.ChunkArgs(rows(), rows(), P, P, 10, 8, 0, 0.125, P, 1 << 40), change)


def cache(**change):
    return changed(attn.Cache(P, P, P, P, 4, 64, 2, 64), change)


def table(**change):
    return changed(attn.Table(P, 3, 3, 2), change)


def bits(*axes):
    """Pairs' axes as entro_rotary holds them."""
    w = [0] * 4
    for i, a in enumerate(axes):
        w[i // 16] |= a << (2 * (i % 16))
    return (ctypes.c_uint32 * 4)(*w)


ROTARY = [
    (dict(d_freqs=None), INVAL), (dict(d_freqs=P + 4), INVAL), (dict(pairs=0), INVAL), (dict(pairs=40), INVAL),
    (dict(pairs=12), UNSUPPORTED), (dict(n_axes=0), INVAL), (dict(n_axes=5), UNSUPPORTED), (dict(interleaved=2), INVAL),
    (dict(gain=float("nan")), INVAL), (dict(gain=float("inf")), INVAL), (dict(axes=bits(0, 1)), INVAL),
    (dict(n_axes=3, axes=bits(*[2] * 31, 3)), INVAL),
]


@pytest.mark.parametrize("change,want", ROTARY)
def test_rotary_refusals(lib, change, want):
    r = rotary(**change)
    assert lib.entro_rope(ctypes.byref(r), ctypes.byref(rope()), None) == want
    assert lib.entro_kv_append(ctypes.byref(cache()), ctypes.byref(table()), ctypes.byref(r), ctypes.byref(append()), P, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(head_dim=80), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(in_type=3), INVAL), (dict(in_type=-1), INVAL),
    (dict(out_type=2), INVAL), (dict(d_pos=None), INVAL), (dict(pos_stride=-1), INVAL), (dict(rows=1 << 31), INVAL),
    (dict(n_heads=65536), UNSUPPORTED), (dict(n_kv_heads=65536), UNSUPPORTED), (dict(q=rows(None)), INVAL),
    (dict(q_out=rows(P + 8)), INVAL), (dict(k=rows(P, 516)), INVAL), (dict(k_out=rows(P, 512, -64)), INVAL),
    (dict(rows=0), OK), (dict(n_heads=0, n_kv_heads=0), OK), (dict(rows=0, q=rows(None), d_pos=None), OK),
    (dict(n_heads=0, q=rows(None), q_out=rows(None), k=rows(None)), INVAL),
])
def test_rope_refusals(lib, change, want):
    assert lib.entro_rope(ctypes.byref(rotary()), ctypes.byref(rope(**change)), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(in_type=3), INVAL), (dict(out_type=2), INVAL), (dict(d_held=None), INVAL), (dict(d_cu_new=None), INVAL),
    (dict(total_new=1 << 31), INVAL), (dict(pos_stride=-1), INVAL), (dict(n_heads=65536), UNSUPPORTED), (dict(k=rows(None)), INVAL),
    (dict(v=rows(P, 100)), INVAL), (dict(q=rows(P + 2)), INVAL), (dict(q_out=rows(None)), INVAL),
])
def test_append_refusals(lib, change, want):
    c, t, r = cache(), table(), rotary()
    assert lib.entro_kv_append(ctypes.byref(c), ctypes.byref(t), ctypes.byref(r), ctypes.byref(append(**change)), P, None) == want


@pytest.mark.parametrize("change,want", [
    (dict(q=rows(P + 4)), INVAL), (dict(out=rows(P, 512, 63)), INVAL), (dict(out=rows(None)), INVAL), (dict(d_lens=None), INVAL),
    (dict(d_cu_q=None), INVAL), (dict(n_heads=9), INVAL), (dict(n_heads=0), INVAL), (dict(n_heads=131072), UNSUPPORTED),
    (dict(dtype=2), INVAL), (dict(dtype=-1), INVAL), (dict(scale=float("nan")), INVAL), (dict(scale=float("inf")), INVAL),
    (dict(d_work=None), INVAL), (dict(d_work=P + 8), INVAL), (dict(work_bytes=1000), INVAL), (dict(total_q=1 << 31), INVAL),
])
def test_chunk_refusals(lib, change, want):
    assert lib.entro_attn_chunk(ctypes.byref(cache()), ctypes.byref(table()), ctypes.byref(chunk(**change)), P, None) == want


@pytest.mark.parametrize("change_c,change_t,want", [
    (dict(page_tokens=0), {}, FORMAT), (dict(page_tokens=48), {}, FORMAT), (dict(head_dim=72), {}, UNSUPPORTED),
    (dict(n_kv_heads=0), {}, INVAL), (dict(n_pages=0), {}, INVAL), (dict(n_pages=1 << 31), {}, INVAL), (dict(d_k_codes=None), {}, INVAL),
    (dict(d_v_codes=P + 4), {}, INVAL), (dict(d_v_scales=None), {}, INVAL), ({}, dict(d_table=None), INVAL),
    ({}, dict(table_pages=0), INVAL), ({}, dict(table_pages=4), INVAL), ({}, dict(table_pages=1 << 26, table_stride=1 << 26), UNSUPPORTED),
    ({}, dict(n_seq=0), OK),
])
def test_cache_refusals(lib, change_c, change_t, want):
    c, t, r = cache(**change_c), table(**change_t), rotary()
    assert lib.entro_attn_chunk(ctypes.byref(c), ctypes.byref(t), ctypes.byref(chunk()), P, None) == want
    assert lib.entro_kv_append(ctypes.byref(c), ctypes.byref(t), ctypes.byref(r), ctypes.byref(append()), P, None) == want


def test_null_arguments(lib):
    c, t, r, x, y, z = (ctypes.byref(v) for v in (cache(), table(), rotary(), append(), chunk(), rope()))
    assert lib.entro_rope(None, z, None) == INVAL and lib.entro_rope(r, None, None) == INVAL
    for i in range(5):
        a = [c, t, r, x, P]
        a[i] = None
        assert lib.entro_kv_append(*a, None) == INVAL, i
    for i in range(4):
        a = [c, t, y, P]
        a[i] = None
        assert lib.entro_attn_chunk(*a, None) == INVAL, i


def test_work_bytes():
    size = ent.attn_chunk_work_bytes
    assert size(0, 8, 8, 2, 64) == 0 and size(1, 0, 8, 2, 64) == 0 and size(1, 8, 7, 2, 64) == 0 and size(1, 8, 8, 2, 80) == 0
    for heads in ((8, 2, 64), (32, 32, 96), (300, 1, 128), (65535, 1, 64)):
        for n, rows_ in ((1, 1), (16, 100), (3, 5000)):
            assert 0 < size(n, rows_, *heads) < 2 << 30


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    f, n = torch.zeros(32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="freqs"):
        ent.Rotary(f)
    with pytest.raises(ValueError, match="tensor"):
        ent.Rotary([1.0])
    with pytest.raises(AttributeError):
        ent.rope(None, x, x, n)
    no = type("NoPlan", (), {"desc": b"short"})()
    with pytest.raises(ValueError, match="Rotary"):
        ent.rope(no, x, x, n)
    with pytest.raises(ValueError, match="KVCache"):
        ent.kv_append(no, no, x, x, n, n, n, n)
    with pytest.raises(ValueError, match="KVCache"):
        ent.attn_chunk(x, no, n, n, n, n)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        ent.rope(no, x, x, n, dtype=torch.float32)
    with pytest.raises(ValueError, match="another type"):
        ent.rope(no, x, x, n, dtype=torch.float16, out=(x, x))
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        ent.rope(no, x.double(), None, n)


# ---------------------------------------------------------------------------
# refusals of the binding: tensors stand in for ones on a GPU, with a shape, a type
# and a device and no memory, and are refused before any would be read
# ---------------------------------------------------------------------------

def placed():
    torch = pytest.importorskip("torch")

    class Placeless(torch.Tensor):
        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise AssertionError(f"{func} of a tensor that is to be refused")

    def on(gpu, *shape, dtype=torch.bfloat16):
        return torch.Tensor._make_wrapper_subclass(Placeless, shape, dtype=dtype, device=torch.device("cuda", gpu))

    class Cache:
        def __init__(self, gpu=0):
            self.desc = bytes(attn.Cache(P, P, P, P, 4, 16, 2, 64)) + ctypes.c_int64(gpu)

    class Plan:
        def __init__(self, gpu=0, axes=1):
            self.desc = bytes(rotary(n_axes=axes)) + ctypes.c_int64(gpu)

    ints = lambda *s, gpu=0: on(gpu, *s, dtype=torch.int32)  # noqa: E731
    rows_ = lambda h=2, gpu=0, **k: on(gpu, 5, h, 64, **k)  # noqa: E731
    calls = {
        "rope": (lambda x: ent.rope(x["rotary"], x["q"], x["k"], x["positions"], out=(x["q_out"], x["k_out"])),
                 dict(rotary=Plan(), q=rows_(8), k=rows_(), positions=ints(5), q_out=rows_(8), k_out=rows_())),
        "append": (lambda x: ent.kv_append(x["cache"], x["rotary"], x["k"], x["v"], x["table"], x["held"], x["cu_new"], x["status"],
                                           positions=x["positions"], q=x["q"], q_out=x["q_out"]),
                   dict(cache=Cache(), rotary=Plan(), k=rows_(), v=rows_(), table=ints(1, 4), held=ints(1), cu_new=ints(2),
                        status=ints(1), positions=ints(5), q=rows_(8), q_out=rows_(8))),
        "chunk": (lambda x: ent.attn_chunk(x["q"], x["cache"], x["table"], x["lens"], x["cu_q"], x["status"], out=x["out"],
                                           work=x["work"]),
                  dict(q=rows_(8), cache=Cache(), table=ints(1, 4), lens=ints(1), cu_q=ints(2), status=ints(1), out=rows_(8),
                       work=on(0, 64, dtype=torch.uint8))),
    }
    return torch, on, Cache, Plan, calls


OPERANDS = {"rope": "rotary q k positions q_out k_out", "append": "cache rotary k v table held cu_new status positions q q_out",
            "chunk": "q cache table lens cu_q status out work"}


@pytest.mark.parametrize("call,what", [(c, w) for c, v in OPERANDS.items() for w in v.split()], ids=lambda x: x)
def test_one_tensor_on_another_device(call, what):
    torch, on, Cache, Plan, calls = placed()
    fn, x = calls[call]
    assert set(x) == set(OPERANDS[call].split())
    old = x[what]
    x[what] = Cache(1) if what == "cache" else Plan(1) if what == "rotary" else on(1, *old.shape, dtype=old.dtype)
    with pytest.raises(ValueError, match="device"):
        fn(x)


@pytest.mark.parametrize("call,change,match", [
    ("rope", dict(positions=(6,)), "positions"), ("rope", dict(positions=(2, 5)), "positions"), ("rope", dict(q=(5, 8, 96)), "shape"),
    ("rope", dict(k=(4, 2, 64)), "same rows"), ("rope", dict(q_out=(4, 8, 64)), "rows of q"), ("rope", dict(k_out=(5, 3, 64)), "shape"),
    ("append", dict(k=(5, 3, 64)), "shape"), ("append", dict(v=(4, 2, 64)), "same rows"), ("append", dict(q=(4, 8, 64)), "rows of k"),
    ("append", dict(q_out=(6, 8, 64)), "rows of q"), ("append", dict(cu_new=(3,)), "cu_new"), ("append", dict(held=(2,)), "held"),
    ("append", dict(status=(2,)), "status"), ("append", dict(positions=(4,)), "positions"), ("append", dict(table=(4,)), "held"),
    ("chunk", dict(q=(5, 8, 96)), "head dimension"), ("chunk", dict(q=(5, 64)), "rows"), ("chunk", dict(out=(4, 8, 64)), "rows of q"),
    ("chunk", dict(out=(5, 4, 64)), "shape"), ("chunk", dict(lens=(2,)), "lens"), ("chunk", dict(cu_q=(1,)), "cu_q"),
    ("chunk", dict(status=(3,)), "status"),
])
def test_shapes(call, change, match):
    torch, on, Cache, Plan, calls = placed()
    fn, x = calls[call]
    for name, shape in change.items():
        x[name] = on(0, *shape, dtype=x[name].dtype)
    with pytest.raises(ValueError, match=match):
        fn(x)


def test_types():
    torch, on, Cache, Plan, calls = placed()
    for call, name, dtype in (("rope", "q", torch.float64), ("rope", "k", torch.float32), ("rope", "positions", torch.int64),
                              ("append", "k", torch.int8), ("append", "v", torch.float32), ("append", "q", torch.float16),
                              ("chunk", "q", torch.float32), ("chunk", "out", torch.float16), ("chunk", "lens", torch.int64)):
        fn, x = placed()[4][call]
        x[name] = on(0, *x[name].shape, dtype=dtype)
        with pytest.raises(ValueError):
            fn(x)
    fn, x = placed()[4]["rope"]
    x["q"] = None
    with pytest.raises(ValueError, match="there is no q"):
        fn(x)
    x["q_out"] = x["k"] = x["k_out"] = None
    with pytest.raises(ValueError):
        ent.rope(x["rotary"], None, None, x["positions"], dtype=torch.bfloat16)


def test_gradients_are_refused():
    torch, on, Cache, Plan, calls = placed()
    for call, name in (("rope", "q"), ("append", "k"), ("chunk", "q")):
        fn, x = placed()[4][call]
        x[name].requires_grad_(True)
        with pytest.raises(ValueError, match="gradient"):
            fn(x)


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

def test_oracle_rotation_by_hand():
    """A quarter turn takes (x, y) to (-y, x); a whole number of them more is no
    different; position 0 turns nothing; what is no pair stays."""
    x = np.arange(1.0, 9.0)[None, None]            # pairs (1, 3), (2, 4) or (1, 2), (3, 4)
    f = np.float32(np.pi / 2)
    got, size = oa.rotate(x, [[1]], [f, 0.0])
    assert np.allclose(got[0, 0], [-3, 2, 1, 4, 5, 6, 7, 8], atol=1e-6) and size[0, 0].tolist() == [4, 6, 4, 6, 0, 0, 0, 0]
    got, _ = oa.rotate(x, [[1]], [f, 0.0], interleaved=True, gain=2.0)
    assert np.allclose(got[0, 0], [-4, 2, 6, 8, 5, 6, 7, 8], atol=1e-6)
    got, _ = oa.rotate(x, [[0], [3]], [f, f], axes=[0, 1])
    assert np.allclose(got[0, 0], [1, 4, 3, -2, 5, 6, 7, 8], atol=1e-6)


def test_oracle_rotation_keeps_relative_positions():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    f = 10000.0 ** (-np.arange(32) / 32)
    dots = [float((oa.rotate(q, [[p + 7]], f)[0] * oa.rotate(k, [[p]], f)[0]).sum()) for p in (0, 5, 1000)]
    assert np.allclose(dots, dots[0])
    assert np.allclose(np.linalg.norm(oa.rotate(q, [[9]], f)[0]), np.linalg.norm(q))


def test_oracle_chunk_is_prompt_over_its_tokens():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    a = oa.chunk(q, [k], [v], [9], [0, 5], 0.3)
    b = oa.prompt(q, k, v, [0, 5], [0, 9], 0.3)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))
    assert not oa.chunk(q, [k[:2]], [v[:2]], [2], [0, 5], 0.3)[0][:3].any()      # more queries than tokens
