"""Host-side checks of the attention and cache entry points (no GPU needed):
every refusal comes before anything is enqueued, and the oracle's cache and
attention agree with their definitions."""
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


def rows(d=P, t=512, h=64):
    return attn.Rows(d, t, h)


def prompt(**change):
    a = attn.PromptArgs(rows(), rows(), rows(), rows(), P, P, 2, 10, 10, 8, 2, 64, 0, 0.125)
    for name, value in change.items():
        setattr(a, name, value)
    return a


def cache(**change):
    c = attn.Cache(P, P, P, P, 4, 64, 2, 64)
    for name, value in change.items():
        setattr(c, name, value)
    return c


def table(**change):
    t = attn.Table(P, 3, 3, 2)
    for name, value in change.items():
        setattr(t, name, value)
    return t


def store(**change):
    a = attn.StoreArgs(rows(), rows(), P, P, 10, 0)
    for name, value in change.items():
        setattr(a, name, value)
    return a


def over(**change):
    a = attn.CacheArgs(rows(), rows(), P, 8, 0, 0.125, P, 1 << 40)
    for name, value in change.items():
        setattr(a, name, value)
    return a


@pytest.mark.parametrize("change,want", [
    (dict(n_heads=7), INVAL), (dict(n_heads=0), INVAL), (dict(n_kv_heads=0), INVAL), (dict(head_dim=80), UNSUPPORTED),
    (dict(head_dim=256), UNSUPPORTED), (dict(n_heads=131072), UNSUPPORTED), (dict(dtype=2), INVAL), (dict(dtype=-1), INVAL),
    (dict(scale=float("nan")), INVAL), (dict(scale=float("inf")), INVAL), (dict(d_cu_q=None), INVAL), (dict(d_cu_k=None), INVAL),
    (dict(total_q=1 << 31), INVAL), (dict(total_k=1 << 31), INVAL), (dict(n_seq=1 << 31), INVAL),
    (dict(q=rows(None)), INVAL), (dict(q=rows(P + 8)), INVAL), (dict(k=rows(P, 516)), INVAL), (dict(v=rows(P, 512, 4)), INVAL),
    (dict(out=rows(P, -512)), INVAL), (dict(out=rows(None)), INVAL),
    (dict(n_seq=0), OK),
])
def test_prompt_refusals(lib, change, want):
    assert lib.entro_attn_prompt(ctypes.byref(prompt(**change)), P, None) == want


def test_null_arguments(lib):
    a, c, t = prompt(), cache(), table()
    assert lib.entro_attn_prompt(None, P, None) == INVAL
    assert lib.entro_attn_prompt(ctypes.byref(a), None, None) == INVAL
    for fn, x in (("entro_kv_store", store()), ("entro_kv_load", store()), ("entro_attn_cache", over())):
        f = getattr(lib, fn)
        assert f(None, ctypes.byref(t), ctypes.byref(x), P, None) == INVAL
        assert f(ctypes.byref(c), None, ctypes.byref(x), P, None) == INVAL
        assert f(ctypes.byref(c), ctypes.byref(t), None, P, None) == INVAL
        assert f(ctypes.byref(c), ctypes.byref(t), ctypes.byref(x), None, None) == INVAL


CACHE_CHANGES = [
    (dict(page_tokens=0), {}, FORMAT), (dict(page_tokens=48), {}, FORMAT), (dict(page_tokens=256), {}, FORMAT),
    (dict(head_dim=72), {}, UNSUPPORTED), (dict(n_kv_heads=0), {}, INVAL), (dict(n_kv_heads=65536), {}, UNSUPPORTED),
    (dict(n_pages=0), {}, INVAL), (dict(n_pages=1 << 31), {}, INVAL), (dict(d_k_codes=None), {}, INVAL),
    (dict(d_v_codes=P + 4), {}, INVAL), (dict(d_k_scales=None), {}, INVAL), (dict(d_v_scales=None), {}, INVAL),
    ({}, dict(d_table=None), INVAL), ({}, dict(table_pages=0), INVAL), ({}, dict(table_pages=4), INVAL),
    ({}, dict(table_pages=1 << 26, table_stride=1 << 26), UNSUPPORTED), ({}, dict(n_seq=0), OK),
]


@pytest.mark.parametrize("change_c,change_t,want", CACHE_CHANGES)
def test_cache_refusals(lib, change_c, change_t, want):
    c, t = cache(**change_c), table(**change_t)
    for fn, x in (("entro_kv_store", store()), ("entro_kv_load", store()), ("entro_attn_cache", over())):
        if fn == "entro_attn_cache" and change_c.get("n_kv_heads") == 65536:
            continue   # 8 query heads are no multiple of it: refused as such
        assert getattr(lib, fn)(ctypes.byref(c), ctypes.byref(t), ctypes.byref(x), P, None) == want, fn


@pytest.mark.parametrize("change", [dict(k=rows(P + 2)), dict(v=rows(P, 100)), dict(k=rows(None)), dict(d_pos=None), dict(d_cu=None),
                                    dict(total=1 << 31), dict(dtype=5)])
def test_store_and_load_refusals(lib, change):
    for fn in ("entro_kv_store", "entro_kv_load"):
        assert getattr(lib, fn)(ctypes.byref(cache()), ctypes.byref(table()), ctypes.byref(store(**change)), P, None) == INVAL


@pytest.mark.parametrize("change", [dict(q=rows(P + 4)), dict(out=rows(P, 512, 63)), dict(d_lens=None), dict(n_heads=9),
                                    dict(n_heads=0), dict(dtype=3), dict(scale=float("nan")), dict(d_work=None), dict(d_work=P + 8),
                                    dict(work_bytes=1000)])
def test_cache_attention_refusals(lib, change):
    assert lib.entro_attn_cache(ctypes.byref(cache()), ctypes.byref(table()), ctypes.byref(over(**change)), P, None) == INVAL


def test_prompt_workspace(lib):
    size = ent.attn_prompt_work_bytes
    assert size(0, 8, 8, 8, 2, 64) == 0 and size(1, 8, 8000, 7, 2, 64) == 0 and size(1, 8, 8000, 8, 2, 80) == 0
    assert size(1, 500, 500, 8, 2, 64) == 0 and size(64, 64, 64 * 1000, 8, 2, 64) == 0    # short ones
    assert size(1, 0, 8000, 8, 2, 64) == 0 and size(1, 8000, 8000, 32, 8, 128) == 0        # nothing, enough workgroups
    one = 32 * 130 * 4
    assert size(1, 1, 16000, 32, 8, 128) % one == 0 and size(1, 1, 16000, 32, 8, 128) // one > 8
    big = dict(total_q=1, total_k=16000, n_seq=1, n_heads=32, n_kv_heads=8, head_dim=128)
    need = size(1, 1, 16000, 32, 8, 128)
    for change in (dict(d_work=P, work_bytes=need - 1), dict(d_work=P, work_bytes=0), dict(d_work=P + 8, work_bytes=need)):
        assert lib.entro_attn_prompt(ctypes.byref(prompt(**big, **change)), P, None) == INVAL


def test_work_bytes():
    assert ent.attn_cache_work_bytes(0, 8, 2, 64) == 0
    assert ent.attn_cache_work_bytes(1, 8, 3, 64) == 0
    assert ent.attn_cache_work_bytes(1, 8, 2, 65) == 0
    one = ent.attn_cache_work_bytes(1, 32, 8, 128)
    assert 0 < one < 32 << 20
    assert ent.attn_cache_work_bytes(65, 32, 8, 128) - one == 64 * 32 * 130 * 4


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        ent.attn_prompt(x, x, x, cu, cu, cu[:2], out=x)
    with pytest.raises(ValueError, match="rows"):
        ent.attn_prompt(x, x, x[:3], cu, cu, cu[:2], out=x)
    with pytest.raises(ValueError):
        ent.KVCache.empty(2, 1, 64, 16, device="cpu")
    with pytest.raises(ValueError, match="four"):
        ent.KVCache(x, x, x, x)
    with pytest.raises(ValueError, match="tensor"):
        ent.attn_prompt([1.0], x, x, cu, cu, cu[:2])
    with pytest.raises(ValueError, match="GPU"):
        ent.attn_prompt(x, x, x, cu, cu, cu[:2])
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        ent.attn_prompt(x.float(), x.float(), x.float(), cu, cu, cu[:2], out=x)
    with pytest.raises(ValueError, match="do not belong together"):
        ent.KVCache(x[None], x[None], x[0], x[0])
    with pytest.raises(AttributeError):
        ent.kv_store(None, x, x, cu, cu, cu, cu)
    assert ent.FLAGS["length"] == 0x40 and ent.FLAGS["page"] == 0x80


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

def test_oracle_attention_by_hand():
    """Two keys with score difference ln 3: weights 1/4 and 3/4; the mean of
    equal values is the value; later tokens do not count."""
    q = np.array([1.0, 0.0])
    k = np.array([[0.0, 5.0], [np.log(3.0), -7.0]])
    v = np.array([[4.0, 1.0], [8.0, 1.0]])
    out, mean, top = oa.attend(q, k, v, 1.0)
    assert np.allclose(out, [7.0, 1.0]) and np.allclose(mean, [7.0, 1.0]) and np.isclose(top, np.log(3.0))
    got, _, _ = oa.prompt(q[None, None].repeat(2, 0), k[:, None], v[:, None], [0, 2], [0, 2], 1.0)
    assert np.allclose(got[0, 0], [4.0, 1.0]) and np.allclose(got[1, 0], [7.0, 1.0])
    assert not oa.attend(q, k[:0], v[:0], 1.0)[0].any()


def test_oracle_page_grows():
    f = np.float32
    codes = np.zeros((4, 2), np.int8)
    codes, s = oa.grow_page(codes, f(9.0), 0, np.array([[127.0, -64.0]], f))
    assert np.isclose(s, 1.0) and codes[0].tolist() == [127, -64]
    codes, s = oa.grow_page(codes, s, 1, np.array([[1.0, 254.0]], f))
    assert np.isclose(s, 2.0)
    assert codes[:2].tolist() == [[64, -32], [0, 127]]      # 63.5 and 0.5 to even
    codes, s2 = oa.grow_page(codes, s, 2, np.array([[np.inf, np.nan]], f))
    assert s2 == s and codes[2].tolist() == [127, 0]


def test_oracle_store_round_trip():
    rng = np.random.default_rng(0)
    page, kv, d = 16, 2, 64
    z = [np.zeros((5, kv, page, d), np.int8), np.zeros((5, kv, d, page), np.int8), np.zeros((5, kv), np.float32),
         np.zeros((5, kv), np.float32)]
    k, v = (rng.standard_normal((50, kv, d)).astype(np.float32) for _ in range(2))
    t = np.array([[4, 0, 2, 1]])
    z = oa.store(*z, k[:20], v[:20], t, [0], [0, 20])
    z = oa.store(*z, k[20:], v[20:], t, [20], [0, 30])
    kk, vv = oa.rows_of(*z, t[0], 0, 50)
    # half a step of the page's scale, twice where a code was rounded again
    assert np.abs(kk - k).max() <= 1.02 * z[2].max() and np.abs(vv - v).max() <= 1.02 * z[3].max()
