"""Refusals of the attention calls' binding (no GPU needed): all tensors of a call
are on one device.  Tensors stand in for ones on two GPUs: they have a shape, a
type and a device, and no memory, and are refused before any would be read."""
import pytest

torch = pytest.importorskip("torch")

import entropy_coded_weight_canonical_amd as ent  # noqa: E402


class Placeless(torch.Tensor):
    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} of a tensor that is to be refused")


def on(gpu, *shape, dtype=torch.bfloat16):
    return torch.Tensor._make_wrapper_subclass(Placeless, shape, dtype=dtype, device=torch.device("cuda", gpu))


def ints(gpu, *shape):
    return on(gpu, *shape, dtype=torch.int32)


def cache_tensors(gpus=(0, 0, 0, 0)):
    a, b, c, d = gpus
    return (on(a, 4, 2, 16, 64, dtype=torch.int8), on(b, 4, 2, 64, 16, dtype=torch.int8),
            on(c, 4, 2, dtype=torch.float32), on(d, 4, 2, dtype=torch.float32))


def calls():
    """name, call, its tensors on one device."""
    rows = lambda h=2: on(0, 5, h, 64)  # noqa: E731
    return {
        "prompt": (lambda x: ent.attn_prompt(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], x["status"], out=x["out"], work=x["work"]),
                   dict(q=rows(8), k=rows(), v=rows(), cu_q=ints(0, 2), cu_k=ints(0, 2), status=ints(0, 1), out=rows(8),
                        work=on(0, 64, dtype=torch.uint8))),
        "store": (lambda x: ent.kv_store(x["cache"], x["k"], x["v"], x["table"], x["held"], x["cu_new"], x["status"]),
                  dict(cache=0, k=rows(), v=rows(), table=ints(0, 1, 4), held=ints(0, 1), cu_new=ints(0, 2), status=ints(0, 1))),
        "load": (lambda x: ent.kv_load(x["cache"], x["table"], x["first"], x["cu_out"], 5, x["status"], out=(x["k"], x["v"])),
                 dict(cache=0, table=ints(0, 1, 4), first=ints(0, 1), cu_out=ints(0, 2), status=ints(0, 1), k=rows(), v=rows())),
        "cache": (lambda x: ent.attn_cache(x["q"], x["cache"], x["table"], x["lens"], x["status"], out=x["out"], work=x["work"]),
                  dict(q=on(0, 1, 8, 64), cache=0, table=ints(0, 1, 4), lens=ints(0, 1), status=ints(0, 1), out=on(0, 1, 8, 64),
                       work=on(0, 64, dtype=torch.uint8))),
    }


NAMES = [(call, what) for call, (_, x) in calls().items() for what in x]


class Cache:
    """What the calls take of a KVCache, of one on the given GPU."""

    def __init__(self, gpu):
        import ctypes

        from entropy_coded_weight_canonical_amd import attn

        c = attn.Cache(1 << 20, 1 << 20, 1 << 20, 1 << 20, 4, 16, 2, 64)
        self.desc = bytes(c) + ctypes.c_int64(gpu)


@pytest.mark.parametrize("call,what", NAMES, ids=lambda x: x)
def test_one_tensor_on_another_device(call, what):
    fn, x = calls()[call]
    x = {k: Cache(0) if k == "cache" else v for k, v in x.items()}
    old = x[what]
    x[what] = Cache(1) if what == "cache" else on(1, *old.shape, dtype=old.dtype)
    with pytest.raises(ValueError, match="device"):
        fn(x)


@pytest.mark.parametrize("which", range(4))
def test_cache_of_two_devices(which):
    gpus = [0, 0, 0, 0]
    gpus[which] = 1
    with pytest.raises(ValueError, match="device"):
        ent.KVCache(*cache_tensors(gpus))


def test_cache_needs_its_description():
    fn, x = calls()["store"]
    x["cache"] = type("NoCache", (), {"desc": b"short"})()
    with pytest.raises(ValueError, match="KVCache"):
        fn(x)
