"""GPU tests of the attention of chunks at the largest sequences that a table of shared
pages can name: the last tile of 64 tokens ends at 2^31."""
import pytest

from tests.test_gpu_attn import ints, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def ent():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import entropy_coded_weight_canonical_amd as e

    e.load()
    return e


# 1 to 48 rows a sequence, to 128, and more: each kernel
@pytest.mark.parametrize("new", [3, 40, 100, 200])
def test_last_tile_of_the_longest_sequence(ent, new):
    """A token's score is the higher the later it is among the last ones, by far: each
    row gives its own token's value, which is its code times the scale.  The 16 tokens
    of the last tile that are past the sequence's end have page 0's keys, whose scores
    would be higher still."""
    say(f"chunk: {new} tokens at the end of 2^31")
    page, d = 16, 64
    pages = (1 << 27) - 1
    n = pages * page
    tail = 14                                       # pages of their own at the end: 224 tokens
    c = ent.KVCache.empty(tail + 2, 1, d, page)
    table = torch.ones(1, pages, dtype=torch.int32, device="cuda")
    table[0, pages - tail:] = torch.arange(2, tail + 2, dtype=torch.int32, device="cuda")
    # 8 (code of dim 0) + code of dim 1: tokens 0 .. 223 of the tail count up from 8 on, times 64
    # for the score; page 0: 320
    i = torch.arange(tail * page, device="cuda")
    c.k_codes[2:, 0, :, 0] = (i // 8 + 1).view(tail, page).to(torch.int8)
    c.k_codes[2:, 0, :, 1] = (i % 8).view(tail, page).to(torch.int8)
    c.k_codes[0, 0, :, 0] = 40
    c.k_scales.fill_(1.0)
    v = (i % 100 + 1).view(tail, page).to(torch.int8)
    c.v_codes[2:, 0] = v[:, None, :]
    c.v_codes[0], c.v_codes[1] = -128, -100
    c.v_scales.fill_(1.0)
    q = torch.zeros(new, 1, d, dtype=torch.float16, device="cuda")
    q[:, 0, 0], q[:, 0, 1] = 8.0, 1.0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ent.attn_chunk(q, c, table, ints([n]), ints([0, new]), status, scale=64.0)
    want = v.view(-1)[-new:].to(torch.float16)
    assert not status.any()
    assert torch.equal(out[:, 0], want[:, None].expand(new, d))
