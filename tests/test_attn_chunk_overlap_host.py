"""Attention of chunks: outputs may not lie where the queries do, which workgroups that
share a block still read (no GPU needed: refused before anything is enqueued)."""
import ctypes

import pytest

import entropy_coded_weight_canonical_amd as ent
from tests.test_attn_chunk_host import INVAL, P, cache, chunk, rows, table


@pytest.fixture(scope="module")
def lib():
    return ent.load()


def call(lib, q, out):
    return lib.entro_attn_chunk(ctypes.byref(cache()), ctypes.byref(table()), ctypes.byref(chunk(q=q, out=out)), P, None)


# rows of 8 heads of 64 values of 2 bytes, 10 of them
@pytest.mark.parametrize("q,out", [
    (rows(P), rows(P)),                                      # the same place
    (rows(P, 1024), rows(P, 512)),                           # other strides
    (rows(P), rows(P + 16)),                                 # a part of it
    (rows(P), rows(P + 9 * 1024)),                           # its last row
    (rows(P + 9 * 1024), rows(P)),
])
def test_refused(lib, q, out):
    assert call(lib, q, out) == INVAL
