"""Attention operators, what needs no GPU: limits that keep the kernels' arithmetic in range, and what the
binding refuses before it launches anything."""
import ctypes as C

import pytest

import bit_affine_quantized_mlx_gb300 as q4
from bit_affine_quantized_mlx_gb300 import build as q4build
from test_kv8_cpu import _batch, _cache


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4.load()


def _size(lib, cache, batch, T, heads):
    return lib.lily_kv8_attention_workspace_bytes(C.byref(cache), C.byref(batch), T, heads)


def test_work_of_every_sequence_is_countable(lib):
    """Row ranges that go backwards can give the same row to 2048 of 4096 sequences, so the count of work
    covers all of them, not just as many as there are rows."""
    cache = _cache(kv_heads=65535, head_dim=256)
    assert _size(lib, cache, _batch(batch=4096, max_q=1, max_kv=1024, table_pages=16), 1, 65535) == 0
    assert _size(lib, cache, _batch(batch=1, max_q=1, max_kv=1024, table_pages=16), 1, 65535) > 0
    # a large server's largest call
    assert _size(lib, _cache(kv_heads=8), _batch(batch=4096, max_q=1, max_kv=1 << 20, table_pages=1 << 14), 4096, 64) > 0
