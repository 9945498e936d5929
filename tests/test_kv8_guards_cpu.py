"""Attention operators, what needs no GPU: limits that keep the kernels' arithmetic in range, and what the
binding refuses before it launches anything."""
import ctypes as C
import struct

import pytest

import bit_affine_quantized_mlx_gb300 as q4
from bit_affine_quantized_mlx_gb300 import build as q4build
from test_kv8_cpu import _batch, _cache, _op


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


# --------------------------------------------------------------------------- numbers beyond 32 bits

@pytest.mark.parametrize("which,at,sizes", [(0, (1, 2, 3), 18), (1, (2, 3), 13), (2, (2, 3), 13), (3, (2, 3, 4, 6, 7), 18)])
def test_packed_call_refuses_wide_integers(lib, which, at, sizes):
    """A word whose low 32 bits would be a valid argument (T = 0 of them: nothing is launched)."""
    cache, batch, op = _cache(), _batch(), _op()
    words = [0] * sizes
    words[0] = C.addressof(op if which == 0 else cache)
    if which:
        words[1] = C.addressof(batch)
    if which == 3:
        words[3], words[5], words[6] = 8, struct.unpack("q", struct.pack("d", 0.1))[0], 1
    pack = lambda: struct.pack(f"{sizes}q", *words)
    assert lib.lily_q4_call(which, pack()) == q4.OK
    for i in at:
        for add in (1 << 32, -(1 << 32), 1 << 40):
            words[i] += add
            assert lib.lily_q4_call(which, pack()) == q4.ERR_INVALID_ARG, (i, add)
            words[i] -= add


def test_binding_refuses_wide_integers(lib):
    torch = pytest.importorskip("torch")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)
    wide = (1 << 32) + 5
    for kw in (dict(max_q=wide, max_kv=5), dict(max_q=5, max_kv=wide)):
        with pytest.raises(q4.Q4Error) as e:
            q4.KV8Batch(i32(0).reshape(1, 1), i32(0, 1), i32(1), **kw)
        assert e.value.status == q4.ERR_INVALID_ARG
    cache = q4.KV8Cache.new(3, 2, 16, 64, device="cpu")
    batch = q4.KV8Batch(i32(0).reshape(1, 1), i32(0, 1), i32(1), 1, 16)
    assert q4.lily_kv8_attention_workspace_bytes(cache, batch, 1, 4) > 0
    for T, heads in ((wide, 4), (1, (1 << 32) + 4)):
        with pytest.raises(q4.Q4Error):
            q4.lily_kv8_attention_workspace_bytes(cache, batch, T, heads)
    with pytest.raises(q4.Q4Error):
        q4.lily_rope_turns((1 << 32) + 64)
