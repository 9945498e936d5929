"""Attention operators, what needs no GPU: the rotation table and the refusals, which come before
anything is launched."""
import ctypes as C
from fractions import Fraction

import numpy as np
import pytest

import bit_affine_quantized_mlx_gb300 as q4
from bit_affine_quantized_mlx_gb300 import build as q4build

FAKE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4.load()


@pytest.mark.parametrize("R,base", [(2, 10000.0), (64, 10000000.0), (128, 500000.0), (256, 1.5)])
def test_rope_turns(lib, R, base):
    t = q4.lily_rope_turns(R, base)
    f = base ** (-2.0 * np.arange(R // 2) / R)
    got = np.array([float(Fraction(int(x), 1 << 64)) for x in t]) * 2 * np.pi
    # pow, the division by 2 pi and its rounding: a few 2^-53 each, of a turn below one
    assert np.all(np.abs(got - f) <= 8 * 2.0 ** -53)


def test_rope_turns_scaling(lib):
    R, base = 128, 10000.0
    plain = q4.lily_rope_turns(R, base).astype(np.float64)
    linear = q4.lily_rope_turns(R, base, "linear", factor=4.0).astype(np.float64)
    # the table drops what is below one of its 2^64 steps: under 4 steps of 4 times an entry
    assert np.allclose(linear * 4, plain, rtol=1e-15, atol=4)
    yarn = q4.lily_rope_turns(R, base, "yarn", factor=4.0, original_len=4096).astype(np.float64)
    n = 4096 * plain / 2.0 ** 64  # turns within the original context
    assert np.array_equal(yarn[n >= 32], plain[n >= 32])
    assert np.allclose(yarn[n <= 1] * 4, plain[n <= 1], rtol=1e-15, atol=4)
    mid = (n > 1) & (n < 32)
    assert mid.sum() > 5
    keep = (n[mid] - 1) / 31
    assert np.allclose(yarn[mid], plain[mid] * (keep + (1 - keep) / 4), rtol=1e-13, atol=2)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=3), dict(rotary_dim=-2), dict(rotary_dim=258), dict(rotary_dim=64, base=0.0),
    dict(rotary_dim=64, base=float("nan")), dict(rotary_dim=64, scaling="linear", factor=0.0),
    dict(rotary_dim=64, scaling="yarn", factor=2.0, original_len=0.0),
    dict(rotary_dim=64, scaling="yarn", factor=2.0, original_len=10.0, slow=5.0, fast=5.0),
    dict(rotary_dim=64, scaling="other"),
])
def test_rope_turns_refuses(lib, kw):
    with pytest.raises(q4.Q4Error) as e:
        q4.lily_rope_turns(**kw)
    assert e.value.status == q4.ERR_INVALID_ARG


def _op(**kw):
    d = dict(head_dim=128, rotary_dim=64, interleaved=0, dtype=0, normalize=1, eps=1e-6,
             weight_offset=0.0, rope_scale=1.0, q_weight=FAKE, k_weight=FAKE, turns=FAKE)
    d.update(kw)
    return q4.lily_qk_rope(*d.values())


def _rope(lib, op, T=2, hq=4, hk=2, pos=FAKE, q=FAKE, ts=1024, hs=128, qo=FAKE, k=FAKE, ko=FAKE):
    return lib.lily_qk_norm_rope(C.byref(op) if op else None, T, hq, hk, pos, q, ts, hs, qo, 512, 128,
                                 k, 256, 128, ko, 256, 128, None)


@pytest.mark.parametrize("op,kw,want", [
    ({}, dict(T=0), q4.OK), ({}, dict(hq=0, hk=0), q4.OK),
    ({}, dict(T=-1), q4.ERR_INVALID_ARG), ({}, dict(hq=-1), q4.ERR_INVALID_ARG),
    (dict(head_dim=4), {}, q4.ERR_UNSUPPORTED), (dict(head_dim=264), {}, q4.ERR_UNSUPPORTED),
    (dict(head_dim=100), {}, q4.ERR_UNSUPPORTED), (dict(rotary_dim=130), {}, q4.ERR_INVALID_ARG),
    (dict(rotary_dim=3), {}, q4.ERR_INVALID_ARG), (dict(dtype=2), {}, q4.ERR_UNSUPPORTED),
    (dict(interleaved=2), {}, q4.ERR_INVALID_ARG), (dict(normalize=-1), {}, q4.ERR_INVALID_ARG),
    (dict(eps=-1.0), {}, q4.ERR_INVALID_ARG), (dict(eps=float("nan")), {}, q4.ERR_INVALID_ARG),
    (dict(q_weight=FAKE + 2), {}, q4.ERR_INVALID_ARG), (dict(turns=None), {}, q4.ERR_INVALID_ARG),
    ({}, dict(pos=None), q4.ERR_INVALID_ARG), ({}, dict(q=None), q4.ERR_INVALID_ARG),
    ({}, dict(q=FAKE + 8), q4.ERR_INVALID_ARG), ({}, dict(ts=1028), q4.ERR_INVALID_ARG),
    ({}, dict(hs=130), q4.ERR_INVALID_ARG), ({}, dict(qo=None), q4.ERR_INVALID_ARG),
    ({}, dict(k=None), q4.ERR_INVALID_ARG), ({}, dict(ko=FAKE + 4), q4.ERR_INVALID_ARG),
])
def test_norm_rope_refuses(lib, op, kw, want):
    assert _rope(lib, _op(**op), **kw) == want


def test_norm_rope_refuses_no_op(lib):
    assert _rope(lib, None) == q4.ERR_INVALID_ARG


def _cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_amax=FAKE, v_amax=FAKE, n_pages=100, kv_heads=2, page=64, head_dim=128)
    d.update(kw)
    return q4.lily_kv8_cache(*d.values())


def _batch(**kw):
    d = dict(block_table=FAKE, q_start=FAKE, kv_len=FAKE, table_pages=10, batch=3, max_q=4, max_kv=600)
    d.update(kw)
    return q4.lily_kv8_batch(*d.values())


CACHE_AND_BATCH = [
    (dict(k=None), {}, {}, q4.ERR_INVALID_ARG), (dict(v=FAKE + 8), {}, {}, q4.ERR_INVALID_ARG),
    (dict(k_amax=None), {}, {}, q4.ERR_INVALID_ARG), (dict(v_amax=FAKE + 2), {}, {}, q4.ERR_INVALID_ARG),
    (dict(n_pages=0), {}, {}, q4.ERR_INVALID_ARG), (dict(kv_heads=0), {}, {}, q4.ERR_INVALID_ARG),
    (dict(page=48), {}, {}, q4.ERR_UNSUPPORTED), (dict(page=256), {}, {}, q4.ERR_UNSUPPORTED),
    (dict(head_dim=96), {}, {}, q4.ERR_UNSUPPORTED), (dict(head_dim=512), {}, {}, q4.ERR_UNSUPPORTED),
    ({}, dict(block_table=None), {}, q4.ERR_INVALID_ARG), ({}, dict(q_start=FAKE + 1), {}, q4.ERR_INVALID_ARG),
    ({}, dict(kv_len=None), {}, q4.ERR_INVALID_ARG), ({}, dict(batch=-1), {}, q4.ERR_INVALID_ARG),
    ({}, dict(batch=0), {}, q4.ERR_INVALID_ARG), ({}, dict(batch=4097), {}, q4.ERR_UNSUPPORTED),
    ({}, dict(max_q=0), {}, q4.ERR_INVALID_ARG), ({}, dict(max_kv=-1), {}, q4.ERR_INVALID_ARG),
    ({}, dict(table_pages=0), {}, q4.ERR_INVALID_ARG),
    ({}, {}, dict(T=-1), q4.ERR_INVALID_ARG), ({}, {}, dict(T=0), q4.OK),
    ({}, {}, dict(dtype=3), q4.ERR_UNSUPPORTED), ({}, {}, dict(dtype=-1), q4.ERR_UNSUPPORTED),
    ({}, {}, dict(a=None), q4.ERR_INVALID_ARG), ({}, {}, dict(b=FAKE + 8), q4.ERR_INVALID_ARG),
    ({}, {}, dict(ts=1001), q4.ERR_INVALID_ARG), ({}, {}, dict(ws=None), q4.ERR_INVALID_ARG),
    ({}, {}, dict(ws=FAKE + 16), q4.ERR_INVALID_ARG),
    ({}, {}, dict(ws_bytes=128), q4.ERR_WORKSPACE_TOO_SMALL),
]


def _call(lib, name, cache, batch, T=6, dtype=0, a=FAKE, b=FAKE, ts=1024, ws=FAKE, ws_bytes=1 << 30,
          heads=8, scale=0.1, causal=1, window=0, lse=FAKE):
    head = [C.byref(cache), C.byref(batch), T]
    rows = [a, ts, 128, b, 1024, 128]
    if name == "attention":
        return lib.lily_kv8_attention(*head, heads, dtype, scale, causal, window, *rows, lse, ws, ws_bytes, None)
    return getattr(lib, "lily_kv8_" + name)(*head, dtype, *rows, ws, ws_bytes, None)


@pytest.mark.parametrize("name", ["append", "read", "attention"])
@pytest.mark.parametrize("cache,batch,kw,want", CACHE_AND_BATCH)
def test_kv8_refuses(lib, name, cache, batch, kw, want):
    assert _call(lib, name, _cache(**cache), _batch(**batch), **kw) == want


def test_types_of_each_call(lib):
    """fp32 rows are for read alone, and their strides count in fours."""
    assert _call(lib, "append", _cache(), _batch(), dtype=2) == q4.ERR_UNSUPPORTED
    assert _call(lib, "attention", _cache(), _batch(), dtype=2) == q4.ERR_UNSUPPORTED
    assert _call(lib, "read", _cache(), _batch(), dtype=2, ts=1002) == q4.ERR_INVALID_ARG


@pytest.mark.parametrize("kw,want", [
    (dict(heads=7), q4.ERR_INVALID_ARG), (dict(heads=0), q4.ERR_INVALID_ARG),
    (dict(heads=258), q4.ERR_UNSUPPORTED), (dict(causal=2), q4.ERR_INVALID_ARG),
    (dict(window=-1), q4.ERR_INVALID_ARG), (dict(scale=float("nan")), q4.ERR_INVALID_ARG),
    (dict(scale=float("inf")), q4.ERR_INVALID_ARG), (dict(lse=FAKE + 2), q4.ERR_INVALID_ARG),
    (dict(ws_bytes=256), q4.ERR_WORKSPACE_TOO_SMALL),
])
def test_attention_refuses(lib, kw, want):
    assert _call(lib, "attention", _cache(), _batch(), **kw) == want


def test_attention_workspace(lib):
    size = lambda c, b, T, h: lib.lily_kv8_attention_workspace_bytes(C.byref(c), C.byref(b), T, h)
    assert size(_cache(), _batch(), 6, 7) == 0
    assert size(_cache(page=8), _batch(), 6, 8) == 0
    assert size(_cache(), _batch(max_q=1, max_kv=1 << 30, batch=4096), 4096, 8) == 0  # uncountable
    last = 0
    for max_q, T in ((1, 3), (4, 12), (200, 600), (4096, 9000)):
        n = size(_cache(), _batch(max_q=max_q, max_kv=5000), T, 16)
        assert n >= last > -1
        last = n


def test_status_of_bad_indices(lib):
    assert "out of range" in q4.status_string(q4.ERR_INDEX)


# --------------------------------------------------------------------------- the packed call

def test_packed_call_forwards(lib):
    """The same statuses as the typed calls, from the words in their order."""
    import struct
    op, cache, batch = _op(), _cache(), _batch()
    rows = [FAKE, 1024, 128]
    rope = lambda T, q: struct.pack("18q", C.addressof(op), T, 4, 2, FAKE, q, 1024, 128, *rows, *rows, *rows, 0)
    assert lib.lily_q4_call(0, rope(0, 0)) == q4.OK
    assert lib.lily_q4_call(0, rope(2, 0)) == q4.ERR_INVALID_ARG
    for which in (1, 2):
        words = lambda T, dt, n: struct.pack("13q", C.addressof(cache), C.addressof(batch), T, dt, *rows, *rows, FAKE, n, 0)
        assert lib.lily_q4_call(which, words(0, 0, 256)) == q4.OK
        assert lib.lily_q4_call(which, words(6, 3, 256)) == q4.ERR_UNSUPPORTED
        assert lib.lily_q4_call(which, words(6, 0, 255)) == q4.ERR_WORKSPACE_TOO_SMALL
    att = lambda T, scale, n: struct.pack("5qd12q", C.addressof(cache), C.addressof(batch), T, 8, 0, scale, 1, 0,
                                          *rows, *rows, 0, FAKE, n, 0)
    assert lib.lily_q4_call(3, att(0, 0.1, 0)) == q4.OK
    assert lib.lily_q4_call(3, att(6, float("nan"), 1 << 30)) == q4.ERR_INVALID_ARG
    assert lib.lily_q4_call(3, att(6, 0.1, 256)) == q4.ERR_WORKSPACE_TOO_SMALL
    assert lib.lily_q4_call(4, att(0, 0.1, 0)) == q4.ERR_INVALID_ARG
    assert lib.lily_q4_call(0, None) == q4.ERR_INVALID_ARG


class _Stream:
    cuda_stream = 0


def _tensors():
    import torch
    cache = q4.KV8Cache.new(3, 2, 16, 64, device="cpu")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)
    batch = q4.KV8Batch(i32(0, 1).reshape(1, 2), i32(0, 1), i32(1), 1, 20)
    return torch, cache, batch


@pytest.mark.parametrize("bad", ["heads", "dim", "dtype", "mixed", "dense", "lse", "no workspace"])
def test_binding_refuses_attention(lib, bad):
    torch, cache, batch = _tensors()
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    out, lse, ws = q.clone(), torch.zeros((1, 4)), torch.zeros(1 << 20, dtype=torch.uint8)
    if bad == "heads":
        out = out[:, :3]
    elif bad == "dim":
        q, out = (torch.zeros((1, 4, 128), dtype=torch.bfloat16) for _ in "qo")
    elif bad == "dtype":
        q, out = q.float(), out.float()
    elif bad == "mixed":
        out = out.half()
    elif bad == "dense":
        q = torch.zeros((1, 64, 4), dtype=torch.bfloat16).transpose(1, 2)
    elif bad == "lse":
        lse = lse.double()
    else:
        ws = None
    with pytest.raises(q4.Q4Error):
        q4.lily_kv8_attention(cache, batch, q, out, 0.1, lse=lse, ws=ws, stream=_Stream)


def test_binding_refuses_the_rest(lib):
    torch, cache, batch = _tensors()
    ws = torch.zeros(256, dtype=torch.uint8)
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    for a, b in ((k[:, :1], k), (k, k.half()), (k.float(), k.float()), (k[..., :32], k[..., :32])):
        with pytest.raises(q4.Q4Error):
            q4.lily_kv8_append(cache, batch, a, b, ws=ws, stream=_Stream)
    op = q4.QKNormRope(64, 64, torch.zeros(32, dtype=torch.int64))
    pos = torch.zeros(1, dtype=torch.int32)
    for q, o, p in ((k, k, pos.long()), (k, k.half(), pos), (k, k[:, :1], pos), (k[..., :32], k[..., :32], pos),
                    (k, k, torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(q4.Q4Error):
            q4.lily_qk_norm_rope(op, q, None, p, o, None, stream=_Stream)
    with pytest.raises(q4.Q4Error):
        q4.QKNormRope(64, 64, torch.zeros(31, dtype=torch.int64))
    with pytest.raises(q4.Q4Error):
        q4.KV8Cache(cache.k, cache.v, cache.k_amax[:2], cache.v_amax)
    with pytest.raises(q4.Q4Error):
        q4.KV8Batch(torch.zeros((1, 2), dtype=torch.int64), pos, pos, 1, 1)
