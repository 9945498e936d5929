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


# --------------------------------------------------------------------------- tensors on other devices

class _Stream:
    cuda_stream = 0


def _on(torch, device, *tensors):
    """CPU tensors that say they are on GPU `device`."""
    class Placed(torch.Tensor):
        def get_device(self):
            return device
    return [t.as_subclass(Placed) for t in tensors]


@pytest.fixture
def calls(lib, monkeypatch):
    """What reaches the C ABI, with GPU 0 as the current one and nothing launched."""
    pytest.importorskip("torch")
    q4._first_use()
    seen = []
    monkeypatch.setattr(q4, "_call", lambda which, words: seen.append(which) or q4.OK)
    monkeypatch.setattr(q4, "_current", lambda: 0)
    return seen


def _operands(torch, move=None, to=-1):
    """Operands of every call, all on GPU 0 but for the one named by `move`."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    i32 = lambda *s: z(*s, dtype=torch.int32)
    made = dict(k8=z(2, 2, 16, 64, dtype=torch.int8), ka=z(2, 2, dtype=torch.float32), table=i32(1, 2),
                start=i32(2), length=i32(1), ws=z(1 << 20, dtype=torch.uint8), q=z(1, 4, 64), out=z(1, 4, 64),
                lse=z(1, 4, dtype=torch.float32), k=z(1, 2, 64), v=z(1, 2, 64), pos=i32(1),
                turns=z(16, dtype=torch.int64), w=z(64))
    return {n: _on(torch, to if n == move else 0, t)[0] for n, t in made.items()}


def _run(name, o):
    op = lambda: q4.QKNormRope(64, 32, o["turns"], o["w"], o["w"])
    cache = lambda: q4.KV8Cache(o["k8"], o["k8"], o["ka"], o["ka"])
    batch = lambda: q4.KV8Batch(o["table"], o["start"], o["length"], 1, 16)
    if name == "rope":
        return q4.lily_qk_norm_rope(op(), o["q"], o["k"], o["pos"], o["out"], o["v"], stream=_Stream)
    if name == "attention":
        return q4.lily_kv8_attention(cache(), batch(), o["q"], o["out"], 0.1, lse=o["lse"], ws=o["ws"], stream=_Stream)
    return getattr(q4, "lily_kv8_" + name)(cache(), batch(), o["k"], o["v"], ws=o["ws"], stream=_Stream)


USED = {"rope": ["q", "k", "pos", "out", "v", "turns", "w"],
        "append": ["k8", "ka", "table", "start", "length", "k", "v", "ws"],
        "read": ["k8", "ka", "table", "start", "length", "k", "v", "ws"],
        "attention": ["k8", "ka", "table", "start", "length", "q", "out", "lse", "ws"]}


@pytest.mark.parametrize("name", USED)
def test_tensors_have_to_be_on_the_current_gpu(calls, monkeypatch, name):
    import torch
    assert _run(name, _operands(torch)) == q4.OK and len(calls) == 1
    for move in USED[name]:
        for to in (-1, 1):
            with pytest.raises(q4.Q4Error) as e:
                _run(name, _operands(torch, move, to))
            assert e.value.status == q4.ERR_INVALID_ARG and len(calls) == 1, (move, to)
    monkeypatch.setattr(q4, "_current", lambda: 1)
    with pytest.raises(q4.Q4Error):
        _run(name, _operands(torch))
    assert len(calls) == 1


@pytest.mark.parametrize("name", USED)
def test_host_tensors_are_refused(calls, name):
    import torch
    o = {n: t.as_subclass(torch.Tensor) for n, t in _operands(torch).items()}
    with pytest.raises(q4.Q4Error) as e:
        _run(name, o)
    assert e.value.status == q4.ERR_INVALID_ARG and not calls


def test_a_rotation_without_tensors_takes_any_gpus_heads(calls):
    import torch
    o = _operands(torch)
    op = q4.QKNormRope(64, 0, None)
    assert q4.lily_qk_norm_rope(op, o["q"], None, None, o["out"], None, stream=_Stream) == q4.OK and len(calls) == 1


# --------------------------------------------------------------------------- one operator, two types

def test_one_rotation_serves_two_types_at_once(lib):
    """The struct that a call was given stays as it is when another thread takes the other type's."""
    torch = pytest.importorskip("torch")
    read = lambda at: q4.lily_qk_rope.from_address(at).dtype
    op = q4.QKNormRope(64, 32, torch.zeros(16, dtype=torch.int64))
    first, second = op.c(q4.BF16), op.c(q4.F16)
    assert (read(first), read(second)) == (q4.BF16, q4.F16)
    assert (op.c(q4.BF16), op.c(q4.F16)) == (first, second)
    for code, dtype in ((q4.BF16, torch.bfloat16), (q4.F16, torch.float16)):
        op = q4.QKNormRope(64, 32, torch.zeros(16, dtype=torch.int64), torch.ones(64, dtype=dtype))
        assert read(op.c(code)) == code
        with pytest.raises(q4.Q4Error) as e:
            op.c(q4.F16 if code == q4.BF16 else q4.BF16)
        assert e.value.status == q4.ERR_INVALID_ARG


# --------------------------------------------------------------------------- workspaces

def test_prompt_workspace_has_room_for_parts_that_there_can_be(lib):
    """Keys are split more than once an SM only where one sequence fills the SMs.  Many short prompts need no
    more than a part an SM: 152 of 256 rows of 128 outputs, a maximum and a sum, in fp32."""
    part = 256 * (128 + 2) * 4
    many = _size(lib, _cache(kv_heads=8), _batch(batch=100, max_q=300, max_kv=5000, table_pages=100), 30000, 32)
    one = _size(lib, _cache(kv_heads=8), _batch(batch=1, max_q=4096, max_kv=50000, table_pages=1000), 4096, 32)
    assert 152 * part <= many < 2 * 152 * part
    assert 8 * 152 * part <= one < 9 * 152 * part


def test_smaller_calls_need_no_more_space(lib):
    """Over a grid of bounds: fewer sequences, rows, tokens or keys never need more than the larger call."""
    grid = [(b, n, t, kv) for b in (1, 3, 20, 300) for n in (1, 7, 33, 97, 300, 2500) for t in (1, 40, 900, 20000)
            for kv in (20, 600, 9000, 200000)]
    for heads, group, D in ((1, 1, 64), (2, 8, 256), (8, 4, 128), (1, 48, 64), (16, 1, 256)):
        size = {}
        for b, n, t, kv in grid:
            size[b, n, t, kv] = _size(lib, _cache(kv_heads=heads, head_dim=D),
                                      _batch(batch=b, max_q=n, max_kv=kv, table_pages=1 << 14), t, heads * group)
        for at in grid:
            for axis in range(4):
                less = [g for g in grid if g[axis] < at[axis] and all(g[i] == at[i] for i in range(4) if i != axis)]
                if less:
                    assert max(size[g] for g in less) <= size[at], (heads, group, D, at, axis)
