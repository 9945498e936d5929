"""GPU tests of the attention operators (lily_qk_norm_rope, lily_kv8_append, lily_kv8_read,
lily_kv8_attention) against plain 64-bit forms.

Tolerances.  A result rounded to type t is off by finfo(t).eps / 2 of its value, or of the type's
smallest normal number where the value is below that.
Rotation: besides, fp32 products and sums of a pair (8 roundings of 2^-24) and the angle's
rounding (2^-24 of half a turn), of |a| + |b|.
Append: codes and magnitudes are those of exact arithmetic: equal.
Read: fp32, two roundings; then the output's.
Attention: the weight of a key is off by 2^-11 of itself (fp16), or 2^-25 of the largest
weight-times-magnitude where that is more; by the error of its score, 2^-21 of sum |q k| at most
(fp32 sums of the products, which may drop bits instead of rounding), twice (sum of weights too);
and by 2^-18 for exponentials and the fp32 sums of many weights."""
import numpy as np
import pytest

import bit_affine_quantized_mlx_gb300 as q4
import kv8_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    return torch


def _f64(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, tol, what):
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} {want[bad][0]} tolerance {np.broadcast_to(tol, got.shape)[bad][0]}")


# --------------------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("T,hq,hk,D,R,inter,dtype,norm,scaling", [
    (1, 1, 1, 64, 64, False, "bfloat16", True, "none"),
    (1, 16, 2, 256, 64, False, "bfloat16", True, "none"),
    (7, 5, 3, 128, 128, True, "float16", True, "yarn"),
    (3, 40, 8, 128, 128, False, "float16", False, "linear"),
    (400, 9, 1, 96, 48, False, "bfloat16", True, "none"),
    (33, 4, 4, 80, 50, False, "bfloat16", True, "none"),    # R / 2 odd: pairs across lanes
    (33, 4, 2, 80, 22, True, "float16", True, "none"),
    (700, 6, 2, 8, 4, False, "float16", True, "none"),
    (2, 3, 1, 40, 0, False, "bfloat16", True, "none"),
    (5, 48, 8, 256, 256, False, "bfloat16", True, "none"),
    (5, 2, 0, 192, 2, True, "bfloat16", True, "none"),
])
def test_norm_rope(torch, T, hq, hk, D, R, inter, dtype, norm, scaling):
    dt = getattr(torch, dtype)
    g = torch.Generator().manual_seed(T * 1000 + D + R)
    rows = (torch.randn((T, hq + 2 * hk + 1, D), generator=g) * 3).to(dt).cuda()
    q, k = rows[:, :hq], rows[:, hq:hq + hk]
    wq, wk = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt).cuda() for _ in range(2)]
    pos = torch.randint(0, 1 << 31, (T,), generator=g).to(torch.int32)
    pos[0] = (1 << 31) - 1
    if T > 2:
        pos[1], pos[2] = 0, -5
    kw = dict(scaling=scaling, factor=8.0, original_len=4096)
    turns = q4.lily_rope_turns(R, 500000.0, **kw)
    freq = turns.astype(np.float64) / 2.0 ** 64 * 2 * np.pi
    op = q4.QKNormRope(D, R, q4.to_device(turns), wq, wk if hk else None, eps=1e-5, interleaved=inter,
                       weight_offset=0.5, rope_scale=1.25, normalize=norm)
    qo = torch.full_like(q, 7)
    ko = torch.full_like(k, 7)
    q4.lily_qk_norm_rope(op, q, k if hk else None, pos.cuda(), qo, ko if hk else None)
    # the 64-bit angle: pos * turn in whole integers, so that the oracle loses nothing either
    ang = [(int(p) * int(t)) % (1 << 64) for p in pos for t in turns]
    ang = np.array(ang, dtype=np.float64).reshape(T, R // 2) / 2.0 ** 64 * 2 * np.pi
    for x, o, w, what in ((q, qo, wq, "q"), (k, ko, wk, "k")):
        if x.shape[1] == 0:
            continue
        want, size = plain.rope(_f64(x), _f64(w), 0.5, 1e-5, norm, freq * 0 + 1, np.zeros(T), inter, 1.0)
        y = want  # normalised, not turned; turn it by the exact angles
        a_at, b_at = ((np.arange(R // 2) * 2, np.arange(R // 2) * 2 + 1) if inter
                      else (np.arange(R // 2), np.arange(R // 2) + R // 2))
        a, b = y[..., a_at].copy(), y[..., b_at].copy()
        c, s = np.cos(ang)[:, None] * 1.25, np.sin(ang)[:, None] * 1.25
        y[..., a_at], y[..., b_at] = a * c - b * s, a * s + b * c
        tol = torch.finfo(dt).eps / 2 * np.abs(y) + (8 + 3.2) * 2.0 ** -24 * 1.25 * size + 2.0 ** -25
        _close(_f64(o), y, tol, what)
    # in place gives the same bits
    q2, k2 = q.clone(), k.clone()
    q4.lily_qk_norm_rope(op, q2, k2 if hk else None, pos.cuda(), q2, k2 if hk else None)
    assert torch.equal(q2, qo) and (hk == 0 or torch.equal(k2, ko))


def test_norm_rope_against_plain_angles(torch):
    """Small positions: the table's frequencies against base^(-2i/R) itself."""
    T, D, R = 50, 64, 32
    x = torch.randn((T, 2, D)).bfloat16().cuda()
    pos = torch.arange(T, dtype=torch.int32)
    op = q4.QKNormRope(D, R, q4.to_device(q4.lily_rope_turns(R, 10000.0)))
    out = torch.empty_like(x)
    q4.lily_qk_norm_rope(op, x, None, pos.cuda(), out, None)
    freq = 10000.0 ** (-np.arange(R // 2) / (R // 2))
    want, size = plain.rope(_f64(x), None, 0, 1e-6, True, freq, pos.numpy(), False, 1.0)
    _close(_f64(out), want, 2.0 ** -8 * np.abs(want) + 12 * 2.0 ** -24 * size, "rope")


# --------------------------------------------------------------------------- cache

class Setup:
    """Sequences of `old` tokens and `new` more: pages in random order, stale numbers everywhere
    that nothing may read (NaN magnitudes, wild page numbers)."""

    def __init__(self, torch, old, new, hk, D, page, dtype, seed=0, spare=3, first_page=0, total=None):
        rs = np.random.RandomState(seed)
        self.torch, self.page, self.hk, self.D = torch, page, hk, D
        self.dt = getattr(torch, dtype)
        self.old, self.new = np.array(old), np.array(new)
        self.len = np.maximum(self.old + self.new, 0)
        pages = -(-self.len // page)
        used = int(pages.sum())
        n = total or used + spare
        ids = first_page + rs.permutation(n - first_page)[:used]
        self.table = np.full((len(old), int(pages.max()) + 2), 1 << 30, np.int32)
        self.table[:, -1] = -7
        at = 0
        for b, p in enumerate(pages):
            self.table[b, :p] = ids[at:at + p]
            at += p
        self.codes = {x: np.zeros((n, hk, page, D), np.int8) for x in "kv"} if total is None else None
        self.amax = {x: np.full((n, hk), np.nan) for x in "kv"} if total is None else None
        self.q_start = np.concatenate([[0], np.cumsum(self.new)])
        self.T = int(self.new.sum())
        self.rs = rs
        if total is None:
            for x in "kv":
                self.codes[x][:] = rs.randint(-127, 128, self.codes[x].shape)
                for b, p in enumerate(pages):
                    own = self.table[b, :p]
                    mag = np.exp(rs.randn(p, hk) * (1.0 if x == "k" else 2.0))
                    self.amax[x][own] = self.rounded(mag)

    def rounded(self, x):
        return _f64(self.torch.from_numpy(np.asarray(x, np.float64)).to(self.dt))

    def rows(self, heads, scale=1.0):
        x = self.rs.randn(self.T, heads, self.D) * scale
        return self.torch.from_numpy(x).to(self.dt)

    def upload(self):
        t = self.torch
        up = lambda a, d: t.from_numpy(np.ascontiguousarray(a)).to(d).cuda()
        self.cache = q4.KV8Cache(up(self.codes["k"], t.int8), up(self.codes["v"], t.int8),
                                 up(self.amax["k"], t.float32), up(self.amax["v"], t.float32))
        self.batch = self.make_batch(self.q_start, int(self.new.max()))
        return self

    def make_batch(self, q_start, max_q, length=None):
        t = self.torch
        up = lambda a: t.from_numpy(np.ascontiguousarray(a)).to(t.int32).cuda()
        length = self.len if length is None else length
        return q4.KV8Batch(up(self.table), up(q_start), up(length), max_q, int(max(length)))


APPEND = [
    # old, new, hk, D, page, dtype
    ([0], [1], 1, 64, 16, "bfloat16"),
    ([5, 0, 16, 31, 100], [1, 1, 1, 1, 1], 2, 256, 16, "bfloat16"),
    ([3, 0, 7], [4, 0, 2], 3, 64, 32, "float16"),
    ([100, 0, 63, 64, 65], [37, 300, 0, 1, 200], 2, 128, 64, "bfloat16"),
    ([1, 2, 3, 127], [129, 500, 1, 2], 1, 256, 128, "float16"),
    ([0, 15], [17, 1000], 8, 128, 32, "float16"),
    ([7] * 70, [2] * 70, 1, 64, 16, "bfloat16"),
    ([9] * 40 + [0], [1] * 40 + [700], 2, 128, 128, "bfloat16"),
]


@pytest.mark.parametrize("old,new,hk,D,page,dtype", APPEND)
def test_append_and_read(torch, old, new, hk, D, page, dtype):
    s = Setup(torch, old, new, hk, D, page, dtype, seed=len(old) + D)
    # halves of the magnitude give exact ties; some pages grow, some do not, one head is all zeros
    kv = {x: s.rows(hk) * (0.05 if x == "k" else 3.0) for x in "kv"}
    for x in kv.values():
        x[..., 1::7] = x.abs().amax() / 2
        x[:, -1, :] *= 0 if hk > 1 else 1
    s.upload()
    view = torch.empty((s.T, 2 * hk + 1, D), dtype=s.dt).cuda()
    view[:, :hk], view[:, hk:2 * hk] = kv["k"].cuda(), kv["v"].cuda()
    ws = q4.new_workspace(256)
    q4.lily_kv8_append(s.cache, s.batch, view[:, :hk], view[:, hk:2 * hk], ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    for x, codes, amax in (("k", s.cache.k, s.cache.k_amax), ("v", s.cache.v, s.cache.v_amax)):
        plain.append(s.codes[x], s.amax[x], s.table, s.q_start, s.len, _f64(kv[x]))
        assert np.array_equal(amax.cpu().numpy(), s.amax[x].astype(np.float32), equal_nan=True)
        assert np.array_equal(codes.cpu().numpy(), s.codes[x])
    # the whole sequences read back, in every type
    start = np.concatenate([[0], np.cumsum(s.len)])
    every = s.make_batch(start, int(s.len.max()))
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        if dt == torch.float16 and dtype != "float16":
            continue
        k, v = (torch.full((int(start[-1]), hk + 1, D), 9, dtype=dt, device="cuda")[:, :hk] for _ in "kv")
        q4.lily_kv8_read(s.cache, every, k, v, ws=ws)
        for x, got in (("k", k), ("v", v)):
            want = np.concatenate([plain.values(s.codes[x], s.amax[x], s.table[b], n).transpose(1, 0, 2)
                                   for b, n in enumerate(s.len)])
            half = torch.finfo(dt).eps / 2
            _close(_f64(got), want, (half + 2.0 ** -24) * np.abs(want) + (2.0 ** -25 if dt == torch.float16 else 0), x)
    assert q4.lily_q4_workspace_status(ws) == q4.OK


def test_append_extreme_magnitudes(torch):
    """Magnitudes near both ends of bf16's range, and a page that turns non-finite."""
    s = Setup(torch, [4, 4, 0, 2], [2, 2, 2, 2], 1, 64, 16, "bfloat16").upload()
    x = s.rows(1)
    x[0:2] *= 1e-30
    x[2:4] = (x[2:4].double() / x[2:4].double().abs().max() * 3e38).to(s.dt)
    x[4:6] = (x[4:6].double() * 1e-39).to(s.dt)
    x[6, 0, 3], x[7, 0, 5] = float("inf"), float("nan")
    ws = q4.new_workspace(256)
    q4.lily_kv8_append(s.cache, s.batch, x.cuda(), x.cuda(), ws=ws)
    plain_codes, plain_amax = s.codes["k"].copy(), s.amax["k"].copy()
    plain.append(plain_codes, plain_amax, s.table[:3], s.q_start[:4], s.len[:3], _f64(x))
    own = s.table[:3, 0]
    assert np.array_equal(s.cache.k.cpu().numpy()[own], plain_codes[own])
    assert np.array_equal(s.cache.k_amax.cpu().numpy()[own], plain_amax[own].astype(np.float32))
    bad = int(s.table[3, 0])
    assert np.isnan(s.cache.k_amax[bad, 0].item())
    assert (s.cache.k[bad, 0, :4] == 0).all()


# --------------------------------------------------------------------------- attention

def expected(torch, s, q, b, scale, causal=True, window=0):
    """Output, lse and their tolerances of sequence b."""
    r0, r1, n = int(s.q_start[b]), int(s.q_start[b + 1]), int(s.len[b])
    k, v = (plain.values(s.codes[x], s.amax[x], s.table[b], n) for x in "kv")
    mag = np.repeat(s.amax["v"][s.table[b][:-(-n // s.page)]].T, s.page, 1)[:, :n]
    o, l, size, top, reach = plain.attention(_f64(q[r0:r1]), k, v, mag, scale, causal, window)
    d = 2.0 ** -21 * reach
    tol = (torch.finfo(s.dt).eps / 2 * np.abs(o) + (2.0 ** -11 + 2.0 ** -18 + 2 * d[..., None]) * size
           + n * 2.0 ** -25 * top[..., None]
           + torch.finfo(s.dt).smallest_normal * torch.finfo(s.dt).eps / 2)
    return o, l, tol, d + 2.0 ** -18 + 2.0 ** -22 * np.abs(np.where(np.isneginf(l), 0, l))


def check_attention(torch, s, hq, scale, causal=True, window=0, q=None, ws=None, stream=None):
    q = s.rows(hq, 1.5) if q is None else q
    view = torch.zeros((s.T, hq + 2, s.D), dtype=s.dt).cuda()
    view[:, 1:hq + 1] = q.cuda()
    out = torch.full((s.T, hq + 1, s.D), 7, dtype=s.dt, device="cuda")
    lse = torch.full((s.T, hq), 7.0, device="cuda")
    if ws is None:
        n = q4.lily_kv8_attention_workspace_bytes(s.cache, s.batch, s.T, hq)
        ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
        ws[:256] = 0  # only the header has to be clean
    torch.cuda.synchronize()
    q4.lily_kv8_attention(s.cache, s.batch, view[:, 1:hq + 1], out[:, :hq], scale, lse=lse,
                          causal=causal, window=window, ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    assert (out[:, hq] == 7).all()
    got, glse = _f64(out[:, :hq]), _f64(lse)
    for b in range(len(s.len)):
        r0, r1 = int(s.q_start[b]), int(s.q_start[b + 1])
        if r0 == r1:
            continue
        o, l, tol, ltol = expected(torch, s, q, b, scale, causal, window)
        _close(got[r0:r1], o, tol, f"out of sequence {b}")
        empty = np.isneginf(l)
        assert np.array_equal(empty, np.isneginf(glse[r0:r1]))
        _close(np.where(empty, 0, glse[r0:r1]), np.where(empty, 0, l), ltol, f"lse of sequence {b}")
    return out[:, :hq], lse


ATTENTION = [
    # old, new, hk, group, D, page, dtype, window, causal
    ([0], [1], 1, 1, 64, 16, "bfloat16", 0, True),
    ([776], [1], 2, 8, 256, 64, "bfloat16", 0, True),
    ([5000], [1], 1, 8, 128, 32, "float16", 0, True),
    ([15, 16, 17, 0, 1, 255, 256, 999], [1] * 8, 2, 4, 128, 16, "bfloat16", 0, True),
    ([15, 16, 17, 0, 1, 255, 256, 999], [1] * 8, 2, 8, 64, 128, "float16", 0, True),
    ([300, 0, 2000, 63], [3, 1, 0, 2], 1, 5, 256, 64, "bfloat16", 0, True),
    ([300, 10, 2000, 63], [3, 4, 1, 2], 2, 8, 128, 32, "bfloat16", 100, True),
    ([4000, 9, 0], [3, 3, 3], 6, 1, 64, 16, "float16", 64, True),
    ([900, 1], [2, 2], 1, 16, 256, 16, "float16", 0, True),
    ([900, 1], [8, 3], 2, 4, 128, 64, "bfloat16", 0, False),
    ([900, 31], [8, 3], 2, 3, 64, 64, "bfloat16", 17, False),
    ([500, 129], [40, 7], 2, 7, 256, 64, "bfloat16", 0, True),
    ([0, 129, 1000], [130, 70, 1], 2, 6, 128, 32, "float16", 0, True),
    ([0, 700], [300, 33], 1, 16, 64, 16, "bfloat16", 90, True),
    ([0], [257], 1, 1, 128, 128, "float16", 0, True),
    ([64, 5], [200, 64], 1, 48, 64, 32, "bfloat16", 0, True),
    ([3], [5], 1, 128, 64, 16, "float16", 0, True),
    ([1800], [310], 8, 8, 256, 64, "bfloat16", 0, True),    # one sequence fills the SMs: keys in halves
    ([1000, 0], [64, 200], 1, 3, 128, 16, "float16", 300, True),  # few row tiles in a window
    ([700], [97], 1, 1, 256, 32, "bfloat16", 0, True),      # heads of 256 from 97 rows, few sequences
    ([700], [96], 1, 1, 256, 32, "bfloat16", 0, True),
]


@pytest.mark.parametrize("old,new,hk,group,D,page,dtype,window,causal", ATTENTION)
def test_attention(torch, old, new, hk, group, D, page, dtype, window, causal):
    s = Setup(torch, old, new, hk, D, page, dtype, seed=len(old) * 7 + D + group).upload()
    check_attention(torch, s, hk * group, D ** -0.5, causal, window)


@pytest.mark.parametrize("D,new", [(64, 5), (128, 6), (256, 3), (128, 150), (256, 40), (64, 70)])
def test_attention_rows_that_see_nothing(torch, D, new):
    """Tokens at positions before the first (more rows than cached tokens), and a length of zero."""
    s = Setup(torch, [-2, -new, 40], [new, new, new], 2, D, 16, "bfloat16").upload()
    out, lse = check_attention(torch, s, 4, 0.3)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    assert (out[new:2 * new] == 0).all() and torch.isneginf(lse[new:2 * new]).all()


@pytest.mark.parametrize("new", [1, 60])
def test_attention_magnitudes_of_values(torch, new):
    """Value pages of very different size, all zeros among them: the small ones count where the
    softmax says so."""
    s = Setup(torch, [400], [new], 1, 128, 16, "bfloat16")
    own = s.table[0, :-(-int(s.len[0]) // 16)]
    s.amax["v"][own, 0] = s.rounded(10.0 ** s.rs.uniform(-6, 4, len(own)))
    s.amax["v"][own[3], 0] = 0
    s.amax["k"][own[5], 0] = 0
    s.amax["k"][own[7], 0] = 30.0  # scores that single out one small page
    s.amax["v"][own[7], 0] = s.rounded(1e-6)
    check_attention(torch, s.upload(), 4, 1.0)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_large_and_small_queries(torch, new):
    s = Setup(torch, [100], [new], 1, 64, 32, "bfloat16").upload()
    q = s.rows(8)
    q[:, 1] *= 1e4
    q[:, 2] *= 1e-20
    q[:, 3] = 0
    q[:, 4, 1:] *= 1e-12
    check_attention(torch, s, 8, 0.125, q=q)


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "bfloat16"), (256, "bfloat16")])
@pytest.mark.parametrize("growth", [1.05, 1.4, 3.0])
def test_prompt_form_growing_scores(torch, D, dtype, growth):
    # the rows' maxima rise from one 128-key tile to the next, by less and by more than 2^14
    s = Setup(torch, [1500], [70], 1, D, 128, dtype, seed=D)
    own = s.table[0, :-(-int(s.len[0]) // 128)]
    s.amax["k"][own, 0] = s.rounded(0.3 * np.minimum(growth ** np.arange(len(own)), 30.0))
    q = s.rows(5)
    q[:, 1] *= 0.05
    check_attention(torch, s.upload(), 5, 0.5, q=q)


def test_attention_repeats_bit_for_bit_and_on_another_stream(torch):
    for new in (1, 80):
        s = Setup(torch, [3000, 50, 700], [new] * 3, 2, 128, 32, "bfloat16").upload()
        q = s.rows(8)
        a = check_attention(torch, s, 8, 0.1, q=q)
        b = check_attention(torch, s, 8, 0.1, q=q, stream=torch.cuda.Stream())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("D,tokens", [(256, 310), (128, 310), (64, 310), (256, 40)])
def test_prompt_form_repeats_bit_for_bit(torch, D, tokens):
    # many blocks at once, whose products and conversions end in another order each time
    s = Setup(torch, [1800], [tokens], 8, D, 64, "float16", seed=D + tokens).upload()
    q = s.rows(64, 1.5).cuda()
    ws = q4.new_workspace(q4.lily_kv8_attention_workspace_bytes(s.cache, s.batch, s.T, 64))
    runs = []
    for _ in range(12):
        out = torch.empty((s.T, 64, D), dtype=s.dt, device="cuda")
        lse = torch.empty((s.T, 64), dtype=torch.float32, device="cuda")
        q4.lily_kv8_attention(s.cache, s.batch, q, out, D ** -0.5, lse=lse, ws=ws)
        runs.append((out, lse))
    torch.cuda.synchronize()
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])


@pytest.mark.parametrize("new", [1, 33])
def test_attention_graph_follows_lengths(torch, new):
    """A captured call replayed after the device's lengths changed."""
    s = Setup(torch, [600, 90], [new, new], 2, 128, 32, "bfloat16").upload()
    hq, q = 8, None
    q = s.rows(hq).cuda()
    out = torch.empty_like(q)
    lse = torch.empty((s.T, hq), device="cuda")
    ws = q4.new_workspace(q4.lily_kv8_attention_workspace_bytes(s.cache, s.batch, s.T, hq))
    call = lambda: q4.lily_kv8_attention(s.cache, s.batch, q, out, 0.1, lse=lse, ws=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([new + 1, 400][:1] + [new + 60], [new + 300, new]):
        s.batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        keep = s.len
        s.len = np.array(lens)
        want, wl = check_attention(torch, s, hq, 0.1, q=q.cpu())
        s.len = keep
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("new", [1, 90])
def test_far_pages(torch, new):
    """Pages beyond 2^32 bytes of codes."""
    hk, D, page = 1, 256, 128
    total = (1 << 32) // (hk * D * page) + 40
    s = Setup(torch, [300], [new], hk, D, page, "bfloat16", first_page=total - 20, total=total)
    codes = [torch.empty((total, hk, page, D), dtype=torch.int8, device="cuda") for _ in "kv"]
    amax = [torch.zeros((total, hk), dtype=torch.float32, device="cuda") for _ in "kv"]
    s.cache = q4.KV8Cache(*codes, *amax)
    s.batch = s.make_batch(s.q_start, new)
    # written by append from nothing, checked by read and attention
    n = int(s.len[0])
    fill = s.make_batch([0, n], n)
    x = {y: torch.from_numpy(s.rs.randn(n, hk, D)).to(s.dt) for y in "kv"}
    ws = q4.new_workspace(256)
    q4.lily_kv8_append(s.cache, fill, x["k"].cuda(), x["v"].cuda(), ws=ws)
    ids = s.table[0, :-(-n // page)].copy()
    s.table[0, :len(ids)] = np.arange(len(ids))
    s.codes = {y: np.zeros((len(ids), hk, page, D), np.int8) for y in "kv"}
    s.amax = {y: np.zeros((len(ids), hk)) for y in "kv"}
    for i, y in enumerate("kv"):
        plain.append(s.codes[y], s.amax[y], s.table, [0, n], [n], _f64(x[y]))
        got = codes[i][torch.from_numpy(ids).long().cuda()].cpu().numpy()
        tail = n - (len(ids) - 1) * page
        assert np.array_equal(got[:-1], s.codes[y][:-1]) and np.array_equal(got[-1, :, :tail], s.codes[y][-1, :, :tail])
    check_attention(torch, s, 4, 0.06)


def test_lengths_and_pages_out_of_range_are_recorded(torch):
    """Nothing outside the cache or the rows is touched: the call passes over them and says so."""
    for new in (1, 40):
        s = Setup(torch, [200, 100, 300], [new] * 3, 2, 128, 32, "bfloat16").upload()
        q = s.rows(8).cuda()
        kv = s.rows(2).cuda()
        ws = q4.new_workspace(q4.lily_kv8_attention_workspace_bytes(s.cache, s.batch, s.T, 8))
        out0 = torch.full_like(q, 7)
        q4.lily_kv8_attention(s.cache, s.batch, q, out0, 0.1, ws=ws)
        good_table, good_len = s.batch.block_table.clone(), s.batch.kv_len.clone()
        for what in ("page", "negative page", "length", "negative length", "rows"):
            b = q4.KV8Batch(good_table.clone(), s.batch.q_start.clone(), good_len.clone(), new, int(s.len.max()))
            if what == "page":
                b.block_table[1, 1] = s.cache.n_pages
            elif what == "negative page":
                b.block_table[1, 1] = -1
            elif what == "length":
                b.kv_len[1] = 1 << 30
            elif what == "negative length":
                b.kv_len[1] = -1
            else:
                b.q_start[2] = 1 << 20
            out = torch.full_like(q, 7)
            q4.lily_kv8_attention(s.cache, b, q, out, 0.1, ws=ws)
            assert q4.lily_q4_workspace_status(ws) == q4.ERR_INDEX, what
            assert q4.lily_q4_workspace_status(ws) == q4.OK
            for other in (0, 2):  # the others are not disturbed (but their keys may be shared out otherwise)
                if what == "rows" and other == 2:
                    continue  # its rows begin where the bad range ends
                o, _, tol, _ = expected(torch, s, q.cpu(), other, 0.1)
                _close(_f64(out[other * new:(other + 1) * new]), o, tol, f"{what}: sequence {other}")
            if what in ("length", "negative length", "rows"):
                assert (out[new:2 * new] == 7).all()
            ko, vo = torch.full_like(kv, 7), torch.full_like(kv, 7)
            q4.lily_kv8_read(s.cache, b, ko, vo, ws=ws)
            st = q4.lily_q4_workspace_status(ws)
            assert st == (q4.OK if "page" in what else q4.ERR_INDEX), what
            held = (s.cache.k, s.cache.v, s.cache.k_amax, s.cache.v_amax)
            before = [x.clone() for x in held]
            q4.lily_kv8_append(s.cache, b, kv, kv, ws=ws)
            st = q4.lily_q4_workspace_status(ws)
            assert st == (q4.OK if "page" in what else q4.ERR_INDEX), what
            for x, y in zip(held, before):
                x.copy_(y)


def test_masked_pages_out_of_range_read_as_zero(torch):
    s = Setup(torch, [40], [3], 1, 64, 16, "bfloat16").upload()
    s.batch.block_table[0, 2] = 1 << 29
    ko = torch.full((s.T, 1, 64), 7, dtype=torch.bfloat16, device="cuda")
    ws = q4.new_workspace(256)
    q4.lily_kv8_read(s.cache, s.batch, ko, ko.clone(), ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.ERR_INDEX
    assert (ko == 0).all()


def test_bad_weights_stay_in_their_rows(torch):
    """A NaN query row does not reach the others."""
    for new in (2, 70):
        s = Setup(torch, [200], [new], 1, 128, 32, "bfloat16").upload()
        q = s.rows(4)
        good, _ = check_attention(torch, s, 4, 0.1, q=q)
        q = q.cuda()
        q[1, 2, 5] = float("nan")
        out = torch.empty_like(q)
        ws = q4.new_workspace(q4.lily_kv8_attention_workspace_bytes(s.cache, s.batch, s.T, 4))
        q4.lily_kv8_attention(s.cache, s.batch, q, out, 0.1, ws=ws)
        assert torch.isnan(out[1, 2]).all()
        out[1, 2] = good[1, 2]
        assert torch.equal(out, good)
