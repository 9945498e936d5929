"""GPU tests of the attention operators where the plain range ends: NaN and infinity in pages that a row
does not see, softmax weights far below the largest, magnitudes and queries near the ends of their
types, positions near 2^31.  Setups, oracles and tolerances are those of test_gpu_kv8.py unless a test says
otherwise."""
import numpy as np
import pytest

import bit_affine_quantized_mlx_gb300 as q4
import kv8_plain as plain
from test_gpu_kv8 import Setup, _close, _f64, check_attention, expected
from test_gpu_kv8 import torch  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------- what a row does not see

@pytest.mark.parametrize("bad", ["v nan", "v inf", "k nan", "k inf"])
@pytest.mark.parametrize("D,new,side", [(64, 3, "ahead"), (128, 3, "behind"), (256, 3, "ahead"), (256, 3, "behind"),
                                        (64, 70, "ahead"), (128, 70, "behind"), (128, 40, "ahead"),
                                        (256, 130, "ahead"), (256, 130, "behind")])
def test_bad_pages_stay_with_the_rows_that_see_them(torch, D, new, side, bad):
    """One page that is not finite, ahead of the first rows (causal) or behind the last ones (a window):
    every row that sees no token of it is as it is without it, and one that does is NaN."""
    page, old, window = 16, 303, 0 if side == "ahead" else 81
    s = Setup(torch, [old], [new], 1, D, page, "bfloat16", seed=D + new)
    n = int(s.len[0])
    pos = old + np.arange(new)
    first = np.maximum(0, pos - window + 1) if window else np.zeros(new, int)
    at = (n - 1) // page if side == "ahead" else int(first[0]) // page
    sees = (first < (at + 1) * page) & (pos >= at * page)
    assert sees.any() and not sees.all()
    q = s.rows(4, 1.5)
    want, lse, tol, ltol = expected(torch, s, q, 0, D ** -0.5, True, window)
    which, what = bad.split()
    s.amax[which][s.table[0, at], 0] = float(what)  # as lily_kv8_append leaves such a page
    s.codes[which][s.table[0, at], 0] = 0
    s.upload()
    out = torch.empty((new, 4, D), dtype=s.dt, device="cuda")
    got_lse = torch.empty((new, 4), device="cuda")
    ws = q4.new_workspace(q4.lily_kv8_attention_workspace_bytes(s.cache, s.batch, new, 4))
    q4.lily_kv8_attention(s.cache, s.batch, q.cuda(), out, D ** -0.5, lse=got_lse, window=window, ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    got, got_lse = _f64(out), _f64(got_lse)
    _close(got[~sees], want[~sees], tol[~sees], "rows that see only finite pages")
    _close(got_lse[~sees], lse[~sees], ltol[~sees], "their lse")
    assert np.isnan(got[sees]).all()


# --------------------------------------------------------------------------- weights far below the largest

def one_key_draws(torch, keys, new, copies, D, dtype, at, gap, group=4, page=64, size=1.0, rest=None):
    """`copies` sequences that share their pages and queries, so that one block goes through many keys.  Key
    `at` has a score `gap` (and up to a quarter more, head by head) above all others, which tie.  Its own value
    is small and of both signs; the others' are positive.  `rest`: the value magnitude of pages other than
    that of `at`, where it is not `size`."""
    pages = -(-keys // page)
    s = Setup(torch, [keys - new], [new], 1, D, page, dtype, seed=keys + D, total=pages + 2)
    shape = (pages + 2, 1, page, D)
    s.codes = {x: s.rs.randint(-127, 128, shape).astype(np.int8) for x in "kv"}
    s.codes["v"] = np.abs(s.codes["v"])
    s.amax = {"k": np.ones(shape[:2]), "v": np.full(shape[:2], float(s.rounded(size if rest is None else rest)))}
    own = s.table[0, at // page]
    s.amax["v"][own] = float(s.rounded(size))
    s.codes["k"][:, :, :, 0] = 0
    s.codes["k"][own, 0, at % page, 0] = 127
    s.codes["v"][own, 0, at % page] = s.rs.randint(-5, 6, D)
    s.table, s.len, s.new = s.table.repeat(copies, 0), s.len.repeat(copies), s.new.repeat(copies)
    s.T, s.q_start = new * copies, new * np.arange(copies + 1)
    q = s.rows(group) * 0
    q[:, :, 0] = torch.linspace(1.0, 1.25, group).to(s.dt)
    return s.upload(), q


def check_small_weights(torch, s, q, scale, floor, step):
    """As check_attention, for weights that are off by `floor` of the largest weight-times-magnitude where that
    is more than 2^-11 of their own, and sums that take `step` keys at a time: fp32 additions, 2^-25 (the
    products' may drop bits: 2^-23) of the total each."""
    n, new, heads = int(s.len[0]), int(s.new[0]), q.shape[1]
    out = torch.empty((s.T, heads, s.D), dtype=s.dt, device="cuda")
    lse = torch.empty((s.T, heads), device="cuda")
    ws = q4.new_workspace(q4.lily_kv8_attention_workspace_bytes(s.cache, s.batch, s.T, heads))
    q4.lily_kv8_attention(s.cache, s.batch, q.cuda(), out, scale, lse=lse, ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    k, v = (plain.values(s.codes[x], s.amax[x], s.table[0], n) for x in "kv")
    mag = np.repeat(s.amax["v"][s.table[0][:-(-n // s.page)]].T, s.page, 1)[:, :n]
    o, l, size, top, reach = plain.attention(_f64(q[:new]), k, v, mag, scale, True, 0)
    d, sums = 2.0 ** -21 * reach, n / step * 2.0 ** -25
    tol = (torch.finfo(s.dt).eps / 2 * np.abs(o) + (2.0 ** -11 + 2.0 ** -18 + 5 * sums + 2 * d[..., None]) * size
           + n * floor * top[..., None] + torch.finfo(s.dt).smallest_normal * torch.finfo(s.dt).eps / 2)
    copies = len(s.len)
    for b in {0, copies // 2, copies - 1}:
        _close(_f64(out[b * new:(b + 1) * new]), o, tol, "out")
        _close(_f64(lse[b * new:(b + 1) * new]), l, d + 2.0 ** -18 + sums + 2.0 ** -22 * np.abs(l), "lse")


@pytest.mark.parametrize("keys,copies,D,dtype,at,gap", [
    (33000, 300, 128, "bfloat16", 5, 17.5), (40000, 200, 256, "bfloat16", 39999, 17.5), (30000, 400, 64, "float16", 15000, 17.0),
    (1000, 1, 64, "float16", 500, 13.0), (262144, 1, 256, "bfloat16", 0, 17.5),
])
def test_small_weights_count(torch, keys, copies, D, dtype, at, gap):
    """One key draws most of the weight and carries little; what all others add is about 2^-25 of it
    each.  Weights are at most 2^14 in fp16, whose last step is 2^-24: half of it is 2^-39 of the largest.
    A block's four warps take 16 keys at a time each."""
    s, q = one_key_draws(torch, keys, 1, copies, D, dtype, at, gap)
    check_small_weights(torch, s, q, gap, 2.0 ** -39, 64)


@pytest.mark.parametrize("keys,copies,D,dtype,at,gap", [
    (65536, 160, 128, "float16", 0, 17.5), (65536, 160, 256, "bfloat16", 30000, 17.5), (33000, 160, 64, "float16", 32900, 17.0),
    (131072, 1, 256, "float16", 65536, 17.5),
])
def test_small_weights_count_in_prompts(torch, keys, copies, D, dtype, at, gap):
    """The same for prompts of 40 tokens: the first maximum is at weight 2^6, so the fp16 weights' last half step
    is 2^-31 of the largest at most.  Products take 16 keys at a time."""
    s, q = one_key_draws(torch, keys, 40, copies, D, dtype, at, gap)
    check_small_weights(torch, s, q, gap, 2.0 ** -31, 16)


@pytest.mark.parametrize("keys,new,copies,D,at,gap", [
    (33000, 1, 300, 128, 7, 17.5), (33000, 1, 200, 256, 30000, 17.5), (262144, 1, 1, 128, 7, 18.0), (262144, 1, 1, 256, 100000, 18.0),
    (65536, 40, 160, 64, 7, 13.5), (65536, 40, 160, 256, 65000, 13.5), (65536, 40, 160, 128, 40000, 13.5), (131072, 40, 1, 128, 7, 13.5),
])
def test_zero_values_stay_in_the_sum(torch, keys, new, copies, D, at, gap):
    """Pages of zero values beside one of values near fp16's largest: they add nothing to the output, but
    their weights count, in a block's running sum and where parts are joined."""
    s, q = one_key_draws(torch, keys, new, copies, D, "float16", at, gap, size=6e4, rest=0.0)
    check_small_weights(torch, s, q, gap, *((2.0 ** -39, 64) if new == 1 else (2.0 ** -31, 16)))


@pytest.mark.parametrize("new", [1, 60])
def test_small_values_beside_zero_ones(torch, new):
    """Values of 1e-18 keep their bits beside pages of zeros, which count as of 2^-80 (8e-25)."""
    s = Setup(torch, [400], [new], 1, 128, 16, "bfloat16")
    own = s.table[0, :-(-int(s.len[0]) // 16)]
    s.amax["v"][own, 0] = s.rounded(1e-18)
    s.amax["v"][own[::3], 0] = 0
    check_attention(torch, s.upload(), 4, 0.1)


# --------------------------------------------------------------------------- ends of the types' ranges

@pytest.mark.parametrize("top", [1e30, 2.6e36, 2.8e36, 1e37, 3.3e38])
def test_read_near_the_top_of_the_range(torch, top):
    """Finite tokens read back finite, to the code's resolution and the output's rounding."""
    s = Setup(torch, [0], [20], 2, 64, 16, "bfloat16").upload()
    x = s.rows(2)
    x = (x.double() / x.double().abs().max() * top).to(s.dt)
    assert torch.isfinite(x).all()
    ws = q4.new_workspace(256)
    q4.lily_kv8_append(s.cache, s.batch, x.cuda(), x.cuda(), ws=ws)
    plain.append(s.codes["k"], s.amax["k"], s.table, s.q_start, s.len, _f64(x))
    want = plain.values(s.codes["k"], s.amax["k"], s.table[0], 20).transpose(1, 0, 2)
    for dt in (torch.float32, torch.bfloat16):
        k, v = (torch.empty((20, 2, 64), dtype=dt, device="cuda") for _ in "kv")
        q4.lily_kv8_read(s.cache, s.batch, k, v, ws=ws)
        # q amax is exact; the reciprocal of 127 and the product with it are rounded; then the output's rounding
        _close(_f64(k), want, (2.0 ** -23 + torch.finfo(dt).eps / 2) * np.abs(want), str(dt))
        assert torch.equal(k, v)
    assert q4.lily_q4_workspace_status(ws) == q4.OK


@pytest.mark.parametrize("new", [1, 50])
def test_queries_near_the_top_of_the_range(torch, new):
    """Queries up to 3e38 with scores of ordinary size (a scale as small as they are large)."""
    s = Setup(torch, [100], [new], 1, 64, 32, "bfloat16").upload()
    q = s.rows(8).double()
    q /= q.abs().amax(-1, keepdim=True)
    q = (q * torch.tensor([1e28, 1e30, 3e30, 1e31, 1e33, 1e36, 1e38, 3.3e38], dtype=torch.float64)[:, None]).to(s.dt)
    assert torch.isfinite(q).all()
    check_attention(torch, s, 8, 2e-36, q=q)


# --------------------------------------------------------------------------- positions and windows near 2^31

@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 4, 1 << 30, 300])
@pytest.mark.parametrize("new,causal", [(8, False), (8, True), (70, False), (70, True)])
def test_widest_windows_and_rows_before_the_first_position(torch, new, causal, window):
    """Rows at negative positions (more of them than tokens) in a window as wide as its type takes: position
    less window stays in range."""
    s = Setup(torch, [3 - new, 60], [new, new], 2, 64, 16, "bfloat16").upload()
    check_attention(torch, s, 8, 0.2, causal, window)


@pytest.mark.parametrize("new", [1, 40])
def test_tables_wider_than_positions(torch, new):
    """A block table whose pages' tokens pass 2^31, of which few are used."""
    s = Setup(torch, [30], [new], 1, 64, 128, "bfloat16").upload()
    wide = torch.full((1, 1 << 24), -9, dtype=torch.int32, device="cuda")
    used = -(-int(s.len[0]) // 128)
    wide[0, :used] = s.batch.block_table[0, :used]
    s.batch = q4.KV8Batch(wide, s.batch.q_start, s.batch.kv_len, new, (1 << 31) - 1)
    x = s.rows(1)
    ws = q4.new_workspace(256)
    q4.lily_kv8_append(s.cache, s.batch, x.cuda(), x.cuda(), ws=ws)
    k, v = (torch.empty((new, 1, 64), dtype=torch.float32, device="cuda") for _ in "kv")
    q4.lily_kv8_read(s.cache, s.batch, k, v, ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    for y in "kv":
        plain.append(s.codes[y], s.amax[y], s.table, s.q_start, s.len, _f64(x))
    for y, got in (("k", k), ("v", v)):
        want = plain.values(s.codes[y], s.amax[y], s.table[0], int(s.len[0])).transpose(1, 0, 2)[-new:]
        _close(_f64(got), want, 2.0 ** -22 * np.abs(want), y)
    check_attention(torch, s, 4, 0.1)


@pytest.mark.parametrize("page,length", [(16, (1 << 29) - 3), (128, (1 << 31) - 65600)])
def test_last_tokens_of_a_far_sequence(torch, page, length):
    """Append and read at positions near the end of a table of 2^25 and 2^24 entries."""
    new, D = 5, 64
    s = Setup(torch, [0], [new], 1, D, page, "bfloat16").upload()
    table = torch.full((1, 1 << 25 if page == 16 else 1 << 24), -9, dtype=torch.int32, device="cuda")
    first = (length - new) // page
    table[0, first], table[0, (length - 1) // page] = 1, 2 if (length - 1) // page != first else 1
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    batch = q4.KV8Batch(table, i32(0, new), i32(length), new, length)
    s.cache = q4.KV8Cache.new(4, 1, page, D)
    x = s.rows(1).cuda()
    k, v = (torch.empty((new, 1, D), dtype=torch.float32, device="cuda") for _ in "kv")
    ws = q4.new_workspace(256)
    q4.lily_kv8_append(s.cache, batch, x, x, ws=ws)
    q4.lily_kv8_read(s.cache, batch, k, v, ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    # a code is off by half a step of the page's largest magnitude
    _close(_f64(k), _f64(x), np.abs(_f64(x)).max() * (0.5 / 127 + 2.0 ** -22), "keys")
    assert torch.equal(k, v)


# --------------------------------------------------------------------------- status

def test_status_reports_an_index_error_beside_a_time_out(torch):
    """Both errors in one workspace: each is reported once, the time-out first."""
    s = Setup(torch, [40], [1], 1, 64, 16, "bfloat16").upload()
    s.batch.block_table[0, 2] = 1 << 29
    ko = torch.empty((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    ws = q4.new_workspace(4096)
    q4.lily_q4_selftest_timeout(ws, 1)  # a bounded wait on a barrier that nothing completes
    q4.lily_kv8_read(s.cache, s.batch, ko, ko.clone(), ws=ws)
    assert [q4.lily_q4_workspace_status(ws) for _ in range(3)] == [q4.ERR_TIMEOUT, q4.ERR_INDEX, q4.OK]


# --------------------------------------------------------------------------- threads

def test_small_and_large_batches_from_several_threads(torch):
    """A kernel's first launches, with little and with much shared memory, from threads on streams of their own."""
    import threading
    for D in (64, 128, 256):
        for group in (1, 9, 17):
            jobs = []
            for batch in (1, 4096, 2, 3000):
                s = Setup(torch, [20] * batch, [1] * batch, 1, D, 16, "float16", seed=batch).upload()
                jobs.append((s, s.rows(group), torch.cuda.Stream()))
            failed, start = [], threading.Barrier(len(jobs), timeout=60)

            def work(s, q, stream):
                try:
                    q = q.cuda()
                    out, ws = torch.empty_like(q), q4.new_workspace(
                        q4.lily_kv8_attention_workspace_bytes(s.cache, s.batch, s.T, group))
                    torch.cuda.synchronize()
                    start.wait()
                    for _ in range(20):
                        q4.lily_kv8_attention(s.cache, s.batch, q, out, 0.1, ws=ws, stream=stream)
                    torch.cuda.synchronize()
                    assert q4.lily_q4_workspace_status(ws) == q4.OK
                    for b in (0, len(s.len) - 1):
                        o, _, tol, _ = expected(torch, s, q.cpu(), b, 0.1)
                        _close(_f64(out[b:b + 1]), o, tol, f"sequence {b} of {len(s.len)}")
                except Exception as e:  # reported by the main thread
                    failed.append(e)

            threads = [threading.Thread(target=work, args=j) for j in jobs]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
            assert not failed, failed
