"""The operators around a step's products where elements lie more than 2^31 from the first: rows far apart, and many rows."""
import numpy as np
import pytest

import bit_affine_quantized_mlx_gb300 as q4
import mx_plain as plain
from test_gpu_mx4_linear import torch  # noqa: F401 (fixture)
from test_gpu_sample import plain_row

pytestmark = pytest.mark.gpu
FAR = (1 << 30) + 8  # a row's stride in elements: the third row is beyond 2^31


@pytest.fixture(autouse=True)
def free(torch):  # noqa: F811
    yield
    torch.cuda.empty_cache()


def _np(t):
    return t.double().cpu().numpy()


def _rows(torch, n, stride, count, dtype):  # noqa: F811
    return torch.zeros(n * stride, dtype=dtype, device="cuda").view(n, stride)[:, 16:16 + count]


def test_norm_of_rows_far_apart(torch):  # noqa: F811
    H, g = 256, torch.Generator().manual_seed(1)
    x, y = (_rows(torch, 3, FAR, H, torch.bfloat16) for _ in "xy")
    x.copy_(torch.randn((3, H), generator=g))
    add = torch.randn((3, H), generator=g).bfloat16().cuda()
    before, mx, v = _np(x), q4.DeviceMX.new(3, H, 8), torch.empty((3, H), device="cuda")
    op = q4.RMSNorm(torch.ones(H, dtype=torch.bfloat16, device="cuda"))
    q4.lily_add_rms_norm(op, x, y=y, add=add, total=x, mx=mx)
    s, n = plain.norm(before, _np(add), np.ones(H), 0.0, 1e-6, "bf16")
    q4.lily_mx_read(mx, v)
    assert np.array_equal(_np(x), s) and np.array_equal(_np(y), n) and np.array_equal(_np(v), plain.quantize(n, 8)[2])
    # quantised from there and read to there
    other = q4.DeviceMX.new(3, H, 4)
    q4.lily_mx_quantize(y, other)
    q4.lily_mx_read(other, x)
    assert np.array_equal(_np(x), plain.quantize(n, 4)[2])


@pytest.mark.parametrize("bits", [8, 4])
def test_norm_and_blocks_of_many_rows(torch, bits):  # noqa: F811
    H, T = 2048, (1 << 20) * (8 // bits) + 5  # the codes alone pass 2^31 bytes
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    y, back, mx = torch.empty_like(x), torch.empty_like(x), q4.DeviceMX.new(T, H, bits)
    q4.lily_add_rms_norm(q4.RMSNorm(torch.ones(H, dtype=torch.bfloat16, device="cuda")), x, y=y, mx=mx)
    q4.lily_mx_read(mx, back)
    at = torch.tensor([0, 1, T // 2, (1 << 20) - 1, 1 << 20, T - 7, T - 2, T - 1], device="cuda")
    n = plain.norm(_np(x[at]), None, np.ones(H), 0.0, 1e-6, "bf16")[1]
    assert np.array_equal(_np(y[at]), n)
    assert np.array_equal(_np(back[at]), plain.quantize(n, bits)[2])
    again = q4.DeviceMX.new(T, H, bits)
    q4.lily_mx_quantize(y, again)
    assert bool((again.codes == mx.codes).all()) and bool((again.scales == mx.scales).all())


def _matrix(torch, rows, cols, bits, seed):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (rows, cols * bits // 8), dtype=torch.uint8, device="cuda", generator=g)
    if bits == 8:
        codes &= 0xBF  # below 2, and no NaN
    return q4.DeviceMX(codes, torch.randint(124, 131, (rows, cols // 32), dtype=torch.uint8, device="cuda", generator=g), bits)


def _values(m, at):
    return plain.values(m.codes[at].cpu().numpy(), m.scales[at].cpu().numpy(), m.bits)


def _check(out, W, x, ts, ns):
    """Some rows and columns, within the bound of test_gpu_mx4_linear.py."""
    w, v = _values(W, ns), _values(x, ts)
    got = _np(out[ts][:, ns])
    assert np.all(np.abs(got - v @ w.T) <= W.cols * 2.0 ** -23 * (np.abs(v) @ np.abs(w).T) + 2.0 ** -24 * np.abs(v @ w.T))


@pytest.mark.parametrize("bits", [8, 4])
def test_product_with_many_weights(torch, bits):  # noqa: F811
    K, T = 1024, 2
    N = (1 << 31) // (K // 2) + 130
    W, x = _matrix(torch, N, K, 4, 3), _matrix(torch, T, K, bits, 4)
    out = torch.empty((T, N), device="cuda")
    ws = q4.new_workspace(256)
    q4.lily_mx4_linear(W, x, out, ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    _check(out, W, x, slice(None), torch.tensor([0, 5, N // 2, N - 200, N - 129, N - 2, N - 1], device="cuda"))


@pytest.mark.parametrize("bits", [8, 4])
def test_product_with_many_rows(torch, bits):  # noqa: F811
    K, N = 256, 40
    T = (1 << 31) // (K * bits // 8) + 77
    W, x = _matrix(torch, N, K, 4, 5), _matrix(torch, T, K, bits, 6)
    out = torch.empty((T, N), device="cuda", dtype=torch.float32)
    ws = q4.new_workspace(256)
    q4.lily_mx4_linear(W, x, out, ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    _check(out, W, x, torch.tensor([0, 7, T // 2, T - 100, T - 2, T - 1], device="cuda"), slice(None))


@pytest.mark.parametrize("T", [3, 200])
def test_product_to_rows_far_apart(torch, T):  # noqa: F811
    W, x = _matrix(torch, 150, 256, 4, 7), _matrix(torch, T, 256, 8, 8)
    out = _rows(torch, T, FAR if T == 3 else (1 << 24) + 3, 150, torch.bfloat16)
    near = torch.empty((T, 150), dtype=torch.bfloat16, device="cuda")
    ws = q4.new_workspace(256)
    for o in (out, near):
        q4.lily_mx4_linear(W, x, o, ws=ws)
    assert bool((out == near).all()) and float(near.abs().max()) > 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sampling_of_rows_far_apart(torch, dtype):  # noqa: F811
    l = _rows(torch, 3, FAR + 1, 5000, getattr(torch, dtype))
    l.copy_(torch.randn((3, 5000), generator=torch.Generator().manual_seed(9)))
    u, token = torch.tensor([0.2, 0.5, 0.9], device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    for k in (0, 20):
        q4.lily_sample(q4.Sampling(top_k=torch.full((3,), k, dtype=torch.int32, device="cuda")), l, u, token, ws=q4.new_workspace(256))
        assert token.tolist() == [plain_row(_np(l[b]), 1.0, k, 1.0, 0.0, float(u[b]))[0] for b in range(3)]


def test_sampling_of_many_rows(torch):  # noqa: F811
    V, B = 151936, (1 << 31) // 151936 + 9
    some = torch.randn((7, V), generator=torch.Generator().manual_seed(10)).bfloat16().cuda()
    l = some.repeat(-(-B // 7), 1)[:B]
    u = torch.tensor([0.1, 0.4, 0.6, 0.8, 0.99], device="cuda").repeat(-(-B // 5))[:B].contiguous()
    token = torch.empty(B, dtype=torch.int32, device="cuda")
    q4.lily_sample(q4.Sampling(top_p=torch.full((B,), 0.5, device="cuda")), l, u, token, ws=q4.new_workspace(256))
    want = {(i, j): plain_row(_np(some[i]), 1.0, 0, 0.5, 0.0, float(u[j]))[0] for i in range(7) for j in range(5)}
    assert token.tolist() == [want[b % 7, b % 5] for b in range(B)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("K", [(1 << 31) - 128, (1 << 31) - 256])
def test_product_of_the_longest_rows(torch, K, bits):  # noqa: F811
    """Zeros but for a few places, whose products are exact."""
    W, x = q4.DeviceMX.new(2, K, 4), q4.DeviceMX.new(1, K, bits)
    W.scales.fill_(127)
    x.scales.fill_(127)
    at = [0, 129, 1 << 20, (1 << 30) - 1, 1 << 30, K - 257, K - 130, K - 1]
    for i, k in enumerate(at):  # 2^(i % 3) in x, 1 and 2^(i % 2) in W
        one = lambda m, row, e: m.codes[row, k // 2].add_((2 + 2 * e) << (4 * (k % 2))) if m.bits == 4 else m.codes[row, k].fill_((7 + e) << 3)
        one(x, 0, i % 3)
        one(W, 0, 0)
        one(W, 1, i % 2)
    out, ws = torch.empty((1, 2), device="cuda"), q4.new_workspace(256)
    q4.lily_mx4_linear(W, x, out, ws=ws)
    assert q4.lily_q4_workspace_status(ws) == q4.OK
    assert out.tolist() == [[sum(2.0 ** (i % 3) for i in range(len(at))), sum(2.0 ** (i % 3 + i % 2) for i in range(len(at)))]]
