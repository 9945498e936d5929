"""The norm of rows at both ends of bf16 and with any eps, against its plain 64-bit form, whose numbers reach from 2^-1022 to
2^1023, far beyond the squares of any row here.

The kernel rounds a value that is right to 2^-40, so its result is what one of v (1 - 2^-40) and v (1 + 2^-40) rounds to, v the plain
form before its rounding (right to 2^-50).  That is the same number everywhere but at borders: where eps is a power of four and
far above the mean square, the root is a power of two to 2^-70, products of two 8-bit numbers lie on borders, and which side the
exact value is on neither form can tell.  The codes are those of the kernel's own rows, bit for bit."""
import numpy as np
import pytest

import bit_affine_quantized_mlx_gb300 as q4
import mx_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    return torch


def _np(t):
    return t.double().cpu().numpy()


def _check(torch, x, eps, bits=8, add=None, offset=0.0, seed=0):
    """x, add: float64 arrays that are rounded to bf16."""
    T, H = x.shape
    up = lambda a: torch.from_numpy(a).float().bfloat16().cuda()
    x, add = up(x), None if add is None else up(add)
    w = up((1 - offset) + 0.2 * np.random.default_rng(seed).standard_normal(H))
    y, total = torch.empty_like(x), torch.empty_like(x)
    mx = q4.DeviceMX.new(T, H, bits) if H % 32 == 0 else None
    q4.lily_add_rms_norm(q4.RMSNorm(w, eps=eps, weight_offset=offset), x, y=y, add=add, total=total, mx=mx)
    s, n = plain.norm(_np(x), None if add is None else _np(add), _np(w), offset, eps, "bf16")
    assert np.isfinite(n).all()
    assert np.array_equal(_np(total), s)
    exact = s / np.sqrt((s * s).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * (_np(w) + offset)
    got, low, high = _np(y), plain.round16(exact * (1 - 2.0 ** -40), "bf16"), plain.round16(exact * (1 + 2.0 ** -40), "bf16")
    wrong = np.argwhere((got != low) & (got != high))
    assert len(wrong) == 0, (len(wrong), wrong[:4].tolist(), got[tuple(wrong[0])], n[tuple(wrong[0])])
    assert np.array_equal(np.signbit(got), np.signbit(n))
    if mx is not None:
        codes, scales, _ = plain.quantize(got, bits)
        assert np.array_equal(mx.scales.cpu().numpy(), scales)
        assert np.array_equal(mx.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("T,H", [(700, 512), (40, 5120)])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_zeros_keep_their_signs(torch, T, H, offset):
    """Whatever their neighbours are: next to some of these the plain products leave a rounding open."""
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, H))
    x[:, 1::3], x[:, 2::3] = -0.0, 0.0
    _check(torch, x, 1e-6, offset=offset)


SHAPES = [(3, 8), (5, 256), (2, 2048), (3, 5120), (1500, 512), (700, 2048), (2, 32768)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("power", [-126, -100, -81, -80, -76, -73, -66, -60, -41, 49, 52, 63, 70, 100, 118])
def test_rows_of_one_size_without_eps(torch, T, H, power):
    _check(torch, np.random.default_rng(T + H + 1000 - power).standard_normal((T, H)) * 2.0 ** power, 0.0)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("eps", [0.0, 1e-42, 2.0 ** -120, 2.0 ** -99, 1e-6, 2.0 ** 99, 2.0 ** 101, 3e38])
def test_rows_of_all_sizes(torch, T, H, eps):
    """Neighbours of every size in one call, elements of many sizes in one row."""
    rng = np.random.default_rng(T * H)
    power = rng.integers(-125, 118, (T, 1)).astype(float)
    power[:2, 0] = -90.0, 90.0
    x = rng.standard_normal((T, H)) * np.exp2(power + rng.integers(-25, 1, (T, H)))
    # norms next to the end of the normal numbers may lose bits
    x = np.where(np.abs(x) < 2.0 ** -100 * np.sqrt((x * x).mean(-1, keepdims=True) + eps), 0.0, x)
    _check(torch, x, eps, bits=4)


def test_the_smallest_numbers(torch):
    x = np.zeros((6, 64))
    x[0], x[1, 5], x[2, :32], x[3] = 2.0 ** -133, 2.0 ** -133, 3 * 2.0 ** -133, 2.0 ** -126
    x[4] = np.where(np.arange(64) % 2, -2.0 ** -127, 2.0 ** -130)
    x[5] = 3.3895313892515355e38
    _check(torch, x, 0.0)
    _check(torch, x[:5], 1e-45)


def test_one_warp_small_the_others_not(torch):
    """A row whose parts lie far apart: what is small does not count, and is as exact as the rest."""
    x = np.full((4, 4096), 2.0 ** -70)
    x[1, 4000:] = 1.5
    x[2, :8] = 2.0 ** 80
    x[3, ::2] = 2.0 ** -45
    _check(torch, x, 0.0)


def test_sum_and_offset(torch):
    rng = np.random.default_rng(5)
    for power in (-110, -75, 55, 110):
        x, add = (rng.standard_normal((40, 1024)) * 2.0 ** power for _ in "xa")
        _check(torch, x, 0.0, add=add, offset=1.0)


def test_rows_that_are_not_finite_stay_by_themselves(torch):
    x = torch.ones((6, 512), dtype=torch.bfloat16, device="cuda") * 2.0 ** -90
    x[1, 3], x[3, 500] = float("inf"), float("nan")
    y = torch.empty_like(x)
    q4.lily_add_rms_norm(q4.RMSNorm(torch.ones(512, dtype=torch.bfloat16, device="cuda"), eps=0.0), x, y=y)
    assert bool((y[[0, 2, 4, 5]] == 1).all()) and bool(y[[1, 3]].isnan().any(1).all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("eps", [1e-45, 1e-42, 1e-38, 1e-20, 1e30])
@pytest.mark.parametrize("H", [64, 4096])
def test_rows_of_zeros(torch, H, eps, dtype):
    """Zeros with any eps above 0, beside a row that is not."""
    x = torch.zeros((3, H), dtype=getattr(torch, dtype), device="cuda")
    x[0], x[2] = 1.0, -0.0
    y = torch.full_like(x, 7.0)
    q4.lily_add_rms_norm(q4.RMSNorm(torch.ones(H, dtype=x.dtype, device="cuda"), eps=eps), x, y=y)
    assert bool((y[1:] == 0).all()) and bool(y[2].signbit().all()) and not bool(y[1].signbit().any())
    one = plain.round16(np.ones(1) / np.sqrt(1.0 + np.float64(np.float32(eps))), "bf16" if dtype == "bfloat16" else "fp16")
    assert np.array_equal(_np(y[0]), np.repeat(one, H))
