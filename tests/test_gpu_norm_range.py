"""The sign of zeros in the norm, against its plain 64-bit form, bit for bit."""
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
    wrong = np.argwhere(_np(y) != n)
    assert len(wrong) == 0, (len(wrong), wrong[:4].tolist(), _np(y)[tuple(wrong[0])], n[tuple(wrong[0])])
    assert np.array_equal(np.signbit(_np(y)), np.signbit(n))
    if mx is not None:
        codes, scales, _ = plain.quantize(n, bits)
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
