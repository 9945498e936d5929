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
