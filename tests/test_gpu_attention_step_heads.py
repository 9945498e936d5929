"""The attention stack with heads of 128 and 256: a prompt fed at once against the same prompt fed in
pieces and token by token, in both forms of attention.  The tolerance is that of
test_gpu_attention_step.py: a score's error from codes off by half a step of their page falls with the
width of a head, so that what holds for heads of 64 holds here."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head_dim", [128, 256])
def test_pieces_agree_with_the_whole(head_dim):
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from bit_affine_quantized_mlx_gb300.attention_step import Stack
    lengths = [150, 40]
    tokens = [torch.randint(0, 4096, (n,), generator=torch.Generator().manual_seed(n)).cuda() for n in lengths]
    stack = lambda: Stack(capacity=256, experts=2, sequences=2, head_dim=head_dim)
    whole = stack()
    h = whole.forward(torch.cat(tokens), lengths, lengths)
    whole.check()
    want = h[torch.from_numpy(np.cumsum(lengths) - 1).cuda()].float()
    pieces, fed = stack(), [0, 0]
    for more in ([100, 39], [47, 0], [1, 1], [2, 0]):
        fed = [a + b for a, b in zip(fed, more)]
        out = pieces.forward(torch.cat([t[n - m:n] for t, n, m in zip(tokens, fed, more)]), more, fed).split(more)
        for b, n in enumerate(lengths):
            if more[b] and fed[b] == n:
                err = (out[b][-1].float() - want[b]).norm() / want[b].norm()
                assert err < 0.03, (b, float(err))
    pieces.check()
    assert fed == lengths
