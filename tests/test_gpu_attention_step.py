"""The attention operators together with the mixture-of-experts layers and the LM head: a prompt fed
at once against the same prompt fed in pieces and token by token.

The two orders quantise pages at different times (a page's codes are re-rounded when its magnitude
grows), so hidden states agree to the 8-bit cache's resolution, not bit for bit: a code is off by
half a step of its page (1/254 of the largest magnitude) once, and by another half for every growth;
over 64 x 2 rounded elements of a score and a mean of many values that stays below 3% of the hidden
state's norm in two layers, where a wrong position, page or mask is off by its own size.  Both of the
layers' two experts are taken for every token: a choice among more would flip on such differences,
and a flip is as large as an expert's output."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def test_pieces_agree_with_the_whole():
    import torch
    import __graft_entry__
    __graft_entry__.build()
    from bit_affine_quantized_mlx_gb300.attention_step import Stack
    lengths = [150, 40, 3]
    tokens = [torch.randint(0, 4096, (n,), generator=torch.Generator().manual_seed(n)).cuda() for n in lengths]
    whole = Stack(capacity=256, experts=2)
    h = whole.forward(torch.cat(tokens), lengths, lengths)
    whole.check()
    last = h[torch.from_numpy(np.cumsum(lengths) - 1).cuda()].float()

    pieces = Stack(capacity=256, experts=2)
    fed = [100, 39, 1]
    pieces.forward(torch.cat([t[:n] for t, n in zip(tokens, fed)]), fed, fed)
    more = [48, 0, 1]
    fed = [a + b for a, b in zip(fed, more)]
    pieces.forward(torch.cat([t[n - m:n] for t, n, m in zip(tokens, fed, more)]), more, fed)
    got = [None] * 3
    while fed != lengths:
        step = [int(a < b) for a, b in zip(fed, lengths)]
        fed = [a + b for a, b in zip(fed, step)]
        out = pieces.forward(torch.cat([t[n - m:n] for t, n, m in zip(tokens, fed, step)]), step, fed)
        rows = out.split(step)
        for b in range(3):
            if step[b] and fed[b] == lengths[b]:
                got[b] = rows[b][0].float()
    pieces.check()
    for b in range(3):
        err = (got[b] - last[b]).norm() / last[b].norm()
        assert err < 0.03, (b, float(err))


def test_command(capsys):
    from bit_affine_quantized_mlx_gb300 import attention_step
    attention_step.main(["--prompts", "70", "5", "--steps", "3"])
    out = capsys.readouterr().out.splitlines()
    assert len(out) == 2 and all(len(line.split(":")[1].split()) == 3 for line in out)
