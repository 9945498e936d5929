"""The 4-bit product at every width of tiles that it has (16 to 192 tokens), of more K than its ring of stages holds, with a
remainder in tokens, weights and K.  The width follows from the sizes and the GPU's SMs, so the sizes are sought here; the bound is
that of test_gpu_mx4_linear.py."""
import pytest

from test_gpu_mx4_linear import _run, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
WIDTHS = [16, 32, 64, 96, 128, 160, 192]


def width(T, N, sms):
    """The rule of the launch: the least of (128 + width) times rounds of tiles over the SMs; and how many tiles."""
    cost = lambda nt: -(-(-(-N // 128) * -(-T // nt)) // sms) * (128 + nt)
    best = min(WIDTHS, key=cost)  # the first of the least
    return best, -(-N // 128) * -(-T // best)


def sizes(nt, sms, rows):
    """Tokens and weights of the least work with this width and a remainder in both: more tiles than SMs, or more than one
    of tokens."""
    found = []
    for N in (1030, 2100, 5000, 128 * (sms + 1) + 66):
        for T in range(3, 9000):
            if T % nt and width(T, N, sms)[0] == nt and (width(T, N, sms)[1] > sms if rows else T > nt):
                found.append((T * N, T, N))
                break
    return min(found)[1:]


def test_every_width_has_sizes():
    for sms in (132, 148, 152, 160):
        for nt in WIDTHS:
            for rows in (False, True):
                T, N = sizes(nt, sms, rows)
                assert N % 128 and T % nt


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("nt", WIDTHS)
@pytest.mark.parametrize("rows", [False, True])
def test_widths(torch, nt, rows, bits):  # noqa: F811
    T, N = sizes(nt, torch.cuda.get_device_properties(0).multi_processor_count, rows)
    # 23 blocks of 8-bit rows and 12 of 4-bit ones (half of the last); ten stages at most
    _, _, out, _ = _run(torch, T, N, 2944, bits, torch.float32)
    # and in rows of a wider buffer, nothing beside them
    wide = torch.full((T + 1, N + 9), 7.0, device="cuda")
    _run(torch, T, N, 2944, bits, torch.float32, out=wide[:T, 3:3 + N])
    assert bool((wide[:T, 3:3 + N] == out).all())
    wide[:T, 3:3 + N] = 7.0
    assert bool((wide == 7.0).all())
