"""GPU: the norms around a block where values are no numbers, infinite or nothing: they stay in their row, and what
follows from the new residual is what h3q_residual_rmsnorm_adaln_nvfp4 makes of it."""
import pytest
import torch

import nvfp4_activation_quantize_gb300 as h3q
from parity import gsf_tensor

pytestmark = pytest.mark.gpu

ROWS = 150


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def logical(scales, rows, cols):
    """The block scales [rows, cols / 16] of the swizzled layout."""
    tiles = scales.view(-1, cols // 64, 32, 4, 4)   # row tile, columns / 64, row % 32, row / 32, column
    return tiles.permute(0, 3, 2, 1, 4).reshape(-1, cols // 16)[:rows]


@pytest.mark.parametrize("cols", [64, 1024, 7168, 8128])
@pytest.mark.parametrize("tables", [False, True])
def test_they_stay_in_their_row(dev, cols, tables):
    g = torch.Generator(device=dev)
    g.manual_seed(cols)
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    h, o, post, gamma, bias = r(ROWS, cols), r(ROWS, cols).bfloat16(), r(cols).bfloat16(), r(cols).bfloat16(), r(cols).bfloat16()
    kw = {"gate_table": r(2, cols).bfloat16(), "mod_table": r(2, 2, cols).bfloat16(), "rows_per_frame": 75} if tables else {}
    gsf = gsf_tensor(200.0, dev)
    call = lambda h, o: h3q.h3q_postnorm_residual_adaln_nvfp4(h, o, post, gamma, gsf, bias=bias, **kw)  # noqa: E731
    want_h = h.clone()
    want = call(want_h, o)
    bad_h, bad_o = h.clone(), o.clone()
    bad_o[3, 5], bad_o[20, cols - 1], bad_o[127, 7] = float("nan"), float("inf"), -float("inf")
    bad_h[40, 8], bad_h[41, cols - 1], bad_h[128, 0], bad_h[ROWS - 1, 9] = (float(x) for x in ("nan", "inf", "-inf", "3e38"))
    hit = torch.zeros(ROWS, dtype=torch.bool, device=dev)
    hit[[3, 20, 127, 40, 41, 128, ROWS - 1]] = True
    got = call(bad_h, bad_o)
    assert torch.equal(bad_h[~hit], want_h[~hit]) and torch.equal(got[0][~hit], want[0][~hit])
    assert torch.equal(logical(got[1], ROWS, cols)[~hit], logical(want[1], ROWS, cols)[~hit])
    # a value of o that is none makes the row none; an infinite one, whose mean square is infinite, leaves a norm of 0
    # beside itself; those of h stay where they are
    assert bool(torch.isnan(bad_h[3]).all())
    for row, col in ((20, cols - 1), (127, 7)):
        assert bool(torch.isnan(bad_h[row, col])) and int(torch.isnan(bad_h[row]).sum()) == 1
        rest = torch.arange(cols, device=dev) != col
        assert torch.equal(bad_h[row][rest], h[row][rest])
    assert bool(torch.isnan(bad_h[40, 8])) and int((~torch.isfinite(bad_h[40])).sum()) == 1
    assert float(bad_h[41, cols - 1]) == float("inf") and float(bad_h[128, 0]) == -float("inf")
    # the rest, from the new residual
    zero = torch.zeros_like(o)
    no_gate, still = torch.zeros((2, cols), device=dev).bfloat16(), torch.zeros((2, 2, cols), device=dev).bfloat16()
    still[:, 0] = -0.0   # (a shift of 0 makes 0 of the -0 that a row with an infinite mean square has; its absence does not)
    again = h3q.h3q_residual_rmsnorm_adaln_nvfp4(bad_h.clone(), zero, no_gate, gamma, kw.get("mod_table", still), gsf,
                                                 rows_per_frame=75)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_rows_of_zeros_without_eps(dev):
    """With eps = 0 a row of zeros has no norm: no numbers in its row alone."""
    cols = 1024
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    h, o = torch.randn((9, cols), generator=g, device=dev), torch.randn((9, cols), generator=g, device=dev).bfloat16()
    ones, gsf = torch.ones(cols, device=dev).bfloat16(), gsf_tensor(100.0, dev)
    o[2], h[5] = 0, 0
    keep = h.clone()
    h3q.h3q_postnorm_residual_adaln_nvfp4(h, o, ones, ones, gsf, eps=0.0)
    assert bool(torch.isnan(h[2]).all())
    rest = torch.arange(9, device=dev) != 2
    want = keep[rest].double() + o[rest].double() / o[rest].double().pow(2).mean(1, keepdim=True).sqrt()
    assert float((h[rest].double() - want).abs().max()) <= 2.0 ** -20 * float(want.abs().max())
