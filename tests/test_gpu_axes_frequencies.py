"""GPU: rotary axes with frequencies far from one and positions far away: angles within what the header states, against
powers and turns in 60 digits; and rows of values that are no numbers, or nothing."""
import decimal
import math

import pytest
import torch

import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu

D = decimal.Decimal
PI = D("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


CASES = [  # theta, scale, farthest position
    (10000.0, 1.0, 2 ** 31 - 1), (10000.0, -1.0, 10 ** 6), (0.5, 1.0, 10 ** 6), (1e-3, 3.0, 2 ** 31 - 1),
    (10000.0, 2.0 ** 20, 10 ** 5), (3.0, 2.0 ** 20, 2 ** 30), (1e6, -2.0 ** 12, 2 ** 31 - 1), (1e300, 1.0, 10 ** 9),
]


@pytest.mark.parametrize("theta, scale, far", CASES)
@pytest.mark.parametrize("sections", [False, True])
def test_angles_against_sixty_digits(dev, theta, scale, far, sections):
    decimal.getcontext().prec = 60
    dim, rows = 64, 24
    g = torch.Generator().manual_seed(7)
    positions = torch.randint(-far, far + 1, (rows, 1), generator=g)
    positions[0], positions[1], positions[2] = far, -far, 1
    q = torch.zeros((rows, dim), device=dev, dtype=torch.bfloat16)
    q[:, :dim // 2] = 1.0                                    # (1, 0) turned: cosine and sine
    out = h3q.h3q_qkv_epilogue_axes(q, q, q, positions.int().to(dev), (dim,), 1, theta=theta, scale=scale, norm=False,
                                    sections=sections)[0].double().cpu().view(rows, 2, dim // 2)
    for i in range(dim // 2):
        f = D(scale) * (D(theta).ln() * D(-2 * i) / D(dim)).exp()
        for r, p in enumerate(positions[:, 0].tolist()):
            angle = float((f * D(p)) % (2 * PI))
            off = abs(p) * (abs(float(f)) * (2 + abs(math.log2(theta))) * 2.0 ** -51 + 2.0 ** -50) + 2 * math.pi * 2.0 ** -23
            for got, want in zip(out[r, :, i].tolist(), (math.cos(angle), math.sin(angle))):
                assert abs(got - want) <= off + abs(want) * 2.0 ** -8 + 2.0 ** -22, (i, p)


def test_values_that_are_no_numbers_stay_in_their_head(dev):
    """A value that is none, or infinite, reaches its own head's (with a norm) or pair's outputs alone."""
    rows, heads, dim = 40, 4, 64
    g = torch.Generator(device=dev)
    g.manual_seed(8)
    x = torch.randn((rows, heads * dim), generator=g, device=dev).bfloat16()
    pos = torch.arange(rows, device=dev, dtype=torch.int32)[:, None].contiguous() + 1
    for norm in (True, False):
        for interleaved in (True, False):
            call = lambda t: h3q.h3q_qkv_epilogue_axes(t, t, t, pos, (32,), heads, norm=norm, interleaved=interleaved)  # noqa: E731
            want = call(x)
            bad = x.clone()
            bad[5, 2 * dim + 3], bad[7, dim + 40], bad[9, 3] = float("nan"), float("inf"), -float("inf")
            got = call(bad)
            partner = 2 if interleaved else 3 + 16
            hit = torch.zeros((rows, heads, dim), dtype=torch.bool, device=dev)
            if norm:
                hit[5, 2], hit[7, 1], hit[9, 0] = True, True, True
            else:
                hit[5, 2, [3, partner]], hit[7, 1, 40], hit[9, 0, [3, partner]] = True, True, True
            for a, b in zip(got[:2], want[:2]):
                assert torch.equal(a[~hit], b[~hit])
                assert bool(torch.isnan(a[5, 2][hit[5, 2]]).all())
                if norm:   # an infinite mean square: 0 for the others, no number for its own (and its pair)
                    assert bool(torch.isnan(a[7, 1, 40])) and bool(torch.isnan(a[9, 0, [3, partner]]).all())
                    rest = torch.ones(dim, dtype=torch.bool, device=dev)
                    rest[40] = False
                    assert bool((a[7, 1][rest] == 0).all())
                else:
                    assert float(a[7, 1, 40]) == float("inf") and bool(torch.isinf(a[9, 0, [3, partner]]).all())
            v = got[2].view(rows, -1)
            assert torch.equal(v.isnan(), bad.isnan()) and torch.equal(v[~v.isnan()], bad[~bad.isnan()])


def test_heads_of_zeros(dev):
    """With eps = 0 no numbers, with any other eps zeros."""
    x = torch.zeros((3, 128), device=dev, dtype=torch.bfloat16)
    x[1] = 1.0
    pos = torch.ones((3, 1), device=dev, dtype=torch.int32)
    q, k, v = h3q.h3q_qkv_epilogue_axes(x, x, x, pos, (128,), 1, eps=0.0)
    for t in (q, k):
        assert bool(torch.isnan(t[0]).all()) and bool(torch.isnan(t[2]).all()) and bool(torch.isfinite(t[1]).all())
    assert bool((v.view(3, 128) == x).all())
    q, _, _ = h3q.h3q_qkv_epilogue_axes(x, x, x, pos, (128,), 1, eps=1e-30)
    assert bool((q[0] == 0).all())
