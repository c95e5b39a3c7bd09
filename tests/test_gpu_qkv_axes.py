"""GPU: the QKV epilogue with rotary positions of several axes, against the formula in 64 bits: head sizes and
groups, splits of the axes, both pairings, sections, scales, positions far away and negative, strided views, and rows
that do not fill the GPU."""
import numpy as np
import pytest
import torch

import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def _inputs(dev, rows, heads, kv_heads, dim, dims, far, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    d, dk = heads * dim, kv_heads * dim
    packed = torch.randn((rows, d + 2 * dk + 16), generator=g, device=dev).bfloat16()   # q, k, v and something else
    r = lambda n: torch.randn(n, generator=g, device=dev).bfloat16()  # noqa: E731
    return {"q": packed[:, :d], "k": packed[:, d:d + dk], "v": packed[:, d + dk:d + 2 * dk], "biases": (r(d), r(dk), r(dk)),
            "weights": (r(dim), r(dim)),
            "positions": torch.randint(-far, far + 1, (rows, len(dims)), generator=g, device=dev).int()}


def _want(x, bias, weight, positions, dims, theta, scale, sections, pairs, norm, eps, heads):
    """The formula in 64 bits, and the size that its fp32 errors are counted in."""
    rows = x.shape[0]
    x = x.double().unflatten(1, (heads, -1))
    if bias is not None:
        x = x + bias.double().view(heads, -1)
    dim = x.shape[-1]
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double()
    rot = sum(dims)
    f = []
    for a, d in enumerate(dims):
        for i in range(d // 2):
            power = 2 * len(f) / rot if sections else 2 * i / d
            f.append((a, scale[a] * (theta[0] if sections else theta[a]) ** -power))
    angle = torch.stack([positions[:, a].double() * w for a, w in f], 1)[:, None]   # [rows, 1, rot / 2]
    c, s = torch.cos(angle), torch.sin(angle)
    j = torch.arange(rot // 2, device=x.device)
    lo, hi = (2 * j, 2 * j + 1) if pairs else (j, j + rot // 2)
    out, size = x.clone(), x.abs()
    out[..., lo] = x[..., lo] * c - x[..., hi] * s
    out[..., hi] = x[..., hi] * c + x[..., lo] * s
    both = x[..., lo].abs() + x[..., hi].abs()
    size[..., lo] = both
    size[..., hi] = both
    assert out.shape == (rows, heads, dim)
    return out, size


def _check(got, want, size, what):
    """One rounding to bf16 (2^-8), and fp32's own: the mean of at most 256 squares in 8 products and 5 sums (2^-20), the
    square root's reciprocal, weights, cosines and sines (each 2^-22 of the pair), the angle, rounded in turns
    (pi 2^-24), and four products and sums: 2^-18 of the pair's magnitudes covers them.  Angles that come from
    doubles on both sides differ by 2^-50 of a position of 2^30 at most: 2^-20."""
    tol = want.abs() * 2.0 ** -8 + size * 2.0 ** -18 + 1e-38
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: off by {float((err / tol).max()):.3g} of what is allowed"


CASES = [  # rows, heads, kv heads, dim, axis dims, far
    (1, 1, 1, 128, (128,), 5),
    (37, 8, 2, 64, (16, 24, 24), 50),
    (5, 56, 56, 128, (44, 42, 42), 100),
    (130, 3, 3, 128, (30, 34), 1000),            # 64 of 128 turn
    (41, 7, 1, 64, (16,), 30),
    (29, 5, 5, 256, (62, 68, 14, 96), 1_000_000),
    (33, 4, 4, 256, (2, 14), 2_000_000_000),
    (1000, 12, 4, 128, (16, 56, 56), 3000),
    (3, 64, 8, 128, (2, 2, 12), 7),
    (20_000, 2, 1, 64, (20, 44), 100_000),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm, bias, weights", [(True, True, True), (True, False, False), (False, True, False)])
def test_against_the_formula(dev, case, pairs, norm, bias, weights):
    rows, heads, kv_heads, dim, dims, far = CASES[case]
    w = _inputs(dev, rows, heads, kv_heads, dim, dims, far, case)
    sections = case % 4 == 2
    theta = [10000.0, 500.0, 1e6, 3.0][:len(dims)] if case % 2 else [10000.0] * len(dims)
    scale = [1.0, 0.25, 1.7, -1.0][:len(dims)] if case % 3 == 1 else [1.0] * len(dims)
    got = h3q.h3q_qkv_epilogue_axes(
        w["q"], w["k"], w["v"], w["positions"], dims, heads, kv_heads=kv_heads, theta=theta, scale=scale,
        sections=sections, biases=w["biases"] if bias else None, weights=w["weights"] if weights else None, norm=norm,
        interleaved=pairs)
    for i, (name, h) in enumerate((("q", heads), ("k", kv_heads))):
        want, size = _want(w[name], w["biases"][i] if bias else None, w["weights"][i] if weights else None, w["positions"],
                           dims, theta, scale, sections, pairs, norm, 1e-6, h)
        _check(got[i], want, size, f"case {case} {name}")
    v = w["v"].double() + (w["biases"][2].double() if bias else 0)
    assert torch.equal(got[2], v.bfloat16().unflatten(1, (kv_heads, dim)))


def test_whole_turns_leave_nothing(dev):
    """Positions that are multiples of a period of 2^k turn by nothing, however far."""
    import math

    rows, dim = 64, 64
    w = _inputs(dev, rows, 1, 1, dim, (64,), 0, 30)
    # theta = 1: every pair turns by scale a step; a scale of 2 pi / 8 is an eighth of a turn
    w["positions"][:, 0] = torch.arange(rows, device=dev) * 8 * 1_000_003
    got = h3q.h3q_qkv_epilogue_axes(w["q"], w["k"], w["v"], w["positions"], (64,), 1, theta=1.0, scale=2 * math.pi / 8,
                                    norm=False)
    # (an eighth of a turn as a double is off by 2^-53 of it: 2^-27 of a turn at 2^29)
    assert float((got[0].double().view(rows, dim) - w["q"].double()).abs().max()) <= 2.0 ** -8 * float(w["q"].abs().max())


def test_an_existing_epilogue_of_one_axis(dev):
    """One axis, no weights, rotate-half: what h3q_qkv_epilogue gives with tables, within its bf16 steps."""
    rows, heads, dim = 300, 4, 128
    w = _inputs(dev, rows, heads, heads, dim, (64,), 0, 31)
    w["positions"][:, 0] = torch.arange(rows, device=dev)
    got = h3q.h3q_qkv_epilogue_axes(w["q"], w["k"], w["v"], w["positions"], (64,), heads, biases=w["biases"])
    f = 10000.0 ** (-2 * torch.arange(32, device=dev).double() / 64)
    angle = (torch.arange(rows, device=dev).double()[:, None] * f).repeat(1, 2)
    old = h3q.h3q_qkv_epilogue(w["q"], w["k"], w["v"], w["biases"], angle.cos().bfloat16(), angle.sin().bfloat16(), heads,
                               1e-6)
    for a, b in zip(got[:2], old[:2]):
        # there x', n, cos, sin, two products and the sum are each rounded to bf16, here the result alone: 8 halves of
        # a step of the pair's size, which is at most sqrt(2) times the norm of its two values
        pair = torch.stack((b[..., :32].float(), b[..., 32:64].float())).norm(dim=0).repeat(1, 1, 2)
        assert bool(((a[..., :64].float() - b[..., :64].float()).abs() <= 8 * 2.0 ** -8 * 1.5 * pair + 1e-6).all())
    assert torch.equal(got[2], old[2])


def test_stream_and_graph(dev):
    rows, heads, dim, dims = 200, 4, 128, (44, 42, 42)
    w = _inputs(dev, rows, heads, 2, dim, dims, 100, 32)
    want = h3q.h3q_qkv_epilogue_axes(w["q"], w["k"], w["v"], w["positions"], dims, heads, kv_heads=2)
    stream = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    got = h3q.h3q_qkv_epilogue_axes(w["q"], w["k"], w["v"], w["positions"], dims, heads, kv_heads=2, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3q.h3q_qkv_epilogue_axes(w["q"], w["k"], w["v"], w["positions"], dims, heads, kv_heads=2, outs=outs)
    w["positions"] += 3
    graph.replay()
    want = h3q.h3q_qkv_epilogue_axes(w["q"], w["k"], w["v"], w["positions"], dims, heads, kv_heads=2)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_rows_past_2_31_elements(dev):
    rows, heads, dim = 300_000, 56, 128
    x = torch.empty((rows, heads * dim), dtype=torch.bfloat16, device=dev)
    g = torch.Generator(device=dev)
    g.manual_seed(33)
    x[:] = torch.randn((1, heads * dim), generator=g, device=dev).bfloat16()
    kv = x[:, :128]
    positions = torch.arange(rows, device=dev, dtype=torch.int32)[:, None].contiguous()
    q, k, v = h3q.h3q_qkv_epilogue_axes(x, kv, kv, positions, (128,), heads, kv_heads=1)
    at = torch.tensor([0, 1, 299_593, 299_999], device=dev)   # 2^31 / 7,168 = 299,593
    want, size = _want(x[at], None, None, positions[at], (128,), [10000.0], [1.0], False, False, True, 1e-6, heads)
    _check(q[at], want, size, "far rows")
    assert torch.equal(v[at].flatten(1), kv[at])
    assert np.isfinite(float(k.float().sum()))
