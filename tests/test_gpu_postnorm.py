"""GPU: the norm after a block, gate and scaled residual, the next norm and its modulation -> NVFP4, bit for bit
against numpy in binary32 with the oracle's row statistics and block quantize: widths, ragged rows, tables and biases
that are there or not, strides, frames by rows, in place, graphs."""
import numpy as np
import pytest
import torch

import nvfp4_activation_quantize_gb300 as h3q
import oracle
from parity import bits, check_rows, fill, gsf_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def _inputs(dev, rows, cols, frames, bias, gate, table, seed, strided=False):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    wide = cols + 32 if strided else cols
    return {"h": (2 * r(rows, wide))[:, :cols], "o": r(rows, wide).bfloat16()[:, :cols], "post": r(cols).bfloat16(),
            "gamma": r(cols).bfloat16(), "bias": r(cols).bfloat16() if bias else None,
            "gate": r(frames, cols).bfloat16() if gate else None,
            "table": (0.5 * r(frames, 2, cols)).bfloat16() if table else None}


def _f32(t):
    return t.detach().float().cpu().numpy()


def _want(w, frames, keep, eps, gsf):
    """h', codes, logical scales and rstd: one binary32 rounding an operation."""
    o = w["o"]
    if w["bias"] is not None:
        o = (o.float() + w["bias"].float()).bfloat16()
    u = _f32(o)
    rstd_u = np.array([oracle.row_rstd(b, eps) for b in bits(o)], np.float32)[:, None]
    n = u * rstd_u * _f32(w["post"])
    if w["gate"] is not None:
        n = n * _f32(w["gate"])[frames]
    h = _f32(w["h"]) * np.float32(keep) + n
    rstd = np.array([oracle.row_rstd_f32(x, eps) for x in h], np.float32)
    y = h * rstd[:, None] * _f32(w["gamma"])
    if w["table"] is not None:
        t = _f32(w["table"])
        y = y * (np.float32(1) + t[frames, 1]) + t[frames, 0]
    codes, sf = oracle.quantize_rows(oracle.bf16_bits(y.astype(np.float32)), gsf)
    return h, codes, sf, rstd


def _check(dev, w, frames, keep=1.0, eps=1e-6, gsf=200.0, **kw):
    rows, cols = w["o"].shape
    want_h, codes_ref, sf_ref, rstd_ref = _want(w, frames, keep, eps, gsf)
    codes = fill(torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev))
    scales = fill(torch.empty((h3q.padded_rows(rows), cols // 16), dtype=torch.uint8, device=dev))
    rstd = torch.empty(rows, device=dev)
    h3q.h3q_postnorm_residual_adaln_nvfp4(w["h"], w["o"], w["post"], w["gamma"], gsf_tensor(gsf, dev), bias=w["bias"],
                                          gate_table=w["gate"], mod_table=w["table"], residual_scale=keep, eps=eps,
                                          codes=codes, scales=scales, row_rstd=rstd, **kw)
    got = w["h"].cpu().numpy()
    assert (got.view(np.uint32) == want_h.view(np.uint32)).all(), "h differs"
    assert (rstd.cpu().numpy().view(np.uint32) == rstd_ref.view(np.uint32)).all(), "rstd differs"
    check_rows(codes, scales, np.arange(rows), cols, codes_ref, sf_ref, f"{rows} x {cols}")


CASES = [(1, 64), (5, 128), (37, 1024), (64, 960), (130, 1088), (300, 2048), (64, 4096), (33, 5120), (129, 7168), (200, 7104),
         (31, 8192), (17, 8128)]


@pytest.mark.parametrize("rows, cols", CASES)
@pytest.mark.parametrize("bias, gate, table", [(True, True, True), (False, False, False), (False, True, False),
                                               (True, False, True)])
def test_bit_exact(dev, rows, cols, bias, gate, table):
    frames = 3
    w = _inputs(dev, rows, cols, frames, bias, gate, table, rows + cols, strided=rows % 2 == 1)
    per = -(-rows // frames)
    kw = {"rows_per_frame": per} if gate or table else {}
    _check(dev, w, np.arange(rows) // per, keep=[1.0, 0.9375, 0.7][rows % 3], **kw)


def test_frames_by_rows(dev):
    rows, cols = 300, 1024
    w = _inputs(dev, rows, cols, 7, True, True, True, 1)
    frames = torch.randint(0, 7, (rows,), device=dev, dtype=torch.int32)
    _check(dev, w, frames.cpu().numpy(), keep=1.25, row_frame=frames)


def test_rows_of_zero_and_one_value(dev):
    """A block that adds nothing, a residual of nothing, and a residual scale of zero."""
    w = _inputs(dev, 64, 1024, 1, False, False, False, 2)
    w["o"][:20] = 0
    w["h"][10:30] = 0
    w["o"][40] = 1.0
    _check(dev, w, np.zeros(64, int))
    w = _inputs(dev, 64, 1024, 1, False, False, False, 3)
    _check(dev, w, np.zeros(64, int), keep=0.0)


def test_without_the_first_norm_it_is_the_residual_fold(dev):
    """Rows of o whose norm is 1 under a gamma_post of ones: what h3q_residual_rmsnorm_adaln_nvfp4 gives."""
    rows, cols, frames = 128, 1024, 4
    w = _inputs(dev, rows, cols, frames, False, True, True, 4)
    w["o"] = torch.where(torch.rand((rows, cols), device=dev) < 0.5, -1.0, 1.0).bfloat16()
    w["post"] = torch.ones(cols, device=dev).bfloat16()
    one = gsf_tensor(100.0, dev)
    h = w["h"].clone()
    a = h3q.h3q_postnorm_residual_adaln_nvfp4(w["h"], w["o"], w["post"], w["gamma"], one, gate_table=w["gate"],
                                              mod_table=w["table"], rows_per_frame=32, eps=0.0)
    b = h3q.h3q_residual_rmsnorm_adaln_nvfp4(h, w["o"], w["gate"], w["gamma"], w["table"], one, rows_per_frame=32, eps=0.0)
    assert torch.equal(h, w["h"]) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_every_row_of_many(dev):
    """More rows than CTAs, frames that change within a CTA's rows: against the same call in pieces."""
    rows, cols, frames = 3001, 7168, 32
    w = _inputs(dev, rows, cols, frames, True, True, True, 5)
    gsf = gsf_tensor(150.0, dev)
    frame = (torch.arange(rows, device=dev) * frames // rows).int()
    h = w["h"].clone()
    call = lambda h, o, f: h3q.h3q_postnorm_residual_adaln_nvfp4(  # noqa: E731
        h, o, w["post"], w["gamma"], gsf, bias=w["bias"], gate_table=w["gate"], mod_table=w["table"], row_frame=f)
    codes, scales = call(w["h"], w["o"], frame)
    for at in range(0, rows, 128):
        end = min(rows, at + 128)
        c, s = call(h[at:end], w["o"][at:end], frame[at:end].contiguous())
        assert torch.equal(codes[at:end], c) and torch.equal(scales[at:at + 128], s)
    assert torch.equal(h, w["h"])


def test_stream_and_graph(dev):
    w = _inputs(dev, 100, 1024, 1, True, False, False, 6)
    gsf = gsf_tensor(150.0, dev)
    h = w["h"].clone()
    call = lambda h, **kw: h3q.h3q_postnorm_residual_adaln_nvfp4(  # noqa: E731
        h, w["o"], w["post"], w["gamma"], gsf, bias=w["bias"], residual_scale=0.5, **kw)
    want = [t.clone() for t in (*call(h), h)]
    stream = torch.cuda.Stream(dev)
    other = w["h"].clone()
    torch.cuda.synchronize()
    got = call(other, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, other), want))
    third = w["h"].clone()
    codes, scales = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(third, codes=codes, scales=scales)
    third.copy_(w["h"])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((codes, scales, third), want))
