"""GPU: the calls of rotary axes, norms around a block and attention over blocks through the C module and without it:
the same results, and the same refusals in words."""
import pytest
import torch

import block_cases as bc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def args():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    torch.cuda.set_device(0)
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()  # noqa: E731
    c = bc.sequences(dev, [(200, 500), (64, 300)], 4, 2, 128, seed=1)
    return {**c, "x": r(40, 512), "kv": r(40, 256), "pos": torch.randint(-9, 9, (40, 2), generator=g, device=dev).int(),
            "bias": r(512), "kv_bias": r(256), "weight": r(128), "h": torch.randn((40, 512), generator=g, device=dev),
            "gamma": r(512), "gate": r(3, 512), "table": r(3, 2, 512), "frame": torch.zeros(40, device=dev).int(),
            "gsf": torch.full((1,), 90.0, device=dev), "lists": bc.random_lists(c, 2, 64, 64, 4, 1)}


CALLS = {
    "axes": lambda a: h3q.h3q_qkv_epilogue_axes(a["x"], a["kv"], a["kv"], a["pos"], (64, 48), 4, kv_heads=2,
                                                theta=(1e4, 100), scale=[1, 0.5], biases=(a["bias"], None, a["kv_bias"]),
                                                weights=(a["weight"], None)),
    "postnorm": lambda a: h3q.h3q_postnorm_residual_adaln_nvfp4(
        a["h"].clone(), a["x"], a["gamma"], a["gamma"], a["gsf"], bias=a["bias"], gate_table=a["gate"],
        mod_table=a["table"], row_frame=a["frame"], residual_scale=0.5),
    "select": lambda a: [h3q.h3q_select_blocks(a["q"], a["k"], a["cu_q"], a["cu_k"], 4, block_q=64, block_k=64,
                                               causal=True, first=1)],
    "blocks": lambda a: [h3q.h3q_attention_blocks(a["q"], a["k"], a["v"], a["cu_q"], a["cu_k"], a["lists"], block_q=64,
                                                  block_k=64, causal=True)[:264]],
}


class NoShortWay:
    axes = postnorm = select = blocks = staticmethod(lambda *a: None)


def test_both_ways_agree(args, monkeypatch):
    short = {name: [t.clone() for t in call(args)] for name, call in CALLS.items()}
    monkeypatch.setattr(h3q, "_native", NoShortWay)
    for name, call in CALLS.items():
        for a, b in zip(short[name], call(args)):
            assert torch.equal(a, b), name


BAD = [  # argument, how it is spoilt, the calls that take it, what is raised
    ("x", lambda t: t.float(), ("axes", "postnorm"), TypeError, "bfloat16"),
    ("x", lambda t: t.t(), ("axes", "postnorm"), ValueError, "contiguous rows"),
    ("x", lambda t: t[:39], ("axes", "postnorm"), ValueError, "rows|shape"),
    ("x", lambda t: t.cpu(), ("axes", "postnorm"), ValueError, "CUDA"),
    ("kv", lambda t: t[:, :128], ("axes",), ValueError, "kv_heads"),
    ("pos", lambda t: t.long(), ("axes",), TypeError, "int32"),
    ("pos", lambda t: t[:, :1], ("axes",), ValueError, "positions"),
    ("bias", lambda t: t[:256], ("axes", "postnorm"), ValueError, "bias"),
    ("weight", lambda t: t.float(), ("axes",), TypeError, "bfloat16"),
    ("h", lambda t: t.bfloat16(), ("postnorm",), TypeError, "float32"),
    ("gamma", lambda t: t[None], ("postnorm",), ValueError, "gamma"),
    ("gate", lambda t: t[:2], ("postnorm",), ValueError, "frames"),
    ("gate", lambda t: t[:, :256], ("postnorm",), ValueError, "gate_table"),
    ("table", lambda t: t[:, :1], ("postnorm",), ValueError, "mod_table"),
    ("frame", lambda t: t.long(), ("postnorm",), TypeError, "int32"),
    ("gsf", lambda t: torch.cat((t, t)), ("postnorm",), ValueError, "global_scale"),
    ("q", lambda t: t.half(), ("select", "blocks"), TypeError, "bfloat16"),
    ("q", lambda t: t.transpose(0, 1), ("select", "blocks"), ValueError, "contiguous rows"),
    ("q", lambda t: t[:, :3].contiguous(), ("select", "blocks"), h3q.H3QError, "multiple of kv_heads"),
    ("q", lambda t: t[:, :, :64].contiguous(), ("select", "blocks"), ValueError, "head_dim"),
    ("k", lambda t: t[0], ("select", "blocks"), ValueError, "rows, heads"),
    ("v", lambda t: t[:9], ("blocks",), ValueError, "k and v"),
    ("cu_q", lambda t: t.long(), ("select", "blocks"), TypeError, "int32"),
    ("cu_q", lambda t: t[None], ("select", "blocks"), ValueError, "cu_q"),
    ("cu_k", lambda t: t[:2], ("select", "blocks"), ValueError, "cu_k"),
    ("lists", lambda t: t.long(), ("blocks",), TypeError, "int32"),
    ("lists", lambda t: t[:, :3].contiguous(), ("blocks",), ValueError, "blocks must be"),
    ("lists", lambda t: t[:, :, ::2], ("blocks",), ValueError, "blocks must be"),
]


@pytest.mark.parametrize("short", [True, False])
@pytest.mark.parametrize("case", range(len(BAD)))
def test_refusals_in_words(args, monkeypatch, case, short):
    name, spoil, calls, error, what = BAD[case]
    if not short:
        monkeypatch.setattr(h3q, "_native", NoShortWay)
    for call in calls:
        with pytest.raises(error, match=what):
            CALLS[call]({**args, name: spoil(args[name])})


def test_outputs_that_do_not_fit(args):
    a = args
    with pytest.raises(ValueError, match="workspace"):
        h3q.h3q_select_blocks(a["q"], a["k"], a["cu_q"], a["cu_k"], 4, block_q=64, block_k=64,
                              workspace=torch.empty(100, dtype=torch.uint8, device=a["q"].device))
    with pytest.raises(ValueError, match="out"):
        h3q.h3q_attention_blocks(a["q"], a["k"], a["v"], a["cu_q"], a["cu_k"], a["lists"], block_q=64, block_k=64,
                                 out=a["q"][:5].contiguous())
    with pytest.raises(ValueError, match="q_out|k_out"):
        h3q.h3q_qkv_epilogue_axes(a["x"], a["kv"], a["kv"], a["pos"], (64, 48), 4, kv_heads=2,
                                  outs=[a["q"], a["q"], a["q"]])
    with pytest.raises(h3q.H3QError, match="overlap"):
        h3q.h3q_attention_blocks(a["q"], a["k"], a["v"], a["cu_q"], a["cu_k"], a["lists"], block_q=64, block_k=64,
                                 out=a["q"])
    for top in (-1, 0, 4097):
        with pytest.raises(ValueError, match="top"):
            h3q.h3q_select_blocks(a["q"], a["k"], a["cu_q"], a["cu_k"], top, block_q=64, block_k=64)
    with pytest.raises(ValueError, match="cu_q"):
        h3q.h3q_select_blocks(a["q"], a["k"], a["cu_q"][:0], a["cu_k"], 4, block_q=64, block_k=64)
    with pytest.raises(h3q.H3QError, match="no room"):
        h3q.h3q_select_blocks(a["q"], a["k"], a["cu_q"], a["cu_k"], 2, block_q=64, block_k=64, causal=True, first=1)
