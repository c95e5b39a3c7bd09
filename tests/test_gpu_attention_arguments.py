"""GPU: what the Python binding of the cache and attention calls refuses, and that the way through its C module
and the way through Python's own checks give the same."""
import pytest
import torch

import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.fixture
def args(dev):
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    rows = lambda n, h: torch.randn((n, h, 64), generator=g, device=dev).bfloat16()  # noqa: E731
    cache = h3q.kv_cache_nvfp4(4, 2, 16, 64, dev)
    return {"q": rows(5, 4), "k": rows(5, 2), "v": rows(5, 2), "cache": cache, "cu": cc.ints([0, 2, 5], dev),
            "len": cc.ints([2, 20], dev), "table": cc.ints([[3, 0], [1, 2]], dev), "one": torch.ones(1, device=dev)}


def _calls(a):
    lists = a["cu"], a["len"], a["table"], a["one"], a["one"]
    return {
        "write": lambda: h3q.h3q_kv_cache_write_nvfp4(a["k"], a["v"], a["cache"], *lists),
        "read": lambda: h3q.h3q_kv_cache_read_nvfp4(a["cache"], *lists, rows=5),
        "cached": lambda: h3q.h3q_attention_cache_nvfp4(a["q"], a["cache"], *lists, max_rows=3),
        "varlen": lambda: h3q.h3q_attention_varlen(a["q"], a["k"], a["v"], a["cu"], a["cu"]),
    }


def test_both_ways_agree(dev, args, monkeypatch):
    def results():
        for t in args["cache"]:
            t.zero_()
        out = [t.clone() for t in _calls(args)["write"]()]
        for name in ("read", "cached", "varlen"):
            got = _calls(args)[name]()
            out += list(got) if isinstance(got, tuple) else [got]
        return out

    short = results()

    class NoShortWay:
        write = read = cached = varlen = staticmethod(lambda *a: None)

    monkeypatch.setattr(h3q, "_native", NoShortWay)
    for a, b in zip(short, results()):
        assert torch.equal(a, b)


BAD = [  # argument, how it is spoilt, the calls that take it, what they say
    ("k", lambda t: t.float(), ("write", "varlen"), TypeError, "bfloat16"),
    ("k", lambda t: t[:, :, :32], ("write", "varlen"), ValueError, "contiguous rows|head"),
    ("v", lambda t: t[:4], ("write", "varlen"), ValueError, "k and v"),
    ("k", lambda t: t.cpu(), ("write", "varlen"), ValueError, "CUDA"),
    ("q", lambda t: t.transpose(0, 1), ("cached", "varlen"), ValueError, "contiguous rows"),
    ("q", lambda t: t.half(), ("cached", "varlen"), TypeError, "bfloat16"),
    ("q", lambda t: t[:, :3].contiguous(), ("cached", "varlen"), h3q.H3QError, "multiple of kv_heads"),
    ("cu", lambda t: t.long(), ("write", "read", "cached", "varlen"), TypeError, "int32"),
    ("cu", lambda t: t[:2], ("write", "read", "cached"), ValueError, "cu_rows"),
    ("len", lambda t: t[None], ("write", "read", "cached"), ValueError, "kv_len"),
    ("table", lambda t: t[:1], ("write", "read", "cached"), ValueError, "block_table"),
    ("table", lambda t: t.t(), ("write", "read", "cached"), ValueError, "block_table"),
    ("one", lambda t: t.double(), ("write", "read", "cached"), TypeError, "float32"),
    ("one", lambda t: t.repeat(2), ("write", "read", "cached"), ValueError, "one fp32"),
    ("cache", lambda c: c[:3], ("write", "read", "cached"), ValueError, "cache must be"),
    ("cache", lambda c: (c[0], c[1][:, :, :, :2], c[2], c[3]), ("write", "read", "cached"), ValueError, "k_scales"),
    ("cache", lambda c: (c[0].int(), *c[1:]), ("write", "read", "cached"), TypeError, "uint8"),
    ("cache", lambda c: tuple(t[:, :, :8].contiguous() for t in c), ("write", "read", "cached"), h3q.H3QError,
     "page_size"),
]


@pytest.mark.parametrize("case", range(len(BAD)))
def test_refusals(dev, args, case):
    name, spoil, calls, error, words = BAD[case]
    args[name] = spoil(args[name])
    for call in calls:
        with pytest.raises(error, match=words):
            _calls(args)[call]()


def test_outputs_are_checked(dev, args):
    lists = args["cu"], args["len"], args["table"], args["one"], args["one"]
    out = torch.empty((5, 4, 64), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((4, 5), device=dev)
    with pytest.raises(ValueError, match="out"):
        h3q.h3q_attention_varlen(args["q"], args["k"], args["v"], args["cu"], args["cu"], out=out[:4])
    with pytest.raises(ValueError, match="lse"):
        h3q.h3q_attention_varlen(args["q"], args["k"], args["v"], args["cu"], args["cu"], lse=lse.t())
    with pytest.raises(ValueError, match="tree_mask"):
        h3q.h3q_attention_cache_nvfp4(args["q"], args["cache"], *lists, max_rows=3,
                                      tree_mask=torch.zeros(4, dtype=torch.int64, device=dev))
    with pytest.raises(h3q.H3QError, match="max_rows"):
        h3q.h3q_attention_cache_nvfp4(args["q"], args["cache"], *lists, max_rows=65)
    with pytest.raises(ValueError, match="k_out"):
        h3q.h3q_kv_cache_read_nvfp4(args["cache"], *lists, outs=(out, out))
    with pytest.raises(ValueError, match="rows or outs"):
        h3q.h3q_kv_cache_read_nvfp4(args["cache"], *lists)
    with pytest.raises(h3q.H3QError, match="scale"):
        h3q.h3q_attention_varlen(args["q"], args["k"], args["v"], args["cu"], args["cu"], scale=-1.0)


def test_numbers_of_other_types(dev, args):
    """Whole numbers and truth values where Python lets them stand for one another."""
    lists = args["cu"], args["len"], args["table"], args["one"], args["one"]
    a = h3q.h3q_attention_varlen(args["q"], args["k"], args["v"], args["cu"], args["cu"], causal=1, scale=1)
    b = h3q.h3q_attention_varlen(args["q"], args["k"], args["v"], args["cu"], args["cu"], causal=True, scale=1.0)
    assert torch.equal(a, b)
    a = h3q.h3q_attention_cache_nvfp4(args["q"], list(args["cache"]), *lists, max_rows=3.0)
    b = h3q.h3q_attention_cache_nvfp4(args["q"], args["cache"], *lists, max_rows=3)
    assert torch.equal(a, b)
