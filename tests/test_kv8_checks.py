"""Refusals of the 8-bit cache's entry points that need no GPU: bad arguments are turned
down on the host before any CUDA call."""
import pytest
import torch

import speculative_decoding_verification_36_gb300 as sv
from speculative_decoding_verification_36_gb300 import _lib, build

# never dereferenced; the pools lie far apart
K, V, KC, VC, KS, VS, TAB, CTAB, ROWS = (0x100000000 * (i + 1) for i in range(9))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


BASE = dict(k=K, v=V, layers=1, ls=0, pages=4, ps=16, tab=TAB, mp=4, first=ROWS, last=ROWS + 4096, B=2, H=2, D=32, fmt=0, kc=KC, vc=VC,
            cst=0, ks=KS, vs=VS, sst=0, cp=4, block=16, ctab=CTAB, mcp=4, out=ROWS + 8192)


def quantize(lib, fn, **kw):
    a = dict(BASE, **kw)
    return getattr(lib, fn)(a["k"], a["v"], a["layers"], a["ls"], a["pages"], a["ps"], a["tab"], a["mp"], a["first"], a["last"], a["B"], a["H"],
                            a["D"], a["fmt"], a["kc"], a["vc"], a["cst"], a["ks"], a["vs"], a["sst"], a["cp"], a["block"], a["ctab"], a["mcp"],
                            a["out"], None)


def dequantize(lib, fn, **kw):
    a = dict(BASE, **kw)
    return getattr(lib, fn)(a["kc"], a["vc"], a["layers"], a["cst"], a["ks"], a["vs"], a["sst"], a["cp"], a["block"], a["ctab"], a["mcp"], a["first"],
                            a["last"], a["B"], a["H"], a["D"], a["fmt"], a["k"], a["v"], a["ls"], a["pages"], a["ps"], a["tab"], a["mp"], None)


SIZES = [dict(layers=0), dict(layers=32768), dict(B=-1), dict(H=0), dict(D=0), dict(D=8), dict(D=24), dict(D=272), dict(H=2 ** 16 + 1, D=256),
         dict(pages=0), dict(ps=0), dict(mp=0), dict(pages=2 ** 20, ps=2 ** 11), dict(cp=0), dict(block=0), dict(block=65537), dict(mcp=0),
         dict(cp=2 ** 20, block=2 ** 11), dict(mcp=2 ** 23 + 1), dict(mcp=2 ** 20, block=128), dict(fmt=2), dict(fmt=-1)]


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("call,fn", [(quantize, "spec_kv_quantize_"), (dequantize, "spec_kv_dequantize_")])
def test_cache_checks(lib, call, fn, t):
    for bad in SIZES:
        assert call(lib, fn + t, **bad) == _lib.SPEC_ERR_SHAPE, bad
    for name in ("k", "v", "tab", "first", "last", "kc", "vc", "ks", "vs", "ctab"):
        assert call(lib, fn + t, **{name: None}) == _lib.SPEC_ERR_NULL, name
    assert call(lib, fn + t, B=0, k=None, kc=None) == _lib.SPEC_OK
    for name in ("k", "v", "kc", "vc"):  # off a 16-byte boundary
        assert call(lib, fn + t, **{name: BASE[name] + 8}) == _lib.SPEC_ERR_SHAPE, name
    # layers closer together than their sizes, or off boundaries
    e = 4 if t == "f32" else 2
    entry, many = 64, dict(layers=3, ls=4 * 16 * 64, cst=4 * 16 * 64, sst=8)
    for bad in (dict(ls=4 * 16 * 64 - 16), dict(cst=4 * 16 * 64 - 16), dict(sst=7), dict(ls=-1), dict(ls=4 * 16 * 64 + 2), dict(cst=4 * 16 * 64 + 8)):
        assert call(lib, fn + t, **dict(many, **bad)) == _lib.SPEC_ERR_SHAPE, bad
    # what a call writes shares no memory with what it reads or with what else it writes
    size = 4 * 16 * entry
    both = [dict(kc=K), dict(vc=V + size * e - 16), dict(ks=K + 16), dict(k=KC + size - 16)]
    for bad in both + ([dict(kc=ROWS), dict(kc=VC), dict(vs=KS + 16), dict(kc=KS)] if call is quantize else [dict(v=ROWS + 4096), dict(k=V + 16)]):
        assert call(lib, fn + t, **bad) == _lib.SPEC_ERR_OVERLAP, bad
    if call is quantize:
        assert call(lib, fn + t, out=None) == _lib.SPEC_ERR_NULL
        for out in (ROWS, ROWS + 4096 + 4, K, KC + size - 4, KS, TAB, CTAB + 4):
            assert call(lib, fn + t, out=out) == _lib.SPEC_ERR_OVERLAP, hex(out)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_attention_checks(lib, t):
    f = getattr(lib, "spec_kv_attention_" + t)
    Q, OUT = 0xA00000000, 0xB00000000

    def call(q=Q, qs=128, k=K, v=V, pages=4, ps=16, tab=TAB, mp=4, ln=ROWS, n_new=None, par=None, kc=KC, vc=VC, ks=KS, vs=VS, cp=4, block=16,
             ctab=CTAB, mcp=4, st=ROWS + 4096, fmt=1, B=2, T=3, Hq=4, H=2, D=32, scale=1.0, out=OUT):
        return f(q, qs, k, v, pages, ps, tab, mp, ln, n_new, par, kc, vc, ks, vs, cp, block, ctab, mcp, st, fmt, B, T, Hq, H, D, scale, out, None)

    for name in ("q", "k", "v", "tab", "ln", "kc", "vc", "ks", "vs", "ctab", "st", "out"):
        assert call(**{name: None}) == _lib.SPEC_ERR_NULL, name
    for bad in SIZES[2:]:
        if "B" in bad or "layers" in bad:
            continue
        assert call(**{dict(H="H").get(n, n): x for n, x in bad.items()}) == _lib.SPEC_ERR_SHAPE, bad
    for bad in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(Hq=3), dict(qs=127), dict(scale=float("nan")), dict(scale=float("inf")), dict(par=ROWS, T=1026),
                dict(B=2 ** 20, T=2 ** 12), dict(Hq=2 ** 20, qs=2 ** 25), dict(T=2 ** 29, B=1), dict(out=OUT + 8), dict(kc=KC + 4)):
        assert call(**bad) == _lib.SPEC_ERR_SHAPE, bad
    assert call(B=0, q=None) == _lib.SPEC_OK and call(T=0, q=None) == _lib.SPEC_OK
    for out in (Q, Q + 16, K, V + 16, KC, VC + 4096 - 16, KS, VS, TAB, CTAB, ROWS, ROWS + 4096):
        assert call(out=out) == _lib.SPEC_ERR_OVERLAP, hex(out)


def test_binding_checks():
    x = torch.zeros((2, 4, 2, 32))
    with pytest.raises(ValueError):
        sv.spec_kv_quantize(x, x, x, x, x, x, x, x, x, x)
    with pytest.raises(ValueError):
        sv.spec_kv_attention(x, x, x, x, x, x, x, x, x, x, x)
    with pytest.raises(ValueError):
        sv.spec_kv_dequantize(x, x, x, x, x, x[0, 0, 0], x, x, x, x)
