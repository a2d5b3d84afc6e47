"""Sizes past which the 8-bit cache's kernels would count wrongly are refused on the host, before any
CUDA call."""
import pytest

from speculative_decoding_verification_36_gb300 import _lib
from test_kv8_checks import BASE, CTAB, K, KC, KS, ROWS, TAB, V, VC, VS, dequantize, lib, quantize  # noqa: F401 (lib: a fixture)


def attention(lib, t, **kw):
    a = dict(q=0x10000000000, qs=128, B=2, T=3, Hq=4, H=2, D=32, n_new=None, par=None, scale=1.0, out=0x20000000000, st=0x30000000000)
    a.update(kw)
    return getattr(lib, "spec_kv_attention_" + t)(a["q"], a["qs"], K, V, 4, 16, TAB, 4, ROWS, a["n_new"], a["par"], KC, VC, KS, VS, 4, 16, CTAB, 4,
                                                  a["st"], 1, a["B"], a["T"], a["Hq"], a["H"], a["D"], a["scale"], a["out"], None)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("B", [2 ** 30 + 1, 2 ** 31 - 128, 2 ** 31 - 1])
def test_batches(lib, t, B):
    """A round of sequences that starts below B may not end past 2^31."""
    far = dict(tab=0x100000000000, ctab=0x200000000000, first=0x300000000000, last=0x400000000000, out=0x500000000000)
    assert quantize(lib, "spec_kv_quantize_" + t, B=B, **far) == _lib.SPEC_ERR_SHAPE
    assert dequantize(lib, "spec_kv_dequantize_" + t, B=B, **far) == _lib.SPEC_ERR_SHAPE
    assert attention(lib, t, B=B, T=1, out=0x600000000000) == _lib.SPEC_ERR_SHAPE


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.4e38, -3.0e38])
def test_scales_past_the_exponent_s_range(lib, t, scale):
    """The scale is taken times log2(e), which has to be finite in fp32 too."""
    assert attention(lib, t, scale=scale) == _lib.SPEC_ERR_SHAPE


@pytest.mark.parametrize("t,e", [("f32", 4), ("bf16", 2)])
def test_token_strides_past_the_address_range(lib, t, e):
    """A stride whose bytes wrap around 2^64 to 0 ended the process in the look for shared memory.  Between tokens
    such strides are refused; a single token has none, and its queries may lie anywhere."""
    for stride in (2 ** 44 + 1, 2 ** 61, 2 ** 62, 2 ** 63 - 1):
        assert attention(lib, t, qs=stride) == _lib.SPEC_ERR_SHAPE
        assert attention(lib, t, qs=stride, B=1, T=1, out=ROWS) == _lib.SPEC_ERR_OVERLAP
        append = getattr(lib, "spec_kv_append_" + t)
        far, n = 1 << 45, 1 << 40

        def call(ks, qs, B, out=far + 6 * n):
            return append(far, far + n, ks, far + 2 * n, qs, out, None, None, ROWS, TAB, B, 1, 4, 2, 32, 0, 0, None, far + 3 * n, far + 4 * n, 4, 16, 4, None)

        assert call(stride, 128, 2) == _lib.SPEC_ERR_SHAPE and call(64, stride, 2) == _lib.SPEC_ERR_SHAPE
        assert call(stride, stride, 1, out=ROWS) == _lib.SPEC_ERR_OVERLAP
