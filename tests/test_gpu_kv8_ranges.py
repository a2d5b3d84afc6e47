"""Attention to the 8-bit cache where its inputs' sizes lie far apart: against 64 bits, with a
tolerance that goes by the weighted values, so that what has almost no weight excuses nothing."""
import numpy as np
import pytest
import torch

import plain_kv8 as plain
import speculative_decoding_verification_36_gb300 as sv
from test_gpu_kv8 import BF16, F32, attend, attend_case, dev, host, rows_of

pytestmark = pytest.mark.gpu


def value_scales(x, b, n):
    """What a key's weight is multiplied by, for each key and head: the scale of its block, or a power
    of two above 1/256 of a plain entry's largest magnitude and at most 1/128 of it."""
    s = np.arange(x["lengths"][b] + n)
    old, new = s[s < x["stored"][b]], s[s >= x["stored"][b]]
    cache = np.abs(host(x["v"])[x["table"][b, new // x["page"]], new % x["page"]]).astype(np.float64)
    return np.concatenate((host(x["v_scales"])[x["code_table"][b, old // x["block"]]].astype(np.float64), cache.max(-1) / 128))


def check_weighted(x, got, only=None):
    """Two parts of the tolerance are those of plain_kv8.tolerance; the others:

    A weight p (the largest p of a row is at least 1, l is their sum) enters the second product as
    w = p s / 2^unit in fp16, s its key's scale.  2^unit follows the largest p s that the row has
    seen: that one is at least 2^7 in these units.  fp16 is off by its relative step (counted with
    the weight) or by 2^-25, which is 2^-32 of the largest p s.  A code is at most 448, a plain
    entry below 256: a key may add 2^-32 * 448 max(p s) / l.
    p below 2^-126 counts as 0: at most 2^-126 * 448 s a key, as l is at least 1."""
    B, T, Hq, D = x["q"].shape
    q, got = x["q"].double().cpu().numpy(), got.double().cpu().numpy()
    two = x["dtype"] == F32
    for b in range(B) if only is None else only:
        n = T if x["n_new"] is None else int(x["n_new"][b])
        k, v, s = rows_of(x, "k", b, n), rows_of(x, "v", b, n), value_scales(x, b, n)
        parents = None if x["parents"] is None else x["parents"][b]
        out, mag, most, _ = plain.attention(q[b], k, v, int(x["lengths"][b]), n, parents, D ** -0.5)
        keys = int(x["lengths"][b]) + n
        see = np.ones((n, keys), bool)
        see[:, x["lengths"][b]:] = plain.step_visible(n, parents)
        tol = plain.tolerance(0 * out, mag, most, 0 * out, D, keys, two)
        for h in range(Hq):
            z = k[:, h // (Hq // k.shape[1])] @ q[b, :n, h].T * D ** -0.5
            z = np.where(see, z.T, -np.inf)
            p = np.exp(z - z.max(1, keepdims=True))
            size = s[:, h // (Hq // k.shape[1])]
            tol[:, h] += 448 * ((2.0 ** -32 * keys * (p * size).max(1) / p.sum(1)) + 2.0 ** -126 * np.where(see, size, 0).sum(1))[:, None]
        tol += (2.0 ** -24 if two else 2.0 ** -8) * (np.abs(out) + tol)
        assert np.isfinite(got[b, :n]).all() and np.isfinite(out).all()
        off = np.abs(got[b, :n] - out)
        assert (off <= tol).all(), (b, float((off / tol).max()), float(off.max()))


def sized_case(rng, B, T, Hq, D, dtype, fmt, block, ctx, key, size, tail=0.0):
    """B sequences of the same ctx stored entries: all keys of a block from slot s on are key(s) in the first channel, the
    queries are 1 there, the values lie between 1 and 2 times size(s); the step's own entries have `tail` for them."""
    x = attend_case(rng, B, T, Hq, 1, D, dtype, fmt, block, 16, [ctx] + [0] * (B - 1))
    x["lengths"][:], x["stored"][:], x["code_table"][:] = ctx, ctx, x["code_table"][0]
    x["table"] = np.full((B, -(-(ctx + T) // 16)), -1, np.int32)
    x["table"][:, ctx // 16:] = np.arange(x["table"].shape[1] - ctx // 16)
    x["q"].zero_()
    x["q"][..., 0] = D ** 0.5
    x["k"], x["v"] = torch.zeros_like(x["k"]), torch.full_like(x["v"], tail)
    s = block * np.arange(ctx // block)
    codes = {c: np.zeros(tuple(x[c + "_codes"].shape), np.float32) for c in ("k", "v")}
    scales = {c: np.zeros(tuple(x[c + "_scales"].shape), np.float32) for c in ("k", "v")}
    pages = x["code_table"][0, :len(s)]
    keys, sizes = np.array([key(i) for i in s]), np.array([size(i) for i in s])
    codes["k"][pages, :, :, 0] = 64 * np.sign(keys)[:, None, None]
    scales["k"][pages] = np.abs(keys)[:, None] / 64
    codes["v"][pages] = rng.integers(64, 128, (len(s), *codes["v"].shape[1:]))
    scales["v"][pages] = sizes[:, None] / 64
    for c in ("k", "v"):
        x[c + "_codes"], x[c + "_scales"] = torch.from_numpy(codes[c]).to(plain.DTYPE[fmt]).to(x["q"].device), dev(scales[c])
    return x


KINDS = [(1, 4, 128, BF16), (9, 4, 128, BF16), (9, 2, 64, BF16), (9, 2, 256, BF16), (5, 2, 80, F32)]


@pytest.mark.parametrize("ctx", [128, 6400])  # a share has all of the sequence; many shares, which are joined
@pytest.mark.parametrize("first,later", [(0.0, 2.0 ** 63), (0.0, 2.0 ** 71), (1.0, 2.0 ** 100), (2.0 ** 71, 0.0), (2.0 ** -60, 2.0 ** 60)])
@pytest.mark.parametrize("T,Hq,D,dtype", KINDS)
def test_the_sum_of_weights_does_not_go_by_the_values(T, Hq, D, dtype, first, later, ctx):
    """Keys of equal scores, half of them with values of another size: each has the same weight."""
    rng = np.random.default_rng(D)
    x = sized_case(rng, 1, T, Hq, D, dtype, "int8", 16, ctx, lambda s: 0.0, lambda s: first if s < ctx // 2 else later)
    check_weighted(x, attend(x))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("B,ctx", [(1, 1024), (1, 6400), (200, 1024)])  # shares of a unit, of a few, of many
@pytest.mark.parametrize("block", [4, 16])  # others beside it in a unit, in a product
@pytest.mark.parametrize("fmt,outlier", [("int8", 2.0 ** 25), ("e4m3", 2.0 ** 36), ("int8", 2.0 ** 60), ("int8", 2.0 ** 120)])
@pytest.mark.parametrize("T,Hq,D,dtype", KINDS)
def test_large_values_of_little_weight(T, Hq, D, dtype, fmt, outlier, block, B, ctx):
    """A block whose values are far larger than all others and whose weight is e^-100 of theirs."""
    rng = np.random.default_rng(D)
    at = 16 * (ctx // 48)
    x = sized_case(rng, B, T, Hq, D, dtype, fmt, block, ctx, lambda s: -100.0 if s == at else 0.0, lambda s: outlier if s == at else 1.0, tail=1.0)
    check_weighted(x, attend(x), only=range(0, B, 67))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("down", [80.0, 120.0])
@pytest.mark.parametrize("T,Hq,D,dtype", KINDS)
def test_large_values_whose_weight_falls(T, Hq, D, dtype, down):
    """The first values are the largest and their scores the lowest: what they add in the end goes down
    with the scores that come after, in small steps and in one."""
    rng = np.random.default_rng(D)
    for steps in (1, 4, 60):
        x = sized_case(rng, 200, T, Hq, D, dtype, "int8", 16, 1024, lambda s: down * (s // 16 * steps // 64 / steps - 1), lambda s: 2.0 ** 80 if s < 32 else 1.0)
        check_weighted(x, attend(x), only=(0, 77, 199))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("T,D,dtype,B,blocks", [(9, 64, BF16, 310, 8192), (9, 256, BF16, 155, 8192), (40, 128, BF16, 305, 8192), (1, 128, BF16, 460, 16384),
                                                (1, 64, F32, 620, 16384)])
def test_sums_of_many_keys_do_not_drift(T, D, dtype, B, blocks):
    """Many sequences of the same 2^19 or 2^20 entries with equal weights: a CTA has a whole sequence or most of one.

    An entry is c * 1027 * 2^-10, exact in the products, and its sum takes more than 24 bits.  These c lie 2^-12 to
    2^-11 above the middle of two bf16 numbers.  A sum may drop 2^-23 for each 16 keys (there are no more
    than 2048 such steps in a row: 2^-12), so that the upper one has to come out.  fp32: 2048 sums of 64 keys in a
    row, each rounded by 2^-24, and the sum of the up to 8 such sums: 2^-13 + 2^-21."""
    block = 64
    code = torch.tensor([47, 48, 49, 50, 51, 94, 95, 96, 97, 98, 99, 100, 101, 102])[torch.arange(D) % 14]
    want = code.double() * 1027 * 2.0 ** -10
    dev_ = "cuda"
    codes = code.to(torch.int8).to(dev_).expand(blocks, block, 1, D).contiguous()
    scales = torch.full((blocks, 1), 1027 * 2.0 ** -10, device=dev_)
    cache = want.to(torch.bfloat16).to(dtype).to(dev_).expand(1, block, 1, D).contiguous()
    code_table = torch.arange(blocks, dtype=torch.int32, device=dev_).expand(B, blocks).contiguous()
    lengths = torch.full((B,), blocks * block, dtype=torch.int32, device=dev_)
    table = torch.zeros((B, blocks + 1), dtype=torch.int32, device=dev_)
    q = torch.zeros((B, T, 1, D), dtype=dtype, device=dev_)
    got = sv.spec_kv_attention(q, cache, cache, table, lengths, codes, codes, scales, scales, code_table, lengths)
    assert sv.spec_get_status() == 0
    if dtype == BF16:
        assert torch.equal(got, want.to(BF16).to(dev_).expand_as(got))
    else:
        assert float((got.double() / want.to(dev_) - 1).abs().max()) <= 2.0 ** -13 + 2.0 ** -21 + 2.0 ** -24
