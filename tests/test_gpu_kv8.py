"""The 8-bit key/value cache on the GPU: quantising and reading back bit for bit,
attention against a plain 64-bit implementation (tolerances: plain_kv8.tolerance)."""
import numpy as np
import pytest
import torch

import plain_kv8 as plain
import speculative_decoding_verification_36_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF16, F32 = torch.bfloat16, torch.float32


def dev(x):
    return None if x is None else torch.as_tensor(np.ascontiguousarray(x)).to(DEV)


def host(x):
    return x.float().cpu().numpy()


def table_of(rng, first, last, most, spare=1):
    """Page tables [B, most] with distinct pages for [first, last) of each sequence; the rest -1."""
    B = len(first)
    table = np.full((B, most), -1, np.int32)
    total = int(sum(max(0, b - a) for a, b in zip(first, last)))
    order = iter(rng.permutation(total + spare))
    for b in range(B):
        for p in range(first[b], last[b]):
            table[b, p] = next(order)
    return table, total + spare


# ---------------------------------------------------------------------------
# quantising and reading back
# ---------------------------------------------------------------------------
def store_case(rng, layers, B, Hkv, D, dtype, fmt, block, page, ctx, new):
    stored = (rng.integers(0, ctx + 1, B) // block * block).astype(np.int32)
    lengths = (stored + rng.integers(0, new + 1, B)).astype(np.int32)
    table, pages = table_of(rng, stored // page, -(-lengths // page), max(1, int(-(-lengths.max() // page))))
    code_table, code_pages = table_of(rng, stored // block, lengths // block, max(1, int(lengths.max() // block)))
    shape = (layers, pages, page, Hkv, D)
    x = dict(stored=stored, lengths=lengths, table=table, code_table=code_table, block=block, page=page, fmt=fmt, dtype=dtype)
    for c in ("k", "v"):
        y = rng.normal(0, 1, shape) * np.exp(rng.normal(0, 2, (layers, pages, page, 1, 1)))
        x[c] = torch.from_numpy(y.astype(np.float32)).to(dtype).to(DEV)
        x[c + "_codes"] = torch.from_numpy(rng.integers(0, 100, (layers, code_pages, block, Hkv, D)).astype(np.uint8)).to(DEV).view(plain.DTYPE[fmt])
        x[c + "_scales"] = torch.from_numpy(rng.normal(0, 1, (layers, code_pages, Hkv)).astype(np.float32)).to(DEV)
    return x


def quantize(x, flat=False, **kw):
    t = [x[c][0] if flat and x[c].shape[0] == 1 else x[c] for c in ("k", "v", "k_codes", "v_codes", "k_scales", "v_scales")]
    return sv.spec_kv_quantize(t[0], t[1], dev(x["table"]), dev(x["stored"]), dev(x["lengths"]), *t[2:], dev(x["code_table"]), **kw)


def expect_store(x, c):
    """The codes (values) and scales after quantising cache c, by the definition."""
    codes, scales = host(x[c + "_codes"]), host(x[c + "_scales"])
    cache = host(x[c])
    block, page = x["block"], x["page"]
    for b in range(len(x["stored"])):
        for i in range(x["stored"][b] // block, x["lengths"][b] // block):
            at = x["code_table"][b, i]
            s = np.arange(i * block, (i + 1) * block)
            y = cache[:, x["table"][b, s // page], s % page]
            codes[:, at], scales[:, at] = plain.quantize(y, x["fmt"])
    return codes, scales


STORES = [
    # layers, B, Hkv, D, dtype, fmt, block, page, ctx, new
    (1, 1, 1, 16, F32, "int8", 1, 1, 0, 3),
    (1, 3, 2, 64, BF16, "int8", 16, 16, 100, 40),
    (2, 3, 2, 80, F32, "e4m3", 24, 16, 100, 60),
    (1, 2, 8, 128, BF16, "int8", 64, 16, 300, 200),
    (3, 4, 1, 256, BF16, "e4m3", 65, 7, 200, 150),
    (1, 2, 3, 48, F32, "int8", 128, 64, 200, 300),   # more than the registers hold
    (1, 150, 1, 32, BF16, "e4m3", 16, 5, 50, 40),    # more sequences than a round takes
    (1, 5, 2, 96, BF16, "int8", 1000, 100, 1000, 2100),
]


@pytest.mark.parametrize("layers,B,Hkv,D,dtype,fmt,block,page,ctx,new", STORES)
def test_store_and_read_back(layers, B, Hkv, D, dtype, fmt, block, page, ctx, new):
    rng = np.random.default_rng(B + D + block)
    x = store_case(rng, layers, B, Hkv, D, dtype, fmt, block, page, ctx, new)
    want = {c: expect_store(x, c) for c in ("k", "v")}
    got = quantize(x, flat=True)
    np.testing.assert_array_equal(got.cpu().numpy(), x["lengths"] // block * block)
    for c in ("k", "v"):
        np.testing.assert_array_equal(host(x[c + "_codes"]), want[c][0])
        np.testing.assert_array_equal(host(x[c + "_scales"]), want[c][1])
    # back to other places, from the middle of a block on
    starts = (x["stored"] + np.minimum(3, got.cpu().numpy() - x["stored"])).astype(np.int32)
    back = {c: torch.full_like(x[c], 7.0) for c in ("k", "v")}
    sv.spec_kv_dequantize(x["k_codes"], x["v_codes"], x["k_scales"], x["v_scales"], dev(x["code_table"]), dev(starts), got,
                          back["k"], back["v"], dev(x["table"]))
    for c in ("k", "v"):
        ref = np.full(x[c].shape, 7.0, np.float32)
        for b in range(B):
            for s in range(starts[b], int(got[b])):
                at = x["code_table"][b, s // block]
                ref[:, x["table"][b, s // page], s % page] = want[c][0][:, at, s % block] * want[c][1][:, at][..., None]
        np.testing.assert_array_equal(host(back[c]), torch.from_numpy(ref).to(dtype).float().numpy())
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block", [4, 200])
def test_blocks_of_zeros_tiny_and_not_finite(dtype, fmt, block):
    rng = np.random.default_rng(3)
    n = 8
    x = dict(stored=np.zeros(1, np.int32), lengths=np.full(1, n * block, np.int32), block=block, page=block, fmt=fmt,
             table=np.arange(n, dtype=np.int32)[None], code_table=np.arange(n, dtype=np.int32)[::-1][None].copy())
    for c in ("k", "v"):
        y = rng.normal(0, 1, (1, n, block, 2, 64)).astype(np.float32)
        y[0, 0] = 0
        y[0, 1] *= 2.0 ** -105
        y[0, 2, 1, 0, 5] = np.nan
        y[0, 3, block - 1, 1, 63] = -np.inf
        y[0, 4] *= 2.0 ** 100
        y[0, 5] = -0.0
        y[0, 6] *= 2.0 ** -98
        x[c] = torch.from_numpy(y).to(dtype).to(DEV)
        x[c + "_codes"] = torch.ones((1, n, block, 2, 64), device=DEV).to(plain.DTYPE[fmt])
        x[c + "_scales"] = torch.ones((1, n, 2), device=DEV)
    want = {c: expect_store(x, c) for c in ("k", "v")}
    got = quantize(x)
    assert int(got[0]) == n * block
    for c in ("k", "v"):
        np.testing.assert_array_equal(host(x[c + "_scales"]), want[c][1])
        np.testing.assert_array_equal(host(x[c + "_codes"]), want[c][0])
        assert np.isnan(want[c][1]).sum() == 2
    back = torch.zeros_like(x["k"]), torch.zeros_like(x["v"])
    sv.spec_kv_dequantize(x["k_codes"], x["v_codes"], x["k_scales"], x["v_scales"], dev(x["code_table"]), dev(x["stored"]), got, *back,
                          dev(x["table"]))
    assert torch.isnan(back[0][0, 2, :, 0]).all() and not torch.isnan(back[0][0, 2, :, 1]).any()
    assert sv.spec_get_status() == 0


def test_store_bad_data():
    """A bad sequence keeps its count, the others are stored; what no block is written to stays."""
    x = dict(block=16, page=16, fmt="int8")
    x["stored"] = np.array([0, 16, 5, 32, -16, 0, 0, 16], np.int32)
    x["lengths"] = np.array([40, 40, 40, 31, 20, 81, 40, 47], np.int32)  # 2: no multiple; 3: above; 4: negative; 5: past the table
    x["table"] = np.arange(40, dtype=np.int32).reshape(8, 5)
    x["code_table"] = np.arange(40, dtype=np.int32).reshape(8, 5)
    x["table"][6, 1], x["code_table"][7, 1] = 40, -1
    for c in ("k", "v"):
        x[c] = torch.randn((2, 40, 16, 2, 32), device=DEV).to(BF16)
        x[c + "_codes"] = torch.full((2, 40, 16, 2, 32), 9, dtype=torch.int8, device=DEV)
        x[c + "_scales"] = torch.full((2, 40, 2), 9.0, device=DEV)
    keep = dict(x, stored=x["stored"].copy(), lengths=x["lengths"].copy())
    for b in (2, 3, 4, 5, 6, 7):  # nothing of them is expected; sequence 6's first block is free to be written
        keep["stored"][b] = keep["lengths"][b] = 0
    want = expect_store(keep, "k")
    got = quantize(x)
    assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA
    assert got.cpu().tolist() == [32, 32, 5, 32, -16, 0, 0, 16]
    free = [x["code_table"][6, 0]]
    rest = [i for i in range(40) if i not in free]
    np.testing.assert_array_equal(host(x["k_codes"])[:, rest], want[0][:, rest])
    np.testing.assert_array_equal(host(x["k_scales"])[:, rest], want[1][:, rest])


def test_read_bad_data():
    codes = torch.randint(-127, 128, (4, 8, 1, 16), dtype=torch.int8, device=DEV)
    scales = torch.ones((4, 1), device=DEV)
    plain_k, plain_v = (torch.full((8, 4, 1, 16), 5.0, device=DEV) for _ in range(2))
    table = np.arange(20, dtype=np.int32).reshape(5, 4) % 8
    table[4] = [0, 1, -1, 3]
    code_table = np.array([[0, 1], [0, 1], [0, 1], [0, 4], [2, 3]], np.int32)
    starts, ends = np.array([-1, 3, 0, 0, 0], np.int32), np.array([4, 2, 17, 0, 16], np.int32)
    sv.spec_kv_dequantize(codes, codes, scales, scales, dev(code_table), dev(starts), dev(ends), plain_k, plain_v, dev(table))
    assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA
    want = np.full((8, 4, 1, 16), 5.0, np.float32)
    for s in range(16):
        if s // 4 != 2:
            want[table[4, s // 4], s % 4] = host(codes)[code_table[4, s // 8], s % 8]
    np.testing.assert_array_equal(host(plain_k), want)
    np.testing.assert_array_equal(host(plain_v), want)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attend_case(rng, B, T, Hq, Hkv, D, dtype, fmt, block, page, lengths, tree=False, ragged=False, stored="blocks", joint=False):
    """stored: "blocks" (all whole ones before the step), "none", "some", "step" (also of the step)."""
    lengths = np.array([lengths] * B if np.isscalar(lengths) else lengths, np.int32)
    n_new = rng.integers(0, T + 1, B).astype(np.int32) if ragged else None
    new = np.full(B, T) if n_new is None else n_new
    have = {"blocks": lengths, "none": 0 * lengths, "step": lengths + new}.get(stored)
    have = rng.integers(0, lengths + 1) if have is None else have
    have = (have // block * block).astype(np.int32)
    x = dict(lengths=lengths, n_new=n_new, stored=have, block=block, page=page, dtype=dtype, parents=None, D=D)
    if tree:
        x["parents"] = np.stack([[int(rng.integers(max(-1, j - 4), j)) if j else -1 for j in range(T - 1)] for _ in range(B)]).reshape(B, T - 1).astype(np.int32)
    x["code_table"], code_pages = table_of(rng, 0 * have, have // block, max(1, int(have.max()) // block))
    end = lengths + new
    x["table"], pages = table_of(rng, have // page, -(-end // page), max(1, int(-(-(lengths + T).max() // page))))
    for c in ("k", "v"):
        size = rng.normal(0, 1, (code_pages, block, Hkv, D)) * np.exp(rng.normal(0, 1, (code_pages, 1, Hkv, 1)))
        codes, scales = plain.quantize(size, fmt)
        cache = torch.from_numpy((rng.normal(0, 1, (pages, page, Hkv, D)) * np.exp(rng.normal(0, 1, (pages, page, 1, 1)))).astype(np.float32)).to(dtype)
        x[c + "_codes"], x[c + "_scales"], x[c] = torch.from_numpy(codes).to(plain.DTYPE[fmt]).to(DEV), dev(scales), cache.to(DEV)
    if joint:
        x["q"] = torch.from_numpy(rng.normal(0, 1, (B, T, Hq + 2 * Hkv, D)).astype(np.float32)).to(dtype).to(DEV)[:, :, Hkv:Hkv + Hq]
    else:
        x["q"] = torch.from_numpy(rng.normal(0, 1, (B, T, Hq, D)).astype(np.float32)).to(dtype).to(DEV)
    return x


def attend(x, **kw):
    return sv.spec_kv_attention(x["q"], x["k"], x["v"], dev(x["table"]), dev(x["lengths"]), x["k_codes"], x["v_codes"], x["k_scales"],
                                x["v_scales"], dev(x["code_table"]), dev(x["stored"]), parent_idx=dev(x["parents"]), n_new=dev(x["n_new"]), **kw)


def rows_of(x, c, b, n):
    """The entries [lengths + n, Hkv, D] of sequence b in 64 bits."""
    s = np.arange(x["lengths"][b] + n)
    old, new = s[s < x["stored"][b]], s[s >= x["stored"][b]]
    codes, scales, cache = host(x[c + "_codes"]), host(x[c + "_scales"]), host(x[c])
    p, e = x["code_table"][b, old // x["block"]], x["table"][b, new // x["page"]]
    return np.concatenate((codes[p, old % x["block"]].astype(np.float64) * scales[p][..., None], cache[e, new % x["page"]].astype(np.float64)))


def check(x, got, scale=None, skip=()):
    B, T, _, D = x["q"].shape
    q = x["q"].double().cpu().numpy()
    got = got.double().cpu().numpy()
    for b in range(B):
        if b in skip:
            continue
        n = T if x["n_new"] is None else int(x["n_new"][b])
        out, mag, most, top = plain.attention(q[b], rows_of(x, "k", b, n), rows_of(x, "v", b, n), int(x["lengths"][b]), n,
                                              None if x["parents"] is None else x["parents"][b], D ** -0.5 if scale is None else scale)
        np.testing.assert_array_equal(np.isnan(got[b, :n]), np.isnan(out))
        ok = ~np.isnan(out)
        tol = plain.tolerance(out, mag, most, top, D, int(x["lengths"][b]) + n, x["dtype"] == F32)
        off = np.abs(got[b, :n] - out)
        assert (off[ok] <= tol[ok]).all(), (b, (off[ok] / tol[ok]).max(), off[ok].max())
        assert (got[b, n:] == 5.0).all()


def run_and_check(x, **kw):
    out = torch.full(x["q"].shape, 5.0, dtype=x["dtype"], device=DEV)
    got = attend(x, out=out, **kw)
    check(x, got, kw.get("scale"))
    assert sv.spec_get_status() == 0
    return got


ATTENDS = [
    # B, T, Hq, Hkv, D, block, page, lengths, tree, ragged, stored
    (1, 1, 1, 1, 16, 1, 1, 0, False, False, "blocks"),          # a first token
    (1, 1, 4, 1, 64, 16, 16, 1, False, False, "blocks"),
    (2, 1, 8, 2, 128, 16, 16, [700, 64], False, False, "blocks"),
    (3, 1, 2, 2, 80, 24, 7, [5, 1000, 23], False, False, "blocks"),
    (2, 5, 8, 2, 128, 64, 16, [300, 129], False, False, "blocks"),
    (2, 5, 3, 1, 48, 1, 3, [40, 0], False, False, "some"),
    (4, 9, 8, 8, 96, 32, 16, [63, 64, 65, 0], False, True, "some"),
    (2, 7, 12, 4, 64, 65, 16, [130, 200], False, False, "none"),
    (3, 31, 8, 2, 128, 16, 16, [100, 5, 333], True, False, "blocks"),
    (2, 40, 6, 2, 64, 16, 5, [17, 90], True, True, "some"),
    (2, 2, 4, 1, 32, 8, 8, [8, 9], True, False, "step"),         # codes of a tree's own nodes
    (2, 70, 8, 2, 128, 16, 16, [100, 0], False, True, "step"),  # codes that early tokens do not see
    (1, 200, 4, 4, 64, 64, 16, [333], False, False, "step"),
    (2, 3, 8, 1, 256, 16, 16, [1000, 77], False, False, "blocks"),
    (1, 20, 6, 3, 208, 24, 16, [150], False, False, "blocks"),
    (200, 2, 2, 1, 32, 16, 16, list(range(200)), False, False, "blocks"),  # more sequences than a round counts
    (1, 4, 8, 2, 128, 16, 16, [9000], False, False, "blocks"),  # one segment over many CTAs
    (1, 300, 2, 2, 64, 16, 16, [40], True, False, "blocks"),    # a large tree
]


@pytest.mark.parametrize("dtype,fmt", [(BF16, "int8"), (BF16, "e4m3"), (F32, "int8"), (F32, "e4m3")])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,block,page,lengths,tree,ragged,stored", ATTENDS)
def test_attention_matches_plain(B, T, Hq, Hkv, D, block, page, lengths, tree, ragged, stored, dtype, fmt):
    rng = np.random.default_rng(T + D + B)
    run_and_check(attend_case(rng, B, T, Hq, Hkv, D, dtype, fmt, block, page, lengths, tree, ragged, stored, joint=T % 2 == 1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.0, 2.0, -0.5])
def test_attention_scales(dtype, scale):
    rng = np.random.default_rng(8)
    run_and_check(attend_case(rng, 2, 6, 4, 2, 64, dtype, "int8", 16, 16, [100, 41]), scale=scale)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_wide_ranges(T, dtype):
    """Scores that grow along the sequence (the running maximum moves), queries and values of
    very different sizes, blocks of zeros."""
    rng = np.random.default_rng(9)
    x = attend_case(rng, 2, T, 4, 2, 64, dtype, "int8", 16, 16, [400, 333])
    x["q"].mul_(torch.exp2(torch.arange(T, device=DEV) % 7 * 3 - 10).to(dtype)[None, :, None, None])
    grow = np.exp(rng.normal(0, 3, x["v_scales"].shape)).astype(np.float32)
    x["v_scales"].mul_(dev(grow))
    x["k_scales"].mul_(torch.linspace(0.01, 1, x["k_scales"].shape[0], device=DEV)[:, None])
    x["v_scales"][::5] = 0
    x["k_scales"][::7] = 0
    run_and_check(x)
    # heads of zeros only
    x["v_scales"].zero_()
    x["v"].zero_()
    assert (attend(x) == 0).all()


@pytest.mark.parametrize("T,G", [(8, 1), (33, 4)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_not_finite(T, G, dtype):
    """An entry that is not finite reaches the rows that see it and no others; so does a query row."""
    rng = np.random.default_rng(10)
    for tree in (False, True):
        x = attend_case(rng, 2, T, 2 * G, 2, 64, dtype, "int8", 16, 16, [50, 30], tree=tree)
        slot = 50 + T // 2
        x["k"][x["table"][0, slot // 16], slot % 16, 0, 3] = float("nan")
        x["v"][x["table"][0, (slot + 1) // 16], (slot + 1) % 16, 1, 63] = float("inf")
        x["v"][x["table"][0, (slot + 2) // 16], (slot + 2) % 16, 0] = 1e30  # finite, and far from all others
        x["q"][1, 2, 1, 5] = float("-inf")
        x["q"][1, 1, 0, 0] = float("nan")
        got = run_and_check(x)
        nan = torch.isnan(got[0]).all(-1).cpu()
        assert nan.any() and not nan.all()
        x["k_scales"][x["code_table"][1, 0], 1] = float("nan")
        got = run_and_check(x)
        assert torch.isnan(got[1, :, G:]).all() and not torch.isnan(got[1, 0, :G]).any()


@pytest.mark.parametrize("T", [4, 40])
def test_attention_bad_data(T):
    """A bad sequence's rows are NaN, the others' as they would be."""
    rng = np.random.default_rng(11)
    for tree in (False, True):
        x = attend_case(rng, 8, T, 4, 2, 64, BF16, "int8", 16, 16, [64] * 8, tree=tree)
        x["n_new"] = np.full(8, T, np.int32)
        x["lengths"][0] = -1
        x["n_new"][1] = T + 1
        x["stored"][2] = 40          # no multiple of a block
        x["stored"][3] = 64 + T // 16 * 16 + 16  # above what there is
        x["lengths"][4] = 4000       # past the table
        lost = [0, 1, 2, 3, 4]
        if tree:
            x["parents"][5, T - 2] = T - 2
            lost.append(5)
        out = torch.full(x["q"].shape, 5.0, dtype=BF16, device=DEV)
        got = attend(x, out=out)
        assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA
        assert torch.isnan(got[lost]).all()
        check(x, got, skip=lost)
        # pages outside their pools
        x = attend_case(rng, 3, T, 4, 2, 64, BF16, "int8", 16, 16, [64] * 3, tree=tree)
        good = attend(x)
        x["code_table"][0, 2] = x["k_codes"].shape[0]
        x["table"][1, (64 + T - 1) // 16] = -1
        got = attend(x)
        assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA
        assert torch.isnan(got[0]).all() and torch.equal(got[2], good[2])
        first = (64 + T - 1) // 16 * 16 - 64
        assert torch.isnan(got[1, T - 1]).all()
        if first > 0 and not tree:
            assert torch.equal(got[1, :first], good[1, :first]) and torch.isnan(got[1, first:]).all()


def test_attention_is_the_same_on_every_run_and_stream():
    rng = np.random.default_rng(12)
    for T in (1, 6, 40):
        x = attend_case(rng, 3, T, 8, 2, 128, BF16, "int8", 16, 16, [900, 5000, 17])
        first = attend(x)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        outs = [attend(x) for _ in range(3)]
        with torch.cuda.stream(side):
            outs += [attend(x) for _ in range(3)]
        torch.cuda.synchronize()
        outs.append(attend(x, stream=side))
        side.synchronize()
        assert all(torch.equal(first, o) for o in outs)
    assert sv.spec_get_status() == 0


def test_attention_in_graphs():
    """Captured calls read what their inputs hold at each replay; two graphs run side by side."""
    rng = np.random.default_rng(13)
    xs = [attend_case(rng, 2, T, 8, 2, 128, BF16, "e4m3", 16, 16, [700, 90]) for T in (5, 20)]
    args = []
    for x in xs:
        args.append([x["q"], x["k"], x["v"], dev(x["table"]), dev(x["lengths"]), x["k_codes"], x["v_codes"], x["k_scales"], x["v_scales"],
                     dev(x["code_table"]), dev(x["stored"])])
    want = [sv.spec_kv_attention(*a) for a in args]
    outs = [torch.empty_like(w) for w in want]
    graphs = []
    for a, o in zip(args, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.spec_kv_attention(*a, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for a in args:
        a[0].neg_()
    want = [sv.spec_kv_attention(*a) for a in args]
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert sv.spec_get_status() == 0
