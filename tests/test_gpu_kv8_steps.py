"""The 8-bit key/value cache on the GPU as a server uses it, and the edges of its calls:
outputs between canaries, pools past 32 bits, pages outside, waits and allocations that fail."""
import numpy as np
import pytest
import torch

import plain_kv8 as plain
import speculative_decoding_verification_36_gb300 as sv
from speculative_decoding_verification_36_gb300 import _lib
from test_gpu_guards import Guarded
from test_gpu_kv8 import BF16, DEV, F32, attend, attend_case, check, dev, host, quantize, store_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,fmt,Hq,Hkv,D,block,page", [(BF16, "int8", 8, 2, 128, 16, 16), (BF16, "e4m3", 2, 1, 256, 24, 8), (F32, "int8", 4, 4, 64, 16, 5)])
def test_a_server_s_steps(dtype, fmt, Hq, Hkv, D, block, page):
    """A prompt, then tree steps: append, attention, verify, commit, quantise.  Pages whose tokens have all
    become codes are filled with NaN and leave the table; at the end all is read back."""
    rng = np.random.default_rng(D)
    B, layers, N, V, most = 3, 2, 6, 50, 160
    pages = -(-most // page) * B
    x = dict(block=block, page=page, fmt=fmt, dtype=dtype, D=D)
    table = rng.permutation(pages).astype(np.int32).reshape(B, -1)
    x["code_table"] = rng.permutation(-(-most // block) * B).astype(np.int32).reshape(B, -1)
    for c in ("k", "v"):
        x[c] = torch.zeros((layers, pages, page, Hkv, D), dtype=dtype, device=DEV)
        x[c + "_codes"] = torch.zeros((layers, x["code_table"].size, block, Hkv, D), device=DEV).to(plain.DTYPE[fmt])
        x[c + "_scales"] = torch.zeros((layers, x["code_table"].size, Hkv), device=DEV)
    lengths, x["stored"] = np.zeros(B, np.int32), np.zeros(B, np.int32)
    truth = {c: [np.zeros((layers, 0, Hkv, D), np.float32) for _ in range(B)] for c in ("k", "v")}  # committed entries as they were appended

    def step(T, parents, n_new):
        """Appends and attends in all layers; returns what was appended."""
        new = {c: torch.from_numpy((rng.normal(0, 1, (layers, B, T, Hkv, D)) * np.exp(rng.normal(0, 1, (layers, B, T, 1, 1)))).astype(np.float32))
               .to(dtype).to(DEV) for c in ("k", "v")}
        for layer in range(layers):
            q = torch.from_numpy(rng.normal(0, 1, (B, T, Hq, D)).astype(np.float32)).to(dtype).to(DEV)
            sv.spec_kv_append(new["k"][layer], new["v"][layer], x["k"][layer], x["v"][layer], dev(table), dev(lengths), parent_idx=dev(parents),
                              n_new=dev(n_new))
            y = dict(x, q=q, lengths=lengths, n_new=n_new, parents=parents, table=table)
            for c in ("k", "v", "k_codes", "v_codes", "k_scales", "v_scales"):
                y[c] = x[c][layer]
            out = torch.full(q.shape, 5.0, dtype=dtype, device=DEV)
            check(y, attend(y, out=out))
        return {c: host(new[c]) for c in new}

    def store():
        nonlocal lengths
        got = quantize(dict(x, lengths=lengths, table=table)).cpu().numpy()
        np.testing.assert_array_equal(got, lengths // block * block)
        for b in range(B):
            for p in range(int(got[b]) // page):
                if table[b, p] >= 0:
                    x["k"][:, table[b, p]] = x["v"][:, table[b, p]] = float("nan")
                    table[b, p] = -1
        x["stored"] = got.astype(np.int32)

    n_new = np.array([50, 33, 7], np.int32)
    new = step(50, None, n_new)
    for c in ("k", "v"):
        truth[c] = [new[c][:, b, :n_new[b]] for b in range(B)]
    lengths = lengths + n_new
    store()
    for _ in range(4):
        parents = np.stack([[int(rng.integers(-1, j)) if j else -1 for j in range(N)] for _ in range(B)]).astype(np.int32)
        new = step(N + 1, parents, None)
        tokens = torch.randint(0, V, (B, N), dtype=torch.int32, device=DEV)
        logits = torch.randn((B, N + 1, V), device=DEV)
        for j in range(N):  # every other draft is what the target wants
            if j % 2 == 0:
                for b in range(B):
                    logits[b, parents[b, j] + 1, tokens[b, j]] = 20.0 + j
        path, n, _ = sv.spec_tree_verify_greedy(logits, tokens, dev(parents))
        nodes, after = sv.spec_kv_commit(x["k"], x["v"], dev(table), dev(lengths), tokens, dev(parents), path, n)
        nodes, after = nodes.cpu().numpy(), after.cpu().numpy().astype(np.int32)
        for b in range(B):
            kept = [0] + [int(j) + 1 for j in nodes[b, :after[b] - lengths[b] - 1]]
            assert len(kept) == after[b] - lengths[b]
            for c in ("k", "v"):
                truth[c][b] = np.concatenate((truth[c][b], new[c][:, b, kept]), 1)
        lengths = after
        store()
    assert (x["stored"] > 0).any()
    back = {c: torch.zeros((layers, pages, page, Hkv, D), dtype=dtype, device=DEV) for c in ("k", "v")}
    whole = np.arange(pages, dtype=np.int32).reshape(B, -1)
    sv.spec_kv_dequantize(x["k_codes"], x["v_codes"], x["k_scales"], x["v_scales"], dev(x["code_table"]), dev(0 * lengths), dev(x["stored"]), back["k"],
                          back["v"], dev(whole))
    for c in ("k", "v"):
        for b in range(B):
            s = np.arange(x["stored"][b])
            got = host(back[c])[:, whole[b, s // page], s % page]
            for layer in range(layers):
                codes, scales = plain.quantize(truth[c][b][layer, :len(s)].reshape(-1, block, Hkv, D), fmt)
                want = torch.from_numpy((codes * scales[:, None, :, None]).reshape(-1, Hkv, D)).to(dtype).float().numpy()
                np.testing.assert_array_equal(got[layer], want)
            s = np.arange(x["stored"][b], lengths[b])  # the tail is as it was appended
            np.testing.assert_array_equal(host(x[c])[:, table[b, s // page], s % page], truth[c][b][:, x["stored"][b]:])
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("B,T,Hq,Hkv,D", [(700, 3, 4, 1, 64), (600, 12, 1, 1, 128), (3, 5, 2, 1, 112), (2, 1025, 1, 1, 16)])
def test_attention_of_more_shapes(B, T, Hq, Hkv, D):
    """More sequences than a round counts, 9 to 16 rows a head, heads that are no power of two, a long prompt."""
    rng = np.random.default_rng(B)
    x = attend_case(rng, B, T, Hq, Hkv, D, BF16, "int8", 16, 16, rng.integers(0, 90, B), ragged=True)
    out = torch.full(x["q"].shape, 5.0, dtype=BF16, device=DEV)
    check(x, attend(x, out=out))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,block,page,lengths,tree,ragged,stored", [
    (2, 31, 8, 1, 256, 16, 16, [700, 33], True, False, "blocks"),
    (1, 200, 2, 1, 160, 24, 7, [333], False, False, "step"),
    (3, 9, 4, 2, 144, 64, 16, [1000, 63, 0], False, True, "some"),
    (2, 128, 2, 2, 192, 16, 5, [50, 400], True, True, "blocks"),   # the largest tree of the tiles
    (1, 129, 1, 1, 208, 16, 16, [90], True, False, "blocks"),      # a larger one
    (1, 16, 1, 1, 256, 16, 16, [20000], False, False, "blocks"),   # one segment over all CTAs: a quarter of its shares to a warp
])
def test_attention_of_wide_heads(B, T, Hq, Hkv, D, block, page, lengths, tree, ragged, stored, fmt):
    rng = np.random.default_rng(T + D + B)
    x = attend_case(rng, B, T, Hq, Hkv, D, BF16, fmt, block, page, lengths, tree, ragged, stored)
    out = torch.full(x["q"].shape, 5.0, dtype=BF16, device=DEV)
    check(x, attend(x, out=out))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("T,Hkv,D,dtype,tree", [(1, 2, 128, BF16, False), (5, 1, 80, BF16, True), (5, 1, 80, F32, True), (37, 3, 48, BF16, False), (3, 1, 240, BF16, False)])
def test_outputs_are_guarded(T, Hkv, D, dtype, tree):
    rng = np.random.default_rng(T)
    x = attend_case(rng, 3, T, 4 * Hkv, Hkv, D, dtype, "int8", 24, 7, [130, 0, 47], tree=tree, ragged=True)
    out = Guarded(tuple(x["q"].shape), dtype)
    keep = out.t.clone()
    attend(x, out=out.t)
    assert out.intact()
    for b in range(3):
        assert torch.equal(out.t[b, x["n_new"][b]:], keep[b, x["n_new"][b]:])
    x = store_case(rng, 2, 3, Hkv, D, dtype, "int8", 24, 7, 100, 90)
    guards = {}
    for c in ("k_codes", "v_codes"):
        buf = torch.full((x[c].numel() + 512,), 33, dtype=torch.int8, device=DEV)
        guards[c], x[c] = buf, buf[256:-256].view(x[c].shape)
    for c in ("k_scales", "v_scales"):
        guards[c] = Guarded(tuple(x[c].shape), F32)
        x[c] = guards[c].t
    got = quantize(x)
    back = [Guarded(tuple(x["k"].shape), dtype) for _ in range(2)]
    sv.spec_kv_dequantize(x["k_codes"], x["v_codes"], x["k_scales"], x["v_scales"], dev(x["code_table"]), dev(x["stored"]), got, back[0].t, back[1].t,
                          dev(x["table"]))
    torch.cuda.synchronize()
    assert all((guards[c][:256] == 33).all() and (guards[c][-256:] == 33).all() for c in ("k_codes", "v_codes"))
    assert all(g.intact() for g in (guards["k_scales"], guards["v_scales"], *back))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("T,D,dtype", [(1, 128, BF16), (20, 128, BF16), (3, 128, F32)])
def test_pools_past_32_bits(T, D, dtype):
    """The same pages at the end of pools of more than 2^32 bytes give the same bits."""
    rng = np.random.default_rng(T)
    x = attend_case(rng, 2, T, 16, 8, D, dtype, "int8", 16, 16, [300, 77])
    want = attend(x)
    y = dict(x)
    pages = 2 ** 32 // (16 * 8 * D) + 1000
    for c in ("k", "v", "k_codes", "v_codes", "k_scales", "v_scales"):
        y[c] = torch.empty((pages, *x[c].shape[1:]), dtype=x[c].dtype, device=DEV)
        y[c][-x[c].shape[0]:] = x[c]
    for t, c in (("table", "k"), ("code_table", "k_codes")):
        y[t] = np.where(x[t] >= 0, x[t] + pages - x[c].shape[0], -1).astype(np.int32)
    assert y["k_codes"].numel() > 2 ** 32
    assert torch.equal(attend(y), want)
    # read back, then quantised anew: int8 codes whose largest is 127 come back as they were
    first, last = 0 * x["stored"], x["stored"]
    y["table"] = np.arange(pages - 64, pages, dtype=np.int32).reshape(2, 32)
    sv.spec_kv_dequantize(y["k_codes"], y["v_codes"], y["k_scales"], y["v_scales"], dev(y["code_table"]), dev(first), dev(last), y["k"], y["v"], dev(y["table"]))
    codes = y["k_codes"][-x["k_codes"].shape[0]:].clone()
    y["k_codes"][-x["k_codes"].shape[0]:] = 0
    y["stored"], y["lengths"] = first, last
    quantize(y)
    back = y["k_codes"][-x["k_codes"].shape[0]:]
    used = torch.from_numpy(np.sort(x["code_table"][x["code_table"] >= 0])).long().to(DEV)
    # a bf16 entry is off by 2^-8 of its code, so less than half a step up to 128 * 2^-8; fp32 gives the codes themselves
    assert (back[used].int() - codes[used].int()).abs().max() <= (1 if dtype == BF16 else 0)
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("T,Hq,D,dtype", [(40, 2, 64, BF16), (40, 2, 64, F32), (40, 1, 256, BF16)])
def test_what_lies_on_other_pages_does_not_matter(T, Hq, D, dtype):
    """A block outside the pool makes NaN of the rows that see it alone, also where the pool's first page holds NaN codes."""
    rng = np.random.default_rng(T)
    x = attend_case(rng, 2, T, Hq, 1, D, dtype, "e4m3", 16, 16, [32, 50], stored="step")
    for c in ("k", "v"):
        x[c + "_codes"] = torch.cat((torch.full_like(x[c + "_codes"][:1].view(torch.uint8), 0x7f), x[c + "_codes"].view(torch.uint8))).view(torch.float8_e4m3fn)
        x[c + "_scales"] = torch.cat((torch.full_like(x[c + "_scales"][:1], float("nan")), x[c + "_scales"]))
        x[c] = torch.cat((torch.full_like(x[c][:1], float("nan")), x[c]))
    x["table"], x["code_table"] = (np.where(x[t] >= 0, x[t] + 1, -1).astype(np.int32) for t in ("table", "code_table"))
    good = attend(x)
    check(x, good)
    assert x["stored"][0] == 64
    x["code_table"][0, 3] = -1  # slots 48 .. 63: tokens 16 on
    got = attend(x)
    assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA
    assert torch.isnan(got[0, 16:]).all() and torch.equal(got[0, :16], good[0, :16]) and torch.equal(got[1], good[1])


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (256, BF16), (64, F32)])
def test_a_whole_unit_without_a_page(D, dtype):
    """The step's own second block of 64 has no page: tokens before it are as they were, the rest NaN."""
    rng = np.random.default_rng(D)
    x = attend_case(rng, 3, 140, 2, 1, D, dtype, "e4m3", 64, 16, [0, 64, 5], stored="step")
    good = attend(x)
    check(x, good)
    lost = x["code_table"].copy()
    lost[:, 1] = -1
    got = attend(dict(x, code_table=lost))
    assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA
    for b, first in enumerate((64, 0, 59)):
        assert torch.equal(got[b, :first], good[b, :first]) and torch.isnan(got[b, first:]).all()


@pytest.mark.parametrize("T,dtype", [(2, BF16), (30, BF16), (4, F32)])
def test_queries_off_16_byte_boundaries(T, dtype):
    rng = np.random.default_rng(T)
    x = attend_case(rng, 2, T, 4, 2, 64, dtype, "int8", 16, 16, [100, 41])
    want = attend(x)
    wide = torch.zeros((2, T, 4 * 64 + 3), dtype=dtype, device=DEV)
    wide[..., 1:257] = x["q"].reshape(2, T, 256)
    x["q"] = wide[..., 1:257].view(2, T, 4, 64)
    assert torch.equal(attend(x), want)


def test_calls_side_by_side():
    """Calls of different head sizes on three streams share the SMs and their tensor memory."""
    rng = np.random.default_rng(4)
    xs = [attend_case(rng, 3, T, 8, 2, D, BF16, "int8", 16, 16, [3000, 10, 500]) for T, D in ((9, 256), (20, 128), (7, 64))]
    args = [[x["q"], x["k"], x["v"], dev(x["table"]), dev(x["lengths"]), x["k_codes"], x["v_codes"], x["k_scales"], x["v_scales"],
             dev(x["code_table"]), dev(x["stored"])] for x in xs]
    want = [sv.spec_kv_attention(*a) for a in args]
    outs = [[torch.empty_like(w) for _ in range(8)] for w in want]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for i in range(8):
        for a, o, s in zip(args, outs, streams):
            sv.spec_kv_attention(*a, out=o[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for w, many in zip(want, outs) for o in many)
    assert sv.spec_get_status() == 0


def test_nothing_to_do():
    rng = np.random.default_rng(0)
    x = attend_case(rng, 2, 3, 4, 2, 64, BF16, "int8", 16, 16, [100, 41])
    x["q"] = x["q"][:, :0]
    assert attend(x).shape == (2, 0, 4, 64)
    x = attend_case(rng, 2, 3, 4, 2, 64, BF16, "int8", 16, 16, [100, 41])
    x["n_new"] = np.zeros(2, np.int32)
    out = torch.full(x["q"].shape, 5.0, dtype=BF16, device=DEV)
    assert (attend(x, out=out) == 5.0).all()
    assert sv.spec_get_status() == 0


def test_store_and_read_back_in_a_graph():
    rng = np.random.default_rng(1)
    x = store_case(rng, 2, 4, 2, 64, BF16, "int8", 16, 16, 100, 90)
    args = [x["k"], x["v"], dev(x["table"]), dev(x["stored"]), dev(x["lengths"]), x["k_codes"], x["v_codes"], x["k_scales"], x["v_scales"], dev(x["code_table"])]
    stored = torch.empty(4, dtype=torch.int32, device=DEV)
    back = [torch.zeros_like(x["k"]) for _ in range(2)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_kv_quantize(*args, out_stored=stored)
        sv.spec_kv_dequantize(*args[5:9], args[9], args[3], stored, *back, args[2])
    for _ in range(2):
        for c in ("k", "v"):
            x[c].normal_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*args[5:9], *back, stored)]
        sv.spec_kv_quantize(*args, out_stored=stored)
        sv.spec_kv_dequantize(*args[5:9], args[9], args[3], stored, *back, args[2])
        assert all(torch.equal(a, b) for a, b in zip(got, (*args[5:9], *back, stored)))
    assert sv.spec_get_status() == 0


def test_a_lowered_wait_limit_never_writes_out_of_place():
    """Waits of one poll: whether one runs out depends on timing.  The call returns, says so in the status
    word and writes nothing beside its output; with the default limit back the next call is right."""
    rng = np.random.default_rng(2)
    x = attend_case(rng, 4, 20, 8, 2, 128, BF16, "int8", 16, 16, [3000, 200, 0, 917])
    want = attend(x)
    out = Guarded(tuple(x["q"].shape), BF16)
    assert sv.spec_get_status() == 0
    try:
        sv.spec_test_spin_limit(1)
        for _ in range(3):
            attend(x, out=out.t)
            torch.cuda.synchronize()
            status = sv.spec_get_status()
            assert status in (0, sv.SPEC_FLAG_TIMEOUT), status
            assert out.intact()
            if status == 0:
                assert torch.equal(out.t, want)
    finally:
        sv.spec_test_spin_limit(0)
    attend(x, out=out.t)
    assert sv.spec_get_status() == 0
    assert torch.equal(out.t, want)


@pytest.mark.parametrize("T", [1, 20])
def test_a_failed_allocation(T):
    rng = np.random.default_rng(3)
    x = attend_case(rng, 2, T, 8, 2, 128, BF16, "int8", 16, 16, [300, 20])
    want = attend(x)
    out = torch.full(x["q"].shape, 5.0, dtype=BF16, device=DEV)
    torch.cuda.synchronize()
    try:
        _lib.load().spec_test_fail_allocations(1)
        with pytest.raises(sv.SpecError):
            attend(x, out=out)
    finally:
        _lib.load().spec_test_fail_allocations(0)
    torch.cuda.synchronize()
    assert (out == 5.0).all()
    assert torch.equal(attend(x, out=out), want)
    assert sv.spec_get_status() == 0
