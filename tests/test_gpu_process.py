"""Token counts and logit processing on the GPU against a plain 64-bit
implementation.

Tolerance: z * rep, f * c + p and the additions are at most eight fp32
operations (the reciprocal of rep, its product, f * c, two penalties joined,
the drafts' share, the biases' sum of up to 3 terms, the last addition), each
off by at most 2^-24 of the magnitudes it adds: 8 * 2^-24 of their sum.  A bf16
output adds half a step of the result, 2^-8 of it."""
import numpy as np
import pytest
import torch

import plain_ops
import speculative_decoding_verification_36_gb300 as sv
from speculative_decoding_verification_36_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def dev(x):
    return None if x is None else torch.as_tensor(np.ascontiguousarray(x)).to(DEV)


def random_parents(rng, B, N, kind):
    if kind == "chain":
        return np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))
    if kind == "star":
        return np.full((B, N), -1, np.int32)
    return np.stack([[int(rng.integers(-1, j)) if j else -1 for j in range(N)] for _ in range(B)]).astype(np.int32)


def make(rng, B, R, V, dtype, tree=None, hist=40, bias=6, mask="rows", dups=True, alphabet=None):
    """Inputs as numpy arrays (logits: exactly representable in dtype)."""
    hi = min(V, alphabet or V)
    z = torch.from_numpy(rng.normal(0, 4, (B, R, V)).astype(np.float32)).to(dtype)
    x = dict(logits=z, drafts=None, parents=None, state=None, rep=None, freq=None, pres=None, bias_tokens=None,
             bias_values=None, mask=None)
    if R > 1:
        x["drafts"] = rng.integers(0, hi, (B, R - 1)).astype(np.int32)
        if tree:
            x["parents"] = random_parents(rng, B, R - 1, tree)
    if hist:
        tok = rng.integers(0, hi, (B, hist)).astype(np.int32)
        ln = rng.integers(0, hist + 1, B).astype(np.int32)
        x["state"] = plain_ops.count(tok, ln, (ln * 0.6).astype(np.int32), V)
    x["rep"] = rng.uniform(0.8, 1.6, B).astype(np.float32)
    x["freq"] = rng.uniform(-0.5, 1, B).astype(np.float32)
    x["pres"] = rng.uniform(-0.5, 1, B).astype(np.float32)
    if bias:
        x["bias_tokens"] = rng.integers(-1, V, (B, bias)).astype(np.int32)
        if dups and bias > 2:
            x["bias_tokens"][:, 1:3] = x["bias_tokens"][:, :1]  # the same token three times
        x["bias_values"] = rng.normal(0, 3, (B, bias)).astype(np.float32)
    if mask:
        W = (V + 31) // 32
        shape = (B, R, W) if mask == "rows" else (B, W)
        m = rng.integers(0, 2 ** 32, shape, dtype=np.uint32)
        if mask == "rows":
            m[:, ::2] |= rng.integers(0, 2 ** 32, m[:, ::2].shape, dtype=np.uint32)
            m[0, 0] = 0xffffffff
            m[-1, -1] = 0  # nothing allowed
        x["mask"] = m.view(np.int32)
    return x


def call(x, out=None, logits=None, stream=None):
    return sv.spec_process_logits(
        x["logits"].to(DEV) if logits is None else logits, draft_tokens=dev(x["drafts"]), parent_idx=dev(x["parents"]),
        token_state=dev(x["state"]), repetition=dev(x["rep"]), frequency=dev(x["freq"]), presence=dev(x["pres"]),
        bias_tokens=dev(x["bias_tokens"]), bias_values=dev(x["bias_values"]), allowed_mask=dev(x["mask"]), out=out,
        stream=stream)


def check(x, got):
    kw = {k: v for k, v in x.items() if k != "logits"}
    ref, mag = plain_ops.process(x["logits"].double().numpy(), **kw)
    g = got.cpu().double().numpy()
    np.testing.assert_array_equal(np.isnan(g), np.isnan(ref))
    inf = np.isinf(ref)
    np.testing.assert_array_equal(g[inf], ref[inf])
    ok = np.isfinite(ref)
    tol = 8 * 2.0 ** -24 * mag[ok]
    if x["logits"].dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref[ok]) + tol)
    err = np.abs(g[ok] - ref[ok])
    assert (err <= tol).all(), (err - tol).max()


SHAPES = [
    # B, R, V, dtype, tree, hist
    (1, 1, 1, torch.float32, None, 3),
    (2, 3, 7, torch.bfloat16, None, 5),
    (3, 5, 1000, torch.bfloat16, None, 40),
    (3, 5, 1000, torch.float32, None, 400),
    (2, 4, 4096, torch.bfloat16, None, 100),
    (2, 4, 4097, torch.float32, None, 100),
    (2, 3, 8200, torch.bfloat16, None, 1000),
    (1, 9, 32000, torch.float32, None, 512),
    (5, 2, 12345, torch.bfloat16, None, 300),
    (2, 7, 1003, torch.float32, "tree", 30),
    (2, 31, 5000, torch.bfloat16, "tree", 200),
    (1, 70, 600, torch.bfloat16, "tree", 20),      # more rows than one group of a tree holds
    (1, 90, 96, torch.float32, "chain", 20),       # a tree that is one long path
    (2, 40, 50, torch.float32, "star", 20),
    (1, 256, 200, torch.bfloat16, None, 10),       # the longest chain
    (70, 2, 40, torch.float32, None, 10),
    (2, 41, 9000, torch.bfloat16, "tree", 100),    # several chunks of the vocabulary and row groups
    (3, 3, 1000, torch.bfloat16, None, 9000),      # a history in which nearly every token occurs
    (2, 14, 16390, torch.float32, "tree", 4000),
    (5, 1, 20000, torch.bfloat16, None, 700),      # single rows
]


@pytest.mark.parametrize("B,R,V,dtype,tree,hist", SHAPES)
@pytest.mark.parametrize("mask", [None, "rows", "shared"])
def test_process_matches_plain(B, R, V, dtype, tree, hist, mask):
    rng = np.random.default_rng(B * 1000 + R * 10 + V)
    x = make(rng, B, R, V, dtype, tree, hist, mask=mask)
    got = call(x)
    check(x, got)
    # in place: the same bits
    z = x["logits"].to(DEV).clone()
    assert call(x, out=z, logits=z) is z
    assert torch.equal(z.view(torch.int16 if dtype == torch.bfloat16 else torch.int32),
                       got.view(torch.int16 if dtype == torch.bfloat16 else torch.int32))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("keep", [(), ("state", "rep"), ("state", "freq"), ("state", "pres"), ("drafts", "rep", "pres"),
                                  ("bias_tokens", "bias_values"), ("mask",), ("state", "drafts", "parents", "rep")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_each_part_alone(keep, dtype):
    rng = np.random.default_rng(3)
    x = make(rng, 3, 6, 2056, dtype, "tree", 60)
    x = {k: v if k in keep or k == "logits" else None for k, v in x.items()}
    got = call(x)
    check(x, got)
    if not keep:
        assert torch.equal(got.cpu().view(torch.uint8), x["logits"].view(torch.uint8))
    assert sv.spec_get_status() == 0


def test_largest_tree_many_equal_tokens():
    rng = np.random.default_rng(8)
    x = make(rng, 1, 1025, 50, torch.float32, "tree", 30, mask=None, alphabet=7)
    check(x, call(x))


def test_many_drafts_that_share_tokens():
    """More drafts in a chunk than a warp has lanes, and fewer, with repeats."""
    for R, V, alphabet in ((33, 5000, 5), (34, 5000, 5), (60, 9000, 9), (20, 300, 3)):
        for tree in (None, "tree", "star", "chain"):
            rng = np.random.default_rng(R)
            x = make(rng, 2, R, V, torch.bfloat16, tree, 60, alphabet=alphabet)
            got = call(x)
            check(x, got)
            z = x["logits"].to(DEV).clone()
            call(x, out=z, logits=z)
            assert torch.equal(z.view(torch.int16), got.view(torch.int16))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("dups", [False, True])
def test_long_bias_lists(dups):
    """More biases than a CTA has ahead, up to one for every token."""
    rng = np.random.default_rng(21)
    for V, n in ((6000, 1500), (700, 700), (5000, 5000)):
        x = make(rng, 2, 3, V, torch.float32, None, 40, bias=n, dups=False)
        x["bias_tokens"] = np.stack([rng.permutation(V)[:n] for _ in range(2)]).astype(np.int32)
        if dups:
            x["bias_tokens"][:, 1:3] = x["bias_tokens"][:, :1]
            x["bias_tokens"][:, -1] = x["bias_tokens"][:, 0]  # four times one token
        check(x, call(x))
    assert sv.spec_get_status() == 0


def test_a_lowered_wait_limit_ends_and_the_next_call_is_right():
    """Waits that give up after one poll: the launch ends, says so, and writes
    nothing next to its output; with the limit restored all is as before."""
    rng = np.random.default_rng(22)
    x = make(rng, 16, 7, 50000, torch.bfloat16, None, 500)
    n = 16 * 7 * 50000
    buf = torch.full((n + 128,), 77.0, dtype=torch.bfloat16, device=DEV)
    out = buf[64:64 + n].view(16, 7, 50000)
    z = x["logits"].to(DEV)
    before = call(x, logits=z)
    torch.cuda.synchronize()
    sv.spec_get_status()
    sv.spec_test_spin_limit(1)
    try:
        call(x, logits=z, out=out)
        torch.cuda.synchronize()
    finally:
        sv.spec_test_spin_limit(0)
    assert sv.spec_get_status() in (0, sv.SPEC_FLAG_TIMEOUT)
    assert bool((buf[:64] == 77).all()) and bool((buf[64 + n:] == 77).all())
    call(x, logits=z, out=out)
    assert torch.equal(out.view(torch.int16), before.view(torch.int16))
    assert sv.spec_get_status() == 0


def test_extreme_values_and_masks():
    rng = np.random.default_rng(5)
    for dtype in (torch.float32, torch.bfloat16):
        x = make(rng, 2, 4, 300, dtype, None, 50)
        low = torch.finfo(dtype).min
        x["logits"][0, :, ::7] = float("-inf")
        x["logits"][0, :, 1::11] = low
        x["logits"][1, :, 2::13] = torch.finfo(dtype).max / 4
        x["mask"][1] = 0  # a sequence whose mask leaves nothing, and NaN and infinities under it
        x["logits"][1, 0, ::3] = float("nan")
        x["logits"][1, 1, ::3] = float("inf")
        x["bias_values"][0, 3] = float("-inf")
        x["rep"][0] = 1.0  # the lowest value times a factor would overflow
        x["freq"][:] = np.abs(x["freq"])
        got = call(x)
        check(x, got)
        assert bool((got[1] == float("-inf")).all())
        # what a verify says of rows with nothing left
        tok, n = sv.spec_verify(got.float().contiguous(), got[:, :3].float().contiguous(), dev(x["drafts"]), 1.0, 0)
        assert int(n[1]) == -1
        assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA


def test_nan_allowed_reaches_the_verify():
    z = torch.zeros((2, 2, 64), device=DEV)
    z[0, 1, 5] = float("nan")
    out = sv.spec_process_logits(z)
    assert bool(torch.isnan(out[0, 1, 5])) and int(torch.isnan(out).sum()) == 1
    _, n = sv.spec_verify(out, None, torch.zeros((2, 1), dtype=torch.int32, device=DEV), 0.0, 0)
    assert n.tolist()[0] == -1 and n.tolist()[1] >= 0
    sv.spec_get_status()


@pytest.mark.parametrize("what,value", [("rep", 0.0), ("rep", -1.0), ("rep", np.nan), ("rep", np.inf), ("freq", np.nan),
                                        ("pres", np.inf), ("parent", 5), ("parent", -2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_bad_data_makes_the_sequence_nan(what, value, in_place):
    rng = np.random.default_rng(9)
    x = make(rng, 3, 6, 5000, torch.bfloat16, "tree", 30)
    if what == "parent":
        x["parents"][1, 2] = value
    else:
        x[what][1] = value
    z = x["logits"].to(DEV)
    got = call(x, logits=z, out=z if in_place else None)
    check(x, got)
    assert bool(torch.isnan(got[1].float()).all())
    assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA


def test_drafts_outside_the_vocabulary_count_for_nothing():
    rng = np.random.default_rng(10)
    x = make(rng, 2, 6, 100, torch.float32, None, 20)
    x["drafts"][0, 1:] = -1
    x["drafts"][1, 2] = 100
    x["drafts"][1, 3] = 2 ** 31 - 1
    check(x, call(x))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift_in,shift_out", [(0, 1), (1, 0), (1, 1), (3, 5), (4, 4), (2, 6)])
@pytest.mark.parametrize("V", [777, 4104])
def test_unaligned_buffers_and_guards(dtype, shift_in, shift_out, V):
    rng = np.random.default_rng(11)
    x = make(rng, 2, 3, V, dtype, None, 50)
    n = 2 * 3 * V
    src = torch.zeros(n + 16, dtype=dtype, device=DEV)
    z = src[shift_in:shift_in + n].view(2, 3, V)
    z.copy_(x["logits"])
    buf = torch.full((n + 16,), 77.0, dtype=dtype, device=DEV)
    out = buf[shift_out:shift_out + n].view(2, 3, V)
    check(x, call(x, logits=z, out=out))
    assert bool((buf[:shift_out] == 77).all()) and bool((buf[shift_out + n:] == 77).all())
    keep = (src[:shift_in].clone(), src[shift_in + n:].clone())
    call(x, logits=z, out=z)
    assert torch.equal(z, out)
    assert torch.equal(src[:shift_in], keep[0]) and torch.equal(src[shift_in + n:], keep[1])


def test_overlapping_output_is_refused():
    buf = torch.zeros(2 * 64 + 8, device=DEV)
    with pytest.raises(sv.SpecError):
        sv.spec_process_logits(buf[:128].view(1, 2, 64), out=buf[8:].view(1, 2, 64))


def test_binding_refuses():
    z = torch.zeros((2, 3, 64), device=DEV)
    i = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    for kw in (dict(draft_tokens=i[:, :1].contiguous()), dict(parent_idx=i), dict(draft_tokens=i.long()),
               dict(token_state=i), dict(repetition=torch.ones(3, device=DEV)), dict(frequency=torch.ones(2)),
               dict(bias_tokens=i), dict(bias_tokens=i, bias_values=torch.zeros((2, 3), device=DEV)),
               dict(allowed_mask=torch.zeros((2, 3, 1), dtype=torch.int32, device=DEV)),
               dict(out=z[:, :2]), dict(out=z.to(torch.bfloat16))):
        with pytest.raises((ValueError, TypeError)):
            sv.spec_process_logits(z, **kw)
    with pytest.raises(ValueError):
        sv.spec_process_logits(z.transpose(0, 1))
    with pytest.raises(TypeError):
        sv.spec_process_logits(z.half())


# ---------------------------------------------------------------------------
# counts
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (3, 17, 5), (4, 300, 33), (2, 5000, 1000), (7, 64, 128256), (1, 70000, 40),
                                   (1, 20000, 100001), (2, 0, 9)])
def test_counts_match_plain(B, S, V):
    rng = np.random.default_rng(B + S + V)
    tok = rng.integers(-1, V + 1, (B, S)).astype(np.int32)  # some just outside
    ln = rng.integers(0, S + 1, B).astype(np.int32)
    pl = (ln * rng.uniform(0, 1, B)).astype(np.int32)
    state = sv.spec_token_state(B, V, DEV)
    state.fill_(-1)
    got = sv.spec_count_tokens(state, dev(tok).reshape(B, S), V, lengths=dev(ln), prompt_lengths=dev(pl), reset=True)
    assert got is state
    ref = plain_ops.count(tok, ln, pl, V)
    np.testing.assert_array_equal(state.cpu().numpy(), ref)
    # added to, as a verify's padded output is
    more = rng.integers(-1, V, (B, 6)).astype(np.int32)
    sv.spec_count_tokens(state, dev(more), V)
    np.testing.assert_array_equal(state.cpu().numpy(), plain_ops.count(more, None, None, V, start=ref))
    assert sv.spec_get_status() == 0


@pytest.mark.parametrize("B,S", [(200, 32767), (200, 32768), (1, 32767), (1, 40000), (3, 32768)])
def test_counts_of_one_token_over_and_over(B, S):
    """The largest counts that 16 bits hold beside the prompt's bit, and the
    next, in a large batch, in a small one and with a cluster's shares."""
    V = 100
    tok = torch.full((B, S), 7, dtype=torch.int32, device=DEV)
    tok[:, 0] = 8
    prompts = torch.full((B,), 1, dtype=torch.int32, device=DEV)
    prompts[-1] = 3
    state = sv.spec_token_state(B, V, DEV)
    sv.spec_count_tokens(state, tok, V, prompt_lengths=prompts, reset=True)
    got = state.cpu().numpy()
    want = np.zeros_like(got)
    want[:, 7], want[:, 8] = S - 1, -2 ** 31
    want[-1, 7] = (S - 3) - 2 ** 31
    want[:, plain_ops.state_words(V)[0]] = 1 << 7 | 1 << 8
    np.testing.assert_array_equal(got, want)
    assert sv.spec_get_status() == 0


def test_counts_at_unaligned_rows():
    rng = np.random.default_rng(23)
    for B, S, V in ((3, 4099, 5000), (1, 20001, 3000), (5, 63, 40000)):
        buf = torch.from_numpy(rng.integers(0, V, B * S + 3).astype(np.int32)).to(DEV)
        for shift in (0, 1, 3):
            tok = buf[shift:shift + B * S].view(B, S)
            ln = rng.integers(0, S + 1, B).astype(np.int32)
            pl = (ln * rng.uniform(0, 1, B)).astype(np.int32)
            state = sv.spec_count_tokens(sv.spec_token_state(B, V, DEV), tok, V, lengths=dev(ln), prompt_lengths=dev(pl), reset=True)
            np.testing.assert_array_equal(state.cpu().numpy(), plain_ops.count(tok.cpu().numpy(), ln, pl, V))


def test_counts_bad_lengths_leave_the_row():
    V = 50
    tok = np.arange(24, dtype=np.int32).reshape(4, 6)
    ln, pl = np.array([6, 7, -1, 3], np.int32), np.array([2, 0, 0, 4], np.int32)
    state = sv.spec_token_state(4, V, DEV)
    sv.spec_count_tokens(state, dev(tok), V, lengths=dev(ln), prompt_lengths=dev(pl))
    np.testing.assert_array_equal(state.cpu().numpy(), plain_ops.count(tok, ln, pl, V))
    assert bool((state[1:] == 0).all())
    assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA


def test_one_row_of_a_state_is_replaced():
    rng = np.random.default_rng(12)
    V, tok = 777, rng.integers(0, 777, (3, 50)).astype(np.int32)
    state = sv.spec_token_state(3, V, DEV)
    sv.spec_count_tokens(state, dev(tok), V)
    new = rng.integers(0, V, (1, 20)).astype(np.int32)
    sv.spec_count_tokens(state[1:2], dev(new), V, prompt_lengths=dev(np.array([20], np.int32)), reset=True)
    ref = plain_ops.count(tok, None, None, V)
    ref[1:2] = plain_ops.count(new, None, np.array([20]), V)
    np.testing.assert_array_equal(state.cpu().numpy(), ref)


# ---------------------------------------------------------------------------
# streams, graphs, the loop
# ---------------------------------------------------------------------------
def test_two_streams_at_once_match_the_calls_alone():
    rng = np.random.default_rng(13)
    xs = [make(rng, 8, 5, 32000, torch.bfloat16, None, 500), make(rng, 4, 9, 20001, torch.float32, "tree", 300)]
    alone = [call(x) for x in xs]
    ins = [x["logits"].to(DEV) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        outs = []
        for x, z, s in zip(xs, ins, streams):
            with torch.cuda.stream(s):
                outs.append(call(x, logits=z))
        torch.cuda.synchronize()
        for o, a in zip(outs, alone):
            assert torch.equal(o.nan_to_num(7.0), a.nan_to_num(7.0))


def test_captured_step_replays_on_new_data():
    """Processing, a greedy verify and the counting of its answer in one graph."""
    rng = np.random.default_rng(14)
    B, K, V = 4, 3, 5000
    x = make(rng, B, K + 1, V, torch.bfloat16, None, 100, mask="rows")
    x["mask"] |= 1  # every row keeps a token
    z, d = x["logits"].to(DEV), dev(x["drafts"])
    start = dev(x["state"])
    state = start.clone()
    pen = [dev(x[k]) for k in ("rep", "freq", "pres")]
    bt, bv, mask = dev(x["bias_tokens"]), dev(x["bias_values"]), dev(x["mask"])
    out = torch.empty_like(z)
    tok = torch.empty((B, K + 1), dtype=torch.int32, device=DEV)
    n = torch.empty((B,), dtype=torch.int32, device=DEV)

    def step():
        sv.spec_process_logits(z, d, None, state, *pen, bias_tokens=bt, bias_values=bv, allowed_mask=mask, out=out)
        sv.spec_verify(out, None, d, 0.0, 0, out_tokens=tok, out_n_accepted=n)
        sv.spec_count_tokens(state, tok, V)

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    state.copy_(start)
    for rep in range(3):
        z.copy_(torch.randn(z.shape, device=DEV) * 4)
        before = state.clone()
        g.replay()
        torch.cuda.synchronize()
        got = (out.clone(), tok.clone(), n.clone(), state.clone())
        state.copy_(before)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, tok, n, state)):
            assert torch.equal(a, b)
        assert not torch.equal(before, state)
    assert sv.spec_get_status() == 0


def test_captured_large_launches_replay():
    """Launches of more units than start at once, and a history shared out over
    a cluster, in one graph; two graphs of the same buffers, replayed by turns."""
    B, R, V = 40, 5, 128256
    o = wl.make_settings(B, R, V, hist=600, n_bias=40, seed=3, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    z = (torch.randn((B, R, V), generator=g, device=DEV) * 4).to(torch.bfloat16)
    d = torch.randint(0, V, (B, R - 1), generator=g, device=DEV, dtype=torch.int32)
    state, out = sv.spec_token_state(B, V, DEV), torch.empty_like(z)
    long = torch.randint(0, V, (1, 60000), generator=g, device=DEV, dtype=torch.int32)
    long_state = sv.spec_token_state(1, V, DEV)

    def step():
        sv.spec_count_tokens(state, o["tokens"], V, o["lengths"], o["prompt_lengths"], reset=True)
        sv.spec_count_tokens(long_state, long, V, reset=True)
        sv.spec_process_logits(z, d, None, state, o["repetition"], o["frequency"], o["presence"], o["bias_tokens"],
                               o["bias_values"], o["allowed_mask"], out=out)

    step()
    torch.cuda.synchronize()
    side, graphs = torch.cuda.Stream(), []
    for _ in range(2):
        with torch.cuda.stream(side):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                step()
    for k in range(4):
        z.copy_((torch.randn((B, R, V), generator=g, device=DEV) * 4).to(torch.bfloat16))
        long.random_(0, V, generator=g)
        o["tokens"].random_(0, V, generator=g)
        out.zero_(), state.fill_(7), long_state.fill_(7)
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, state, long_state)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, state, long_state)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert sv.spec_get_status() == 0


def test_two_large_launches_side_by_side():
    """Two launches that each fill the device, at once: only CTAs that have
    started hold work, and neither takes the other's."""
    B, R, V = 24, 6, 152064
    o = wl.make_settings(B, R, V, hist=2000, n_bias=40, seed=5, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(6)
    zs = [(torch.randn((B, R, V), generator=g, device=DEV) * 4).to(torch.bfloat16) for _ in range(2)]
    state = sv.spec_count_tokens(sv.spec_token_state(B, V, DEV), o["tokens"], V, o["lengths"], o["prompt_lengths"], reset=True)
    outs = [torch.empty_like(z) for z in zs]

    def one(i, stream=None):
        sv.spec_process_logits(zs[i], None, None, state, o["repetition"], o["frequency"], o["presence"], o["bias_tokens"],
                               o["bias_values"], o["allowed_mask"], out=outs[i], stream=stream)

    alone = []
    for i in range(2):
        one(i)
        alone.append(outs[i].clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for x in outs:
            x.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            one(i, streams[i])
        torch.cuda.synchronize()
        for x, y in zip(outs, alone):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert sv.spec_get_status() == 0


def test_empty_batches_and_rows():
    V = 100
    state = sv.spec_token_state(0, V, DEV)
    none = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    sv.spec_count_tokens(state, none, V, reset=True)
    z = torch.empty((0, 5, V), device=DEV)
    assert sv.spec_process_logits(z, none, None, state).shape == (0, 5, V)
    one = torch.zeros((1, 1, V), device=DEV)
    assert torch.equal(sv.spec_process_logits(one, torch.empty((1, 0), dtype=torch.int32, device=DEV)), one)


def test_decode_loop_follows_a_plain_one():
    """N-gram drafts, processed rows, a greedy verify and the counts over
    several steps, against the same loop in numpy: tokens have to agree."""
    rng = np.random.default_rng(15)
    B, K, V, steps, room = 3, 4, 600, 6, 200
    hist = np.full((B, room), -7, np.int32)
    length = np.array([30, 41, 25])
    for b in range(B):
        hist[b, :length[b]] = np.tile(rng.integers(0, 40, 9), 6)[:length[b]]
    prompt = length.copy()
    rep, freq, pres = (np.array(v, np.float32) for v in ([1.2, 1.0, 1.5], [0.1, 0.3, 0.0], [0.2, 0.0, 0.4]))
    state = sv.spec_token_state(B, V, DEV)
    sv.spec_count_tokens(state, dev(hist), V, lengths=dev(length.astype(np.int32)), prompt_lengths=dev(prompt.astype(np.int32)),
                         reset=True)
    for step in range(steps):
        drafts, nd, _ = sv.spec_ngram_draft(dev(hist), dev(length.astype(np.int32)), 1, 4, K)
        d = drafts.clamp(min=0)  # a padded draft is some token: the verify judges it
        z = torch.randn((B, K + 1, V), generator=torch.Generator().manual_seed(step)) * 3
        for b in range(B):  # the model tends to go on with the drafts
            for i in range(K):
                z[b, i, int(d[b, i])] += 14
        mask = torch.from_numpy(rng.integers(0, 2 ** 32, (B, K + 1, (V + 31) // 32), dtype=np.uint32).view(np.int32)) | 0x55555555
        kw = dict(drafts=d.cpu().numpy(), state=state.cpu().numpy(), rep=rep, freq=freq, pres=pres, mask=mask.numpy())
        ref, _ = plain_ops.process(z.double().numpy(), **kw)
        out = sv.spec_process_logits(z.to(DEV), d, None, state, dev(rep), dev(freq), dev(pres), allowed_mask=mask.to(DEV))
        tok, n = sv.spec_verify(out, None, d, 0.0, 0)
        sv.spec_count_tokens(state, tok, V)
        tok, n = tok.cpu().numpy(), n.cpu().numpy()
        for b in range(B):
            want = []
            for i in range(K + 1):
                want.append(int(ref[b, i].argmax()))
                if i == K or want[-1] != int(d[b, i]):
                    break
            assert tok[b, :n[b] + 1].tolist() == want, (step, b)
            hist[b, length[b]:length[b] + len(want)] = want
            length[b] += len(want)
    ref = plain_ops.count(hist, length, prompt, V)
    np.testing.assert_array_equal(state.cpu().numpy(), ref)
    assert (length - prompt).sum() > steps * B  # drafts were accepted


def test_other_stream_argument():
    rng = np.random.default_rng(16)
    x = make(rng, 2, 3, 4000, torch.float32)
    s = torch.cuda.Stream()
    z = x["logits"].to(DEV)
    torch.cuda.synchronize()
    got = call(x, logits=z, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    check(x, got)


def test_workload_shapes_sampled():
    """The largest batch's shape, rows drawn at random against the plain form."""
    p = wl.preset("c3", B=24)
    rng = np.random.default_rng(17)
    g = torch.Generator(device=DEV).manual_seed(1)
    z = (torch.randn((p.B, p.K + 1, p.V), generator=g, device=DEV) * 4).to(torch.bfloat16)
    x = make(rng, p.B, p.K + 1, 64, torch.bfloat16, None, 0, bias=0, mask=None)  # the scalars
    tok = rng.integers(0, p.V, (p.B, 4000)).astype(np.int32)
    tok[:, ::2] //= 200
    ln = rng.integers(2000, 4001, p.B).astype(np.int32)
    x["state"] = plain_ops.count(tok, ln, (ln // 2).astype(np.int32), p.V)
    x["drafts"] = tok[:, :p.K].copy()
    x["mask"] = rng.integers(0, 2 ** 32, (p.B, p.K + 1, p.V // 32), dtype=np.uint32).view(np.int32)
    got = call(x, logits=z)
    for b in (0, 7, p.B - 1):
        sub = {k: v[b:b + 1] if v is not None else None for k, v in x.items()}
        sub["logits"] = z[b:b + 1].cpu()
        check(sub, got[b:b + 1])


# The last piece of the last row then ends inside the 16-byte vector that it
# starts in, or lies across the input's end.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 9, 511, 513, 515, 1027, 4097, 4099])
def test_last_elements_of_rows_off_16_bytes(V, dtype):
    rng = np.random.default_rng(V)
    for B, R in ((1, 1), (1, 2), (1, 3), (2, 3), (1, 5), (3, 3), (7, 1), (2, 7)):
        for mask in (None, "rows"):
            x = make(rng, B, R, V, dtype, mask=mask)
            x["logits"] += 100 * torch.sign(x["logits"])  # far from what other rows or calls left behind
            check(x, call(x))
            plain = {k: None for k in x} | {"logits": x["logits"]}
            assert torch.equal(call(plain).cpu(), x["logits"])
            check(x, call(x, out=(z := x["logits"].to(DEV)), logits=z))


# A padded vocabulary's state has the same size as the rows' own: tokens that
# the rows do not have change nothing, beside the rows least of all.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,counted", [(33, 64), (40, 64), (4097, 4128), (5000, 5024)])
@pytest.mark.parametrize("in_place", [False, True])
def test_state_of_a_padded_vocabulary(V, counted, dtype, in_place):
    rng = np.random.default_rng(V)
    B, R, guard = 3, 4, 64
    x = make(rng, B, R, V, dtype, None, 200)
    tok = np.concatenate([rng.integers(0, V, (B, 50)), np.tile(np.arange(V, counted), (B, 1))], 1).astype(np.int32)
    state = sv.spec_token_state(B, counted, DEV)
    assert state.shape == sv.spec_token_state(B, V, DEV).shape
    sv.spec_count_tokens(state, dev(tok), counted, reset=True)
    x["state"] = plain_ops.count(np.where(tok < V, tok, -1), np.full(B, tok.shape[1], np.int32), np.zeros(B, np.int32), V)
    n = B * R * V
    buf = torch.full((n + guard,), 77.0, dtype=dtype, device=DEV)
    z = buf[:n].view(B, R, V)
    z.copy_(x["logits"])
    got = sv.spec_process_logits(
        z, draft_tokens=dev(x["drafts"]), token_state=state, repetition=dev(x["rep"]), frequency=dev(x["freq"]),
        presence=dev(x["pres"]), bias_tokens=dev(x["bias_tokens"]), bias_values=dev(x["bias_values"]),
        allowed_mask=dev(x["mask"]), out=z if in_place else None)
    check(x, got)
    assert bool((buf[n:] == 77).all())
    assert sv.spec_get_status() == 0


# z / repetition is worked out with the reciprocal, which has to be a normal
# number: outside these limits the call reports bad data instead of a wrong value.
@pytest.mark.parametrize("value,good", [(2.0 ** -126, True), (2.0 ** 126, True), (2.0 ** -127, False),
                                        (2.0 ** -149, False), (1.5 * 2.0 ** 126, False), (3e38, False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_smallest_and_largest_repetitions(value, good, in_place):
    rng = np.random.default_rng(21)
    B, R, V = 2, 2, 64
    z = torch.from_numpy((rng.uniform(0.5, 1, (B, R, V)) * 2.0 ** -4).astype(np.float32))
    if value > 1:
        z = z * 2.0 ** 100  # the quotient stays a normal number
    rep = np.array([1.0, value], np.float32)
    tok = np.tile(np.arange(V, dtype=np.int32), (B, 1))
    st = dev(plain_ops.count(tok, np.full(B, V, np.int32), np.full(B, V, np.int32), V))
    g = z.to(DEV)
    got = sv.spec_process_logits(g, token_state=st, repetition=dev(rep), out=g if in_place else None).cpu()
    assert torch.equal(got[0], z[0])
    if good:
        ref = z[1].double() / value
        assert bool(((got[1].double() - ref).abs() <= 8 * 2.0 ** -24 * ref.abs()).all())
    else:
        assert bool(torch.isnan(got[1]).all())
    assert sv.spec_get_status() == (0 if good else sv.SPEC_FLAG_BAD_DATA)


@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("lengths,prompts,bad", [([0, 3], None, True), ([0, -1], None, True), ([0, 0], [0, 0], False),
                                                 ([0, 0], [0, 1], True), (None, [-1, 0], True), (None, None, False)])
def test_lengths_of_rows_without_entries_are_judged(lengths, prompts, bad, reset):
    V = 40
    state = sv.spec_count_tokens(sv.spec_token_state(2, V, DEV), dev(np.arange(6, dtype=np.int32).reshape(2, 3)), V)
    want = torch.zeros_like(state) if reset else state.clone()
    i32 = lambda x: None if x is None else dev(np.array(x, np.int32))  # noqa: E731
    none = torch.empty((2, 0), dtype=torch.int32, device=DEV)
    sv.spec_count_tokens(state, none, V, lengths=i32(lengths), prompt_lengths=i32(prompts), reset=reset)
    assert torch.equal(state, want)
    assert sv.spec_get_status() == (sv.SPEC_FLAG_BAD_DATA if bad else 0)


# Launches of more units (chunks of 4096 tokens x groups of rows x sequences) than
# start at once, 456 on 152 SMs: CTAs go on to further units, with the ring, the
# masks, the counts and the gatherings of the next one under way.
def take_over(seed, B, R, V, dtype, tree, mask, bias, shift=(0, 0)):
    rng = np.random.default_rng(seed)
    x = make(rng, B, R, V, dtype, tree, 400, bias=bias, mask=mask)
    for b in range(1, B, 3):  # many in the first chunks; no token over three times
        x["bias_tokens"][b, 3:] = rng.permutation(np.setdiff1d(np.arange(min(V, 5000)), x["bias_tokens"][b, :3]))[:bias - 3]
    x["rep"][B // 3] = np.nan  # a bad sequence between good ones
    if tree:
        x["parents"][B // 2, 0] = 0
    n = B * R * V
    src = torch.zeros(n + 16, dtype=dtype, device=DEV)
    z = src[shift[0]:shift[0] + n].view(B, R, V)
    z.copy_(x["logits"])
    buf = torch.full((n + 16,), 77.0, dtype=dtype, device=DEV)
    out = buf[shift[1]:shift[1] + n].view(B, R, V)
    check(x, call(x, logits=z, out=out))
    assert bool((buf[:shift[1]] == 77).all()) and bool((buf[shift[1] + n:] == 77).all())
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    got = out.clone()
    out.fill_(5)
    call(x, logits=z, out=out)
    assert torch.equal(out.view(bits), got.view(bits))
    assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA


@pytest.mark.parametrize("B,R,V,dtype,tree,mask,bias", [
    (24, 4, 96001, torch.bfloat16, None, "shared", 20),     # rows off 16 bytes, 576 units
    (24, 5, 96003, torch.float32, None, "rows", 600),       # ... in fp32, a long bias list
    (16, 31, 40001, torch.bfloat16, "tree", "rows", 30),    # three groups of rows: 480 units
    (16, 14, 60000, torch.float32, "tree", None, 6),        # two groups: 480 units
    (40, 1, 96000, torch.float32, None, "shared", 6),       # single rows, 960 units
    (48, 3, 50003, torch.float32, None, "rows", 40),        # 624 units
    (1000, 3, 4000, torch.bfloat16, None, "rows", 12),      # a chunk a sequence
    (7, 2, 300000, torch.bfloat16, None, None, 6),          # 518 units of a few long rows
    (36, 40, 5000, torch.bfloat16, "tree", "shared", 9),    # many groups, two chunks
])
def test_units_taken_over_match_plain(B, R, V, dtype, tree, mask, bias):
    take_over(V + R, B, R, V, dtype, tree, mask, bias)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [(1, 1), (3, 2)])
def test_units_taken_over_off_16_bytes(dtype, shift):
    take_over(7, 31, 3, 65536, dtype, None, "rows", 20, shift)


def test_waits_that_run_out_write_nothing_wrong():
    """With a limit of one poll some wait of a launch that is bound by memory
    runs out: the call says so, and whatever it has written is right."""
    B, R, V = 64, 9, 128251  # 0.3 GB in and out, rows off 16-byte boundaries
    o = wl.make_settings(B, R, V, hist=2000, n_bias=40, seed=9, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(10)
    state = sv.spec_count_tokens(sv.spec_token_state(B, V, DEV), o["tokens"], V, o["lengths"], o["prompt_lengths"], reset=True)
    d = torch.randint(0, V, (B, R - 1), generator=g, device=DEV, dtype=torch.int32)
    ran_out = 0
    for dtype, bits in ((torch.bfloat16, torch.int16), (torch.float32, torch.int32)):
        z = (torch.randn((B, R, V), generator=g, device=DEV) * 4).to(dtype)
        buf = torch.full((B * R * V + 128,), 77.0, dtype=dtype, device=DEV)  # no logit is 77
        out = buf[64:-64].view(B, R, V)

        def one(out):
            return sv.spec_process_logits(z, d, None, state, o["repetition"], o["frequency"], o["presence"], o["bias_tokens"],
                                          o["bias_values"], o["allowed_mask"], out=out)

        right = one(torch.empty_like(z))
        assert sv.spec_get_status() == 0 and not bool((right == 77).any())
        for _ in range(4):
            buf.fill_(77.0)
            torch.cuda.synchronize()
            sv.spec_test_spin_limit(1)
            try:
                one(out)
                torch.cuda.synchronize()
            finally:
                sv.spec_test_spin_limit(0)
            status = sv.spec_get_status()
            assert status in (0, sv.SPEC_FLAG_TIMEOUT)
            same = out.view(bits) == right.view(bits)
            assert bool((same | (out == 77)).all())
            if status:
                ran_out += 1
            else:
                assert bool(same.all())
            assert bool((buf[:64] == 77).all()) and bool((buf[-64:] == 77).all())
        one(out)
        assert torch.equal(out.view(bits), right.view(bits)) and sv.spec_get_status() == 0
    assert ran_out > 0


@pytest.mark.parametrize("in_place", [False, True])
def test_rows_past_32_bit_offsets(in_place):
    """Over 2^32 logits: the last sequences against the same call on them alone."""
    B, R, V, last = 3200, 9, 152063, 3  # rows off 16-byte boundaries
    assert B * R * V > 2 ** 32
    o = wl.make_settings(B, R, V, hist=64, n_bias=8, mask=False, seed=11, device=DEV)
    mask = torch.full((B, (V + 31) // 32), -2, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(12)
    z = torch.empty((B, R, V), dtype=torch.bfloat16, device=DEV)
    z[:-last] = 1.0
    z[-last:] = (torch.randn((last, R, V), generator=g, device=DEV) * 4).to(torch.bfloat16)
    d = torch.randint(0, V, (B, R - 1), generator=g, device=DEV, dtype=torch.int32)
    state = sv.spec_count_tokens(sv.spec_token_state(B, V, DEV), o["tokens"], V, o["lengths"], o["prompt_lengths"], reset=True)

    def call(s, z, out):
        return sv.spec_process_logits(z, d[s], None, state[s], o["repetition"][s], o["frequency"][s], o["presence"][s],
                                      o["bias_tokens"][s], o["bias_values"][s], mask[s], out=out)

    tail = slice(B - last, B)
    want = call(tail, z[tail].clone(), None)
    got = call(slice(0, B), z, z if in_place else None)
    assert torch.equal(got[tail].view(torch.int16), want.view(torch.int16))
    assert bool((got[:, :, ::32] == float("-inf"))[::101].all())
    assert sv.spec_get_status() == 0
