"""Refusals of the logit-processing, token-count and paged-cache entry points
that need no GPU: bad arguments are turned down on the host before any CUDA
call."""
import pytest
import torch

import speculative_decoding_verification_36_gb300 as sv
from speculative_decoding_verification_36_gb300 import _lib, build
import plain_ops

FAKE = 0x100000  # never dereferenced
FAR = 0x900000000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_state_words(lib):
    for V in (1, 31, 32, 33, 127, 128, 129, 32000, 128256, 152064, 96001):
        assert lib.spec_token_state_words(V) == plain_ops.state_words(V)[1]
        assert lib.spec_token_state_words(V) % 4 == 0
    for V in (0, -1, 2 ** 30 + 1):
        assert lib.spec_token_state_words(V) == _lib.SPEC_ERR_SHAPE
    assert lib.spec_token_state_words(2 ** 30) > 0


def test_count_checks(lib):
    def call(tok=FAKE, ln=None, pl=None, B=2, S=4, V=10, st=FAKE):
        return lib.spec_count_tokens(tok, ln, pl, B, S, V, 0, st, None)

    assert call(tok=None) == _lib.SPEC_ERR_NULL
    assert call(st=None) == _lib.SPEC_ERR_NULL
    for bad in (dict(B=-1), dict(S=-1), dict(S=2 ** 30 + 1), dict(V=0), dict(V=2 ** 30 + 1)):
        assert call(**bad) == _lib.SPEC_ERR_SHAPE
    assert call(B=0, tok=None, st=None) == _lib.SPEC_OK
    assert call(st=FAKE + 8) == _lib.SPEC_ERR_SHAPE  # off a 16-byte boundary


@pytest.mark.parametrize("fn", ["spec_process_logits_f32", "spec_process_logits_bf16"])
def test_process_checks(lib, fn):
    f = getattr(lib, fn)

    def call(z=FAKE, d=FAKE, p=None, n_bias=0, bt=None, bv=None, mask=None, rows=0, B=2, R=3, V=16, out=FAKE):
        return f(z, d, p, None, None, None, None, n_bias, bt, bv, mask, rows, B, R, V, out, None)

    assert call(z=None) == _lib.SPEC_ERR_NULL
    assert call(out=None) == _lib.SPEC_ERR_NULL
    assert call(d=None, p=FAKE) == _lib.SPEC_ERR_NULL
    assert call(n_bias=1, bt=FAKE) == _lib.SPEC_ERR_NULL
    assert call(n_bias=1, bv=FAKE) == _lib.SPEC_ERR_NULL
    for bad in (dict(B=-1), dict(R=0), dict(R=1026), dict(V=0), dict(V=2 ** 30 + 1), dict(n_bias=-1),
                dict(mask=FAKE, rows=0), dict(mask=FAKE, rows=2), dict(B=2 ** 30, R=1025, V=2 ** 30)):
        assert call(**bad) == _lib.SPEC_ERR_SHAPE, bad
    assert call(B=0, z=None, out=None) == _lib.SPEC_OK
    # 2 * 3 * 16 values: an output that starts inside the input, or ends in it
    size = 2 * 3 * 16 * (4 if fn.endswith("f32") else 2)
    assert call(out=FAKE + 16) == _lib.SPEC_ERR_OVERLAP
    assert call(out=FAKE + size - 1) == _lib.SPEC_ERR_OVERLAP
    assert call(out=FAKE - 16) == _lib.SPEC_ERR_OVERLAP


@pytest.mark.parametrize("fn", ["spec_kv_append_f32", "spec_kv_append_bf16"])
def test_append_checks(lib, fn):
    f = getattr(lib, fn)

    def call(k=FAKE, v=FAKE, ks=32, q=None, qs=0, oq=None, par=None, ln=FAKE, tab=FAKE, B=2, T=3, Hq=0, Hkv=2, D=16,
             rot=16, turns=FAKE, kc=FAR, vc=FAR, pages=4, ps=16, mp=2):
        return f(k, v, ks, q, qs, oq, par, None, ln, tab, B, T, Hq, Hkv, D, rot, 0, turns, kc, vc, pages, ps, mp, None)

    for name in ("k", "v", "ln", "tab", "kc", "vc", "turns"):
        assert call(**{name: None}) == _lib.SPEC_ERR_NULL, name
    assert call(Hq=2, qs=32, q=FAKE) == _lib.SPEC_ERR_NULL
    assert call(Hq=2, qs=32, oq=FAKE) == _lib.SPEC_ERR_NULL
    for bad in (dict(B=-1), dict(T=-1), dict(Hq=-1), dict(Hkv=0), dict(D=0), dict(D=1025), dict(rot=-2), dict(rot=3),
                dict(rot=18), dict(pages=0), dict(ps=0), dict(mp=0), dict(ks=31), dict(Hq=2, qs=31, q=FAKE, oq=FAKE),
                dict(par=FAKE, T=1026), dict(B=2 ** 20, T=2 ** 20), dict(Hq=2 ** 14 + 1, D=1024, ks=2 ** 12, qs=2 ** 25, q=FAKE, oq=FAKE, rot=0),
                dict(Hkv=2 ** 14 + 1, D=1024, ks=2 ** 25, rot=0)):
        assert call(**bad) == _lib.SPEC_ERR_SHAPE, bad
    assert call(B=0) == _lib.SPEC_OK
    assert call(T=0) == _lib.SPEC_OK


def test_commit_checks(lib):
    def call(kc=FAKE, vc=FAKE, layers=1, lb=4 * 16 * 64, pages=4, ps=16, eb=64, tab=FAR, mp=2, ln=FAR, tok=FAR, par=FAR,
             path=FAR, plen=FAR, B=2, N=3, nodes=FAR, oln=FAR + 4096):
        return lib.spec_kv_commit(kc, vc, layers, lb, pages, ps, eb, tab, mp, ln, tok, par, path, plen, B, N, nodes, oln,
                                  None)

    for name in ("kc", "vc", "tab", "ln", "tok", "par", "path", "plen", "nodes", "oln"):
        assert call(**{name: None}) == _lib.SPEC_ERR_NULL, name
    for bad in (dict(B=-1), dict(N=-1), dict(N=1025), dict(layers=0), dict(layers=32768), dict(pages=0), dict(ps=0),
                dict(eb=0), dict(mp=0), dict(lb=4 * 16 * 64 - 1)):
        assert call(**bad) == _lib.SPEC_ERR_SHAPE, bad
    assert call(oln=FAR) == _lib.SPEC_ERR_OVERLAP
    assert call(oln=FAR + 4) == _lib.SPEC_ERR_OVERLAP
    assert call(B=0) == _lib.SPEC_OK


def test_binding_refuses_host_tensors(lib):
    i = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.spec_count_tokens(i, i, 10)
    with pytest.raises(ValueError):
        sv.spec_process_logits(torch.zeros(2, 3, 8))
    with pytest.raises(ValueError):
        sv.spec_kv_append(torch.zeros(1, 2, 1, 4), torch.zeros(1, 2, 1, 4), None, None, i, i)
    with pytest.raises(ValueError):
        sv.spec_kv_commit(torch.zeros(1, 2, 1, 4), torch.zeros(1, 2, 1, 4), i, i, i, i, i, i)
    with pytest.raises(sv.SpecError):
        sv.spec_token_state(1, 0, "cpu")
    for V in (1, 32, 33, 4095, 152064):
        assert sv.spec_token_state(2, V, "cpu").shape == (2, lib.spec_token_state_words(V))


def test_rope_turns():
    import math
    t = sv.spec_rope_turns([2 * math.pi / 4, 2 * math.pi * 0.75, 0.0, 2 * math.pi], "cpu")
    assert t.dtype == torch.int64
    assert [int(x) % 2 ** 64 for x in t] == [2 ** 62, 3 * 2 ** 62, 0, 0]


def test_caches_that_share_memory_are_refused(lib):
    def append(fn, kc, vc, pages=4):
        return getattr(lib, fn)(FAKE, FAKE, 32, None, 0, None, None, None, FAKE, FAKE, 2, 3, 0, 2, 16, 16, 0, FAKE, kc, vc,
                                pages, 16, 2, None)

    for fn, size in (("spec_kv_append_f32", 4 * 16 * 32 * 4), ("spec_kv_append_bf16", 4 * 16 * 32 * 2)):
        for d in (0, 16, size - 16):
            assert append(fn, FAR, FAR + d) == _lib.SPEC_ERR_OVERLAP
            assert append(fn, FAR + d, FAR) == _lib.SPEC_ERR_OVERLAP

    def commit(kc, vc, layers=1, lb=4 * 16 * 64, nodes=FAR + 8192, oln=FAR + 4096, **at):
        p = dict(ln=FAR, plen=FAR + 64, path=FAR + 128, tok=FAR + 256, par=FAR + 384) | at
        return lib.spec_kv_commit(kc, vc, layers, lb, 4, 16, 64, FAR + 512, 2, p["ln"], p["tok"], p["par"], p["path"],
                                  p["plen"], 2, 3, nodes, oln, None)

    size, base = 4 * 16 * 64, FAR + (1 << 30)
    for d in (0, 64, size - 64):
        assert commit(base, base + d) == _lib.SPEC_ERR_OVERLAP
        assert commit(base + d, base) == _lib.SPEC_ERR_OVERLAP
    # three layers, twice their size apart: by turns they fit, half a layer on they do not
    for d in (0, 2 * size, 4 * size, size // 2, size + size // 2, 3 * size + 64, 5 * size - 64 - size):
        assert commit(base, base + d, 3, 2 * size) == _lib.SPEC_ERR_OVERLAP, d
    for name in ("ln", "plen", "path", "tok", "par"):
        assert commit(base, base + size, **{name: FAR + 4096}) == _lib.SPEC_ERR_OVERLAP, name
        assert commit(base, base + size, **{name: FAR + 8192 + 4}) == _lib.SPEC_ERR_OVERLAP, name
    assert commit(base, base + size, nodes=FAR + 4096) == _lib.SPEC_ERR_OVERLAP
    # what is apart goes past these checks: to the device, which is not there
    if not torch.cuda.is_available():
        for d, layers, lb in ((size, 1, size), (3 * size, 3, size), (size, 3, 2 * size), (5 * size, 3, 2 * size)):
            assert commit(base, base + d, layers, lb) == _lib.SPEC_ERR_CUDA
            assert commit(base + d, base, layers, lb) == _lib.SPEC_ERR_CUDA


@pytest.mark.parametrize("fn", ["spec_process_logits_f32", "spec_process_logits_bf16"])
def test_sizes_past_a_kernels_counters_are_refused(lib, fn):
    def call(B=1, R=1, V=8, n_bias=0):
        return getattr(lib, fn)(FAKE, None, None, None, None, None, None, n_bias, FAKE, FAKE, None, 0, B, R, V, FAKE, None)

    assert call(n_bias=2 ** 30 + 1) == _lib.SPEC_ERR_SHAPE
    assert call(n_bias=2 ** 31 - 1) == _lib.SPEC_ERR_SHAPE
    assert call(B=2 ** 21, R=1024, V=1) == _lib.SPEC_ERR_SHAPE
    assert lib.spec_kv_commit(FAKE, FAR, 1, 2 ** 40, 1, 1, 2 ** 30 + 1, FAR, 2, FAR, FAR, FAR, FAR, FAR, 2, 3, FAR, FAR,
                              None) == _lib.SPEC_ERR_SHAPE


def test_append_refuses_what_is_no_tensor():
    k = torch.empty(1, 2, 1, 4)
    for v in (None, 3, [1.0]):
        with pytest.raises(ValueError, match="v must be"):
            sv._token_stride(v, "v", torch.float32, k.shape, k.device)


# Every token's warps read their own queries, keys and values: turned queries go
# where no other token still reads, or onto the same token's queries.
@pytest.mark.parametrize("fn,e", [("spec_kv_append_f32", 4), ("spec_kv_append_bf16", 2)])
def test_turned_queries_over_memory_in_use_are_refused(lib, fn, e):
    base, Hq, Hkv, D, B, T = FAR + (1 << 32), 4, 2, 16, 2, 3
    row, n = (Hq + 2 * Hkv) * D, B * T * Hq * D * e
    size = 4 * 16 * Hkv * D * e
    kc, vc = FAR, FAR + size

    def call(q, out_q, k=base + Hq * D * e, v=base + (Hq + Hkv) * D * e, ks=row, qs=row, B=B, T=T):
        return getattr(lib, fn)(k, v, ks, q, qs, out_q, None, None, FAKE, FAKE, B, T, Hq, Hkv, D, D, 0, FAKE, kc, vc, 4, 16,
                                2, None)

    # a joint projection's queries, in place: token 1's answer lies over token 0's keys
    assert call(base, base) == _lib.SPEC_ERR_OVERLAP
    dense = dict(k=base + (1 << 20), v=base + (2 << 20), ks=Hkv * D, qs=Hq * D)
    for d in (-n + 16, -16, 16, n - 16):  # its own buffer, shifted
        assert call(base, base + d, **dense) == _lib.SPEC_ERR_OVERLAP, d
    far = base + (1 << 28)
    assert call(base, base - n + e) == _lib.SPEC_ERR_OVERLAP  # the projection's rows
    for at in (base + Hq * D * e, base + 5 * row * e + (Hq + Hkv) * D * e):
        assert call(far, at, qs=Hq * D) == _lib.SPEC_ERR_OVERLAP
        assert call(base, at) == _lib.SPEC_ERR_OVERLAP
    kv = B * T * Hkv * D * e
    for first in (dense["k"], dense["v"]):
        for at in (first, first - n + 16, first + kv - 16):
            assert call(base, at, **dense) == _lib.SPEC_ERR_OVERLAP
    for at in (kc, kc - n + 16, kc + size - 16, vc, vc + size - 16):
        assert call(base, at) == _lib.SPEC_ERR_OVERLAP
    if not torch.cuda.is_available():  # what is apart goes on to the device, which is not there
        assert call(base, base, **dense) == _lib.SPEC_ERR_CUDA
        assert call(base, base, B=1, T=1) == _lib.SPEC_ERR_CUDA  # one token has no stride
        assert call(base, base - n, **dense) == _lib.SPEC_ERR_CUDA
        assert call(base, base + n, **dense) == _lib.SPEC_ERR_CUDA
        assert call(base, base + 6 * row * e) == _lib.SPEC_ERR_CUDA
        assert call(base, vc + size) == _lib.SPEC_ERR_CUDA
        wide = n // e + row  # between two rows that lie this far apart there is room
        assert call(base, base + row * e, ks=wide, qs=wide) == _lib.SPEC_ERR_CUDA


# Every CTA of a sequence looks up its pages while one writes the answers.
def test_commit_answers_over_the_page_table_are_refused(lib):
    base = FAR + (1 << 32)

    def commit(tab, nodes=FAR + 8192, oln=FAR + 4096, B=2, N=3, mp=5):
        return lib.spec_kv_commit(base, base + (1 << 20), 1, 4 * 16 * 64, 4, 16, 64, tab, mp, FAR, FAR + 256, FAR + 384,
                                  FAR + 128, FAR + 64, B, N, nodes, oln, None)

    for at, n in ((FAR + 8192, 2 * 4 * 4), (FAR + 4096, 2 * 4)):
        for d in (0, 4 - 2 * 5 * 4, n - 4):  # the table's last word, or its first
            assert commit(at + d) == _lib.SPEC_ERR_OVERLAP
    if not torch.cuda.is_available():
        for at, n in ((FAR + 8192, 2 * 4 * 4), (FAR + 4096, 2 * 4)):
            for d in (-2 * 5 * 4, n):
                assert commit(at + d) == _lib.SPEC_ERR_CUDA


def expect(lib, call, where, written):
    """`call(**{name: address})` is refused where an input of n bytes shares its
    first or last word with what is written, and goes on next to it."""
    for name, n in where.items():
        for w, m in written:
            for at in (w, w - n + 4, w + m - 4):
                assert call(**{name: at}) == _lib.SPEC_ERR_OVERLAP, (name, at - w)
    if not torch.cuda.is_available():
        assert call() == _lib.SPEC_ERR_CUDA
        for name, n in where.items():
            for w, m in written:
                for at in (w - n, w + m):
                    assert call(**{name: at}) == _lib.SPEC_ERR_CUDA, (name, at - w)


# What a call writes lies apart from the lists, tables and states that its CTAs read meanwhile.
@pytest.mark.parametrize("e", [4, 2])
@pytest.mark.parametrize("in_place", [False, True])
def test_process_output_over_what_it_reads_is_refused(lib, e, in_place):
    B, R, V, nb, W = 2, 3, 64, 6, 2
    z, out, words = FAR, FAR + (1 << 20), plain_ops.state_words(V)[1]
    if in_place:
        out = z
    f = lib.spec_process_logits_f32 if e == 4 else lib.spec_process_logits_bf16
    other = {n: FAR + (2 << 20) + i * 65536 for i, n in enumerate(("d", "p", "st", "rep", "fr", "pr", "bt", "bv", "mask"))}

    def call(**at):
        x = other | at
        return f(z, x["d"], x["p"], x["st"], x["rep"], x["fr"], x["pr"], nb, x["bt"], x["bv"], x["mask"], R, B, R, V, out, None)

    sizes = dict(d=B * (R - 1) * 4, p=B * (R - 1) * 4, rep=B * 4, fr=B * 4, pr=B * 4, bt=B * nb * 4, bv=B * nb * 4,
                 mask=B * R * W * 4)
    expect(lib, call, sizes, [(out, B * R * V * e)])
    for at in (out, out - B * words * 4 + 16, out + B * R * V * e - 16):  # a state lies on 16 bytes
        assert call(st=at) == _lib.SPEC_ERR_OVERLAP


def test_counted_state_over_what_it_reads_is_refused(lib):
    B, S, V = 2, 5, 64
    n = B * plain_ops.state_words(V)[1] * 4

    def call(tok=FAR, ln=FAR + 65536, pl=FAR + 2 * 65536):
        return lib.spec_count_tokens(tok, ln, pl, B, S, V, 0, FAR + (1 << 20), None)

    expect(lib, call, dict(tok=B * S * 4, ln=B * 4, pl=B * 4), [(FAR + (1 << 20), n)])


@pytest.mark.parametrize("e", [4, 2])
def test_append_writes_over_what_it_reads_are_refused(lib, e):
    B, T, Hq, Hkv, D, pages, page, most = 2, 3, 4, 2, 16, 4, 16, 2
    size, nq = pages * page * Hkv * D * e, B * T * Hq * D * e
    kc, vc, oq = FAR + (4 << 20), FAR + (5 << 20), FAR + (6 << 20)
    f = lib.spec_kv_append_f32 if e == 4 else lib.spec_kv_append_bf16
    other = {n: FAR + i * 65536 for i, n in enumerate(("k", "v", "q", "par", "new", "ln", "tab", "turns"))}

    def call(**at):
        x = other | at
        return f(x["k"], x["v"], Hkv * D, x["q"], Hq * D, oq, x["par"], x["new"], x["ln"], x["tab"], B, T, Hq, Hkv, D, D, 0,
                 x["turns"], kc, vc, pages, page, most, None)

    expect(lib, call, dict(par=B * (T - 1) * 4, new=B * 4, ln=B * 4, tab=B * most * 4, turns=D // 2 * 8),
           [(kc, size), (vc, size), (oq, nq)])
    expect(lib, call, dict(q=nq), [(kc, size), (vc, size)])
    expect(lib, call, dict(k=B * T * Hkv * D * e), [(vc, size)])  # in its own cache a token may lie at its slot
    expect(lib, call, dict(v=B * T * Hkv * D * e), [(kc, size)])
    if not torch.cuda.is_available():
        assert call(k=kc) == _lib.SPEC_ERR_CUDA
        assert call(v=vc) == _lib.SPEC_ERR_CUDA


def test_commit_writes_over_what_it_reads_are_refused(lib):
    B, N, layers, most = 2, 3, 3, 5
    size, step = 4 * 16 * 64, 3 * 4 * 16 * 64
    kc, vc = FAR + (4 << 20), FAR + (4 << 20) + size  # layers by turns, with room between them
    other = {n: FAR + i * 65536 for i, n in enumerate(("tab", "ln", "tok", "par", "path", "plen", "nodes", "oln"))}

    def call(**at):
        x = other | at
        return lib.spec_kv_commit(kc, vc, layers, step, 4, 16, 64, x["tab"], most, x["ln"], x["tok"], x["par"], x["path"],
                                  x["plen"], B, N, x["nodes"], x["oln"], None)

    both = [(kc + l * step, 2 * size) for l in range(layers)]
    expect(lib, call, dict(tab=B * most * 4, ln=B * 4, tok=B * N * 4, par=B * N * 4, path=B * (N + 1) * 4, plen=B * 4,
                           nodes=B * (N + 1) * 4, oln=B * 4), both)


def test_empty_inputs_share_no_memory(lib):
    """A tree without nodes has no tokens, wherever its pointers point."""
    if not torch.cuda.is_available():
        nodes = FAR + 4096
        assert lib.spec_kv_commit(FAR + (1 << 20), FAR + (2 << 20), 1, 4096, 4, 16, 64, FAR, 2, FAR + 64, nodes + 4, nodes + 4,
                                  FAR + 128, FAR + 192, 2, 0, nodes, FAR + 256, None) == _lib.SPEC_ERR_CUDA


class Huge(torch.Tensor):
    """A tensor of any size, without memory, that passes for one on a GPU."""
    is_cuda = True


def huge(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="meta").as_subclass(Huge)


BIG = 2 ** 32 + 8  # 8 in a C int


@pytest.mark.parametrize("call", [
    lambda i, f: sv.spec_process_logits(f(1, 1, BIG)),
    lambda i, f: sv.spec_process_logits(f(1, BIG, 8)),
    lambda i, f: sv.spec_process_logits(f(BIG, 1, 8)),
    lambda i, f: sv.spec_process_logits(f(1, 1, 8), bias_tokens=i(1, BIG), bias_values=f(1, BIG)),
    lambda i, f: sv.spec_count_tokens(i(1, 40), i(1, BIG), 8),
    lambda i, f: sv.spec_count_tokens(i(BIG, 40), i(BIG, 1), 8),
    lambda i, f: sv.spec_kv_append(f(1, 2, 1, 8), f(1, 2, 1, 8), f(BIG, 4, 1, 8), f(BIG, 4, 1, 8), i(1, 2), i(1)),
    lambda i, f: sv.spec_kv_append(f(1, 2, 1, 8), f(1, 2, 1, 8), f(4, BIG, 1, 8), f(4, BIG, 1, 8), i(1, 2), i(1)),
    lambda i, f: sv.spec_kv_append(f(1, 2, 1, 8), f(1, 2, 1, 8), f(4, 4, 1, 8), f(4, 4, 1, 8), i(1, BIG), i(1)),
    lambda i, f: sv.spec_kv_append(f(1, BIG, 1, 8), f(1, BIG, 1, 8), f(4, 4, 1, 8), f(4, 4, 1, 8), i(1, 2), i(1)),
    lambda i, f: sv.spec_kv_append(f(BIG, 1, 1, 8), f(BIG, 1, 1, 8), f(4, 4, 1, 8), f(4, 4, 1, 8), i(BIG, 2), i(BIG)),
    lambda i, f: sv.spec_kv_append(f(1, 2, BIG, 8), f(1, 2, BIG, 8), f(4, 4, BIG, 8), f(4, 4, BIG, 8), i(1, 2), i(1)),
    lambda i, f: sv.spec_kv_append(f(1, 2, 1, BIG), f(1, 2, 1, BIG), f(4, 4, 1, BIG), f(4, 4, 1, BIG), i(1, 2), i(1)),
    lambda i, f: sv.spec_kv_append(f(1, 2, 1, 8), f(1, 2, 1, 8), f(4, 4, 1, 8), f(4, 4, 1, 8), i(1, 2), i(1), q=f(1, 2, BIG, 8)),
    lambda i, f: sv.spec_kv_append(f(1, 2, 1, 8), f(1, 2, 1, 8), f(4, 4, 1, 8), f(4, 4, 1, 8), i(1, 2), i(1),
                                   turns=i(2 ** 31 + 4).to(torch.int64)),
    lambda i, f: sv.spec_kv_commit(f(BIG, 4, 1, 8), f(BIG, 4, 1, 8), i(1, 2), i(1), i(1, 3), i(1, 3), i(1, 4), i(1)),
    lambda i, f: sv.spec_kv_commit(f(4, 4, 1, 8), f(4, 4, 1, 8), i(1, BIG), i(1), i(1, 3), i(1, 3), i(1, 4), i(1)),
    lambda i, f: sv.spec_kv_commit(f(4, 4, 1, 8), f(4, 4, 1, 8), i(1, 2), i(1), i(1, BIG), i(1, BIG), i(1, BIG + 1), i(1)),
    lambda i, f: sv.spec_kv_commit(f(4, 4, 1, 8), f(4, 4, 1, 8), i(BIG, 2), i(BIG), i(BIG, 3), i(BIG, 3), i(BIG, 4), i(BIG)),
    lambda i, f: sv.spec_verify(f(1, 2, BIG), None, i(1, 1), 0.0, 0),
    lambda i, f: sv.spec_verify(f(BIG, 2, 8), f(BIG, 1, 8), i(BIG, 1), 1.0, 0),
    lambda i, f: sv.spec_verify_early_exit(f(1, 2, BIG), f(1, 1, BIG), i(1, 1), 1.0, 0),
    lambda i, f: sv.spec_verify_khint(f(1, 2, 8), f(1, 1, 8), i(1, 1), 1.0, 0, 0.5, 1.0, 2 ** 32, 4),
    lambda i, f: sv.spec_verify_khint(f(1, 2, 8), f(1, 1, 8), i(1, 1), 1.0, 0, 0.5, 1.0, 1, 2 ** 32 + 4),
    lambda i, f: sv.spec_verify_greedy_argmax(f(1, 2, BIG), i(1, 1)),
    lambda i, f: sv.spec_tree_verify_greedy(f(1, 2, BIG), i(1, 1), i(1, 1)),
    lambda i, f: sv.spec_tree_verify_sampling(f(1, 2, BIG), f(1, 2, BIG), i(1, 1), i(1, 1), 1.0, 0),
    lambda i, f: sv.spec_acceptance_stats(i(BIG), 4),
    lambda i, f: sv.spec_acceptance_stats(i(2), -2 ** 32 + 4),
    lambda i, f: sv.spec_ngram_draft(i(2, BIG), i(2), 1, 4, 8),
    lambda i, f: sv.spec_ngram_draft(i(BIG, 9), i(BIG), 1, 4, 8),
    lambda i, f: sv.spec_ngram_draft(i(2, 9), i(2), 2 ** 32 + 1, 4, 8),
    lambda i, f: sv.spec_ngram_draft(i(2, 9), i(2), 1, 2 ** 32 + 4, 8),
    lambda i, f: sv.spec_ngram_draft(i(2, 9), i(2), 1, 4, -2 ** 32 + 8),
])
def test_binding_refuses_sizes_past_a_c_int(lib, call):
    with pytest.raises(sv.SpecError) as e:
        call(huge, lambda *s: huge(*s, dtype=torch.bfloat16))
    assert e.value.code == _lib.SPEC_ERR_SHAPE


def test_one_token_has_no_stride(lib, monkeypatch):
    """Keys from a joint projection and values of their own: with one token
    there is no distance between tokens that they could differ in."""
    calls = []
    monkeypatch.setattr(sv, "_invoke", lambda fn, device, stream, *args: calls.append(args))
    i, f = huge, lambda *s: huge(*s, dtype=torch.bfloat16)

    def call(B, T, k, v):
        sv.spec_kv_append(k, v, f(4, 4, 2, 8), f(4, 4, 2, 8), i(B, 2), i(B))
        return calls.pop()[2]

    joint, own = f(1, 1, 6, 8), f(1, 1, 2, 8)
    assert joint[:, :, :2].stride() != own.stride()
    for k, v in ((joint[:, :, :2], own), (own, joint[:, :, 4:]), (joint[:, :, :2], joint[:, :, 2:4]), (own, own)):
        assert call(1, 1, k, v) >= 16  # the C entry point wants room for a token
    assert call(2, 1, f(2, 1, 6, 8)[:, :, :2], f(2, 1, 6, 8)[:, :, 2:4]) == 48
    for B, T in ((2, 1), (1, 2)):
        with pytest.raises(ValueError, match="share a token stride"):
            call(B, T, f(B, T, 6, 8)[:, :, :2], f(B, T, 2, 8))
