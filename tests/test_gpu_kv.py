"""The paged cache's append (with rotation) and a tree's commit on the GPU
against a plain 64-bit implementation.

Tolerance of a turned value: the angle's fraction is cut to 32 bits and rounded
to fp32 (at most pi 2^-25 + pi 2^-31 radians), sin and cos are within 2 ulp of
values up to 1 (2^-23 each), and three fp32 operations follow (two products, of
which one may be fused, and a sum): (pi 2^-25 + pi 2^-31 + 2^-23 + 3 * 2^-24) of
|x0| + |x1|; a bf16 result adds half a step, 2^-8 of itself."""
import math

import numpy as np
import pytest
import torch

import plain_ops
import speculative_decoding_verification_36_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
ANGLE = math.pi * 2.0 ** -25 + math.pi * 2.0 ** -31 + 2.0 ** -23 + 3 * 2.0 ** -24


def dev(x):
    return None if x is None else torch.as_tensor(np.ascontiguousarray(x)).to(DEV)


def make(rng, B, T, Hq, Hkv, D, rot, dtype, page, ctx, tree=False, ragged=False, joint=True):
    t = lambda *s: torch.from_numpy(rng.normal(0, 1, s).astype(np.float32)).to(dtype)  # noqa: E731
    lengths = rng.integers(0, ctx + 1, B).astype(np.int32)
    span = (T + page - 1) // page + 1
    most = ctx // page + span + 1
    pages = B * span + 2
    table = np.full((B, most), 0, np.int32)
    order = rng.permutation(pages - 2).astype(np.int32) + 1
    for b in range(B):
        f = lengths[b] // page
        table[b, f:f + span] = order[b * span:(b + 1) * span]
    x = dict(lengths=lengths, table=table, pages=pages, page=page, parents=None, n_new=None, dtype=dtype, q=None,
             inv=[10000.0 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)])
    if joint:
        qkv = t(B, T, Hq + 2 * Hkv, D).to(DEV)
        x["q"] = qkv[:, :, :Hq] if Hq else None
        x["k"], x["v"] = qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    else:
        x["q"] = t(B, T, Hq, D).to(DEV) if Hq else None
        x["k"], x["v"] = t(B, T, Hkv, D).to(DEV), t(B, T, Hkv, D).to(DEV)
    x["kc"], x["vc"] = t(pages, page, Hkv, D).to(DEV), t(pages, page, Hkv, D).to(DEV)
    if tree:
        x["parents"] = np.stack([[int(rng.integers(-1, j)) if j else -1 for j in range(T - 1)] for _ in range(B)]).reshape(
            B, T - 1).astype(np.int32)
    if ragged:
        x["n_new"] = rng.integers(0, T + 1, B).astype(np.int32)
    return x


def run_and_check(x, interleaved=False, in_place_q=False):
    turns = sv.spec_rope_turns(x["inv"], DEV) if x["inv"] else None
    n = lambda v: None if v is None else v.cpu().double().numpy()  # noqa: E731
    out_q = None
    if x["q"] is not None:
        out_q = x["q"].contiguous() if in_place_q else torch.full(x["q"].shape, 3.0, dtype=x["dtype"], device=DEV)
    tv = [] if turns is None else [int(v) for v in turns.cpu()]
    kc, vc, oq, km, qm = plain_ops.append(n(x["k"]), n(x["v"]), n(x["kc"]), n(x["vc"]), x["table"], x["lengths"], tv,
                                          q=n(x["q"]), out_q=n(out_q), parents=x["parents"], n_new=x["n_new"],
                                          interleaved=interleaved)
    got = sv.spec_kv_append(x["k"], x["v"], x["kc"], x["vc"], dev(x["table"]), dev(x["lengths"]), turns=turns,
                            q=out_q if in_place_q else x["q"], parent_idx=dev(x["parents"]), n_new=dev(x["n_new"]),
                            interleaved=interleaved, out_q=out_q)
    half = 2.0 ** -8 if x["dtype"] == torch.bfloat16 else 0.0

    def near(a, ref, mag):
        a = n(a)
        np.testing.assert_array_equal(np.isnan(a), np.isnan(ref))
        ok = ~np.isnan(ref)
        tol = ANGLE * mag[ok]
        tol = tol + half * (np.abs(ref[ok]) + tol) * (mag[ok] > 0)
        assert (np.abs(a[ok] - ref[ok]) <= tol).all(), (np.abs(a[ok] - ref[ok]) - tol).max()

    near(x["kc"], kc, km)
    np.testing.assert_array_equal(n(x["vc"]), vc)
    if x["q"] is not None:
        near(got, oq, qm)
    return got


APPENDS = [
    # B, T, Hq, Hkv, D, rot, dtype, page, ctx, tree, ragged, joint
    (1, 1, 0, 1, 1, 0, torch.float32, 1, 0, False, False, False),
    (1, 1, 2, 1, 2, 2, torch.float32, 1, 5, False, False, True),
    (1, 5, 32, 8, 128, 128, torch.bfloat16, 16, 2000, False, False, True),
    (3, 9, 4, 2, 64, 64, torch.bfloat16, 16, 40, False, False, True),
    (3, 9, 0, 2, 64, 32, torch.float32, 24, 100, False, True, False),
    (4, 70, 4, 4, 80, 80, torch.bfloat16, 16, 50, False, True, True),    # half of 80: pairs off the vectors
    (4, 7, 4, 4, 96, 48, torch.float32, 7, 50, True, False, True),
    (2, 31, 8, 1, 256, 256, torch.bfloat16, 64, 1000, True, False, True),
    (2, 5, 3, 3, 7, 6, torch.bfloat16, 3, 9, False, False, True),
    (2, 5, 1, 1, 1024, 1024, torch.float32, 16, 9, False, False, False),
    (2, 130, 2, 2, 64, 64, torch.bfloat16, 1, 1000, True, False, True),
    (5, 33, 2, 2, 16, 8, torch.bfloat16, 16, 1000000, False, True, True),  # far positions
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,dtype,page,ctx,tree,ragged,joint", APPENDS)
def test_append_matches_plain(B, T, Hq, Hkv, D, rot, dtype, page, ctx, tree, ragged, joint, interleaved):
    rng = np.random.default_rng(B * 100 + T + D)
    x = make(rng, B, T, Hq, Hkv, D, rot, dtype, page, ctx, tree, ragged, joint)
    run_and_check(x, interleaved)
    assert sv.spec_get_status() == 0


def test_queries_in_place():
    rng = np.random.default_rng(2)
    x = make(rng, 2, 6, 4, 2, 64, 64, torch.bfloat16, 16, 30, joint=False)
    run_and_check(x, in_place_q=True)
    x = make(rng, 2, 6, 4, 2, 64, 32, torch.float32, 16, 30, joint=False)
    run_and_check(x, interleaved=True, in_place_q=True)


def test_last_positions():
    """Positions next to 2^31: the fraction of a turn is still exact."""
    rng = np.random.default_rng(3)
    x = make(rng, 2, 4, 2, 2, 64, 64, torch.float32, 1 << 20, 10, joint=False)
    far = 2 ** 31 - 8
    x["lengths"][:] = [far, far - 1]
    x["table"] = np.zeros((2, 2 ** 11), np.int32)
    x["table"][:, -1] = [0, 1]
    x["pages"] = 2
    x["kc"], x["vc"] = (torch.zeros((2, 1 << 20, 2, 64), device=DEV) for _ in range(2))
    turns = sv.spec_rope_turns(x["inv"], DEV)
    q = sv.spec_kv_append(x["k"], x["v"], x["kc"], x["vc"], dev(x["table"]), dev(x["lengths"]), turns=turns, q=x["q"])
    tv = [int(v) for v in turns.cpu()]
    for b in range(2):
        for i in range(4):
            pos = int(x["lengths"][b]) + i
            for got, src in ((x["kc"][b, pos % (1 << 20)], x["k"][b, i]), (q[b, i], x["q"][b, i])):
                ref, mag = plain_ops.rotate(src.cpu().double().numpy(), pos, tv, False)
                assert (np.abs(got.cpu().double().numpy() - ref) <= ANGLE * mag).all()
    assert sv.spec_get_status() == 0


def test_cache_past_32_bit_offsets():
    """A cache of over 2^32 bytes and 2^31 elements: its last page is written."""
    rng = np.random.default_rng(4)
    Hkv, D, page = 8, 128, 64
    pages = 2 ** 31 // (Hkv * D * page) + 3
    kc, vc = (torch.empty((pages, page, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    x = make(rng, 1, 3, 0, Hkv, D, D, torch.bfloat16, page, 0, joint=False)
    table = dev(np.array([[pages - 1]], np.int32))
    kc[pages - 1].zero_(), vc[pages - 1].zero_()
    sv.spec_kv_append(x["k"], x["v"], kc, vc, table, dev(np.array([5], np.int32)),
                      turns=sv.spec_rope_turns(x["inv"], DEV))
    assert torch.equal(vc[pages - 1, 5:8], x["v"][0])
    assert bool((vc[pages - 1, :5] == 0).all()) and bool((vc[pages - 1, 8:] == 0).all())
    # and a commit there: node 1 (slot 7) under node 0 rejected, moved to slot 6
    tok, par = dev(np.array([[4, 9]], np.int32)), dev(np.array([[-1, -1]], np.int32))
    sv.spec_kv_commit(kc, vc, table, dev(np.array([5], np.int32)), tok, par, dev(np.array([[9, 3, -1]], np.int32)),
                      dev(np.array([2], np.int32)))
    assert torch.equal(vc[pages - 1, 6], x["v"][0, 2])
    assert sv.spec_get_status() == 0


def test_append_bad_data_is_left_out():
    rng = np.random.default_rng(5)
    for what in ("length", "past", "n_new", "n_new_neg", "page", "page_big", "parent"):
        x = make(rng, 3, 6, 2, 2, 64, 64, torch.bfloat16, 4, 20, tree=what == "parent", ragged=what.startswith("n_new"))
        if what == "length":
            x["lengths"][1] = -1
        elif what == "past":
            x["lengths"][1] = x["table"].shape[1] * 4 - 5
        elif what == "n_new":
            x["n_new"][1] = 7
        elif what == "n_new_neg":
            x["n_new"][1] = -1
        elif what == "page":
            x["table"][1, (x["lengths"][1] + 3) // 4] = -1
        elif what == "page_big":
            x["table"][1, (x["lengths"][1] + 3) // 4] = x["pages"]
        else:
            x["parents"][1, 2] = 2
        got = run_and_check(x)
        if not what.startswith("page"):
            assert bool(torch.isnan(got[1].float()).all())
        assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA, what


def test_empty_steps():
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    kc = torch.full((3, 4, 2, 16), 5.0, device=DEV)
    for B, T in ((0, 3), (2, 0), (0, 0)):
        k = torch.zeros((B, T, 2, 16), device=DEV)
        q = sv.spec_kv_append(k, k, kc, kc.clone(), i(B, 2), i(B), turns=sv.spec_rope_turns([0.5] * 8, DEV), q=k)
        assert q.shape == (B, T, 2, 16)
    assert bool((kc == 5).all())
    nodes, new = sv.spec_kv_commit(kc, kc.clone(), i(0, 2), i(0), i(0, 3), i(0, 3), i(0, 4), i(0))
    assert nodes.shape == (0, 4) and new.shape == (0,)
    assert sv.spec_get_status() == 0


def test_products_depend_on_the_distance():
    """The rotation preserves lengths and angles between equal positions: the
    product of a turned query and key depends on their distance alone."""
    D, far = 64, 1000003
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k = (torch.randn((1, 1, 1, D), generator=g, device=DEV) for _ in range(2))
    turns = sv.spec_rope_turns([10000.0 ** (-2 * i / D) for i in range(D // 2)], DEV)
    kc, vc = (torch.zeros((1, 16, 1, D), device=DEV) for _ in range(2))
    table = torch.zeros((1, 1 << 17), dtype=torch.int32, device=DEV)

    def turned(x, pos):
        at = torch.tensor([pos], dtype=torch.int32, device=DEV)
        return sv.spec_kv_append(k, k, kc, vc, table, at, turns=turns, q=x)[0, 0, 0].double()

    for gap in (0, 1, 37):
        near, away = (float(turned(q, p + gap) @ turned(k, p)) for p in (5, far))
        # 2 D products of values off by ANGLE of |x0| + |x1| each
        bound = 4 * ANGLE * float(q.abs().sum() * k.abs().max() + k.abs().sum() * q.abs().max())
        assert abs(near - away) <= bound


def test_append_refusals():
    rng = np.random.default_rng(6)
    x = make(rng, 2, 3, 2, 2, 16, 16, torch.float32, 4, 8, joint=False)
    tab, ln, turns = dev(x["table"]), dev(x["lengths"]), sv.spec_rope_turns(x["inv"], DEV)

    def call(k=x["k"], v=x["v"], kc=x["kc"], vc=x["vc"], tab=tab, ln=ln, **kw):
        sv.spec_kv_append(k, v, kc, vc, tab, ln, **kw)

    call(turns=turns)
    for kw in (dict(k=x["k"].half()), dict(v=x["v"].to(torch.bfloat16)), dict(v=x["v"][:, :, :1]),
               dict(k=x["k"].transpose(1, 2)), dict(kc=x["kc"][:, :, :1]), dict(vc=x["vc"][:-1]), dict(tab=tab.long()),
               dict(ln=ln[:1]), dict(turns=turns.float()), dict(q=x["q"][:, :2]), dict(out_q=x["q"]),
               dict(parent_idx=ln), dict(n_new=tab)):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    with pytest.raises(sv.SpecError):  # more frequencies than a head has pairs
        call(turns=sv.spec_rope_turns([0.1] * 9, DEV))


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
def random_tree(rng, B, N, kind):
    if kind == "chain":
        return np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))
    lo = (lambda j: -1) if kind == "any" else (lambda j: max(-1, j - 3))
    return np.stack([[int(rng.integers(lo(j), j)) if j else -1 for j in range(N)] for _ in range(B)]).reshape(B, N).astype(np.int32)


def make_commit(rng, B, N, layers, page, dtype, H, D, kind="any", alphabet=4):
    parents = random_tree(rng, B, N, kind)
    tokens = rng.integers(0, alphabet, (B, N)).astype(np.int32)
    path = np.full((B, N + 1), -1, np.int32)
    plen = np.zeros(B, np.int32)
    for b in range(B):
        node, toks = int(rng.integers(-1, N)), []
        j = node
        while j >= 0:
            toks.insert(0, int(tokens[b, j]))
            j = int(parents[b, j])
        path[b, :len(toks)] = toks
        path[b, len(toks)] = 77
        plen[b] = len(toks) + 1
    lengths = rng.integers(0, 50, B).astype(np.int32)
    span = (N + 1 + page - 1) // page + 1
    most = 50 // page + span + 1
    pages = B * most
    table = rng.permutation(pages).astype(np.int32).reshape(B, most)
    if dtype == torch.uint8:
        caches = [torch.from_numpy(rng.integers(0, 256, (layers, pages, page, H, D), dtype=np.uint8)) for _ in range(2)]
    else:
        caches = [torch.from_numpy(rng.normal(size=(layers, pages, page, H, D)).astype(np.float32)).to(dtype) for _ in range(2)]
    return dict(parents=parents, tokens=tokens, path=path, plen=plen, lengths=lengths, table=table, caches=caches)


def commit_and_check(x, layered=True):
    raw = {torch.uint8: torch.uint8, torch.bfloat16: torch.int16, torch.float32: torch.int32}[x["caches"][0].dtype]
    ref, nodes, new = plain_ops.commit([c.view(raw).numpy() for c in x["caches"]], x["table"], x["lengths"], x["tokens"],
                                       x["parents"], x["path"], x["plen"])
    k, v = (c.to(DEV) for c in x["caches"])
    args = (dev(x["table"]), dev(x["lengths"]), dev(x["tokens"]), dev(x["parents"]), dev(x["path"]), dev(x["plen"]))
    if layered:
        gn, gl = sv.spec_kv_commit(k, v, *args)
    else:
        for layer in range(k.shape[0]):
            gn, gl = sv.spec_kv_commit(k[layer], v[layer], *args)
    np.testing.assert_array_equal(gn.cpu().numpy(), nodes)
    np.testing.assert_array_equal(gl.cpu().numpy(), new)
    for g, r in zip((k, v), ref):
        np.testing.assert_array_equal(g.view(raw).cpu().numpy(), r)


@pytest.mark.parametrize("B,N,layers,page,dtype,H,D,kind", [
    (1, 1, 1, 1, torch.float32, 1, 1, "any"),
    (4, 0, 2, 4, torch.bfloat16, 2, 8, "any"),
    (6, 14, 2, 4, torch.bfloat16, 2, 64, "any"),
    (5, 30, 3, 16, torch.bfloat16, 8, 128, "deep"),
    (4, 40, 2, 7, torch.float32, 2, 6, "chain"),     # every entry is where it belongs
    (5, 33, 2, 3, torch.uint8, 3, 5, "deep"),        # 15-byte entries
    (3, 200, 1, 16, torch.float32, 1, 16, "deep"),   # long paths that move over each other
    (2, 1024, 1, 64, torch.bfloat16, 1, 64, "deep"),
])
def test_commit_matches_plain(B, N, layers, page, dtype, H, D, kind):
    rng = np.random.default_rng(B * 10 + N)
    x = make_commit(rng, B, N, layers, page, dtype, H, D, kind)
    commit_and_check(x)
    commit_and_check(x, layered=False)
    assert sv.spec_get_status() == 0


def test_commit_bad_data_is_left():
    rng = np.random.default_rng(7)
    for what in ("verify", "len", "len0", "path", "parent", "past", "page", "length"):
        x = make_commit(rng, 3, 12, 2, 4, torch.bfloat16, 2, 16, "deep")
        x["path"][1], x["plen"][1] = -1, 3
        x["path"][1, 0] = x["tokens"][1, 0]
        kids = [j for j in range(12) if x["parents"][1, j] == 0]
        x["parents"][1, 1] = 0
        x["path"][1, 1] = x["tokens"][1, 1]
        assert kids is not None
        if what == "verify":
            x["plen"][1] = -1
        elif what == "len":
            x["plen"][1] = 14
        elif what == "len0":
            x["plen"][1] = 0
        elif what == "path":
            x["path"][1, 1] = 1000
        elif what == "parent":
            x["parents"][1, 11] = 11
        elif what == "past":
            x["lengths"][1] = x["table"].shape[1] * 4 - 12
        elif what == "page":
            x["table"][1, (x["lengths"][1] + 1) // 4] = -1
        else:
            x["lengths"][1] = -3
        commit_and_check(x)
        assert sv.spec_get_status() == (0 if what == "verify" else sv.SPEC_FLAG_BAD_DATA), what


def test_tree_step_in_a_graph():
    """Append of a tree, greedy verify, commit: captured once, replayed on new
    data, equal to the eager calls and to the entries that a chain of the
    accepted tokens would have written."""
    rng = np.random.default_rng(8)
    B, N, V, Hkv, D, page, layers = 4, 14, 400, 2, 64, 8, 2
    par_row = np.array([i // 2 - 1 for i in range(N)], np.int32)
    parents = dev(np.tile(par_row, (B, 1)))
    lengths = dev(rng.integers(0, 60, B).astype(np.int32))
    most = 60 // page + 4
    table = dev(rng.permutation(B * most).astype(np.int32).reshape(B, most))
    k, v = (torch.randn((layers, B, N + 1, Hkv, D), device=DEV, dtype=torch.float32).to(torch.bfloat16) for _ in range(2))
    kc, vc = (torch.zeros((layers, B * most, page, Hkv, D), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    turns = sv.spec_rope_turns([10000.0 ** (-2 * i / D) for i in range(D // 2)], DEV)
    z = torch.empty((B, N + 1, V), device=DEV)
    tokens = torch.empty((B, N), dtype=torch.int32, device=DEV)
    path, plen = torch.empty((B, N + 1), dtype=torch.int32, device=DEV), torch.empty((B,), dtype=torch.int32, device=DEV)
    mask = torch.empty((B, N, 1), dtype=torch.int32, device=DEV)
    nodes, new = torch.empty((B, N + 1), dtype=torch.int32, device=DEV), torch.empty((B,), dtype=torch.int32, device=DEV)

    def fresh(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        z.copy_(torch.randn(z.shape, generator=g, device=DEV))
        for j in range(N):  # the second child carries the argmax most of the time
            best = z[:, par_row[j] + 1].argmax(-1).int()
            other = torch.randint(0, V, (B,), generator=g, device=DEV, dtype=torch.int32)
            good = torch.rand((B,), generator=g, device=DEV) < (0.85 if j % 2 else 0.0)
            tokens[:, j] = torch.where(good, best, other)
        k.copy_(torch.randn(k.shape, generator=g, device=DEV))
        v.copy_(torch.randn(v.shape, generator=g, device=DEV))

    def step():
        for i in range(layers):
            sv.spec_kv_append(k[i], v[i], kc[i], vc[i], table, lengths, turns=turns, parent_idx=parents)
        sv.spec_tree_verify_greedy(z, tokens, parents, out_path=path, out_len=plen, out_mask=mask)
        sv.spec_kv_commit(kc, vc, table, lengths, tokens, parents, path, plen, out_nodes=nodes, out_lengths=new)

    fresh(0)
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    moved = 0
    for seed in range(1, 5):
        fresh(seed)
        kc.zero_(), vc.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (kc, vc, nodes, new)]
        kc.zero_(), vc.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (kc, vc, nodes, new)):
            assert torch.equal(a, b)
        # a chain of the accepted tokens' keys and values
        kk, vv = torch.zeros_like(kc), torch.zeros_like(vc)
        for b in range(B):
            n = int(plen[b]) - 1
            pick = torch.tensor([0] + [int(c) + 1 for c in nodes[b, :n]], device=DEV)
            moved += n
            for i in range(layers):
                sv.spec_kv_append(k[i, b:b + 1].index_select(1, pick), v[i, b:b + 1].index_select(1, pick), kk[i], vv[i],
                                  table[b:b + 1], lengths[b:b + 1], turns=turns)
            for s in range(int(lengths[b]), int(new[b])):
                at = (slice(None), int(table[b, s // page]), s % page)
                assert torch.equal(kc[at], kk[at]) and torch.equal(vc[at], vv[at])
    assert moved > 8
    assert sv.spec_get_status() == 0


def test_appends_on_two_streams():
    rng = np.random.default_rng(9)
    xs = [make(rng, 4, 50, 4, 2, 128, 128, torch.bfloat16, 16, 100, joint=False) for _ in range(2)]
    turns = sv.spec_rope_turns(xs[0]["inv"], DEV)
    args = [(x["k"], x["v"], dev(x["table"]), dev(x["lengths"])) for x in xs]
    start = [(x["kc"].clone(), x["vc"].clone()) for x in xs]
    alone = []
    for x, (k, v, tab, ln) in zip(xs, args):
        q = sv.spec_kv_append(k, v, x["kc"], x["vc"], tab, ln, turns=turns, q=x["q"])
        alone.append((q, x["kc"].clone(), x["vc"].clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for x, (a, b) in zip(xs, start):
            x["kc"].copy_(a), x["vc"].copy_(b)
        torch.cuda.synchronize()
        qs = [None, None]
        for i, (x, (k, v, tab, ln)) in enumerate(zip(xs, args)):
            with torch.cuda.stream(streams[i]):
                qs[i] = sv.spec_kv_append(k, v, x["kc"], x["vc"], tab, ln, turns=turns, q=x["q"])
        torch.cuda.synchronize()
        for x, q, (a, b, c) in zip(xs, qs, alone):
            assert torch.equal(q, a) and torch.equal(x["kc"], b) and torch.equal(x["vc"], c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_keys_and_values_at_their_own_slots(dtype, interleaved):
    """A projection that wrote into consecutive pages is turned where it lies."""
    rng = np.random.default_rng(11)
    T, H, D, page, length = 37, 3, 32, 8, 13
    x = make(rng, 1, T, 0, H, D, 24, dtype, page, 0, joint=False)
    x["lengths"][:] = length
    x["table"] = np.arange(7, dtype=np.int32)[None]
    x["kc"], x["vc"] = (torch.randn((7, page, H, D), device=DEV).to(dtype) for _ in range(2))
    x["k"], x["v"] = (x[c].view(1, -1, H, D)[:, length:length + T] for c in ("kc", "vc"))
    run_and_check(x, interleaved)
    assert sv.spec_get_status() == 0


def test_one_token_from_two_projections():
    rng = np.random.default_rng(12)
    x = make(rng, 1, 1, 4, 2, 64, 64, torch.bfloat16, 16, 30)
    x["v"] = x["v"].clone(memory_format=torch.contiguous_format)
    assert x["v"].stride() != x["k"].stride()
    run_and_check(x)
    x = make(rng, 1, 1, 4, 2, 64, 64, torch.bfloat16, 16, 30)
    x["k"] = x["k"].clone(memory_format=torch.contiguous_format)
    run_and_check(x, interleaved=True)
    # and a joint projection's queries turned where they lie: one token
    x = make(rng, 1, 1, 4, 2, 64, 64, torch.float32, 16, 30)
    want = sv.spec_kv_append(x["k"], x["v"], x["kc"].clone(), x["vc"].clone(), dev(x["table"]), dev(x["lengths"]),
                             turns=sv.spec_rope_turns(x["inv"], DEV), q=x["q"])
    got = sv.spec_kv_append(x["k"], x["v"], x["kc"], x["vc"], dev(x["table"]), dev(x["lengths"]),
                            turns=sv.spec_rope_turns(x["inv"], DEV), q=x["q"], out_q=x["q"])
    assert got is x["q"] and torch.equal(got, want)
    assert sv.spec_get_status() == 0


def test_queries_of_a_joint_projection_in_place_are_refused():
    rng = np.random.default_rng(13)
    x = make(rng, 1, 4, 2, 1, 64, 64, torch.float32, 16, 30, joint=False)
    whole = torch.zeros((1, 16, 2, 64), device=DEV)
    q = whole[:, ::4]  # four tokens of every fourth row
    with pytest.raises(sv.SpecError) as e:  # its answer, next to each other, would lie over later tokens' queries
        sv.spec_kv_append(x["k"], x["v"], x["kc"], x["vc"], dev(x["table"]), dev(x["lengths"]),
                          turns=sv.spec_rope_turns(x["inv"], DEV), q=q, out_q=whole[:, :4])
    assert e.value.code == sv._lib.SPEC_ERR_OVERLAP
