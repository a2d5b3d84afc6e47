"""The operators around a verify step, as they are measured: token counts, logit
processing (penalties, biases, masks), and the paged key/value cache's append and
commit for drafted chains and trees.

`run` computes them in plain torch operations, or, where `own` is true, by the
package's entry points.  Both take the same state.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _process(name, B, R, V, dtype, hist, bias, mask, tree, in_place=False):
    """mask: "none", "rows" (one mask a row) or "shared" (one a sequence); tree: a
    complete binary tree of R - 1 nodes in breadth-first order, else a chain."""
    c = dict(op="process", B=B, R=R, V=V, dtype=dtype, hist=hist, bias=bias, mask=mask, tree=tree, in_place=in_place)
    return dict(c, name=name) if name else c


def _count(name, B, V, hist):
    c = dict(op="count", B=B, V=V, hist=hist)
    return dict(c, name=name) if name else c


def _append(name, B, T, Hq, Hkv, D, rot, dtype, page, ctx, tree, interleaved, ragged):
    c = dict(op="append", B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, dtype=dtype, page=page, ctx=ctx, tree=tree,
             interleaved=interleaved, ragged=ragged)
    return dict(c, name=name) if name else c


def _step(name, layers, B, N, Hkv, D, dtype, page, ctx):
    c = dict(op="step", layers=layers, B=B, N=N, Hkv=Hkv, D=D, rot=D, dtype=dtype, page=page, ctx=ctx)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's chat turn: 4 drafts, a short history, a few biased tokens, fp32 logits; latency is all
        _process("process one sequence", 1, 5, 32000, "f32", 512, 16, "none", False),
        # a serving batch with penalties and OpenAI-style biases, no grammar
        _process("process chain batch", 64, 6, 128256, "bf16", 4096, 64, "none", False),
        # the largest batch, every feature on: long histories, 300 biases, a grammar's mask for every row
        _process("process chain, all on", 256, 9, 152064, "bf16", 8192, 300, "rows", False),
        # structured output alone: only masks, applied where the logits lie
        _process("mask in place", 256, 5, 128256, "bf16", 0, 0, "rows", False, True),
        # a candidate tree of 30 nodes, whose rows see different paths
        _process("process tree", 32, 31, 128256, "bf16", 2048, 32, "rows", True),
        # a vocabulary that no vector width divides; one banned-words mask a sequence
        _process("process odd vocabulary", 24, 4, 96001, "bf16", 1500, 20, "shared", False),
        # a batch's prompts and outputs so far are admitted
        _count("count batch", 256, 152064, 8192),
        # one long document
        _count("count long history", 1, 128256, 131072),
        # one user's chain of 4 drafts: a launch's latency
        _append("append one chain", 1, 5, 32, 8, 128, 128, "bf16", 16, 2048, False, False, False),
        # prompts of very different lengths, in one padded batch, far into the context
        _append("append ragged prompts", 8, 4096, 32, 8, 128, 128, "bf16", 64, 100000, False, False, True),
        # a tree step on a small model: the tree's entries go in, the accepted path's stay
        _step("tree step", 2, 32, 30, 8, 128, "bf16", 16, 1024),
        # a large batch of larger trees, more layers
        _step("tree step, large", 4, 128, 62, 8, 128, "bf16", 64, 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["process", "process", "process", "count", "append", "step"])
    if op == "process":
        V = _log(rng, 1000, 160000)
        if rng.random() < 0.5:
            V = V // 8 * 8
        tree = rng.random() < 0.3
        R = 2 ** rng.randint(2, 5) - 1 if tree else rng.randint(1, 12)
        B = max(1, min(_log(rng, 1, 256), 200_000_000 // (R * V)))
        if rng.random() < 0.2:
            return _process("", B, R, V, rng.choice(["f32", "bf16", "bf16"]), 0, 0, rng.choice(["rows", "shared"]), tree, True)
        return _process("", B, R, V, rng.choice(["f32", "bf16", "bf16"]), _log(rng, 1, 8192), rng.choice([0, _log(rng, 1, 500)]),
                        rng.choice(["none", "rows", "shared"]), tree)
    if op == "count":
        V = _log(rng, 1000, 160000)
        return _count("", _log(rng, 1, 200), V, _log(rng, 1, 16384))
    D = rng.choice([64, 80, 96, 128, 256])
    if op == "append":
        tree = rng.random() < 0.3
        T = 2 ** rng.randint(2, 6) - 1 if tree else _log(rng, 1, 2048)
        B = max(1, min(_log(rng, 1, 256), 16384 // T))
        Hkv = rng.choice([1, 2, 4, 8])
        return _append("", B, T, rng.choice([0, Hkv, 4 * Hkv]), Hkv, D, rng.choice([D, D // 2]), rng.choice(["f32", "bf16", "bf16"]),
                       rng.choice([1, 16, 24, 64]), _log(rng, 1, 1000000), tree, rng.random() < 0.3, not tree and rng.random() < 0.5)
    return _step("", rng.randint(1, 3), _log(rng, 1, 64), 2 ** rng.randint(2, 6) - 2, rng.choice([1, 2, 4, 8]), D,
                 rng.choice(["f32", "bf16", "bf16"]), rng.choice([16, 24, 64]), _log(rng, 1, 100000))


# Grammar masks differ widely from state to state: a quarter of the sequences has no
# grammar, and a row of the others allows one of these shares of the vocabulary.
SHARES = (0.002, 0.1, 0.95)
FREE = 0.25


def _touched(case):
    """About how many tokens of a sequence have a count or a bias."""
    V = case["V"]
    return min(V, int(0.75 * case["hist"])) + case["bias"]


def work(case):
    if case["op"] == "process":
        B, R, V, e = case["B"], case["R"], case["V"], ESIZE[case["dtype"]]
        masks = {"none": 0, "rows": B * R, "shared": B}[case["mask"]]
        small = masks * ((V + 31) // 32) * 4 + (4 * case["B"] * _touched(case) + B * V // 8 if case["hist"] else 0) + 8 * B * case["bias"]
        if case["in_place"]:
            off = (1 - FREE) * (1 - sum(SHARES) / len(SHARES))
            return {"bytes": small + off * B * R * V * e, "flops": B * R * V}
        return {"bytes": small + 2 * B * R * V * e, "flops": B * R * V}
    if case["op"] == "count":
        B, V = case["B"], case["V"]
        return {"bytes": B * (0.75 * case["hist"] * 4 + _words(V) * 4), "flops": B * 0.75 * case["hist"]}
    e = ESIZE[case["dtype"]]
    if case["op"] == "append":
        tokens = case["B"] * case["T"] * (0.55 if case["ragged"] else 1.0)
        n = tokens * case["D"] * (2 * case["Hkv"] + case["Hq"])
        return {"bytes": 2 * n * e, "flops": 3 * tokens * case["rot"] * (case["Hkv"] + case["Hq"])}
    each = case["layers"] * case["B"] * 2 * case["Hkv"] * case["D"] * e
    depth = (case["N"] + 2).bit_length() - 2
    return {"bytes": 2 * each * (case["N"] + 1) + 2 * each * depth / 2, "flops": 3 * case["layers"] * case["B"] * (case["N"] + 1) * case["rot"] * case["Hkv"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
DEV = "cuda"


def _words(V):
    """int32 words of one sequence's token state: V counts, rounded up to 32, then a
    bitmap of the non-zero ones, rounded up to 4 words."""
    P = (V + 31) // 32 * 32
    return P + (P // 32 + 3) // 4 * 4


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(7919 * (int(seed) + 1))
    return g


def _tokens(g, shape, V):
    """Half of the tokens by a law that repeats the frequent ones, half over the whole vocabulary."""
    u = torch.rand(shape, generator=g, device=DEV, dtype=torch.float64)
    often = torch.rand(shape, generator=g, device=DEV) < 0.5
    v = torch.where(often, torch.exp(u * math.log(V)) - 1, u * V)
    return v.to(torch.int64).clamp_(0, V - 1).to(torch.int32)


def _lengths(g, B, most):
    lo = (most + 1) // 2
    return torch.randint(lo, most + 1, (B,), generator=g, device=DEV, dtype=torch.int32)


def _token_state(tokens, lengths, prompts, V):
    """The state of the given histories: counts of the tokens after the prompt, bit 31
    for those in the prompt, and the bitmap behind them."""
    B, L = tokens.shape
    P = (V + 31) // 32 * 32
    at = torch.arange(L, device=DEV)[None]
    ok = (tokens >= 0) & (tokens < V) & (at < lengths[:, None])
    prompt = ok & (at < prompts[:, None])
    where = torch.where(ok, tokens, 0).long()
    out = torch.zeros((B, P), dtype=torch.int32, device=DEV).scatter_add_(1, where, (ok & ~prompt).int())
    inp = torch.zeros((B, P), dtype=torch.int32, device=DEV).scatter_add_(1, where, prompt.int())
    state = torch.zeros((B, _words(V)), dtype=torch.int32, device=DEV)
    state[:, :P] = torch.where(inp > 0, out | -2 ** 31, out)
    state[:, P:P + P // 32] = _pack(state[:, :P] != 0)
    return state


def _pack(bits):
    """[..., 32 W] truth values to [..., W] int32 words, the lowest bit first."""
    w = bits.reshape(*bits.shape[:-1], -1, 32)
    weight = torch.tensor([1 << i for i in range(31)] + [-2 ** 31], dtype=torch.int64, device=bits.device)
    return (w * weight).sum(-1).to(torch.int32)


def _binary_parents(N):
    i = torch.arange(N, device=DEV, dtype=torch.int32)
    return torch.div(i, 2, rounding_mode="floor") - 1


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "process":
        return _prepare_process(case, g)
    if case["op"] == "count":
        B, V, L = case["B"], case["V"], case["hist"]
        lengths = _lengths(g, B, L)
        return dict(case=case, tokens=_tokens(g, (B, L), V), lengths=lengths, prompts=(lengths * 0.7).to(torch.int32),
                    state=torch.zeros((B, _words(V)), dtype=torch.int32, device=DEV))
    return _prepare_cache(case, g)


def _prepare_process(case, g):
    B, R, V, L, nb = case["B"], case["R"], case["V"], case["hist"], case["bias"]
    s = dict(case=case, logits=(4.0 * torch.randn((B, R, V), generator=g, device=DEV)).to(DTYPES[case["dtype"]]),
             draft=None, parents=None, state=None, rep=None, freq=None, pres=None, bias_tokens=None, bias_values=None, mask=None, out=None)
    if not case["in_place"]:
        s["out"] = torch.empty_like(s["logits"])
    if L:
        lengths = _lengths(g, B, L)
        s["state"] = _token_state(_tokens(g, (B, L), V), lengths, (lengths * 0.7).to(torch.int32), V)
        s["rep"] = 1.0 + 0.3 * torch.rand((B,), generator=g, device=DEV)
        s["freq"] = 0.5 * torch.rand((B,), generator=g, device=DEV)
        s["pres"] = 0.5 * torch.rand((B,), generator=g, device=DEV)
        if R > 1:
            s["draft"] = _tokens(g, (B, R - 1), V)
            if case["tree"]:
                s["parents"] = _binary_parents(R - 1).expand(B, R - 1).contiguous()
    if nb:
        first = torch.randint(0, V, (B, 1), generator=g, device=DEV)
        # distinct tokens, spread by a step that is prime to V
        step = next(p for p in (7919, 104729, 7907, 104723) if V % p)
        s["bias_tokens"] = ((first + step * torch.arange(nb, device=DEV)) % V).to(torch.int32)
        s["bias_values"] = 5.0 * torch.randn((B, nb), generator=g, device=DEV)
    if case["mask"] != "none":
        rows = R if case["mask"] == "rows" else 1
        W = (V + 31) // 32
        pick = torch.randint(0, len(SHARES), (B, rows, 1), generator=g, device=DEV)
        share = torch.tensor(SHARES, device=DEV)[pick]
        share = torch.where(torch.rand((B, 1, 1), generator=g, device=DEV) < FREE, 2.0, share)
        bits = torch.rand((B, rows, 32 * W), generator=g, device=DEV) < share
        bits[..., 0] = True  # no row of a working grammar is empty
        s["mask"] = _pack(bits)
        if rows == 1:
            s["mask"] = s["mask"].reshape(B, W)
    return s


def _prepare_cache(case, g):
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    dt = DTYPES[case["dtype"]]
    step = case["op"] == "step"
    T = case["N"] + 1 if step else case["T"]
    layers = case["layers"] if step else 1
    # the pages of the new tokens lie anywhere in the pool; those of the context are of other pools' business
    lengths = _lengths(g, B, case["ctx"])
    first = lengths // page
    span = (T + page - 1) // page + 1
    most = case["ctx"] // page + span + 1
    table = torch.zeros((B, most), dtype=torch.int32, device=DEV)
    pages = B * span + 1
    order = torch.randperm(pages - 1, generator=g, device=DEV).to(torch.int32).reshape(B, span) + 1
    table.scatter_(1, first[:, None].long() + torch.arange(span, device=DEV)[None], order)
    freq = torch.pow(10000.0, -torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    turns = torch.tensor([_turn(f) for f in freq.tolist()], dtype=torch.int64, device=DEV)
    s = dict(case=case, lengths=lengths, table=table, turns=turns, parents=None, q=None, out_q=None, n_new=None)
    Hq = 0 if step else case["Hq"]
    # queries, keys and values as one projection gives them
    qkv = torch.randn((layers, B, T, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dt)
    if Hq:
        s["q"] = qkv[0, :, :, :Hq]
        s["out_q"] = torch.zeros((B, T, Hq, D), dtype=dt, device=DEV)
    s["k"], s["v"] = qkv[:, :, :, Hq:Hq + Hkv], qkv[:, :, :, Hq + Hkv:]
    s["k_cache"] = torch.randn((layers, pages, page, Hkv, D), generator=g, device=DEV).to(dt)
    s["v_cache"] = torch.randn((layers, pages, page, Hkv, D), generator=g, device=DEV).to(dt)
    if step or case["tree"]:
        N = T - 1
        s["parents"] = _binary_parents(N).expand(B, N).contiguous()
    if step:
        # a path as a verify gives it: down from the root, a side at random, for a random number of levels
        depth = (N + 2).bit_length() - 2
        s["tokens"] = torch.arange(N, device=DEV, dtype=torch.int32) * 7 + torch.randint(0, 1000, (B, 1), generator=g, device=DEV, dtype=torch.int32)
        side = torch.randint(0, 2, (B, depth), generator=g, device=DEV)
        n = torch.randint(0, depth + 1, (B, 1), generator=g, device=DEV)
        level = torch.arange(depth, device=DEV)[None]
        # node d of the path is child `side` of the one above: in breadth-first order its place within the level has the sides as bits
        place = torch.stack([(side[:, :d + 1] * (1 << torch.arange(d, -1, -1, device=DEV))).sum(1) for d in range(depth)], 1)
        node = place + (1 << (level + 1)) - 2
        path = torch.full((B, N + 1), -1, dtype=torch.int32, device=DEV)
        path[:, :depth] = torch.where(level < n, torch.gather(s["tokens"], 1, node), -1)
        path.scatter_(1, n, 5)  # the token that the target adds
        s["path"], s["path_len"] = path, (n[:, 0] + 1).to(torch.int32)
    elif case["ragged"]:
        s["n_new"] = torch.randint(max(1, T // 10), T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    return s


def _turn(inv_freq):
    """Radians a position as a 64-bit fraction of a turn, held in an int64."""
    t = int(round(inv_freq / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64
    return t - 2 ** 64 if t >= 2 ** 63 else t


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "process":
        return _plain_process(s)
    if op == "count":
        s["state"].copy_(_token_state(s["tokens"], s["lengths"], s["prompts"], s["case"]["V"]))
        return s["state"]
    if op == "append":
        return _plain_append(s, 0)
    _plain_append_all(s)
    return _plain_commit(s)


def _own(s, op):
    import speculative_decoding_verification_36_gb300 as sv
    if op == "process":
        return sv.spec_process_logits(s["logits"], draft_tokens=s["draft"], parent_idx=s["parents"], token_state=s["state"],
                                      repetition=s["rep"], frequency=s["freq"], presence=s["pres"], bias_tokens=s["bias_tokens"],
                                      bias_values=s["bias_values"], allowed_mask=s["mask"],
                                      out=s["logits"] if s["case"]["in_place"] else s["out"])
    if op == "count":
        return sv.spec_count_tokens(s["state"], s["tokens"], s["case"]["V"], lengths=s["lengths"], prompt_lengths=s["prompts"], reset=True)
    if op == "append":
        sv.spec_kv_append(s["k"][0], s["v"][0], s["k_cache"][0], s["v_cache"][0], s["table"], s["lengths"], turns=s["turns"], q=s["q"],
                          out_q=s["out_q"], parent_idx=s["parents"], n_new=s["n_new"], interleaved=s["case"]["interleaved"])
        return [x for x in (s["out_q"], s["k_cache"], s["v_cache"]) if x is not None]
    for layer in range(s["case"]["layers"]):  # as a model's layers do
        sv.spec_kv_append(s["k"][layer], s["v"][layer], s["k_cache"][layer], s["v_cache"][layer], s["table"], s["lengths"],
                          turns=s["turns"], parent_idx=s["parents"])
    nodes, lengths = sv.spec_kv_commit(s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["tokens"], s["parents"], s["path"],
                                       s["path_len"])
    return [s["k_cache"], s["v_cache"], nodes, lengths]


def _reach(parents):
    """[B, N, N] in 32 bits: 1 where node j is node i or above it."""
    B, N = parents.shape
    up = torch.zeros((B, N, N + 1), device=DEV).scatter_(2, (parents.long() % (N + 1))[..., None], 1.0)[..., :N]
    reach = up + torch.eye(N, device=DEV)
    for _ in range(N.bit_length()):
        reach = (reach @ reach > 0).float()
    return reach


def _plain_process(s):
    B, R, V = s["logits"].shape
    z = s["logits"].float()
    if s["state"] is not None:
        entry = s["state"][:, None, :V]
        count, seen = (entry & 0x7FFFFFFF).expand(B, R, V), entry < 0
        if s["draft"] is not None:
            N = R - 1
            if s["parents"] is None:
                on = torch.ones((N, N), dtype=torch.int32, device=DEV).tril().expand(B, N, N)
            else:
                on = _reach(s["parents"]).int()
            extra = torch.zeros((B, R, V), dtype=torch.int32, device=DEV)
            extra[:, 1:].scatter_add_(2, s["draft"].long()[:, None].expand(B, N, N), on)
            count = count + extra
        seen = seen | (count > 0)
        rep, freq, pres = (s[k][:, None, None] for k in ("rep", "freq", "pres"))
        z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
        z = z - freq * count - pres * (count > 0)
    if s["bias_tokens"] is not None:
        bias = torch.zeros((B, V), device=DEV).scatter_add_(1, s["bias_tokens"].long(), s["bias_values"])
        z = z + bias[:, None]
    if s["mask"] is not None:
        words = s["mask"] if s["mask"].dim() == 3 else s["mask"][:, None]
        bits = (words[..., None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        z = z.masked_fill(bits.reshape(B, words.shape[1], -1)[..., :V] == 0, -math.inf)
    to = s["logits"] if s["case"]["in_place"] else s["out"]
    return to.copy_(z)


def _positions(s, T):
    """Slot and position of each new token [B, T], and the places of the slots in the pool."""
    i = torch.arange(T, device=DEV)[None]
    slot = s["lengths"][:, None].long() + i
    pos = slot
    if s["parents"] is not None:
        depth = torch.nn.functional.pad(_reach(s["parents"]).sum(2), (1, 0)).long()
        pos = s["lengths"][:, None].long() + depth
    return slot, pos


def _place(s, slot):
    page = s["case"]["page"]
    return torch.gather(s["table"], 1, slot // page).long() * page + slot % page


def _rotate(x, cos, sin, rot, interleaved):
    """x [B, T, H, D], cos and sin [B, T, 1, rot / 2], in 32 bits."""
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    lo, hi = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((lo, hi), -1).flatten(-2) if interleaved else torch.cat((lo, hi), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _angles(s, pos):
    # 64 bits: in 32 a far position's angle keeps no digits behind the point
    turns = pos[..., None].double() * (s["turns"].double() * 2.0 ** -64)
    angle = (turns - torch.floor(turns)) * (2 * math.pi)
    return torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]


def _plain_append(s, layer):
    case = s["case"]
    k, v = s["k"][layer], s["v"][layer]
    B, T = k.shape[:2]
    slot, pos = _positions(s, T)
    cos, sin = _angles(s, pos)
    inter = case.get("interleaved", False)
    new = torch.arange(T, device=DEV)[None] < s["n_new"][:, None] if s["n_new"] is not None else torch.ones((B, T), dtype=torch.bool, device=DEV)
    at = _place(s, slot)[new]
    s["k_cache"][layer].flatten(0, 1)[at] = _rotate(k, cos, sin, case["rot"], inter)[new]
    s["v_cache"][layer].flatten(0, 1)[at] = v[new]
    if s["q"] is None:
        return [s["k_cache"], s["v_cache"]]
    s["out_q"].copy_(torch.where(new[..., None, None], _rotate(s["q"], cos, sin, case["rot"], inter), s["out_q"]))
    return [s["out_q"], s["k_cache"], s["v_cache"]]


def _plain_append_all(s):
    for layer in range(s["case"]["layers"]):  # as a model's layers do
        _plain_append(s, layer)


def _plain_commit(s):
    B, N = s["tokens"].shape
    reach = _reach(s["parents"])
    depth = reach.sum(2).long()
    n = s["path_len"].long()[:, None] - 1
    match = (s["tokens"] == torch.gather(s["path"], 1, depth - 1)) & (depth <= n)
    kept = (reach * (~match).float()[:, None]).sum(2) == 0
    i = torch.arange(N, device=DEV)[None]
    last = torch.where(kept & (depth == n), i, N).amin(1)  # the lowest of the path's last nodes
    on = torch.gather(torch.nn.functional.pad(reach, (0, 0, 0, 1)), 1, last[:, None, None].expand(B, 1, N))[:, 0] > 0
    b, node = torch.nonzero(on, as_tuple=True)
    d = depth[b, node]
    nodes = torch.full((B, N + 1), -1, dtype=torch.int32, device=DEV)
    nodes[b, d - 1] = node.int()
    place = _place(s, s["lengths"][:, None].long() + torch.arange(N + 1, device=DEV)[None])
    for cache in (s["k_cache"], s["v_cache"]):
        flat = cache.flatten(1, 2)
        flat[:, place[b, d]] = flat[:, place[b, node + 1]]
    return [s["k_cache"], s["v_cache"], nodes, s["lengths"] + s["path_len"]]


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "process":
        return _exact_process(s)
    if case["op"] == "append":
        _exact_append(s, 0)
        return [x for x in (s["out_q"], s["k_cache"], s["v_cache"]) if x is not None]
    if case["op"] == "step":
        for layer in range(case["layers"]):
            _exact_append(s, layer)
        _exact_commit(s)
        return [s["k_cache"], s["v_cache"], None, None]
    return None  # counts: whole numbers


def _exact_process(s):
    B, R, V = s["logits"].shape
    out = s["logits"].double()
    drafts = s["draft"].tolist() if s["draft"] is not None else None
    parents = s["parents"].tolist() if s["parents"] is not None else None
    bit = torch.arange(V, device=DEV)
    for b in range(B):
        bias = torch.zeros(V, dtype=torch.float64, device=DEV)
        if s["bias_tokens"] is not None:
            bias.index_put_((s["bias_tokens"][b].long(),), s["bias_values"][b].double(), accumulate=True)
        for r in range(R):
            row = out[b, r]
            if s["state"] is not None:
                entry = s["state"][b, :V].long()
                c = entry % 2 ** 31
                node = r - 1
                while drafts is not None and node >= 0:
                    c[drafts[b][node]] += 1
                    node = parents[b][node] if parents is not None else node - 1
                rep, freq, pres = (s[k][b].double() for k in ("rep", "freq", "pres"))
                hit = torch.nonzero((entry < 0) | (c > 0))[:, 0]
                x, m = row[hit], c[hit].double()
                row[hit] = x * torch.where(x > 0, 1 / rep, rep) - freq * m - pres * m.clamp(max=1)
            row += bias
            if s["mask"] is not None:
                words = s["mask"][b, r] if s["mask"].dim() == 3 else s["mask"][b]
                row[(words[bit // 32].long() >> (bit % 32)) % 2 == 0] = -math.inf
    return out


def _exact_append(s, layer):
    import numpy as np
    case = s["case"]
    rot, page = case["rot"], case["page"]
    B, T = s["k"].shape[1:3]
    length, table = s["lengths"].cpu().numpy().astype(np.int64), s["table"].cpu().numpy()
    parents = s["parents"].cpu().numpy() if s["parents"] is not None else None
    new = s["n_new"].cpu().numpy() if s["n_new"] is not None else np.full(B, T)
    turns = s["turns"].cpu().numpy().astype(np.uint64)
    s["k_cache"], s["v_cache"] = s["k_cache"].double(), s["v_cache"].double()
    if s["q"] is not None:
        s["out_q"] = s["out_q"].double()
    for b in range(B):
        n = int(new[b])
        above = np.arange(n)
        if parents is not None:
            above[:] = 0
            for i in range(1, n):
                above[i] = above[parents[b, i - 1] + 1] + 1
        pos = (length[b] + above).astype(np.uint64)
        # whole turns leave at the 64th bit
        part = (pos[:, None] * turns[None]).astype(np.float64) * 2.0 ** -64 * (2 * np.pi)
        wave = torch.from_numpy(np.cos(part) + 1j * np.sin(part)).to(DEV)[:, None]
        slot = length[b] + np.arange(n)
        p, o = (torch.from_numpy(x.astype(np.int64)).to(DEV) for x in (table[b, slot // page], slot % page))

        def turned(x):
            y = x.double().clone()
            even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if case.get("interleaved") else (slice(0, rot // 2), slice(rot // 2, rot))
            z = torch.complex(y[..., even], y[..., odd]) * wave
            y[..., even], y[..., odd] = z.real, z.imag
            return y

        s["k_cache"][layer, p, o] = turned(s["k"][layer, b, :n])
        s["v_cache"][layer, p, o] = s["v"][layer, b, :n].double()
        if s["q"] is not None:
            s["out_q"][b, :n] = turned(s["q"][b, :n])


def _exact_commit(s):
    page = s["case"]["page"]
    length, table = s["lengths"].tolist(), s["table"].tolist()
    tokens, parents, path, size = (s[k].tolist() for k in ("tokens", "parents", "path", "path_len"))
    for b in range(len(length)):
        above, chosen = -1, []
        for d in range(size[b] - 1):  # siblings differ: one child at most carries the token
            above = next(j for j in range(len(tokens[b])) if parents[b][j] == above and tokens[b][j] == path[b][d])
            chosen.append(above)
        for d, node in enumerate(chosen, 1):
            to, at = length[b] + d, length[b] + 1 + node
            for cache in (s["k_cache"], s["v_cache"]):
                cache[:, table[b][to // page], to % page] = cache[:, table[b][at // page], at % page]
