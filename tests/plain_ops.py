"""Plain numpy implementations, in 64 bits, of the operators around a verify
step (token counts, logit processing, the paged cache's append and commit),
written from their definitions for the tests."""
import numpy as np


def state_words(V):
    P = (V + 31) // 32 * 32
    return P, P + (P // 32 + 3) // 4 * 4


def count(tokens, lengths, prompts, V, start=None):
    """The state after counting: int32 [B, words]."""
    P, words = state_words(V)
    B, S = tokens.shape
    st = np.zeros((B, words), np.uint32) if start is None else start.view(np.uint32).copy()
    for b in range(B):
        L = S if lengths is None else int(lengths[b])
        Lp = 0 if prompts is None else int(prompts[b])
        if L < 0 or L > S or Lp < 0 or Lp > L:
            continue
        for i in range(L):
            t = int(tokens[b, i])
            if 0 <= t < V:
                if i < Lp:
                    st[b, t] |= np.uint32(0x80000000)
                else:
                    st[b, t] += np.uint32(1)
                st[b, P + t // 32] |= np.uint32(1 << (t % 32))
    return st.view(np.int32)


def path_of(row, parents):
    """Nodes above row `row` (its own node first)."""
    out, j = [], row - 1
    while j >= 0:
        out.append(j)
        j = j - 1 if parents is None else int(parents[j])
    return out


def process(logits, drafts=None, parents=None, state=None, rep=None, freq=None, pres=None, bias_tokens=None,
            bias_values=None, mask=None):
    """(result float64 [B, R, V], the sum of the magnitudes of its terms)."""
    z = np.asarray(logits, np.float64)
    B, R, V = z.shape
    out, mag = np.empty_like(z), np.empty_like(z)
    with np.errstate(invalid="ignore"):
        for b in range(B):
            p = float(rep[b]) if rep is not None else 1.0
            f = float(freq[b]) if freq is not None else 0.0
            q = float(pres[b]) if pres is not None else 0.0
            bad = not (p > 0 and np.isfinite(p)) or not np.isfinite(f) or not np.isfinite(q)
            if parents is not None:
                bad |= any(not -1 <= int(x) < j for j, x in enumerate(parents[b]))
            if bad:
                out[b], mag[b] = np.nan, 0.0
                continue
            entry = state[b, :V].view(np.uint32) if state is not None else np.zeros(V, np.uint32)
            base = (entry & np.uint32(0x7fffffff)).astype(np.float64)
            bias, bmag = np.zeros(V), np.zeros(V)
            if bias_tokens is not None:
                for t, x in zip(bias_tokens[b], bias_values[b]):
                    if 0 <= t < V:
                        bias[t] += float(x)
                        bmag[t] += abs(float(x))
            for r in range(R):
                c = base.copy()
                if drafts is not None:
                    for j in path_of(r, None if parents is None else parents[b]):
                        if 0 <= drafts[b, j] < V:
                            c[drafts[b, j]] += 1
                seen = (entry >> np.uint32(31) != 0) | (c > 0)
                x = z[b, r]
                y = np.where(seen, np.where(x > 0, x / p, x * p), x)
                pen = np.where(c > 0, f * c + q, 0.0)
                out[b, r] = y - pen + bias
                mag[b, r] = np.abs(y) + np.where(c > 0, abs(f) * c + abs(q), 0.0) + bmag
                if mask is not None:
                    words = (mask[b, r] if mask.ndim == 3 else mask[b]).view(np.uint32)
                    v = np.arange(V)
                    off = (words[v // 32] >> (v % 32).astype(np.uint32)) & 1 == 0
                    out[b, r][off] = -np.inf
                    mag[b, r][off] = 0.0
    return out, mag


def depths(T, parents):
    """Depth of each of a step's T tokens."""
    if parents is None:
        return np.arange(T)
    d = np.zeros(T, np.int64)
    for j, p in enumerate(parents):
        d[j + 1] = d[p + 1] + 1
    return d


def rotate(x, pos, turns, interleaved):
    """(x [H, D] turned to a position, the magnitudes of its terms), float64."""
    y = np.array(x, np.float64)
    mag = np.abs(y)
    half = len(turns)
    frac = np.array([(int(pos) * (int(t) % 2 ** 64)) % 2 ** 64 for t in turns], dtype=object)
    ang = np.array([float(f) / 2.0 ** 64 * 2 * np.pi for f in frac])
    c, s = np.cos(ang), np.sin(ang)
    i0 = np.arange(half) * 2 if interleaved else np.arange(half)
    i1 = i0 + 1 if interleaved else i0 + half
    a, b = y[:, i0].copy(), y[:, i1].copy()
    y[:, i0], y[:, i1] = a * c - b * s, a * s + b * c
    mag[:, i0] = mag[:, i1] = np.abs(a) + np.abs(b)
    return y, mag


def append(k, v, k_cache, v_cache, table, lengths, turns, q=None, out_q=None, parents=None, n_new=None,
           interleaved=False):
    """Writes into float64 copies of the caches [pages, page, H, D]; returns
    (key cache, value cache, out_q, magnitudes of the key cache's and out_q's new terms)."""
    B, T = k.shape[:2]
    pages, page = k_cache.shape[:2]
    kc, vc = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    km = np.zeros_like(kc)
    oq = None if q is None else np.array(out_q, np.float64)
    qm = None if q is None else np.zeros_like(oq)
    for b in range(B):
        n = T if n_new is None else int(n_new[b])
        L = int(lengths[b])
        par = None if parents is None else parents[b]
        if L < 0 or not 0 <= n <= T or L + n > table.shape[1] * page or (
                par is not None and any(not -1 <= int(x) < j for j, x in enumerate(par))):
            if oq is not None:
                oq[b] = np.nan
            continue
        d = depths(T, par)
        for i in range(n):
            if q is not None:
                oq[b, i], qm[b, i] = rotate(q[b, i], L + d[i], turns, interleaved)
            p = int(table[b, (L + i) // page])
            if not 0 <= p < pages:
                continue
            kc[p, (L + i) % page], km[p, (L + i) % page] = rotate(k[b, i], L + d[i], turns, interleaved)
            vc[p, (L + i) % page] = v[b, i]
    return kc, vc, oq, km, qm


def commit(caches, table, lengths, tokens, parents, path, path_len):
    """Moves in copies of the caches (each [layers, pages, page, ...]); returns
    (caches, nodes [B, N+1], new lengths [B])."""
    caches = [c.copy() for c in caches]
    pages, page = caches[0].shape[1:3]
    B, N = tokens.shape
    nodes = np.full((B, N + 1), -1, np.int32)
    new = np.array(lengths, np.int32)
    for b in range(B):
        n, L = int(path_len[b]) - 1, int(lengths[b])
        if n < 0 or n > N or L < 0 or L + N + 1 > table.shape[1] * page:
            continue
        if any(not -1 <= int(x) < j for j, x in enumerate(parents[b])):
            continue
        level = {-1: 0}
        for j in range(N):
            d = level.get(int(parents[b, j]))
            if d is not None and d < n and tokens[b, j] == path[b, d]:
                level[j] = d + 1
        last = [j for j in range(N) if level.get(j) == n] if n else [-1]
        if not last:
            continue
        chosen, j = [], last[0]
        while j >= 0:
            chosen.insert(0, j)
            j = int(parents[b, j])
        places = [(L + 1 + d, L + 1 + c) for d, c in enumerate(chosen)]
        if any(not 0 <= int(table[b, s // page]) < pages for pair in places for s in pair):
            continue
        nodes[b, :n], new[b] = chosen, L + n + 1
        for c in caches:
            src = [c[:, table[b, f // page], f % page].copy() for _, f in places]
            for (t, _), x in zip(places, src):
                c[:, table[b, t // page], t % page] = x
    return caches, nodes, new
