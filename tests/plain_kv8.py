"""The 8-bit key/value cache in plain numpy: quantising in 32 bits as it is defined,
attention in 64 bits with a bound on what fp32 sums and fp16 operands may be off."""
import numpy as np
import torch

TOP = {"int8": np.float32(127), "e4m3": np.float32(448)}
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def quantize(x, fmt):
    """Codes (as the float32 values that they stand for) and scales of blocks x [n, block, H, D] float32."""
    x = np.asarray(x, np.float32)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = np.abs(x).max((1, 3)).astype(np.float32)
        top = np.where(np.isnan(x).any((1, 3)), np.float32(np.nan), top)
        finite = np.isfinite(top)
        some = finite & (top >= np.float32(2.0 ** -100))
        inv = np.where(some, TOP[fmt] / np.where(some, top, 1), np.float32(0)).astype(np.float32)
        y = np.where(some[:, None, :, None], x * inv[:, None, :, None], np.float32(0)).astype(np.float32)
        scale = np.where(some, top * (np.float32(1) / TOP[fmt]), np.float32(0)).astype(np.float32)
    scale = np.where(finite, scale, np.float32(np.nan))
    if fmt == "int8":
        code = np.clip(np.rint(y), -127, 127).astype(np.float32)
    else:
        code = torch.from_numpy(np.clip(y, -448, 448)).to(torch.float8_e4m3fn).float().numpy()
    return code, scale


def step_visible(T, parents):
    """[T, T] truth: token i sees the step's token j."""
    see = np.zeros((T, T), bool)
    for i in range(T):
        if parents is None:
            see[i, :i + 1] = True
        else:
            see[i, 0] = True
            node = i - 1
            while node >= 0:
                see[i, node + 1] = True
                node = int(parents[node])
    return see


def attention(q, k, v, length, n, parents, scale):
    """One sequence: q [T, Hq, D], k and v [length + n, Hkv, D] in 64 bits.  Returns
    out [n, Hq, D], sum of weights times |v|, the largest sum |q k| scale of a row, and the
    largest |v| that it sees."""
    Hq, Hkv = q.shape[1], k.shape[1]
    see = np.ones((n, length + n), bool)
    see[:, length:] = step_visible(n, parents)
    out, mag, most, top = (np.zeros((n, Hq, q.shape[2])) for _ in range(4))
    for h in range(Hq):
        kk, vv = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)]
        for i in range(n):
            s = see[i]
            with np.errstate(invalid="ignore"):
                z = kk[s] @ q[i, h] * scale
            if not np.isfinite(z).all() or not np.isfinite(vv[s]).all() or not np.isfinite(q[i, h]).all():
                out[i, h] = np.nan
                continue
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h] = p @ vv[s]
            mag[i, h], top[i, h] = p @ np.abs(vv[s]), np.abs(vv[s]).max()
            most[i, h] = (np.abs(kk[s]) @ np.abs(q[i, h])).max() * abs(scale)
    return out, mag, most, top


def tolerance(out, mag, most, top, D, keys, two):
    """What a row may be off.  A score's fp32 sum of D products: D + 8 roundings of at
    most 2^-23 of sum |q k|; fp16 operands in two parts drop 3 * 2^-22 of it (one part
    of bf16 is exact).  A weight is off by that, by its own fp16 rounding (2^-11, or
    2^-22 in two parts) and by 2^-20 for the exponential and the scales; the sums over
    the keys add 2^-23 for each key, in the weights and in the products.  Then one rounding to
    the result's type.
    fp16 ends at 2^-24, so a weight is also off by 2^-25 at least.  Weights are p sv 2^11 /
    ref with p of the largest key >= 1 and ref a power of two up to twice the largest scale sv
    of the values that the row sees, so in the result that is 2^-36 ref |code| a key: at most
    2^-36 * 2 * max sv * |code|, where |code| max sv <= 448 / 128 top (codes to 448; the scales
    of plain entries are powers of two up to top / 128, those of codes top / 127 or less):
    7 * 2^-36 top, under 2^-33 top, a key."""
    score = most * ((D + 8) * 2.0 ** -23 + (3 * 2.0 ** -22 if two else 0))
    weight = 2 * score + (2.0 ** -22 if two else 2.0 ** -11) + 2.0 ** -20 + 2 * (keys + 8) * 2.0 ** -23
    tol = weight * mag + keys * 2.0 ** -33 * top
    return tol + (2.0 ** -24 if two else 2.0 ** -8) * (np.abs(out) + tol)
