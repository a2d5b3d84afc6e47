"""GB300-native speculative-decoding verify step.

A thin binding over libspecverify.so (C ABI in include/specverify.h).  Each
function checks and marshals torch CUDA tensors (device, dtype, contiguity,
shapes), allocates outputs that were not given, and calls the C entry point of
the same name on the current stream; every step of the verify path runs in the
library's CUDA kernels.  There is no CPU fallback.

stream= (a torch stream or a cudaStream_t as an int) runs a call on another
stream: its inputs have to be ready there and to stay until it is done, and its
outputs are complete there.  Outputs that it allocates are that stream's memory.

    spec_verify(target_logits, draft_logits, draft_tokens, temperature, seed)
    spec_verify_early_exit(...)       # reads only the rows the result depends on
    spec_verify_static_scratch(...)   # no allocation: a fixed per-device scratch buffer
    spec_verify_stats(...)            # plus row statistics, p(x), q(x), mass
    spec_verify_khint(..., h_lo, h_hi, k_min, k_max)  # plus a suggested next draft length
    spec_verify_greedy_argmax(...)    # greedy chain plus every row's argmax
    spec_tree_verify_greedy(target_logits, tree_tokens, parent_idx)
    spec_tree_verify_sampling(target_logits, draft_logits, tree_tokens, parent_idx, T, seed)
    spec_acceptance_stats(n_accepted, K)  # histogram, alpha, mean tokens
    spec_ngram_draft(tokens, lengths, n_min, n_max, K)  # prompt-lookup drafts
    spec_token_state(B, V, device)    # zeroed token counts; spec_count_tokens(state, tokens, V) adds to them
    spec_process_logits(logits, draft_tokens, ...)  # penalties, biases and grammar masks on a verify's rows
    spec_kv_append(k, v, key_cache, value_cache, page_table, lengths, ...)  # rotated, into a paged cache
    spec_kv_commit(key_cache, value_cache, page_table, lengths, ...)  # a tree's accepted path stays
    spec_get_status()                 # device status word (bad data, timeouts)
"""
from __future__ import annotations

import math

import torch

from . import _lib
from ._lib import SPEC_FLAG_BAD_DATA, SPEC_FLAG_TIMEOUT, SpecError

__all__ = [
    "spec_verify", "spec_verify_early_exit", "spec_verify_static_scratch", "spec_verify_stats", "spec_verify_khint",
    "spec_verify_greedy_argmax",
    "spec_tree_verify_greedy", "spec_tree_verify_sampling", "spec_acceptance_stats", "spec_ngram_draft",
    "spec_token_state", "spec_count_tokens", "spec_process_logits", "spec_rope_turns", "spec_kv_append",
    "spec_kv_commit",
    "spec_get_status", "spec_test_spin_limit", "spec_test_wait_probe", "SpecError",
    "SPEC_FLAG_BAD_DATA", "SPEC_FLAG_TIMEOUT",
]


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# the handle of a device's current stream without a Stream object around it
# (0.1 us, where torch.cuda.current_stream().cuda_stream takes 2.8)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _is_bf16(t: torch.Tensor, name: str) -> bool:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype == torch.bfloat16:
        return True
    if t.dtype == torch.float32:
        return False
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    if t is None or t.numel() == 0:
        return None
    return t.data_ptr()


def _same_device(t: torch.Tensor, device, name: str):
    # a pointer into another GPU's memory is not readable by this device's kernels
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device} (all tensors of a call share one GPU)")


def _i32(t: torch.Tensor, shape, name: str, device=None):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None:
        _same_device(t, device, name)
    return t


def _new(shape, dtype, device, stream):
    """An output of a call on `stream`.  On another stream than the current one
    it is that stream's memory, which no pending work of the current stream still
    uses and which does not go back to the current stream while the call runs;
    the current stream is noted as a user."""
    handle = None if stream is None else _stream(stream)
    if handle is None or handle == _raw_stream(device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _out(t, shape, dtype, device, name, stream):
    if t is None:
        return _new(shape, dtype, device, stream)
    if t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != tuple(shape) or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _c_ints(*sizes):
    """Refuses what the C entry points' ints do not carry (ctypes would drop the
    upper bits)."""
    for n in sizes:
        if not -2 ** 31 <= n < 2 ** 31:
            _lib.check(_lib.SPEC_ERR_SHAPE)


def _chain_args(target_logits, draft_logits, draft_tokens, temperature):
    bf16 = _is_bf16(target_logits, "target_logits")
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    _c_ints(B, K1, V)
    K = K1 - 1
    if temperature > 0 and K > 0:
        if draft_logits is None:
            raise ValueError("draft_logits is required when temperature > 0")
        if _is_bf16(draft_logits, "draft_logits") != bf16:
            raise TypeError("target_logits and draft_logits must share a dtype")
        if tuple(draft_logits.shape) != (B, K, V):
            raise ValueError(f"draft_logits has shape {tuple(draft_logits.shape)}, expected {(B, K, V)}")
        _same_device(draft_logits, target_logits.device, "draft_logits")
    if K > 0:
        _i32(draft_tokens, (B, K), "draft_tokens", target_logits.device)
    return bf16, B, K, V


def spec_verify(target_logits, draft_logits, draft_tokens, temperature: float, seed: int,
                out_tokens=None, out_n_accepted=None, stream=None):
    """Verify K drafted tokens per sequence; returns (out_tokens [B,K+1], n [B])."""
    bf16, B, K, V = _chain_args(target_logits, draft_logits, draft_tokens, temperature)
    dev = target_logits.device
    out_tokens = _out(out_tokens, (B, K + 1), torch.int32, dev, "out_tokens", stream)
    out_n_accepted = _out(out_n_accepted, (B,), torch.int32, dev, "out_n_accepted", stream)
    lib = _lib.load()
    fn = lib.spec_verify_bf16 if bf16 else lib.spec_verify_f32
    with torch.cuda.device(dev):
        _lib.check(fn(_ptr(target_logits), _ptr(draft_logits) if temperature > 0 else None,
                      _ptr(draft_tokens) if K > 0 else None, B, K, V, float(temperature),
                      int(seed) & (2**64 - 1), _ptr(out_tokens), _ptr(out_n_accepted),
                      _stream(stream)))
    return out_tokens, out_n_accepted


def spec_verify_early_exit(target_logits, draft_logits, draft_tokens, temperature: float, seed: int,
                           out_tokens=None, out_n_accepted=None, stream=None):
    """spec_verify that reads only the rows its result depends on (positions
    up to the first rejection, and the bonus row when every draft is
    accepted); bad data is checked on those rows only.  Temperature 0 is the
    greedy verify with the same early exit (draft_logits may be None).
    Returns (out_tokens [B,K+1], n [B])."""
    bf16, B, K, V = _chain_args(target_logits, draft_logits, draft_tokens, temperature)
    dev = target_logits.device
    out_tokens = _out(out_tokens, (B, K + 1), torch.int32, dev, "out_tokens", stream)
    out_n_accepted = _out(out_n_accepted, (B,), torch.int32, dev, "out_n_accepted", stream)
    lib = _lib.load()
    fn = lib.spec_verify_early_exit_bf16 if bf16 else lib.spec_verify_early_exit_f32
    with torch.cuda.device(dev):
        _lib.check(fn(_ptr(target_logits), _ptr(draft_logits) if temperature > 0 else None,
                      _ptr(draft_tokens) if K > 0 else None, B, K, V, float(temperature),
                      int(seed) & (2**64 - 1), _ptr(out_tokens), _ptr(out_n_accepted),
                      _stream(stream)))
    return out_tokens, out_n_accepted


def spec_verify_static_scratch(target_logits, draft_logits, draft_tokens, temperature: float,
                               seed: int, out_tokens=None, out_n_accepted=None, stream=None):
    """spec_verify for bf16 logits with the library's fixed per-device scratch
    buffer instead of its memory pool (no device allocation by the library).
    Calls that overlap in time on one device race on that buffer.  Pass
    out_tokens / out_n_accepted to keep this wrapper allocation-free too."""
    bf16, B, K, V = _chain_args(target_logits, draft_logits, draft_tokens, temperature)
    if not bf16:
        raise TypeError("spec_verify_static_scratch takes bf16 logits")
    dev = target_logits.device
    out_tokens = _out(out_tokens, (B, K + 1), torch.int32, dev, "out_tokens", stream)
    out_n_accepted = _out(out_n_accepted, (B,), torch.int32, dev, "out_n_accepted", stream)
    lib = _lib.load()
    with torch.cuda.device(dev):
        _lib.check(lib.spec_verify_bf16_static_scratch(
            _ptr(target_logits), _ptr(draft_logits) if temperature > 0 else None,
            _ptr(draft_tokens) if K > 0 else None, B, K, V, float(temperature),
            int(seed) & (2**64 - 1), _ptr(out_tokens), _ptr(out_n_accepted), _stream(stream)))
    return out_tokens, out_n_accepted


def spec_verify_stats(target_logits, draft_logits, draft_tokens, temperature: float, seed: int,
                      stream=None, entropy: bool = False):
    """spec_verify plus the intermediate probabilities (temperature > 0).

    Returns dict(tokens [B,K+1], n [B], row_stats [B,2K+1,2] (max z/tau, sum
    exp(z/tau - max)), pq [B,K,2] (p_i(x_i), q_i(x_i)), resid_mass [B]) and,
    with entropy=True, row_entropy [B,2K+1] (nats)."""
    if not temperature > 0:
        raise ValueError("spec_verify_stats needs temperature > 0")
    bf16, B, K, V = _chain_args(target_logits, draft_logits, draft_tokens, temperature)
    dev = target_logits.device
    tokens = _new((B, K + 1), torch.int32, dev, stream)
    n = _new((B,), torch.int32, dev, stream)
    row_stats = _new((B, 2 * K + 1, 2), torch.float32, dev, stream)
    pq = _new((B, K, 2), torch.float32, dev, stream)
    resid = _new((B,), torch.float32, dev, stream)
    ent = _new((B, 2 * K + 1), torch.float32, dev, stream) if entropy else None
    lib = _lib.load()
    fn = lib.spec_verify_stats_bf16 if bf16 else lib.spec_verify_stats_f32
    with torch.cuda.device(dev):
        _lib.check(fn(_ptr(target_logits), _ptr(draft_logits), _ptr(draft_tokens) if K > 0 else None,
                      B, K, V, float(temperature), int(seed) & (2**64 - 1), _ptr(tokens), _ptr(n),
                      _ptr(row_stats), _ptr(pq), _ptr(resid), _ptr(ent) if entropy else None,
                      _stream(stream)))
    out = dict(tokens=tokens, n=n, row_stats=row_stats, pq=pq, resid_mass=resid)
    if entropy:
        out["row_entropy"] = ent
    return out


def spec_verify_khint(target_logits, draft_logits, draft_tokens, temperature: float, seed: int,
                      h_lo: float, h_hi: float, k_min: int, k_max: int, stream=None, out_tokens=None,
                      out_n_accepted=None, out_k_next=None, out_mean_entropy=None):
    """spec_verify plus a suggested next draft length per sequence (temperature > 0).

    The mean entropy (nats) of target rows 0..n moves K one step up when below
    h_lo, one step down when above h_hi; the result is clamped to [k_min,
    k_max], -1 for a bad sequence.  Returns (tokens [B,K+1], n [B], k_next [B]
    int32, mean_entropy [B] float32)."""
    bf16, B, K, V = _chain_args(target_logits, draft_logits, draft_tokens, temperature)
    _c_ints(int(k_min), int(k_max))
    dev = target_logits.device
    tokens = _out(out_tokens, (B, K + 1), torch.int32, dev, "out_tokens", stream)
    n = _out(out_n_accepted, (B,), torch.int32, dev, "out_n_accepted", stream)
    k_next = _out(out_k_next, (B,), torch.int32, dev, "out_k_next", stream)
    hmean = _out(out_mean_entropy, (B,), torch.float32, dev, "out_mean_entropy", stream)
    lib = _lib.load()
    fn = lib.spec_verify_khint_bf16 if bf16 else lib.spec_verify_khint_f32
    with torch.cuda.device(dev):
        _lib.check(fn(_ptr(target_logits), _ptr(draft_logits), _ptr(draft_tokens) if K > 0 else None,
                      B, K, V, float(temperature), int(seed) & (2**64 - 1), float(h_lo), float(h_hi),
                      int(k_min), int(k_max), _ptr(tokens), _ptr(n), _ptr(k_next), _ptr(hmean),
                      _stream(stream)))
    return tokens, n, k_next, hmean


def spec_verify_greedy_argmax(target_logits, draft_tokens, stream=None):
    """Greedy chain verification that also returns every target row's argmax.

    Returns (out_tokens [B,K+1], n [B], row_argmax [B,K+1])."""
    bf16, B, K, V = _chain_args(target_logits, None, draft_tokens, 0.0)
    dev = target_logits.device
    tokens = _new((B, K + 1), torch.int32, dev, stream)
    n = _new((B,), torch.int32, dev, stream)
    amax = _new((B, K + 1), torch.int32, dev, stream)
    lib = _lib.load()
    fn = lib.spec_verify_greedy_argmax_bf16 if bf16 else lib.spec_verify_greedy_argmax_f32
    with torch.cuda.device(dev):
        _lib.check(fn(_ptr(target_logits), _ptr(draft_tokens) if K > 0 else None, B, K, V,
                      _ptr(tokens), _ptr(n), _ptr(amax), _stream(stream)))
    return tokens, n, amax


def spec_tree_verify_greedy(target_logits, tree_tokens, parent_idx, out_path=None, out_len=None,
                            out_mask=None, stream=None, early_exit: bool = False):
    """Greedy verification of a candidate tree per sequence.

    target_logits [B, N+1, V]; tree_tokens, parent_idx [B, N] int32.
    Returns (out_path [B, N+1], out_len [B], out_mask [B, N, ceil(N/32)] as int32 bits).
    early_exit=True calls spec_tree_verify_greedy_early_exit_*: the rows under
    a rejected node are not read (and bad data there is not reported)."""
    bf16 = _is_bf16(target_logits, "target_logits")
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, N+1, V]")
    B, N1, V = target_logits.shape
    _c_ints(B, N1, V)
    N = N1 - 1
    W = (N + 31) // 32
    dev = target_logits.device
    if N > 0:
        _i32(tree_tokens, (B, N), "tree_tokens", dev)
        _i32(parent_idx, (B, N), "parent_idx", dev)
    out_path = _out(out_path, (B, N + 1), torch.int32, dev, "out_path", stream)
    out_len = _out(out_len, (B,), torch.int32, dev, "out_len", stream)
    # torch has no uint32 arithmetic on every version: the mask words travel as int32 bits
    out_mask = _out(out_mask, (B, N, W), torch.int32, dev, "out_mask", stream)
    lib = _lib.load()
    if early_exit:
        fn = lib.spec_tree_verify_greedy_early_exit_bf16 if bf16 else lib.spec_tree_verify_greedy_early_exit_f32
    else:
        fn = lib.spec_tree_verify_greedy_bf16 if bf16 else lib.spec_tree_verify_greedy_f32
    with torch.cuda.device(dev):
        _lib.check(fn(_ptr(target_logits), _ptr(tree_tokens) if N > 0 else None,
                      _ptr(parent_idx) if N > 0 else None, B, N, V, _ptr(out_path), _ptr(out_len),
                      _ptr(out_mask), _stream(stream)))
    return out_path, out_len, out_mask


def spec_tree_verify_sampling(target_logits, draft_logits, tree_tokens, parent_idx, temperature: float,
                              seed: int, out_path=None, out_len=None, stream=None):
    """Stochastic verification of a candidate tree per sequence (temperature > 0).

    target_logits, draft_logits [B, N+1, V] (draft row u+1: the distribution
    node u's children were drawn from); tree_tokens, parent_idx [B, N] int32.
    Returns (out_path [B, N+1], out_len [B])."""
    if not temperature > 0:
        raise ValueError("spec_tree_verify_sampling needs temperature > 0 (spec_tree_verify_greedy is T = 0)")
    bf16 = _is_bf16(target_logits, "target_logits")
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, N+1, V]")
    if _is_bf16(draft_logits, "draft_logits") != bf16:
        raise TypeError("target_logits and draft_logits must share a dtype")
    if tuple(draft_logits.shape) != tuple(target_logits.shape):
        raise ValueError(f"draft_logits has shape {tuple(draft_logits.shape)}, expected "
                         f"{tuple(target_logits.shape)}")
    B, N1, V = target_logits.shape
    _c_ints(B, N1, V)
    N = N1 - 1
    dev = target_logits.device
    _same_device(draft_logits, dev, "draft_logits")
    if N > 0:
        _i32(tree_tokens, (B, N), "tree_tokens", dev)
        _i32(parent_idx, (B, N), "parent_idx", dev)
    out_path = _out(out_path, (B, N + 1), torch.int32, dev, "out_path", stream)
    out_len = _out(out_len, (B,), torch.int32, dev, "out_len", stream)
    lib = _lib.load()
    fn = lib.spec_tree_verify_sampling_bf16 if bf16 else lib.spec_tree_verify_sampling_f32
    with torch.cuda.device(dev):
        _lib.check(fn(_ptr(target_logits), _ptr(draft_logits), _ptr(tree_tokens) if N > 0 else None,
                      _ptr(parent_idx) if N > 0 else None, B, N, V, float(temperature),
                      int(seed) & (2**64 - 1), _ptr(out_path), _ptr(out_len), _stream(stream)))
    return out_path, out_len


def spec_acceptance_stats(n_accepted, K: int, stream=None):
    """Acceptance statistics of verify outputs on the device.

    n_accepted: int32 [B] (-1 = bad sequence).  Returns dict(hist uint64-valued
    int64 [K+2], alpha float64 [K], mean_tokens float64 scalar tensor)."""
    if (not isinstance(n_accepted, torch.Tensor) or n_accepted.dtype != torch.int32 or n_accepted.dim() != 1
            or not n_accepted.is_contiguous() or not n_accepted.is_cuda):
        raise TypeError("n_accepted must be a contiguous 1-D int32 CUDA tensor")
    dev = n_accepted.device
    B = n_accepted.shape[0]
    _c_ints(B, int(K))
    hist = _new((K + 2,), torch.int64, dev, stream)
    alpha = _new((max(K, 0),), torch.float64, dev, stream)
    mean = _new((1,), torch.float64, dev, stream)
    lib = _lib.load()
    with torch.cuda.device(dev):
        _lib.check(lib.spec_acceptance_stats(_ptr(n_accepted) if B > 0 else None, B, int(K),
                                             _ptr(hist), _ptr(alpha) if K > 0 else None, _ptr(mean),
                                             _stream(stream)))
    return dict(hist=hist, alpha=alpha, mean_tokens=mean[0])


def spec_ngram_draft(tokens, lengths, n_min: int, n_max: int, K: int, out_drafts=None, out_n_drafts=None,
                     out_match_len=None, stream=None):
    """N-gram (prompt-lookup) drafts from token histories on the device.

    tokens: int32 [B, Lmax] (row b's first lengths[b] entries are its history);
    lengths: int32 [B].  Returns (drafts int32 [B, K] (-1 padded), n_drafts
    int32 [B], match_len int32 [B])."""
    if tokens.dim() != 2:
        raise ValueError("tokens must be [B, Lmax]")
    B, Lmax = tokens.shape
    _c_ints(B, Lmax, int(n_min), int(n_max), int(K))
    _i32(tokens, (B, Lmax), "tokens")
    dev = tokens.device
    _i32(lengths, (B,), "lengths", dev)
    drafts = _out(out_drafts, (B, max(int(K), 0)), torch.int32, dev, "out_drafts", stream)  # K < 0: the C layer refuses
    n_drafts = _out(out_n_drafts, (B,), torch.int32, dev, "out_n_drafts", stream)
    match_len = _out(out_match_len, (B,), torch.int32, dev, "out_match_len", stream)
    lib = _lib.load()
    with torch.cuda.device(dev):
        _lib.check(lib.spec_ngram_draft(_ptr(tokens), _ptr(lengths), B, Lmax, int(n_min), int(n_max), int(K),
                                        _ptr(drafts), _ptr(n_drafts), _ptr(match_len), _stream(stream)))
    return drafts, n_drafts, match_len


# The entry points below are called once or more a layer, where a few
# microseconds of checking are a large part of the call: one pass over each
# tensor's properties, and a message only once something is wrong.
def _arg(t, dtype, shape, device, name):
    """The address of a contiguous CUDA tensor of this type, shape and device
    (None for None and for an empty one)."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr() or None
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    _same_device(t, device, name)
    raise ValueError(f"{name} cannot be used")


def _invoke(fn, device, stream, *args):
    """Calls a C entry point on `device`, its current stream by default."""
    index = device.index
    if torch.cuda.current_device() == index:
        code = fn(*args, _raw_stream(index) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(device):
            code = fn(*args, _stream(stream))
    if code:
        _lib.check(code)


# Sizes that the C entry points' ints do not carry are refused: `_too_large if
# (a | b | ...) >> 31`, for sizes that are not negative (a third of the time of _c_ints).
def _too_large():
    _lib.check(_lib.SPEC_ERR_SHAPE)


def _words(V: int) -> int:
    """spec_token_state_words(V), worked out here (the layout is the header's)."""
    if not 1 <= V <= 2 ** 30:
        _lib.check(_lib.SPEC_ERR_SHAPE)
    P = (V + 31) // 32
    return 32 * P + (P + 3) // 4 * 4


def spec_token_state(B: int, V: int, device) -> torch.Tensor:
    """An empty token-count state: int32 [B, words] zeros (spec_count_tokens
    fills it, spec_process_logits reads it; the layout is in specverify.h).
    One row of it, state[b:b+1], is a state too."""
    return torch.zeros((B, _words(int(V))), dtype=torch.int32, device=device)


def spec_count_tokens(state, tokens, V: int, lengths=None, prompt_lengths=None, reset: bool = False, stream=None):
    """Adds tokens [B, S] int32 to the counts in `state` and returns it.

    Row b's first lengths[b] entries count (None: all S); the first
    prompt_lengths[b] of them as prompt (None: none), the rest as output.
    Tokens outside [0, V) are skipped: a verify's padded out_tokens or
    out_path can be passed.  reset=True empties the state first."""
    if not isinstance(tokens, torch.Tensor) or not tokens.is_cuda or tokens.dim() != 2:
        raise ValueError("tokens must be a CUDA tensor [B, S]")
    B, S = tokens.shape
    if (B | S) >> 31:
        _too_large()
    dev, i32, V = tokens.device, torch.int32, int(V)
    _invoke(_lib.load().spec_count_tokens, dev, stream, _arg(tokens, i32, (B, S), dev, "tokens"),
            _arg(lengths, i32, (B,), dev, "lengths"), _arg(prompt_lengths, i32, (B,), dev, "prompt_lengths"), B, S, V,
            1 if reset else 0, _arg(state, i32, (B, _words(V)), dev, "state"))
    return state


def spec_process_logits(logits, draft_tokens=None, parent_idx=None, token_state=None, repetition=None,
                        frequency=None, presence=None, bias_tokens=None, bias_values=None, allowed_mask=None,
                        out=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks on the rows a
    verify reads: logits [B, R, V] (R = K + 1 of a chain, N + 1 of a tree).

    draft_tokens [B, R-1] int32 (with parent_idx [B, R-1] for a tree): row r's
    penalties count the drafts above it too.  token_state: spec_token_state's,
    filled by spec_count_tokens.  repetition, frequency, presence: float32 [B].
    bias_tokens int32 / bias_values float32 [B, n]; tokens outside [0, V) are
    padding.  allowed_mask int32 [B, R, ceil(V/32)], or [B, ceil(V/32)] for
    all rows: a set bit allows the token.  out=logits works in place and
    touches only what changes and the 16 bytes around a token that is not
    allowed (slower than a copy where that is much of a row); out=None
    allocates.  Returns out."""
    bf16 = _is_bf16(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits must be [B, R, V]")
    B, R, V = logits.shape
    dev, i32, f32 = logits.device, torch.int32, torch.float32
    if parent_idx is not None and draft_tokens is None:
        raise ValueError("parent_idx needs draft_tokens")
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values go together")
    n_bias = mask_rows = 0
    if bias_tokens is not None:
        if bias_tokens.dim() != 2:
            raise ValueError("bias_tokens must be [B, n]")
        n_bias = bias_tokens.shape[1]
    if (B | R | V | n_bias) >> 31:
        _too_large()
    mask = None
    if allowed_mask is not None:
        W = (V + 31) // 32
        mask_rows = 1 if allowed_mask.dim() == 2 else R
        mask = _arg(allowed_mask, i32, (B, W) if allowed_mask.dim() == 2 else (B, R, W), dev, "allowed_mask")
    state = None if token_state is None else _arg(token_state, i32, (B, _words(V)), dev, "token_state")
    if out is None:
        out = _new((B, R, V), logits.dtype, dev, stream)
    lib = _lib.load()
    _invoke(lib.spec_process_logits_bf16 if bf16 else lib.spec_process_logits_f32, dev, stream, _ptr(logits),
            _arg(draft_tokens, i32, (B, R - 1), dev, "draft_tokens"), _arg(parent_idx, i32, (B, R - 1), dev, "parent_idx"),
            state, _arg(repetition, f32, (B,), dev, "repetition"), _arg(frequency, f32, (B,), dev, "frequency"),
            _arg(presence, f32, (B,), dev, "presence"), n_bias, _arg(bias_tokens, i32, (B, n_bias), dev, "bias_tokens"),
            _arg(bias_values, f32, (B, n_bias), dev, "bias_values"), mask, mask_rows, B, R, V,
            _arg(out, logits.dtype, (B, R, V), dev, "out"))
    return out


def spec_rope_turns(inv_freq, device) -> torch.Tensor:
    """Rotary frequencies (radians a position, float64-able: theta ** (-2 i /
    rot_dim) or any scaled set) as spec_kv_append takes them: int64 [rot_dim /
    2] holding 2^-64 fractions of a turn (the bits are unsigned)."""
    vals = [int(round(float(f) / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64 for f in inv_freq]
    return torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in vals], dtype=torch.int64, device=device)


def _token_stride(t, name, dtype, shape, device):
    """Elements between successive tokens of a [B, T, H, D] tensor whose tokens
    lie at equal distances and whose heads are contiguous (such as a slice of a
    joint projection)."""
    B, T, H, D = shape
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device:
        sb, st, sh, sd = t.stride()
        if sd == 1 and sh == D and sb == T * st:
            return st
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    _same_device(t, device, name)
    if t.numel() == 0:
        return H * D
    sb, st, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{name}'s heads must be contiguous")
    if T == 1:
        return sb if B > 1 else max(H * D, 1)
    if sb != T * st and B > 1:
        raise ValueError(f"{name}'s tokens must lie at equal distances")
    return st


def spec_kv_append(k, v, key_cache, value_cache, page_table, lengths, turns=None, q=None, parent_idx=None,
                   n_new=None, interleaved: bool = False, out_q=None, stream=None):
    """Appends a step's keys and values [B, T, Hkv, D] to a paged cache
    [pages, page_size, Hkv, D], the keys rotated to their positions, and
    rotates the queries q [B, T, Hq, D].

    Token i goes to slot lengths[b] + i; its position is lengths[b] + i, or,
    with parent_idx [B, T-1] (token 0 the root, token j + 1 node j),
    lengths[b] + its depth.  turns (spec_rope_turns): None rotates nothing.
    n_new [B]: tokens from there on are padding.  k, v and q may be slices of
    a joint projection.  Returns out_q (None without q)."""
    if not isinstance(k, torch.Tensor) or not k.is_cuda or k.dim() != 4:
        raise ValueError("k must be a CUDA tensor [B, T, Hkv, D]")
    dt, dev, i32 = k.dtype, k.device, torch.int32
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError(f"k must be float32 or bfloat16, got {dt}")
    shape = k.shape
    B, T, Hkv, D = shape
    ks = _token_stride(k, "k", dt, shape, dev)
    if _token_stride(v, "v", dt, shape, dev) != ks:
        if B != 1 or T != 1:  # (one token has none)
            raise ValueError("k and v must share a token stride")
        ks = Hkv * D
    if not isinstance(key_cache, torch.Tensor) or key_cache.dim() != 4:
        raise ValueError("key_cache must be [pages, page_size, Hkv, D]")
    pages, page_size = key_cache.shape[:2]
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    max_pages = page_table.shape[1]
    rot = 0
    if turns is not None:
        rot = 2 * turns.numel()
    if (B | T | Hkv | D | rot | pages | page_size | max_pages) >> 31:
        _too_large()
    qp = oq = None
    Hq = qs = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 4:
            raise ValueError("q must be a CUDA tensor [B, T, Hq, D]")
        Hq = q.shape[2]
        if Hq >> 31:
            _too_large()
        qs = _token_stride(q, "q", dt, (B, T, Hq, D), dev)
        if out_q is None:
            out_q = _new((B, T, Hq, D), dt, dev, stream)
        qp, oq = q.data_ptr(), _arg(out_q, dt, (B, T, Hq, D), dev, "out_q")
    elif out_q is not None:
        raise ValueError("out_q needs q")
    cache = (pages, page_size, Hkv, D)
    lib = _lib.load()
    _invoke(lib.spec_kv_append_bf16 if dt is torch.bfloat16 else lib.spec_kv_append_f32, dev, stream, k.data_ptr(),
            v.data_ptr(), ks, qp, qs, oq, _arg(parent_idx, i32, (B, T - 1), dev, "parent_idx"),
            _arg(n_new, i32, (B,), dev, "n_new"), _arg(lengths, i32, (B,), dev, "lengths"),
            _arg(page_table, i32, (B, max_pages), dev, "page_table"), B, T, Hq, Hkv, D, rot, 1 if interleaved else 0,
            _arg(turns, torch.int64, (rot // 2,), dev, "turns"), _arg(key_cache, dt, cache, dev, "key_cache"),
            _arg(value_cache, dt, cache, dev, "value_cache"), pages, page_size, max_pages)
    return out_q


def spec_kv_commit(key_cache, value_cache, page_table, lengths, tree_tokens, parent_idx, out_path, out_len,
                   out_nodes=None, out_lengths=None, stream=None):
    """Keeps a tree verify's accepted path in the paged cache: its nodes'
    entries move to the slots behind the root's.

    key_cache, value_cache: [pages, page_size, H, D] or, with all layers in one
    tensor, [layers, pages, page_size, H, D], any type.  lengths as given to
    spec_kv_append for the step; out_path, out_len: the verify's.  Returns
    (nodes [B, N+1] int32, -1 padded; new lengths [B])."""
    if not isinstance(key_cache, torch.Tensor) or not key_cache.is_cuda or key_cache.dim() not in (4, 5):
        raise ValueError("key_cache must be a CUDA tensor [(layers,) pages, page_size, H, D]")
    dev, dt, i32 = key_cache.device, key_cache.dtype, torch.int32
    shape = key_cache.shape
    pages, page_size, H, D = shape[-4:]
    layers = shape[0] if len(shape) == 5 else 1
    entry = H * D * key_cache.element_size()
    if not isinstance(tree_tokens, torch.Tensor) or tree_tokens.dim() != 2:
        raise ValueError("tree_tokens must be [B, N]")
    B, N = tree_tokens.shape
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    max_pages = page_table.shape[1]
    if (layers | pages | page_size | entry | max_pages | B | N) >> 31:
        _too_large()
    if out_nodes is None:
        out_nodes = _new((B, N + 1), i32, dev, stream)
    if out_lengths is None:
        out_lengths = _new((B,), i32, dev, stream)
    _invoke(_lib.load().spec_kv_commit, dev, stream, _arg(key_cache, dt, shape, dev, "key_cache"),
            _arg(value_cache, dt, shape, dev, "value_cache"), layers, pages * page_size * entry, pages, page_size, entry,
            _arg(page_table, i32, (B, max_pages), dev, "page_table"), max_pages,
            _arg(lengths, i32, (B,), dev, "lengths"), _arg(tree_tokens, i32, (B, N), dev, "tree_tokens"),
            _arg(parent_idx, i32, (B, N), dev, "parent_idx"), _arg(out_path, i32, (B, N + 1), dev, "out_path"),
            _arg(out_len, i32, (B,), dev, "out_len"), B, N, _arg(out_nodes, i32, (B, N + 1), dev, "out_nodes"),
            _arg(out_lengths, i32, (B,), dev, "out_lengths"))
    return out_nodes, out_lengths


def spec_get_status(stream=None, device=None) -> int:
    """Synchronise and return (then clear) the device status word: an OR of
    SPEC_FLAG_BAD_DATA / SPEC_FLAG_TIMEOUT set since the last read."""
    import ctypes
    flags = ctypes.c_uint32(0)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        _lib.check(_lib.load().spec_get_status(_stream(stream), ctypes.addressof(flags)))
    return int(flags.value)


def spec_test_spin_limit(iterations: int, device=None) -> None:
    """Test hook for failure-detection tests: every bounded wait inside the
    kernels of later calls on the device gives up after `iterations` polls and
    flags SPEC_FLAG_TIMEOUT; 0 restores the default limit.  Synchronises the
    device first."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        _lib.check(_lib.load().spec_test_spin_limit(int(iterations)))


def spec_test_wait_probe(device=None) -> tuple:
    """Test hook: runs every bounded-wait helper of the library on a slot that
    nothing writes and on one already written, under the current limit.
    Returns (helpers that gave up on the unwritten slot, helpers that flagged
    the written one) as bit masks; a correct library gives (0x7f, 0)."""
    import ctypes
    flags = (ctypes.c_uint32 * 2)()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        _lib.check(_lib.load().spec_test_wait_probe(ctypes.addressof(flags)))
    return int(flags[0]), int(flags[1])
