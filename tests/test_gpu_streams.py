"""Outputs that a call on another stream allocates: the memory is that stream's.
The current stream's allocator may hand out memory that its own earlier work
still reads, and takes back at once what the call has yet to write."""
import pytest
import torch

import speculative_decoding_verification_36_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
B, K, V = 3, 2, 40


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device=DEV)


def calls():
    z, q, d = torch.randn((B, K + 1, V), device=DEV), torch.randn((B, K, V), device=DEV), i32(B, K)
    zb, qb = z.bfloat16(), q.bfloat16()
    zq, par = torch.randn((B, K + 1, V), device=DEV), torch.full((B, K), -1, dtype=torch.int32, device=DEV)
    path, n = i32(B, K + 1), torch.ones(B, dtype=torch.int32, device=DEV)
    kv, cache = torch.randn((B, K + 1, 2, 16), device=DEV), torch.zeros((B, 8, 2, 16), device=DEV)
    other, table, turns = torch.zeros_like(cache), torch.arange(B, dtype=torch.int32, device=DEV)[:, None], sv.spec_rope_turns([1.0], DEV)
    return {
        "verify": lambda s: sv.spec_verify(z, q, d, 1.0, 0, stream=s),
        "early_exit": lambda s: sv.spec_verify_early_exit(z, q, d, 1.0, 0, stream=s),
        "static": lambda s: sv.spec_verify_static_scratch(zb, qb, d, 1.0, 0, stream=s),
        "stats": lambda s: tuple(sv.spec_verify_stats(z, q, d, 1.0, 0, entropy=True, stream=s).values()),
        "khint": lambda s: sv.spec_verify_khint(z, q, d, 1.0, 0, 0.5, 1.0, 1, 4, stream=s),
        "argmax": lambda s: sv.spec_verify_greedy_argmax(z, d, stream=s),
        "tree": lambda s: sv.spec_tree_verify_greedy(z, d, par, stream=s),
        "tree sampling": lambda s: sv.spec_tree_verify_sampling(z, zq, d, par, 1.0, 0, stream=s),
        "acceptance": lambda s: tuple(sv.spec_acceptance_stats(n, K, stream=s).values()),
        "ngram": lambda s: sv.spec_ngram_draft(path, n, 1, 2, 3, stream=s),
        "process": lambda s: (sv.spec_process_logits(z, d, stream=s),),
        "append": lambda s: (sv.spec_kv_append(kv, kv, cache, other, table, n, turns=turns, q=kv, stream=s),),
        "commit": lambda s: sv.spec_kv_commit(cache, other, table, n, d, par, path, n, stream=s),
    }


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("name", ["verify", "early_exit", "static", "stats", "khint", "argmax", "tree", "tree sampling", "acceptance",
                                  "ngram", "process", "append", "commit"])
def test_outputs_of_another_stream_are_its_memory(name, kind):
    call = calls()[name]
    torch.cuda.synchronize()
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(side if kind == "stream" else side.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    spans = [(t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got, a, b
    # what the current stream is given next is none of it
    for _ in range(3):
        fresh = [torch.empty(shape, dtype=dtype, device=DEV) for shape, dtype in shapes]
        for t in fresh:
            at, n = t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()
            assert all(at + n <= p or p + m <= at for p, m in spans)
    # and without a stream of their own, outputs are the current stream's as before
    with torch.cuda.stream(side):
        mine = call(None)
        theirs = call(side)
    torch.cuda.synchronize()
    for a, b, c in zip(mine, theirs, want):
        assert torch.equal(a, c) and torch.equal(b, c)
    sv.spec_get_status()


def test_an_output_lets_the_current_streams_work_finish():
    """An output of another stream, used and dropped on the current one, is not
    given to that other stream while the use is pending; and a call does not
    write over memory that the current stream still reads."""
    z = torch.randn((1, 4, 1 << 18), device=DEV)
    minus, side = -z, torch.cuda.Stream()
    sv.spec_process_logits(z, out=torch.empty_like(z).copy_(z))  # kernels are loaded
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out = sv.spec_process_logits(z, stream=side)
    side.synchronize()
    at, kept, read = out.data_ptr(), torch.empty_like(out), torch.cuda.Event()
    torch.cuda._sleep(int(2e8))  # some 100 ms
    kept.copy_(out)
    read.record()
    del out
    with torch.cuda.stream(side):
        again = sv.spec_process_logits(minus)
    assert not read.query()  # the use is still pending
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    old, seen = torch.full_like(z, 3.0), torch.empty_like(z)
    torch.cuda.synchronize()
    torch.cuda._sleep(int(2e8))
    seen.copy_(old)
    del old
    new = sv.spec_process_logits(z, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept, z) and torch.equal(again, minus) and torch.equal(new, z) and bool((seen == 3).all())


def test_default_stream_by_its_handle():
    z = torch.randn((1, 4, 1000), device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out = sv.spec_process_logits(z, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, z)


def test_outputs_of_a_forked_stream_in_a_graph():
    """A captured step whose call runs on a stream that was forked from the
    capturing one: the output is the graph's memory, and a replay fills it."""
    z, side, cap = torch.randn((2, 3, 5000), device=DEV), torch.cuda.Stream(), torch.cuda.Stream()
    sv.spec_process_logits(z)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        side.wait_stream(cap)
        out = sv.spec_process_logits(z, stream=side)
        cap.wait_stream(side)
        twice = out * 2
        del out
        again = sv.spec_process_logits(twice)
    for _ in range(3):
        z.normal_()
        again.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, z * 2)
    assert sv.spec_get_status() == 0
