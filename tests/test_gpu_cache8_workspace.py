"""The attention workspace of a context: it grows without taking away what captured
graphs hold, calls of different kinds share it without growing it in turn, and calls that
overlap have a context each."""
import gc

import pytest

from cases import spec
from test_gpu_cache8 import BF, UNSUPPORTED, Pool, i32, kvb, offsets, status_of  # noqa: F401  (kvb: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def call(P, lens, n, g, seed, n_seq=1):
    """An attention call of n tokens for each of n_seq sequences over lens keys, as a function of the context."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((1, P.H * g, n * n_seq, P.d), generator=gen, device="cuda").to(BF)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    seqs = P.kvb.Seqs(P.dtab[:1].repeat(n_seq, 1), i32(offsets([n] * n_seq)), i32([lens - n] * n_seq), max_tokens=n, max_kv=lens)

    def run(ctx=None):
        P.kvb.kvb_cache8_attention(ctx or P.ctx, P.cache, seqs, q, out, lse)
        return out, lse

    return run


def kinds(P):
    """Calls that each need more of something: few keys, partial results of many CTAs, counters, the prompt kernel."""
    return {"few": call(P, 3000, 1, 4, 1), "many": call(P, 3000, 1, 16, 2, 40), "counters": call(P, 20, 1, 1, 3, 9000),
            "prompt": call(P, 3000, 300, 2, 4)}


@pytest.mark.parametrize("first", ["few", "many", "prompt"])
def test_a_captured_call_outlives_larger_ones(kvb, first):  # noqa: F811
    P = Pool(kvb, 1, 2, 128, 16, 1, 3000)
    P.fill([3000])
    run = kinds(P)
    out, lse = run[first]()  # sizes the workspace
    kvb.kvb_ctx_check(P.ctx)
    want = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run[first]()
    for name in run:
        if name != first:
            run[name]()
            torch.cuda.synchronize()
            junk = torch.full((1 << 26,), 1e30, device="cuda")  # on what the calls may have given back
            out.zero_()
            lse.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), name
            assert bool((junk == 1e30).all()), name
            del junk
            torch.cuda.empty_cache()
    kvb.kvb_ctx_check(P.ctx)


def test_calls_of_different_kinds_do_not_grow_it_in_turn(kvb):  # noqa: F811
    P = Pool(kvb, 1, 2, 128, 16, 1, 3000)
    P.fill([3000])
    run = kinds(P)
    want = {}
    for name in run:
        want[name] = [t.clone() for t in run[name]()]
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        for name in reversed(run):
            got = run[name]()
            torch.cuda.synchronize()
            assert torch.cuda.mem_get_info()[0] == free, name
            assert all(torch.equal(a, b) for a, b in zip(got, want[name]))
    kvb.kvb_ctx_check(P.ctx)


def test_growing_on_a_captured_stream_is_refused_and_the_capture_goes_on(kvb):  # noqa: F811
    P = Pool(kvb, 1, 2, 128, 16, 1, 3000)
    P.fill([3000])
    run = kinds(P)
    few = [t.clone() for t in run["few"]()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = run["few"]()
        for name in ("many", "counters", "prompt"):
            assert status_of(kvb, run[name]) == UNSUPPORTED
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, few[0]) and torch.equal(lse, few[1])
    want = run["many"]()[0].clone()
    for _ in range(2):
        assert torch.equal(run["many"]()[0], want)
    kvb.kvb_ctx_check(P.ctx)


def test_a_context_for_each_stream_and_one_context_on_ordered_streams(kvb):  # noqa: F811
    P = Pool(kvb, 1, 2, 128, 16, 1, 3000)
    P.fill([3000])
    run = kinds(P)
    want = {}
    for name in run:
        want[name] = [t.clone() for t in run[name]()]
    torch.cuda.synchronize()

    last = {}

    def check(names):
        torch.cuda.synchronize()
        for name in names:
            assert all(torch.equal(a, b) for a, b in zip(last[name], want[name])), name

    # two contexts of one geometry over one cache, their calls side by side
    s = spec(1, 2, 128, 1e6)
    other = kvb.kvb_ctx_create(s, s, 1, 64)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for a, b in (("many", "prompt"), ("few", "counters"), ("prompt", "many")):
        for _ in range(20):
            for ctx, name, stream in ((P.ctx, a, streams[0]), (other, b, streams[1])):
                with torch.cuda.stream(stream):
                    last[name] = run[name](ctx)
        check((a, b))
    # one context, its calls on two streams in turn, each after the one before
    done = torch.cuda.Event()
    done.record()
    for i in range(20):
        for j, name in enumerate(run):
            stream = streams[(i + j) % 2]
            stream.wait_event(done)
            with torch.cuda.stream(stream):
                last[name] = run[name]()
                done = torch.cuda.Event()
                done.record()
    check(run)
    kvb.kvb_ctx_check(P.ctx)
    kvb.kvb_ctx_check(other)


def test_a_context_that_is_collected_during_a_capture_does_not_end_it(kvb):  # noqa: F811
    P = Pool(kvb, 1, 2, 128, 16, 1, 3000)
    P.fill([3000])
    run = kinds(P)
    want = [t.clone() for t in run["few"]()]
    s = spec(1, 2, 128, 1e6)
    gc.collect()
    gc.disable()
    try:
        left = [kvb.kvb_ctx_create(s, s, 1, 64)]
        left.append(left)
        del left  # a cycle: only the collector finds the context
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, lse = run["few"]()
            assert gc.collect() > 0
    finally:
        gc.enable()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    kvb.kvb_ctx_check(P.ctx)
