"""Captured verify calls without a workspace of the caller's own (GPU): their
graphs stay valid whatever eager calls follow on the stream they were captured
on, and graphs replayed at once do not meet.  Every replay equals the eager
result bit for bit."""
import pytest
import torch

from int4_output_head_amd import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def inputs(R, T, V, H, seed):
    i = synth.int_exact_inputs(R * T, V, H, seed=seed)
    h = torch.from_numpy(i["hidden"]).view(torch.float16).cuda().view(R, T, H)
    w, s = torch.from_numpy(i["packed"]).cuda(), torch.from_numpy(i["scales"]).view(torch.float16).cuda()
    g = torch.Generator().manual_seed(seed)
    d = torch.randint(0, V, (R, T - 1), generator=g, dtype=torch.int32).cuda()
    dp, un = (torch.rand(R, T - 1, generator=g).cuda() for _ in range(2))
    return h, w, s, d, dp, un


def calls(b, x):
    """One list of outputs of every entry point that takes a default workspace."""
    h, w, s, d, dp, un = x
    ids = torch.arange(w.shape[0], dtype=torch.int32, device="cuda")
    out = list(b.verify(h[0], w, s, d[0].contiguous())) + list(b.verify_batch(h, w, s, d, logits=True))
    out += b.verify_mapped(h, w, s, ids, d)
    out += b.verify_sampled(h, w, s, d, dp, un, top_k=5, want_lse=True)
    out += b.verify_ruled(h, w, s, None, d, dp, un, top_k=5, want_lse=True)
    return [t for t in out if t is not None]


def same(got, want):
    for u, v in zip(got, want):
        assert torch.equal(u, v)


@pytest.mark.parametrize("R,T", [(2, 4), (20, 4)])
def test_a_larger_eager_call_behind_a_capture(b, R, T):
    x = inputs(R, T, 3000, 128, R)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        want = [t.clone() for t in calls(b, x)]
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            out = calls(b, x)
        # needs far more than the captured calls, on the stream they were captured on
        big = inputs(40, 4, 20000, 64, 1)
        b.verify_ruled(*big[:3], None, big[3], top_k=3)
        torch.cuda.synchronize()
    kept = []
    for rep in range(3):
        kept += [torch.full((n,), rep, dtype=torch.uint8, device="cuda") for n in (1 << 16, 1 << 20, 8 << 20)]
        for t in out:
            t.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        same(out, want)
        for k, t in enumerate(kept):
            assert int((t != k // 3).sum()) == 0
        with torch.cuda.stream(side):
            same(calls(b, x), want)
        torch.cuda.synchronize()


def test_the_first_call_of_a_stream_is_captured(b):
    """Nothing has run on the stream before; its eager calls come before any
    replay, and between replays."""
    x = inputs(3, 4, 2000, 64, 5)
    want = [t.clone() for t in calls(b, x)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b._ws_cache.pop((torch.cuda.current_device(), side.cuda_stream), None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            out = calls(b, x)
    for _ in range(3):
        with torch.cuda.stream(side):
            same(calls(b, x), want)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        same(out, want)


def test_two_graphs_at_once(b):
    """Two graphs captured on one stream, replayed on two streams beside eager
    calls on the stream of their capture."""
    xs = [inputs(2, 8, 20000, 256, 7), inputs(16, 4, 20000, 256, 8)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    wants, graphs = [], []
    with torch.cuda.stream(side):
        for x in xs:
            wants.append([t.clone() for t in calls(b, x)])
        torch.cuda.synchronize()
        for x in xs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = calls(b, x)
            graphs.append((g, out))
    torch.cuda.synchronize()
    others = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for st, (g, out) in zip(others, graphs):
            with torch.cuda.stream(st):
                for t in out:
                    t.fill_(-7)
                g.replay()
        with torch.cuda.stream(side):
            eager = calls(b, xs[0])
        torch.cuda.synchronize()
        for (_, out), want in zip(graphs, wants):
            same(out, want)
        same(eager, wants[0])
