"""The packed calls captured into CUDA graphs: a captured call owns its workspace."""
import pytest
import torch

import block_sparse_attention_selected_b200 as nsa
import nsa_inputs as ni
from gpu_util import to_device

pytestmark = pytest.mark.gpu


def problem(lens, seed):
    p = ni.make_problem(lens, hq=8, hkv=2, block_size=64, topk=8, seed=seed)
    return p, to_device(p)


def step(p, d):
    out, lse = nsa.nsa_sel_attn_fwd(d["q"], d["k"], d["v"], d["cu"], d["bidx"], 64, p.scale)
    return (out, lse, *nsa.nsa_sel_attn_bwd(d["q"], d["k"], d["v"], out, lse, d["dout"], d["cu"], d["bidx"], 64,
                                            p.scale))


def capture(p, d, stream):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        got = step(p, d)
    return g, got


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


def test_a_replay_writes_nothing_but_its_own_memory():
    p, d = problem([700, 300], 1)
    big, bd = problem([3000], 2)
    s = torch.cuda.Stream()
    want = step(p, d)
    nsa.release_workspaces()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step(p, d)
    torch.cuda.synchronize()
    cached = dict(nsa._ws_cache)
    g, got = capture(p, d, s)
    assert len(nsa._ws_cache) == len(cached) and all(nsa._ws_cache[k] is w for k, w in cached.items())
    # the stream's cached buffer grows, the old one goes back, and other tensors take its place
    size = next(iter(cached.values())).numel()
    with torch.cuda.stream(s):
        step(big, bd)
        cached.clear()
        nsa.release_workspaces()
        fill = [torch.full((size // 4,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    for _ in range(3):
        for x in got:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(got, want)
    assert all(bool((x == 7).all()) for x in fill)


def test_graphs_of_one_stream_may_run_at_once():
    cases = [problem([900, 250], 3), problem([64, 800, 1], 4)]
    want = [step(*c) for c in cases]
    s = torch.cuda.Stream()
    graphs = [capture(*c, s) for c in cases]
    runs = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _), r in zip(graphs, runs):
            with torch.cuda.stream(r):
                g.replay()
        eager = step(*cases[0])
    torch.cuda.synchronize()
    assert same(eager, want[0])
    for (_, got), w in zip(graphs, want):
        assert same(got, w)
