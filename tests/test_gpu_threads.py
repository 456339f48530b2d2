"""Calls of several Python threads on one stream: the binding keeps one workspace per stream, and
a call's kernels hand their results over through it."""
import threading

import pytest
import torch

import block_sparse_attention_selected_b200 as nsa
import nsa_inputs as ni
from gpu_util import to_device
from paged_util import make_case
from test_gpu_paged import attend, tensors

pytestmark = pytest.mark.gpu


def paged(q_lens, kv_lens, hq, seed, topk=0):
    c = make_case(q_lens, kv_lens, hq, 2, 128, 64, seed=seed, topk=topk, poison=False)
    ts = tensors(c)
    return lambda: attend(c, ts)


def packed(lens, seed):
    p = ni.make_problem(lens, hq=8, hkv=2, block_size=64, topk=8, seed=seed)
    d = to_device(p)

    def step():
        out, lse = nsa.nsa_sel_attn_fwd(d["q"], d["k"], d["v"], d["cu"], d["bidx"], 64, p.scale)
        return (out, lse, *nsa.nsa_sel_attn_bwd(d["q"], d["k"], d["v"], out, lse, d["dout"], d["cu"], d["bidx"],
                                                64, p.scale))
    return step


CALLS = {
    "paged": lambda: [paged([1, 1], [9000, 7000], 8, 1), paged([1, 1], [5000, 11000], 8, 2),
                      paged([300], [4000], 8, 3), paged([2], [6000], 64, 4)],
    "selected": lambda: [paged([1, 1], [9000, 7000], 8, 5, topk=16), paged([2, 1], [5000, 9000], 64, 6, topk=16)],
    "packed": lambda: [packed([700, 300], 7), packed([64, 900], 8)],
    "mixed": lambda: [paged([1, 1], [9000, 7000], 8, 9), packed([700, 300], 10)],
}


@pytest.mark.parametrize("kind", list(CALLS))
def test_threads_on_one_stream(kind):
    calls = CALLS[kind]()
    for f in calls:       # the workspace has its size
        f()
    want = [f() for f in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    errors = []
    start = threading.Barrier(len(calls))

    def work(i):
        try:
            start.wait(30)
            for n in range(150):
                got[i].append(calls[i]())
                if n % 25 == 24:
                    torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    assert nsa.nsa_sel_check_status() == 0
    for g, w in zip(got, want):
        for one in g:
            assert all(torch.equal(a, b) for a, b in zip(one, w, strict=True))
