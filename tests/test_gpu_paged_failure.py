"""The paged kernels' bounded waits, made to expire without faulting the GPU: with
NSA_TEST_SKIP_ARRIVE an arrival is missing for the first CTA's first tile of K, the wait for it
expires after two billion cycles (1.02 s at 1.965 GHz), and the call has to report
NSA_ERR_TIMEOUT and leave the device and the workspace usable."""
import ctypes

import pytest
import torch

import block_sparse_attention_selected_b200 as nsa
from block_sparse_attention_selected_b200 import paged as npaged
from paged_util import make_case
from test_gpu_paged import attend, cuda, tensors

pytestmark = pytest.mark.gpu

NSA_ERR_TIMEOUT = 5
NSA_TEST_SKIP_ARRIVE = 0x200

CASES = {   # one per kernel: few rows, one tile and two tiles of rows, selected blocks of both
    "few": dict(q_lens=[1] * 20, kv_lens=[5000] * 20, hq=8, hkv=2),
    "few_one_long": dict(q_lens=[1], kv_lens=[30000], hq=4, hkv=1),
    "one_tile": dict(q_lens=[20, 9], kv_lens=[6000, 4000], hq=8, hkv=2),
    "two_tiles": dict(q_lens=[300, 200], kv_lens=[3000, 2500], hq=8, hkv=2),
    "few_selected": dict(q_lens=[30, 40], kv_lens=[3000, 2500], hq=8, hkv=2, topk=8),
    "tile_selected": dict(q_lens=[30, 40], kv_lens=[3000, 2500], hq=64, hkv=2, topk=8),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", list(CASES))
def test_expired_wait_reports_timeout_and_the_device_stays_usable(kind, d):
    c = make_case(**CASES[kind], d=d, ps=64, seed=1, poison=False)
    q, k, v, cu, kv, table = ts = tensors(c)
    ws = torch.empty(nsa.nsa_sel_paged_attn_workspace_size(c["T"], kv.numel(), q.shape[1], k.shape[2], d),
                     dtype=torch.uint8, device="cuda")
    want = attend(c, ts, workspace=ws)
    assert nsa.nsa_sel_check_status(ws) == 0
    out, lse = torch.empty_like(q), torch.empty(q.shape[1], c["T"], device="cuda")
    cache, _ = npaged._cache_arg(k, v, q.dtype, 0)
    args = [q.data_ptr(), *q.stride()[:2], c["T"], q.shape[1], ctypes.byref(cache), cu.data_ptr(), kv.data_ptr(),
            kv.numel(), table.data_ptr(), table.shape[1], table.stride(0)]
    tail = [c["scale"], 0, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream, NSA_TEST_SKIP_ARRIVE]
    lib = nsa.load_library()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    if c["idx"] is None:
        code = lib.nsa_sel_paged_attn_fwd(*args, *tail)
    else:
        idx = cuda(c["idx"])
        code = lib.nsa_sel_paged_sel_fwd(*args, idx.data_ptr(), idx.shape[2], c["bs"], *tail)
    end.record()
    assert code == 0
    assert nsa.nsa_sel_check_status(ws) == NSA_ERR_TIMEOUT
    # the wait that expires ends the others: one budget, at no less than half of the highest clock
    assert 900 < start.elapsed_time(end) < 2200
    for _ in range(3):
        got = attend(c, ts, workspace=ws)
        assert nsa.nsa_sel_check_status(ws) == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
