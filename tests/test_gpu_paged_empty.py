"""Paged attention where many units see no key: padded requests, queries before the first key,
rows that select nothing, in runs that are longer than a CTA's ring of pieces."""
import numpy as np
import pytest
import torch

import block_sparse_attention_selected_b200 as nsa
from paged_util import make_case
from test_gpu_paged import attend, cuda, run, tensors

pytestmark = pytest.mark.gpu


def places(order, empty, real):
    """`empty` and `real` in one list: the empty ones before, between or after."""
    if order == "before":
        return empty + real
    if order == "after":
        return real + empty
    half, some = len(empty) // 2, len(real) // 2
    return real[:some] + empty[:half] + real[some:-1] + empty[half:] + real[-1:]


@pytest.mark.parametrize("order", ["before", "between", "after"])
@pytest.mark.parametrize("hq, hkv, d", [(32, 8, 128), (16, 8, 64), (256, 8, 128), (160, 8, 64)])
def test_decode_batch_padded_with_requests_without_a_key(hq, hkv, d, order):
    kv = places(order, [0] * 56, [8192, 300, 5000, 1, 8192, 128, 129, 4000])
    got = run(make_case([1] * 64, kv, hq, hkv, d, 64, seed=1))
    for r in np.flatnonzero(np.array(kv) == 0):
        assert torch.all(got[0][r] == 0) and torch.all(torch.isneginf(got[1][:, r]))


@pytest.mark.parametrize("order", ["before", "between", "after"])
def test_many_requests_without_a_key(order):
    run(make_case([1] * 256, places(order, [0] * 250, [2000, 64, 900, 7, 1, 130]), 8, 8, 128, 16, seed=2))


@pytest.mark.parametrize("order", ["before", "between", "after"])
@pytest.mark.parametrize("q_len, hq, d", [(16, 32, 128), (16, 32, 64), (64, 32, 128), (64, 32, 64)],
                         ids=["one_tile_128", "one_tile_64", "two_tiles_128", "two_tiles_64"])
def test_chunks_before_the_first_key(q_len, hq, d, order):
    # every fourth request of those sees its first keys with its last queries
    empty = [3 if i % 16 == 0 else 0 for i in range(60)]
    run(make_case([q_len] * 64, places(order, empty, [12000, 3000, 900, 200]), hq, 8, d, 64, seed=3, pad=2))


def test_a_long_chunk_before_its_first_key():
    run(make_case([6000, 6000, 1], [100, 0, 700], 32, 2, 64, 64, seed=4))


@pytest.mark.parametrize("hq, d", [(8, 128), (8, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("rows", ["none", "runs", "ends"])
def test_selected_rows_without_a_block(rows, hq, d):
    T = 640
    c = make_case([T], [1500], hq, 4, d, 64, seed=5, topk=3, poison=False)
    t = np.arange(T)
    bare = {"none": t >= 0, "runs": (t % 200) < 170, "ends": (t < 300) | (t > 340)}[rows]
    c["idx"][bare] = np.where(t[bare] % 2 == 0, -1, 900)[:, None, None]     # pads, and blocks of the future
    got = run(c)
    bare = torch.from_numpy(bare).cuda()
    assert torch.all(got[0][bare] == 0) and torch.all(torch.isneginf(got[1][:, bare]))


@pytest.mark.parametrize("topk", [0, 3])
def test_requests_that_overlap_are_refused(topk):
    c = make_case([3, 2, 3], [300, 90, 200], 8, 2, 64, 64, seed=6, topk=topk, poison=False)
    ts = list(tensors(c))
    ts[3] = cuda(np.array([0, 6, 1, 8], np.int32))
    attend(c, ts)
    assert nsa.nsa_sel_check_status() == 6
    run(c)


def test_requests_that_overlap_by_more_than_their_sums_hold():
    # every other request has all rows: 2^31 units of one token
    T, R, hq, d = 1 << 18, 16384, 128, 64
    q = torch.zeros(T * 8 + hq * d, dtype=torch.bfloat16, device="cuda").as_strided((T, hq, d), (8, 8, 1))
    k, v = (torch.zeros(4, 16, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    kv = torch.full((R,), 64, dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").expand(R, 4).contiguous()
    out = torch.full((T, hq, d), 77.0, dtype=q.dtype, device="cuda")
    nsa.nsa_sel_paged_attn_fwd(q, k, v, cu, kv, table, out=out, with_lse=False)
    assert nsa.nsa_sel_check_status() == 6
    assert bool((out == 77.0).all())
