"""Paged attention of batches that mix single tokens and chunks, and of caches whose elements pass
32 bits."""
import numpy as np
import pytest
import torch

import block_sparse_attention_selected_b200 as nsa
from paged_util import make_case
from test_gpu_paged import check, cuda, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq, hkv, d", [(32, 8, 128), (8, 8, 64), (64, 2, 128)])
@pytest.mark.parametrize("singles, chunk, behind", [(63, 128, 2000), (200, 512, 1500), (15, 600, 900), (3, 900, 0)])
def test_single_tokens_and_a_chunk(singles, chunk, behind, hq, hkv, d):
    rng = np.random.default_rng(singles)
    q_lens = [1] * singles
    kv_lens = rng.integers(1, 1200, singles).tolist()
    at = singles // 2
    q_lens.insert(at, chunk)
    kv_lens.insert(at, chunk + behind)
    q_lens.append(0)
    kv_lens.append(77)
    run(make_case(q_lens, kv_lens, hq, hkv, d, 64, seed=1, pad=9))


@pytest.mark.parametrize("window", [0, 300])
def test_single_tokens_and_a_chunk_of_selected_blocks(window):
    run(make_case([1] * 40 + [200] + [1] * 20, [900] * 40 + [1500] + [64] * 20, 16, 2, 128, 64, seed=2, topk=6,
                  window=window, pad=3))


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("topk", [0, 5])
def test_a_cache_whose_elements_pass_32_bits(topk, heads_first):
    c = make_case([1, 30, 2], [300, 500, 64], 16, 8, 128, 64, seed=3, topk=topk, poison=False)
    small, (pages, ps, hkv, d) = [c["k"], c["v"]], c["k"].shape
    many = 65536 + 2000                       # 65536 pages are 2^32 elements
    shape = (many, hkv, ps, d) if heads_first else (many, ps, hkv, d)
    big = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    if heads_first:
        big = [x.permute(0, 2, 1, 3) for x in big]
    # page p of the small cache lies at one end or the other of the big one
    to = np.where(np.arange(pages) % 2 == 0, many - 1 - np.arange(pages), np.arange(pages))
    slots = (to[:, None] * ps + np.arange(ps)).reshape(-1)
    nsa.nsa_sel_paged_write_kv(*(cuda(x.reshape(-1, hkv, d)) for x in small), cuda(slots), *big)
    for x, y in zip(small, big):
        assert torch.equal(y[cuda(to)].cpu(), x)
    held = (c["table"] >= 0) & (c["table"] < pages)
    table = np.where(held, to[np.where(held, c["table"], 0)], -1).astype(np.int32)
    args = [cuda(c["q"]), *big, cuda(c["cu"]), cuda(c["kv"]), cuda(table)]
    if topk:
        got = nsa.nsa_sel_paged_sel_fwd(*args, cuda(c["idx"]), c["bs"], scale=c["scale"])
    else:
        got = nsa.nsa_sel_paged_attn_fwd(*args, scale=c["scale"])
    assert nsa.nsa_sel_check_status() == 0
    check(c, got)
