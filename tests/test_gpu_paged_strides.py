"""Strides that the paged calls do not look at, and those that they refuse."""
import pytest
import torch

import block_sparse_attention_selected_b200 as nsa
from block_sparse_attention_selected_b200 import paged as npaged
from paged_util import make_case
from test_gpu_paged import attend, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["compiled", "python"], autouse=True)
def marshalling(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(npaged, "_bind", False)


def odd(t, *dims):
    """t with strides of 3 over its dimensions of one element."""
    strides = list(t.stride())
    for i in dims:
        assert t.shape[i] == 1
        strides[i] = 3
    return t.as_strided(t.shape, strides)


@pytest.mark.parametrize("topk", [0, 3])
def test_dimensions_of_one_element(topk):
    c = make_case([1], [200], 1, 1, 128, 256, seed=1, topk=topk)
    q, k, v, cu, kv, table = tensors(c)
    want = attend(c, (q, k, v, cu, kv, table))
    page = int(c["table"][0, 0])
    k, v, table = k[page:page + 1], v[page:page + 1], torch.zeros_like(table)
    for ts in [(odd(q, 0, 1), odd(k, 0, 2), odd(v, 0, 2), cu, kv, table),
               (q, odd(k, 0), odd(v, 2), cu, kv, table)]:
        got = attend(c, ts)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert nsa.nsa_sel_check_status() == 0


def test_write_dimensions_of_one_element():
    k, v = (torch.randn(1, 1, 64, device="cuda").bfloat16() for _ in range(2))
    kc, vc = (torch.zeros(1, 16, 1, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    slot = torch.tensor([5], device="cuda")
    nsa.nsa_sel_paged_write_kv(odd(k, 0, 1), odd(v, 0, 1), slot, odd(kc, 0, 2), odd(vc, 0))
    assert torch.equal(kc[0, 5], k[0]) and torch.equal(vc[0, 5], v[0])
    assert int((kc != 0).sum()) == int((k != 0).sum())


def test_a_row_repeated_is_written_for_every_token():
    row = torch.randn(1, 2, 64, device="cuda").half()
    kc, vc = (torch.zeros(2, 16, 2, 64, device="cuda", dtype=torch.float16) for _ in range(2))
    slots = torch.tensor([3, -1, 20, 31], device="cuda")
    nsa.nsa_sel_paged_write_kv(row.expand(4, 2, 64), row[:, :1].expand(4, 2, 64), slots, kc, vc)
    at = slots[slots >= 0]
    assert torch.equal(kc.view(32, 2, 64)[at], row.expand(3, 2, 64))
    assert torch.equal(vc.view(32, 2, 64)[at], row[:, :1].expand(3, 2, 64))


@pytest.mark.parametrize("topk", [0, 4])
def test_attention_reads_one_row_for_many(topk):
    c = make_case([2, 1, 40], [100, 40, 300], 4, 2, 64, 16, seed=2, topk=topk, poison=False)
    q, k, v, cu, kv, table = tensors(c)
    for a, b, e in [(q[:1].expand(q.shape), k, v), (q[:, :1].expand(q.shape), k, v),
                    (q, k[:1].expand(k.shape), v[:1].expand(v.shape)),
                    (q, k[:, :1].expand(k.shape), v[:, :1].expand(v.shape)),
                    (q, k[:, :, :1].expand(k.shape), v[:, :, :1].expand(v.shape))]:
        want = attend(c, (a.contiguous(), b.contiguous(), e.contiguous(), cu, kv, table))
        got = attend(c, (a, b, e, cu, kv, table))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert nsa.nsa_sel_check_status() == 0


def test_write_refuses_cache_rows_that_share_memory():
    k, v = (torch.randn(3, 2, 64, device="cuda").half() for _ in range(2))
    c = torch.zeros(4, 16, 2, 64, device="cuda", dtype=torch.float16)
    for one in (c[:1], c[:, :1], c[:, :, :1]):
        with pytest.raises(nsa.NsaError) as err:
            nsa.nsa_sel_paged_write_kv(k, v, torch.arange(3, device="cuda"), one.expand(c.shape), one.expand(c.shape))
        assert err.value.code == 1
    assert not c.any()
