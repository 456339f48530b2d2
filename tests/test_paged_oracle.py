"""Pins of the paged-cache oracle, and the host checks of the nsa_sel_paged_* calls (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_attention_selected_b200 as nsa
import nsa_inputs as ni
import oracle
from block_sparse_attention_selected_b200 import build as nsa_build
from block_sparse_attention_selected_b200 import paged as npaged
from oracle import paged as po
from paged_util import make_case, oracle_of


def test_attend_whole_prompt_equals_sdpa():
    c = make_case([37, 0, 5], [37, 9, 5], 4, 2, 32, 16, seed=1, poison=False)
    out, lse, _ = oracle_of(c)
    for r, n in enumerate(c["kv"]):
        a, b = c["cu"][r], c["cu"][r + 1]
        if a == b:
            continue
        k = torch.from_numpy(po.gather(c["k"].double().numpy(), c["table"][r], n, 16)).permute(1, 0, 2)
        v = torch.from_numpy(po.gather(c["v"].double().numpy(), c["table"][r], n, 16)).permute(1, 0, 2)
        q = c["q"][a:b].double().permute(1, 0, 2)
        ref = torch.nn.functional.scaled_dot_product_attention(
            q, k.repeat_interleave(2, 0), v.repeat_interleave(2, 0), is_causal=True)
        assert np.allclose(out[a:b], ref.permute(1, 0, 2).numpy(), rtol=0, atol=1e-12)


@pytest.mark.parametrize("window", [0, 1, 70])
def test_attend_selected_equals_the_packed_oracle(window):
    # a whole prompt in the cache is the packed problem of the library's first operator
    p = ni.make_problem([200], hq=4, hkv=2, head_dim=64, block_size=64, topk=3, seed=5, with_dout=False)
    ref, rlse = oracle.fwd(p.q, p.k, p.v, p.cu_seqlens, p.block_idx, 64, p.scale, window=window)
    table = np.random.default_rng(0).permutation(15)[None, :13]
    k, v = np.zeros((15, 16, 2, 64)), np.zeros((15, 16, 2, 64))
    j = np.arange(200)
    k[table[0, j // 16], j % 16], v[table[0, j // 16], j % 16] = p.k, p.v
    out, lse, _ = po.attend(p.q, k, v, p.cu_seqlens, [200], table, p.scale, window, p.block_idx, 64)
    assert np.allclose(out, ref, rtol=0, atol=1e-12)
    assert np.allclose(lse.T, rlse, rtol=0, atol=1e-12)


def test_attend_chunk_equals_the_end_of_the_prompt():
    whole = make_case([90], [90], 3, 1, 32, 32, seed=2, poison=False)
    ref, rlse, _ = oracle_of(whole)
    chunk = dict(whole, q=whole["q"][61:], cu=np.array([0, 29], np.int32), T=29)
    out, lse, _ = oracle_of(chunk)
    assert np.array_equal(out, ref[61:]) and np.array_equal(lse, rlse[:, 61:])


def test_attend_rows_without_a_key():
    c = make_case([4], [2], 2, 2, 32, 16, seed=3, poison=False)   # two rows before the first key
    out, lse, _ = oracle_of(c)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:, :2])) and np.all(np.isfinite(lse[:, 2:]))


def test_plan_by_hand():
    cu, kv, slots, pos, used, table = po.plan([3, 0, 1], [15, 4, 16], [9, 5, 7],
                                              [[2, -1], [3, -1], [4, -1]], 16, 6)
    assert cu.tolist() == [0, 3, 3, 4] and kv.tolist() == [18, 4, 17] and used == 2
    assert table.tolist() == [[2, 9], [3, -1], [4, 5]]
    assert slots.tolist() == [2 * 16 + 15, 9 * 16, 9 * 16 + 1, 5 * 16, -1, -1]
    assert pos.tolist() == [15, 16, 17, 16, 0, 0]


# ------------------------------------------------------------------------- host checks

@pytest.fixture(scope="module")
def lib():
    nsa_build.build()
    return nsa.load_library()


FAKE = 1 << 20   # never dereferenced: the checks fail first


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, page_stride=64 * 512, token_stride=512, head_stride=128, num_pages=8,
             page_size=64, hkv=4, head_dim=128)
    f.update(kw)
    return npaged._Cache(**f)


def attend(lib, q=FAKE, qs=(512, 128), T=3, hq=16, c=None, cu=FAKE, kv=FAKE, R=2, table=FAKE, width=4,
           stride=4, scale=0.1, window=0, out=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 30, flags=0, sel=None):
    c = cache() if c is None else c
    args = [q, *qs, T, hq, ctypes.byref(c) if c else None, cu, kv, R, table, width, stride]
    if sel is not None:
        return lib.nsa_sel_paged_sel_fwd(*args, *sel, scale, window, out, lse, ws, nbytes, None, flags)
    return lib.nsa_sel_paged_attn_fwd(*args, scale, window, out, lse, ws, nbytes, None, flags)


@pytest.mark.parametrize("kw, code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(cu=None), 1), (dict(kv=None), 1), (dict(table=None), 1),
    (dict(ws=None), 1), (dict(q=FAKE + 8), 1), (dict(ws=FAKE + 16), 1), (dict(qs=(516, 128)), 1),
    (dict(qs=(512, -128)), 1), (dict(T=-1), 1), (dict(R=0), 1), (dict(hq=6), 1), (dict(hq=0), 1),
    (dict(stride=3), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(window=-1), 1), (dict(flags=1), 1), (dict(flags=0x100), 1),
    (dict(nbytes=255), 3), (dict(R=16385), 2), (dict(T=1 << 25), 2), (dict(hq=4 * 129), 2),
    (dict(width=1 << 26, stride=1 << 26), 2),
    (dict(c=cache(head_dim=96)), 2), (dict(c=cache(page_size=24)), 2), (dict(c=cache(page_size=8)), 2),
    (dict(c=cache(k=0)), 1), (dict(c=cache(v=FAKE + 2)), 1), (dict(c=cache(num_pages=0)), 1),
    (dict(c=cache(token_stride=132)), 1), (dict(c=cache(head_stride=-128)), 1),
    (dict(sel=(FAKE, 0, 64)), 1), (dict(sel=(None, 4, 64)), 1), (dict(sel=(FAKE, 65, 64)), 2),
    (dict(sel=(FAKE, 4, 32)), 2), (dict(sel=(FAKE + 2, 4, 64)), 1),
])
def test_attention_refusals(lib, kw, code):
    assert attend(lib, **kw) == code


def test_attention_valid_arguments_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("fake pointers: only where no device can take the call")
    assert attend(lib) in (4, 7) and attend(lib, sel=(FAKE, 4, 64)) in (4, 7)


def test_workspace_size_domain(lib):
    f = lib.nsa_sel_paged_attn_workspace_size
    assert f(0, 1, 4, 4, 64) > 0 and f(100, 7, 21, 3, 128) > 0
    for bad in [(-1, 1, 4, 4, 128), (1, 0, 4, 4, 128), (1, 1, 6, 4, 128), (1, 1, 4, 4, 96),
                (1, 1, 129, 1, 128), (1 << 25, 1, 4, 4, 128), (1 << 24, 1, 128, 1, 128), (1, 16385, 4, 4, 128)]:
        assert f(*bad) == 0


@pytest.mark.parametrize("kw, code", [
    (dict(new=None), 1), (dict(R=0), 1), (dict(R=16385), 2), (dict(free=None), 1), (dict(nfree=-1), 1),
    (dict(width=0), 1), (dict(stride=3), 1), (dict(ps=48), 2), (dict(ps=0), 1), (dict(T=-1), 1),
    (dict(T=1 << 25), 2), (dict(slots=None), 1), (dict(slots=FAKE + 4), 1), (dict(width=1 << 27, stride=1 << 27), 2),
])
def test_plan_refusals(lib, kw, code):
    a = dict(new=FAKE, R=2, free=FAKE, nfree=4, width=4, stride=4, ps=64, T=3, slots=FAKE)
    a.update(kw)
    assert lib.nsa_sel_paged_plan(a["new"], FAKE, a["R"], a["free"], a["nfree"], FAKE, a["width"], a["stride"],
                                  a["ps"], a["T"], FAKE, FAKE, a["slots"], FAKE, FAKE, None) == code


@pytest.mark.parametrize("kw, code", [
    (dict(k=None), 1), (dict(v=FAKE + 8), 1), (dict(slots=None), 1), (dict(strides=(512, 128, 516, 128)), 1),
    (dict(strides=(-512, 128, 512, 128)), 1), (dict(T=-1), 1), (dict(T=1 << 25), 2),
    (dict(c=cache(head_dim=80)), 2), (dict(c=cache(page_stride=4)), 1),
])
def test_write_refusals(lib, kw, code):
    a = dict(k=FAKE, v=FAKE, strides=(512, 128, 512, 128), slots=FAKE, T=3, c=cache())
    a.update(kw)
    assert lib.nsa_sel_paged_write_kv(a["k"], a["v"], *a["strides"], a["slots"], a["T"], ctypes.byref(a["c"]),
                                      None) == code
    assert lib.nsa_sel_paged_write_kv(FAKE, FAKE, 8, 8, 8, 8, FAKE, 1, None, None) == 1


def test_binding_refuses_host_tensors_and_types():
    q, c = torch.zeros(1, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 16, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        nsa.nsa_sel_paged_attn_fwd(q, c, c, i, i[:1], i.view(1, 2))
    with pytest.raises(TypeError):
        nsa.nsa_sel_paged_attn_fwd(q.float(), c, c, i, i[:1], i.view(1, 2))
    with pytest.raises(TypeError):
        nsa.nsa_sel_paged_write_kv(q.float(), q, i.long(), c, c)
    with pytest.raises(ValueError):
        nsa.nsa_sel_paged_plan(i, i, i, i.view(1, 2), 16, 1)


def test_attention_flags(lib):
    if torch.cuda.is_available():
        pytest.skip("fake pointers: only where no device can take the call")
    # fp16, the missing arrival of the failure tests, both: taken; the other bits are not
    for sel in (None, (FAKE, 4, 64)):
        for flags in (2, 0x200, 0x202):
            assert attend(lib, flags=flags, sel=sel) in (4, 7)
        for flags in (1, 4, 0x100, 0x300, 0x400, 1 << 31):
            assert attend(lib, flags=flags, sel=sel) == 1


def test_plan_refuses_tables_whose_pages_it_cannot_count(lib):
    def call(R, width):
        return lib.nsa_sel_paged_plan(FAKE, FAKE, R, FAKE, 4, FAKE, width, width, 16, 3, FAKE, FAKE, FAKE, FAKE,
                                      FAKE, None)
    assert call(8192, 1 << 18) == 2 and call(16384, (1 << 17) - 8) == 2
    if not torch.cuda.is_available():
        assert call(16384, (1 << 17) - 9) in (4, 7)


@pytest.mark.parametrize("kw", [
    dict(qs=(0, 128)), dict(qs=(512, 0)), dict(c=cache(page_stride=0)), dict(c=cache(token_stride=0)),
    dict(c=cache(head_stride=0)), dict(sel=(FAKE, 4, 64), qs=(0, 128))])
def test_attention_reads_one_row_for_many(lib, kw):
    if torch.cuda.is_available():
        pytest.skip("fake pointers: only where no device can take the call")
    assert attend(lib, **kw) in (4, 7)


def test_write_refuses_cache_rows_that_share_memory(lib):
    for c in (cache(page_stride=0), cache(token_stride=0), cache(head_stride=0)):
        assert lib.nsa_sel_paged_write_kv(FAKE, FAKE, 512, 128, 512, 128, FAKE, 3, ctypes.byref(c), None) == 1


def test_strides_over_one_place_are_not_looked_at(lib):
    if torch.cuda.is_available():
        pytest.skip("fake pointers: only where no device can take the call")
    one = cache(hkv=1, num_pages=1, head_stride=3, page_stride=-5)
    assert attend(lib, T=1, hq=1, qs=(5, -3), c=one) in (4, 7)
    assert attend(lib, T=1, hq=1, qs=(0, 0), c=one, sel=(FAKE, 4, 64)) in (4, 7)
    assert lib.nsa_sel_paged_write_kv(FAKE, FAKE, 5, 3, -1, 0, FAKE, 1, ctypes.byref(one), None) in (4, 7)
    # a row repeated for every token or head can be read
    assert lib.nsa_sel_paged_write_kv(FAKE, FAKE, 0, 0, 512, 0, FAKE, 3, ctypes.byref(cache()), None) in (4, 7)


def test_binding_names_what_is_wrong_with_a_selection():
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for bad in (None, 3):
        with pytest.raises((TypeError, ValueError)):
            nsa.nsa_sel_paged_sel_fwd(q, bad, bad, i, i[:1], i.view(1, 2), i.view(1, 1, 2), 64)


def test_strides_of_an_empty_batch_are_not_looked_at(lib):
    if torch.cuda.is_available():
        pytest.skip("fake pointers: only where no device can take the call")
    assert attend(lib, T=0, qs=(0, 0)) in (4, 7) and attend(lib, T=0, qs=(3, -1), sel=(FAKE, 4, 64)) in (4, 7)
    assert lib.nsa_sel_paged_write_kv(FAKE, FAKE, 0, 3, -1, 0, FAKE, 0, ctypes.byref(cache()), None) in (4, 7)
