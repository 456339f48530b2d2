"""The paged K/V cache on the GPU against the fp64 oracle (oracle/paged.py)."""
import numpy as np
import pytest
import torch

import block_sparse_attention_selected_b200 as nsa
from block_sparse_attention_selected_b200 import paged as npaged
from oracle import paged as po
from paged_util import DTYPES, make_case, oracle_of, rounded, tolerances

pytestmark = pytest.mark.gpu


def cuda(x):
    return torch.as_tensor(x).cuda()


def tensors(c):
    return (cuda(c["q"]), cuda(c["k"]), cuda(c["v"]), cuda(c["cu"]), cuda(c["kv"]), cuda(c["table"]))


def attend(c, ts=None, **kw):
    q, k, v, cu, kv, table = tensors(c) if ts is None else ts
    if c["idx"] is not None:
        return nsa.nsa_sel_paged_sel_fwd(q, k, v, cu, kv, table, cuda(c["idx"]), c["bs"], scale=c["scale"],
                                         window_size=c["window"], **kw)
    return nsa.nsa_sel_paged_attn_fwd(q, k, v, cu, kv, table, scale=c["scale"], window_size=c["window"], **kw)


def check(c, got, ref=None):
    ref = oracle_of(c) if ref is None else ref
    tol, ltol = tolerances(c, ref)
    n = int(c["cu"][-1])
    o = got[0].double().cpu().numpy()[:n]
    assert np.all(np.isfinite(o))
    over = np.abs(o - ref[0][:n]) - tol[:n]
    assert over.max(initial=-1.0) <= 0, (float(over.max()), np.argwhere(over > 0)[:5].tolist(), int((over > 0).sum()))
    if got[1] is not None:
        lse, rl = got[1].double().cpu().numpy()[:, :n], ref[1][:, :n]
        assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
        fin = np.isfinite(rl)
        assert np.all(np.abs(lse[fin] - rl[fin]) <= ltol[:, :n][fin])


def run(c, **kw):
    # outputs start as a value no row has, so that rows left as they were can be told
    out = torch.full(c["q"].shape, 77.0, dtype=c["q"].dtype, device="cuda")
    lse = torch.full((c["q"].shape[1], c["T"]), 77.0, device="cuda")
    got = attend(c, out=out, lse=lse, **kw)
    assert got[0] is out and got[1] is lse
    assert nsa.nsa_sel_check_status() == 0
    n = int(c["cu"][-1])
    assert torch.all(out[n:] == 77.0) and torch.all(lse[:, n:] == 77.0)
    check(c, got)
    return got


# lengths (new, in the cache): one token, whole prompts, chunks, requests without new tokens,
# ends inside a tile and inside a page
LENS = {
    "one": ([1], [1]),
    "decode": ([1, 1, 1, 1], [1, 63, 64, 65]),
    "decode_long": ([1, 1, 1], [2049, 700, 128]),
    "holes": ([0, 1, 0, 0, 3, 1, 0], [5, 130, 0, 64, 100, 17, 300]),
    "prompt": ([130, 1, 64], [130, 1, 64]),
    "chunk": ([100, 33, 1], [357, 290, 1000]),
    "before_first": ([5, 2], [3, 0]),
    "draft": ([3, 9, 5, 2], [700, 77, 1290, 2]),
}


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", list(LENS))
def test_attend_lengths_and_pages(lens, ps):
    run(make_case(*LENS[lens], 8, 2, 128, ps, seed=ps, pad=3))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq, hkv", [(1, 1), (2, 2), (6, 2), (4, 1), (14, 2), (16, 1), (40, 1), (128, 1), (24, 3)])
def test_attend_head_groups(hq, hkv, d):
    run(make_case([1, 40, 7], [150, 200, 7], hq, hkv, d, 64, seed=hq, pad=1))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 64, 70, 200, 5000])
def test_attend_window_and_types(window, d, dtype):
    run(make_case([1, 150, 1, 17], [257, 400, 900, 17], 8, 2, d, 32, dtype=dtype, seed=window, pad=2,
                  window=window))


@pytest.mark.parametrize("gain", [0.0, 0.01, 8.0, 40.0])
def test_attend_score_ranges(gain):
    # equal weights, nearly equal ones, and rows that one key dominates and whose maximum keeps growing
    run(make_case([1, 140, 12], [1500, 1400, 300], 8, 2, 128, 64, seed=7, gain=gain))


def test_attend_growing_maximum():
    # every later key scores higher, by far: each tile raises the running maximum
    c = make_case([1, 70, 200], [1300, 900, 700], 4, 2, 128, 64, seed=8, poison=False)
    c["q"].copy_(rounded(np.abs(c["q"].float().numpy()), "bf16"))
    for r, n in enumerate(c["kv"]):
        j = np.arange(n)
        c["k"][c["table"][r, j // 64], j % 64] = rounded(np.broadcast_to(
            (0.02 * j)[:, None, None], (n, 2, 128)) + 0.0, "bf16")
    run(c)


@pytest.mark.parametrize("hq, hkv, q_lens, kv_lens", [
    (8, 2, [600, 300], [900, 1111]), (4, 4, [513], [2000]), (32, 2, [129, 1, 257], [640, 3000, 257]),
    (12, 4, [701, 44], [1500, 44])])
def test_attend_long_chunks(hq, hkv, q_lens, kv_lens):
    run(make_case(q_lens, kv_lens, hq, hkv, 128, 64, seed=9, pad=5))


@pytest.mark.parametrize("q_lens, topk", [([1, 3], 0), ([100, 40], 0), ([400, 300], 0), ([5, 2], 6)])
def test_window_wider_than_any_cache(q_lens, topk):
    c = make_case(q_lens, [700, 450], 8, 2, 128, 64, seed=24, topk=topk, poison=False)
    plain = run(c)
    for window in (2 ** 31 - 1, 2 ** 31 - 128, 64 * c["table"].shape[1]):
        got = run(dict(c, window=window))
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


@pytest.mark.parametrize("q_len, hq", [(1, 8), (30, 8), (200, 8), (9, 2)])
def test_a_nan_row_of_q_stays_alone(q_len, hq):
    c = make_case([q_len, 2], [600, 130], hq, 2, 128, 64, seed=25, poison=False)
    ref = oracle_of(c)
    tol, ltol = tolerances(c, ref)
    bad = (q_len // 2, hq - 1)
    c["q"][bad] = float("nan")
    out, lse = (x.double().cpu().numpy() for x in attend(c))
    rest = np.ones(out.shape[:2], bool)
    rest[bad] = False
    assert np.all(np.isnan(out[bad])) and np.isnan(lse[bad[1], bad[0]])
    assert np.all(np.abs(out - ref[0])[rest] <= tol[rest])
    assert np.all(np.abs(lse - ref[1]).T[rest] <= ltol.T[rest])


def test_attend_many_requests():
    rng = np.random.default_rng(3)
    kv = rng.integers(1, 300, 333)
    q = np.minimum(kv, rng.integers(0, 4, 333))
    run(make_case(q.tolist(), kv.tolist(), 4, 2, 64, 16, seed=10, pad=1))


def test_attend_one_long_request_is_split():
    run(make_case([1], [20011], 4, 1, 128, 64, seed=11))
    run(make_case([2], [9000], 8, 8, 64, 128, seed=12, window=8000))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_len, group", [(1, 1), (1, 16), (5, 4), (1, 32), (11, 8)])
def test_attend_many_tiles_per_block(q_len, group, d):
    # long runs of key tiles and several units on every SM: the rings of stages, the buffers
    # and their barriers go round many times
    hkv, R = 2, 70
    rng = np.random.default_rng(q_len + group)
    kv = rng.integers(2000, 5000, R)
    kv[:5] = [300, 129, 128, 127, 11]
    run(make_case([q_len] * R, kv.tolist(), group * hkv, hkv, d, 64, seed=30 + group, poison=False))


@pytest.mark.parametrize("hq, hkv, q_lens", [(4, 4, [1] * 150), (32, 8, [3, 1, 2, 5] * 30), (64, 4, [1, 2] * 60)])
def test_attend_many_units_of_one_tile(hq, hkv, q_lens):
    # a unit's only key tile is now one stream's, now the other's
    kv = [n + (37 * i) % 120 for i, n in enumerate(q_lens)]
    for seed in range(3):
        run(make_case(q_lens, kv, hq, hkv, 128, 16, seed=40 + seed))


# ------------------------------------------------------------------------ selected blocks

@pytest.mark.parametrize("bs", [64, 128])
@pytest.mark.parametrize("ps", [16, 64, 128, 256])
@pytest.mark.parametrize("lens", list(LENS))
def test_select_lengths_and_pages(lens, ps, bs):
    run(make_case(*LENS[lens], 8, 2, 128, ps, seed=ps + bs, pad=3, topk=5, bs=bs))


@pytest.mark.parametrize("dtype, d, topk, window, hq, hkv", [
    ("bf16", 64, 1, 0, 4, 4), ("fp16", 128, 16, 0, 16, 4), ("bf16", 128, 64, 0, 32, 2),
    ("bf16", 128, 7, 100, 6, 2), ("fp16", 64, 16, 1, 64, 1), ("bf16", 64, 33, 700, 128, 1), ("bf16", 128, 2, 64, 1, 1)])
def test_select_types_groups_and_windows(dtype, d, topk, window, hq, hkv):
    run(make_case([1, 40, 3], [5000, 300, 901], hq, hkv, d, 64, dtype=dtype, seed=topk, pad=2, topk=topk,
                  window=window))


def test_select_rows_without_a_block():
    c = make_case([3, 1], [300, 200], 8, 2, 128, 64, seed=13, topk=4, poison=False)
    c["idx"][0] = -1
    c["idx"][1, 1] = [9, 8, 7, 6]      # all of the future
    c["idx"][3, 0] = [-1, -5, 4, -1]   # below -1 and past the cache
    got = run(c)
    assert torch.all(got[0][0] == 0) and torch.all(torch.isneginf(got[1][:, 0]))


def test_select_all_blocks_equals_attend():
    c = make_case([50, 1], [333, 1000], 8, 2, 128, 64, seed=14)
    idx = np.full((51, 2, 16), -1, np.int32)
    for t in range(51):
        qb = (283 + t if t < 50 else 999) // 64
        idx[t, :, :qb + 1] = np.arange(qb + 1)[::-1]
    a = run(c)
    b = run(dict(c, idx=idx))
    ref = oracle_of(c)
    tol, _ = tolerances(c, ref)
    assert np.all(np.abs((a[0].double() - b[0].double()).cpu().numpy()) <= 2 * tol)


def test_select_many_tokens():
    run(make_case([300, 211], [2000, 211], 16, 4, 128, 64, seed=15, topk=8, pad=3))


@pytest.mark.parametrize("hq, hkv, topk", [(8, 4, 2), (64, 2, 1), (80, 2, 3), (16, 8, 16), (8, 1, 64)])
def test_select_many_units(hq, hkv, topk):
    rng = np.random.default_rng(hq)
    kv = rng.integers(1, 700, 160)
    q = np.minimum(kv, rng.integers(0, 4, 160))
    run(make_case(q.tolist(), kv.tolist(), hq, hkv, 128, 64, seed=50, topk=topk, pad=1))


# ------------------------------------------------------- layouts, streams, graphs, status

def test_attend_strided_inputs():
    c = make_case([5, 60, 1], [100, 222, 640], 8, 2, 128, 64, seed=16)
    ref = oracle_of(c)
    q, k, v, cu, kv, table = tensors(c)
    # q out of a fused projection; heads before tokens; K and V as halves of one tensor; a
    # table that is a slice of a wider one
    wide = torch.zeros(c["T"], 12, 128, dtype=q.dtype, device="cuda")
    wide[:, 2:10] = q
    kh, vh = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (k, v))
    kv2 = torch.stack([k, v], 1)
    big = torch.full((3, 40), 5, dtype=torch.int32, device="cuda")
    big[:, 3:3 + table.shape[1]] = table
    part = big[:, 3:3 + table.shape[1]]
    plain = attend(c)
    check(c, plain, ref)
    for ts in [(wide[:, 2:10], k, v, cu, kv, table), (q, kh, vh, cu, kv, table),
               (q, kv2[:, 0], kv2[:, 1], cu, kv, part)]:
        got = attend(c, ts)
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


@pytest.mark.parametrize("ps", [16, 64, 256])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,topk", [([2, 1, 0, 4], 0), ([40, 1, 9, 130], 0), ([3, 1, 12, 7], 5)],
                         ids=["few", "chunks", "selected"])
def test_attend_cache_strides(q_lens, topk, d, ps):
    # pages at a distance that is no multiple of 8 tokens, tokens and heads with gaps between
    # them, heads before tokens, K and V side by side: the same bits as packed caches
    c = make_case(q_lens, [300, 129, 17, 513], 8, 2, d, ps, seed=28, topk=topk)
    q, k, v, cu, kv, table = tensors(c)
    plain = run(c)
    pages, hkv = k.shape[0], k.shape[2]

    def placed(shape, size, strides):
        out = []
        for x in (k, v):
            y = torch.full((size,), float("nan"), dtype=x.dtype, device="cuda").as_strided(shape, strides)
            y.copy_(x)
            out.append(y)
        return out

    shape, tok = tuple(k.shape), hkv * d
    gaps = [
        placed(shape, pages * (ps * tok + 8), (ps * tok + 8, tok, d, 1)),                  # after a page
        placed(shape, pages * (ps * tok + 4 * tok), (ps * tok + 4 * tok, tok, d, 1)),      # half a group
        placed(shape, pages * (ps + 8) * tok, ((ps + 8) * tok, tok, d, 1)),                # a whole one
        placed(shape, pages * ps * (tok + 16), (ps * (tok + 16), tok + 16, d, 1)),         # after a token
        placed(shape, pages * ps * hkv * (d + 8), (ps * hkv * (d + 8), hkv * (d + 8), d + 8, 1)),
        placed(shape, pages * ps * tok, (ps * tok, d, ps * d, 1)),                         # heads first
        placed(shape, pages * hkv * (ps * d + 8), (hkv * (ps * d + 8), d, ps * d + 8, 1)),
        placed(shape, pages * ps * tok, (d, pages * tok, pages * d, 1)),                   # pages last
    ]
    both = torch.stack([k, v], 3)
    gaps.append((both[:, :, :, 0], both[:, :, :, 1]))
    for kc, vc in gaps:
        got = attend(c, (q, kc, vc, cu, kv, table))
        n = int(c["cu"][-1])
        assert nsa.nsa_sel_check_status() == 0
        assert torch.equal(got[0][:n], plain[0][:n]) and torch.equal(got[1][:, :n], plain[1][:, :n])


def test_attend_a_cache_of_one_page():
    for stride in (1, 8, 1 << 40):
        c = make_case([3], [200], 8, 2, 128, 256, seed=29)
        q, k, v, cu, kv, table = tensors(c)
        k, v = (x[int(c["table"][0, 0]):][:1] for x in (k, v))
        k, v = (x.as_strided(x.shape, (8 * stride, *x.stride()[1:])) for x in (k, v))
        check(c, nsa.nsa_sel_paged_attn_fwd(q, k, v, cu, kv, torch.zeros_like(table), scale=c["scale"]))
        assert nsa.nsa_sel_check_status() == 0


def test_attend_without_lse_and_repeats_bit_for_bit():
    for topk in (0, 6):
        c = make_case([1, 90, 1, 4], [3000, 500, 64, 1000], 8, 2, 128, 64, seed=17, topk=topk)
        ts = tensors(c)
        first = attend(c, ts)
        got = attend(c, ts, with_lse=False)
        assert got[1] is None and torch.equal(got[0], first[0])
        for _ in range(20):
            again = attend(c, ts)
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_attend_empty_batch():
    c = make_case([0, 0], [5, 0], 4, 2, 64, 16, seed=18)
    got = attend(c)
    assert got[0].shape == (0, 4, 64) and got[1].shape == (4, 0)
    assert nsa.nsa_sel_check_status() == 0


def test_two_streams_at_once():
    cs = [make_case([1] * 8, [4000 - 300 * i for i in range(8)], 8, 2, 128, 64, seed=20 + s) for s in range(2)]
    ts = [tensors(c) for c in cs]
    alone = [attend(c, t) for c, t in zip(cs, ts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(attend(cs[i], ts[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g[0], alone[i][0]) and torch.equal(g[1], alone[i][1])


def test_a_step_captured_and_replayed_with_new_lengths():
    # plan, write and both attentions in one graph; the lengths change between replays
    ps, R, T, hq, hkv, d = 16, 5, 12, 8, 2, 64
    rng = np.random.default_rng(21)
    new, old = (torch.zeros(R, dtype=torch.int32, device="cuda") for _ in range(2))
    table = torch.full((R, 20), -1, dtype=torch.int32, device="cuda")
    free = torch.zeros(60, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(100, ps, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (torch.zeros(T, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    idx = torch.tensor([0, -1], dtype=torch.int32, device="cuda").expand(T, hkv, 2).contiguous()

    def step():
        cu, kv, slots, pos, used = nsa.nsa_sel_paged_plan(new, old, free, table, ps, T)
        nsa.nsa_sel_paged_write_kv(k, v, slots, kc, vc)
        a = nsa.nsa_sel_paged_attn_fwd(q, kc, vc, cu, kv, table)
        b = nsa.nsa_sel_paged_sel_fwd(q, kc, vc, cu, kv, table, idx, 64)
        return cu, kv, slots, pos, used, a, b

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        r1 = step()
    with torch.cuda.graph(g2):
        r2 = step()
    for seed in range(4):
        o = rng.integers(0, 200, R)
        n = np.minimum(rng.integers(0, 5, R), 3)
        while n.sum() > T:
            n[rng.integers(0, R)] = 0
        have = -(-o // ps)
        perm = rng.permutation(100)
        tab = np.full((R, 20), -1, np.int32)
        at = 0
        for r in range(R):
            tab[r, :have[r]] = perm[at:at + have[r]]
            at += have[r]
        fr = np.resize(perm[at:], 60)
        new.copy_(cuda(n.astype(np.int32)))
        old.copy_(cuda(o.astype(np.int32)))
        table.copy_(cuda(tab))
        free.copy_(cuda(fr.astype(np.int32)))
        for x in (q, k, v, kc, vc):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).to(x.dtype))
        g, r = (g1, r1) if seed % 2 else (g2, r2)
        before = kc.clone(), vc.clone()
        g.replay()
        torch.cuda.synchronize()
        cu, kv, slots, pos, used, a, b = r
        ecu, ekv, eslots, epos, eused, etab = po.plan(n, o, fr, tab, ps, T)
        for x, e in ((cu, ecu), (kv, ekv), (slots, eslots), (pos, epos), (used, [eused]), (table, etab)):
            assert np.array_equal(x.cpu().numpy(), e)
        for x, y, src in ((kc, before[0], k), (vc, before[1], v)):
            want = y.view(-1, hkv, d).clone()
            want[cuda(eslots[:n.sum()])] = src[:n.sum()]
            assert torch.equal(x.view(-1, hkv, d), want)
        c = dict(q=q.cpu(), k=kc.cpu(), v=vc.cpu(), cu=ecu, kv=ekv, table=etab, idx=None, bs=64, T=T, ps=ps,
                 window=0, scale=d ** -0.5, dtype="bf16")
        check(c, a)
        check(dict(c, idx=idx.cpu().numpy()), b)


def test_calls_that_read_what_the_call_before_wrote():
    # each kernel starts under the one before it: 25 steps of two layers whose inputs are the
    # outputs of the calls just before give what they give with a wait after every call
    ps, R, hq, hkv, d, steps = 16, 3, 4, 2, 64, 25
    rng = np.random.default_rng(22)
    q0, k0, v0 = (cuda(rng.standard_normal((steps, R, h, d)).astype(np.float32)).bfloat16() for h in (hq, hkv, hkv))
    one = torch.ones(R, dtype=torch.int32, device="cuda")
    idx = torch.tensor([0, -1, 1], dtype=torch.int32, device="cuda").expand(R, hkv, 3).contiguous()

    def go(wait):
        table = torch.full((R, 8), -1, dtype=torch.int32, device="cuda")
        free = torch.arange(60, dtype=torch.int32, device="cuda")
        kc, vc = (torch.zeros(2, 60, ps, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        old = torch.full((R,), 2 * ps - 13, dtype=torch.int32, device="cuda")
        table[:, :2] = 50 + torch.arange(2 * R, device="cuda").view(R, 2)
        seen = []
        torch.cuda.synchronize()
        for i in range(steps):
            cu, old, slots, pos, used = nsa.nsa_sel_paged_plan(one, old, free[R * (i // ps):], table, ps, R)
            wait()
            x = [q0[i], k0[i], v0[i]]
            for layer in range(2):
                nsa.nsa_sel_paged_write_kv(x[1], x[2], slots, kc[layer], vc[layer])
                wait()
                out, lse = nsa.nsa_sel_paged_attn_fwd(x[0], kc[layer], vc[layer], cu, old, table)
                wait()
                out, sel_lse = nsa.nsa_sel_paged_sel_fwd(out, kc[layer], vc[layer], cu, old, table, idx, 64)
                wait()
                seen += [slots, pos, used, out, lse, sel_lse]
                x = [out, out[:, :hkv], out[:, hkv:]]
        torch.cuda.synchronize()
        assert nsa.nsa_sel_check_status() == 0
        return seen + [table, kc, vc, old]

    for x, y in zip(go(lambda: None), go(torch.cuda.synchronize), strict=True):
        assert torch.equal(x, y)


def test_bad_pages_and_lengths_are_reported():
    c = make_case([1, 3], [200, 100], 8, 2, 128, 64, seed=22, poison=False)
    ref = oracle_of(c)
    for broken in ("page", "negative", "length", "cu"):
        b = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in c.items()}
        if broken == "page":
            b["table"][0, 1] = c["k"].shape[0]
        elif broken == "negative":
            b["table"][0, 1] = -1
        elif broken == "length":
            b["kv"][0] = 64 * c["table"].shape[1] + 1
            b["table"][0] = np.clip(b["table"][0], 0, 1)
        else:
            b["cu"][2] = 9
        for topk in (0, 4):
            if topk:
                b["idx"] = np.tile(np.arange(4, dtype=np.int32), (4, 2, 1))
            got = attend(b)
            assert nsa.nsa_sel_check_status() == 6, broken
            if broken in ("page", "negative") and not topk:   # the other request is untouched by it
                tol, _ = tolerances(c, ref)
                assert np.all(np.abs(got[0].double().cpu().numpy() - ref[0])[1:] <= tol[1:])
    check(c, attend(c), ref)
    assert nsa.nsa_sel_check_status() == 0


# ----------------------------------------------------------------------- plan and write

@pytest.mark.parametrize("R, ps, hi_new, hi_old, pad, short", [
    (1, 16, 1, 1, 0, 0), (1, 64, 500, 3000, 7, 0), (3, 16, 4, 100, 2, 0), (64, 64, 2, 5000, 0, 0),
    (1000, 16, 90, 900, 33, 0), (511, 32, 5, 64, 0, 9), (513, 128, 700, 700, 1, 3), (16384, 256, 3, 300, 5, 0)])
def test_plan(R, ps, hi_new, hi_old, pad, short):
    rng = np.random.default_rng(R)
    new, old = rng.integers(0, hi_new + 1, R), rng.integers(0, hi_old + 1, R)
    have, need = -(-old // ps), -(-(old + new) // ps)
    width = int(need.max(initial=1)) + 2
    pages = rng.permutation(int(need.sum()) + 4)
    tab = np.full((R, width + 3), -9, np.int32)
    at = 0
    for r in range(R):
        tab[r, :have[r]] = pages[at:at + have[r]]
        at += have[r]
    free = pages[at:at + max(int((need - have).sum()) - short, 0) + (0 if short else 2)]
    T = int(new.sum()) + pad
    table = cuda(tab)
    got = nsa.nsa_sel_paged_plan(cuda(new.astype(np.int32)), cuda(old.astype(np.int32)),
                                 cuda(free.astype(np.int32)), table[:, :width], ps, T)
    cu, kv, slots, pos, used, etab = po.plan(new, old, free, tab[:, :width], ps, T)
    for x, e in zip(got, (cu, kv, slots, pos, [used])):
        assert np.array_equal(x.cpu().numpy(), e)
    assert np.array_equal(table[:, :width].cpu().numpy(), etab)
    assert torch.all(table[:, width:] == -9)


def test_plan_rows_that_do_not_fit():
    # the second request outgrows its row; negative lengths count as none; too few token rows
    new, old = np.array([3, 40, -5, 2]), np.array([5, 20, 7, -1])
    tab = np.array([[0, -1], [1, 2], [3, -1], [-1, -1]], np.int32)
    free = np.arange(10, 20)
    for T in (45, 50, 4, 0):
        table = cuda(tab)
        got = nsa.nsa_sel_paged_plan(cuda(new.astype(np.int32)), cuda(old.astype(np.int32)),
                                     cuda(free.astype(np.int32)), table, 16, T)
        ref = po.plan(new, old, free, tab, 16, T)
        for x, e in zip(got, (*ref[:4], [ref[4]])):
            assert np.array_equal(x.cpu().numpy(), e)
        assert np.array_equal(table.cpu().numpy(), ref[5])


@pytest.mark.parametrize("T, hkv, d, ps, fused, layout, dtype", [
    (1, 1, 64, 16, False, "nhd", "bf16"), (7, 3, 128, 32, True, "nhd", "fp16"), (300, 8, 128, 64, True, "hnd", "bf16"),
    (1025, 2, 64, 256, False, "pair", "bf16"), (5000, 4, 128, 64, True, "pair", "fp16")])
def test_write(T, hkv, d, ps, fused, layout, dtype):
    g = torch.Generator().manual_seed(T)
    pages = -(-T // ps) + 3
    mk = lambda *s: torch.randn(*s, generator=g).to(DTYPES[dtype]).cuda()
    if layout == "pair":
        both = mk(pages, 2, ps, hkv, d)
        kc, vc = both[:, 0], both[:, 1]
    elif layout == "hnd":
        kc, vc = (mk(pages, hkv, ps, d).permute(0, 2, 1, 3) for _ in range(2))
    else:
        kc, vc = mk(pages, ps, hkv, d), mk(pages, ps, hkv, d)
    if fused:
        qkv = mk(T, 4 * hkv, d)
        k, v = qkv[:, 2 * hkv:3 * hkv], qkv[:, 3 * hkv:]
    else:
        k, v = mk(T, hkv, d), mk(T, hkv, d)
    slots = torch.randperm(pages * ps, generator=g)[:T].cuda()
    slots[::5] = -1
    if T > 6:
        slots[3], slots[6] = pages * ps, 1 << 40    # past the cache: not written
    live = (slots >= 0) & (slots < pages * ps)
    want_k, want_v = kc.contiguous().view(-1, hkv, d).clone(), vc.contiguous().view(-1, hkv, d).clone()
    want_k[slots[live]], want_v[slots[live]] = k[live], v[live]
    nsa.nsa_sel_paged_write_kv(k, v, slots, kc, vc)
    assert torch.equal(kc.contiguous().view(-1, hkv, d), want_k)
    assert torch.equal(vc.contiguous().view(-1, hkv, d), want_v)


@pytest.fixture(params=["compiled", "python"])
def marshalling(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(npaged, "_bind", False)
    else:
        assert npaged._plain(torch.zeros(1, device="cuda")), "_paged_bind.so was not built"


def test_both_marshallings_agree(monkeypatch):
    for topk, window, dtype in ((0, 0, "bf16"), (3, 70, "fp16")):
        c = make_case([1, 30, 0, 2], [300, 200, 5, 64], 6, 2, 64, 32, dtype=dtype, seed=26, topk=topk, pad=3,
                      window=window)
        ts = tensors(c)
        new, old = cuda(np.array([2, 0, 40], np.int32)), cuda(np.array([5, 7, 30], np.int32))
        free = cuda(np.arange(20, 30, dtype=np.int32))
        rows = torch.randn(5, 2, 64, device="cuda").to(DTYPES[dtype])
        slots = torch.tensor([3, -1, 40, 7, 0], device="cuda")
        got = []
        for bind in (None, False):
            monkeypatch.setattr(npaged, "_bind", bind)
            table = torch.tensor([[1, -1, -1], [2, -1, -1], [3, -1, -1]], dtype=torch.int32, device="cuda")
            k, v = ts[1].clone().nan_to_num(), ts[2].clone().nan_to_num()
            nsa.nsa_sel_paged_write_kv(rows, 2 * rows, slots, k, v)
            lse = torch.zeros(6, c["T"], device="cuda")
            out = torch.zeros(c["q"].shape, dtype=DTYPES[dtype], device="cuda")
            a = attend(c, ts, out=out, lse=lse)
            assert a[0] is out and a[1] is lse
            n = int(c["cu"][-1])
            b = attend(c, ts)
            d = attend(c, ts, with_lse=False)
            assert d[1] is None and torch.equal(d[0][:n], out[:n])
            assert torch.equal(b[0][:n], out[:n]) and torch.equal(b[1][:, :n], lse[:, :n])
            got.append([*nsa.nsa_sel_paged_plan(new, old, free, table, 32, 44), table, k, v, out, lse])
        for x, y in zip(*got):
            assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y)


def test_small_cached_workspace_is_grown():
    nsa.release_workspaces()
    c = make_case([1], [50], 4, 2, 64, 16, seed=27)
    nsa.get_workspace(256, "cuda")
    check(c, attend(c))
    assert nsa.nsa_sel_check_status() == 0


def test_refused_workspaces(marshalling):
    c = make_case([2], [50], 4, 2, 64, 16, seed=24)
    args = tensors(c)
    nbytes = nsa.nsa_sel_paged_attn_workspace_size(2, 1, 4, 2, 64)
    good = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    for bad in [torch.empty(nbytes, dtype=torch.uint8), good[None], torch.empty(2 * nbytes, dtype=torch.uint8,
                                                                             device="cuda")[::2]]:
        with pytest.raises(ValueError):
            nsa.nsa_sel_paged_attn_fwd(*args, workspace=bad)
    with pytest.raises(TypeError):
        nsa.nsa_sel_paged_attn_fwd(*args, workspace=good.view(torch.int32))
    with pytest.raises(nsa.NsaError):     # not aligned
        nsa.nsa_sel_paged_attn_fwd(*args, workspace=torch.empty(nbytes + 16, dtype=torch.uint8, device="cuda")[16:])
    nsa.nsa_sel_paged_attn_fwd(*args, workspace=good)


def test_binding_refusals_on_the_device(marshalling):
    c = make_case([2], [50], 4, 2, 64, 16, seed=23)
    q, k, v, cu, kv, table = tensors(c)
    f = nsa.nsa_sel_paged_attn_fwd
    for bad in [(q, k, v[:2], cu, kv, table), (q, k, v, cu[:1], kv, table), (q, k, v, cu, kv, table[:, ::2]),
                (q, k, v.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), cu, kv, table),
                (q[..., :32], k, v, cu, kv, table), (q.transpose(1, 2), k, v, cu, kv, table),
                (q, k.cpu(), v, cu, kv, table), (q[0], k, v, cu, kv, table)]:
        with pytest.raises(ValueError):
            f(*bad)
    for bad in [(q, k.half(), v, cu, kv, table), (q, k, v, cu.long(), kv, table), (q, k, v, cu, kv, table.long())]:
        with pytest.raises(TypeError):
            f(*bad)
    with pytest.raises(nsa.NsaError):
        f(torch.zeros(2, 5, 64, dtype=q.dtype, device="cuda"), k, v, cu, kv, table)
    with pytest.raises(nsa.NsaError):
        f(q, k, v, cu, kv, table, scale=-1.0)
    with pytest.raises(nsa.NsaError):
        f(q, k, v, cu, kv, table, workspace=torch.empty(128, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        nsa.nsa_sel_paged_sel_fwd(q, k, v, cu, kv, table, torch.zeros(2, 1, 3, dtype=torch.int32, device="cuda"), 64)
