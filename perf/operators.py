"""Serving operators over a paged K/V cache, as they are measured.

Four operators of one serving step (hq query heads over hkv KV heads, pages of
page_size tokens, a block table row per request):

  plan      block tables, slot maps and cumulative lengths from request lengths
  write     new K/V rows scattered into their cache slots
  attend    attention of each request's new tokens over its whole paged cache
            (causal, optionally with a sliding window)
  select    the same, over the key blocks that each (token, KV head) selects

``own`` false: plain torch forms.  ``own`` true: the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of a running server: 64 requests, one token each
        dict(name="plan_decode_64", op="plan", requests=64, new_lo=1, new_hi=1, kv_lo=1024,
             kv_hi=32768, page=64, pad=0, lens=1),
        # a prefill-heavy scheduler step: ragged chunks (some empty), small pages, a batch
        # padded to a fixed number of rows
        dict(name="plan_mixed_1000", op="plan", requests=1000, new_lo=0, new_hi=257, kv_lo=0,
             kv_hi=9000, page=16, pad=77, lens=2),
        # K/V of one decode step, 64 requests
        dict(name="write_decode_64", op="write", tokens=64, hkv=8, d=128, page=64, pages=2048,
             fused=False, pad=0, dtype="bf16"),
        # K/V of a prefill step, sliced out of a fused QKV projection
        dict(name="write_prefill_16k", op="write", tokens=16384, hkv=8, d=128, page=64, pages=2048,
             fused=True, pad=19, dtype="bf16"),
        # one user, one token: latency
        dict(name="attend_decode_1", op="attend", requests=1, q_lo=1, q_hi=1, kv_lo=8192,
             kv_hi=8192, hq=32, hkv=8, d=128, page=64, window=0, dtype="bf16", lens=3),
        # a decode step of 64 requests of very different lengths
        dict(name="attend_decode_64", op="attend", requests=64, q_lo=1, q_hi=1, kv_lo=512,
             kv_hi=32768, hq=32, hkv=8, d=128, page=64, window=0, dtype="bf16", lens=4),
        # a few tokens per request (checking drafted tokens), small pages, fp16
        dict(name="attend_draft_16", op="attend", requests=16, q_lo=3, q_hi=9, kv_lo=700,
             kv_hi=16000, hq=16, hkv=4, d=128, page=16, window=0, dtype="fp16", lens=5),
        # ragged chunks with a sliding window, an odd group of heads, head dimension 64
        dict(name="attend_window_8", op="attend", requests=8, q_lo=1, q_hi=701, kv_lo=701,
             kv_hi=5000, hq=12, hkv=4, d=64, page=32, window=512, dtype="bf16", lens=6),
        # a chunk of a long prompt: 2048 tokens, the last of 32768
        dict(name="attend_chunk_2k", op="attend", requests=1, q_lo=2048, q_hi=2048, kv_lo=32768,
             kv_hi=32768, hq=32, hkv=8, d=128, page=64, window=0, dtype="bf16", lens=7),
        # selected blocks, one user at a long context, one token
        dict(name="select_decode_1", op="select", requests=1, q_lo=1, q_hi=1, kv_lo=65536,
             kv_hi=65536, hq=16, hkv=4, d=128, page=64, block=64, topk=16, window=0, dtype="bf16",
             lens=8),
        # selected blocks, a decode step of 64 requests
        dict(name="select_decode_64", op="select", requests=64, q_lo=1, q_hi=1, kv_lo=2000,
             kv_hi=32768, hq=64, hkv=8, d=128, page=64, block=64, topk=16, window=0, dtype="bf16",
             lens=9),
        # selected blocks, a chunk of 512 tokens of a long prompt
        dict(name="select_chunk_512", op="select", requests=1, q_lo=512, q_hi=512, kv_lo=32768,
             kv_hi=32768, hq=64, hkv=8, d=128, page=64, block=64, topk=16, window=0, dtype="bf16",
             lens=10),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "attend", "attend", "attend", "select", "select"])
    if op == "plan":
        new_hi = _log_uniform(rng, 1, 257)
        return dict(op=op, requests=_log_uniform(rng, 1, 1000), new_lo=rng.choice([0, 1]), new_hi=new_hi,
                    kv_lo=rng.choice([0, 500]), kv_hi=_log_uniform(rng, 1000, 9000),
                    page=rng.choice([16, 32, 64, 128]), pad=rng.choice([0, 0, 13]),
                    lens=rng.randrange(1 << 20))
    if op == "write":
        return dict(op=op, tokens=_log_uniform(rng, 1, 16384), hkv=rng.choice([1, 2, 4, 8]),
                    d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), pages=2048,
                    fused=rng.random() < 0.5, pad=rng.choice([0, 0, 5]),
                    dtype=rng.choice(["bf16", "bf16", "fp16"]))
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 8, 16])
    case = dict(op=op, hq=hkv * group, hkv=hkv, d=rng.choice([64, 128, 128, 128]),
                page=rng.choice([16, 32, 64, 64, 128]), window=rng.choice([0, 0, 0, 512, 1000]),
                dtype=rng.choice(["bf16", "bf16", "fp16"]), lens=rng.randrange(1 << 20))
    if op == "attend":
        kv_hi = _log_uniform(rng, 256, 32768)
        q_hi = rng.choice([1, 1, _log_uniform(rng, 2, 16), _log_uniform(rng, 17, min(kv_hi, 2048))])
        # the padded plain form's rows x keys and the cache stay below the largest listed case's
        most = max(1, min(64, (1 << 31) // (q_hi * kv_hi * hkv * group), (1 << 23) // (kv_hi * hkv)))
        case.update(requests=_log_uniform(rng, 1, most), q_lo=1 if rng.random() < 0.5 else q_hi, q_hi=q_hi,
                    kv_lo=max(q_hi, kv_hi // rng.choice([1, 4, 16])), kv_hi=kv_hi)
    else:
        kv_hi = _log_uniform(rng, 256, 32768)
        q_hi = rng.choice([1, 1, _log_uniform(rng, 2, min(kv_hi, 512))])
        most = max(1, min(64, 512 // q_hi, (1 << 23) // (kv_hi * hkv)))
        case.update(requests=_log_uniform(rng, 1, most), q_lo=1 if rng.random() < 0.5 else q_hi, q_hi=q_hi,
                    kv_lo=max(q_hi, kv_hi // rng.choice([1, 4, 16])), kv_hi=kv_hi,
                    block=rng.choice([64, 64, 128]), topk=rng.choice([4, 8, 16]))
    return case


def _lengths(case):
    """Host lists (new tokens, tokens after the step) per request, from the case alone."""
    r = random.Random(case["lens"])
    if case["op"] == "plan":
        new = [r.randint(case["new_lo"], max(case["new_lo"], case["new_hi"])) for _ in range(case["requests"])]
        old = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in new]
        return new, [a + b for a, b in zip(new, old)]
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["requests"])]
    kv = [max(n, r.randint(case["kv_lo"], case["kv_hi"])) for n in q]
    return q, kv


def _pages(n, page):
    return -(-n // page)


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = torch.device("cuda")
    s = dict(case)
    page = case["page"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=_TYPES[case["dtype"]])

    def int32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if case["op"] == "plan":
        new, kv = _lengths(case)
        have = [_pages(b - a, page) for a, b in zip(new, kv)]
        need = [_pages(b, page) for b in kv]
        total = sum(need) + 37
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        width = max(max(need), 1) + 3
        table = torch.full((len(new), width), -1, dtype=torch.int32, device=dev)
        held = torch.arange(width, device=dev)[None, :] < int32(have)[:, None]
        table[held] = ids[:sum(have)]
        s.update(new_lens=int32(new), cached_lens=int32([b - a for a, b in zip(new, kv)]),
                 free_pages=ids[sum(have):].contiguous(), block_table=table,
                 total_tokens=sum(new) + case["pad"])
        return s
    if case["op"] == "write":
        n, hkv, d = case["tokens"], case["hkv"], case["d"]
        rows = case["pages"] * page
        slots = torch.randperm(rows, generator=g, device=dev)[:n]
        # the rows behind the last token of a padded batch have no slot
        slots = torch.cat([slots, torch.full((case["pad"],), -1, dtype=slots.dtype, device=dev)])
        if case["fused"]:   # q | k | v columns of one projection, 4 query heads per KV head
            qkv = randn(n + case["pad"], 6 * hkv, d)
            k, v = qkv[:, 4 * hkv:5 * hkv], qkv[:, 5 * hkv:]
        else:
            k, v = randn(n + case["pad"], hkv, d), randn(n + case["pad"], hkv, d)
        s.update(k=k, v=v, slots=slots, valid=n, k_cache=randn(case["pages"], page, hkv, d),
                 v_cache=randn(case["pages"], page, hkv, d))
        return s
    q_lens, kv_lens = _lengths(case)
    hkv, d = case["hkv"], case["d"]
    need = [_pages(n, page) for n in kv_lens]
    # a server's cache: the requests' pages lie scattered among others'
    ids = torch.randperm(sum(need) + 5, generator=g, device=dev).to(torch.int32)
    width = max(need) + 1
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=dev)
    table[torch.arange(width, device=dev)[None, :] < int32(need)[:, None]] = ids[:sum(need)]
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s.update(q=randn(cu[-1], case["hq"], d), k_cache=randn(sum(need) + 5, page, hkv, d),
             v_cache=randn(sum(need) + 5, page, hkv, d), cu_seqlens=int32(cu), kv_lens=int32(kv_lens),
             block_table=table, max_q=max(q_lens), max_kv=max(kv_lens), scale=float(d) ** -0.5)
    if case["op"] == "select":
        bs, topk = case["block"], case["topk"]
        req = torch.repeat_interleave(torch.arange(len(q_lens), device=dev), int32(q_lens).long())
        pos = (s["kv_lens"] - int32(q_lens))[req] + torch.arange(cu[-1], device=dev) - s["cu_seqlens"][req]
        nb = _pages(max(kv_lens), bs)
        qb = (pos // bs)[:, None, None]
        b = torch.arange(nb, device=dev)
        # the first block, the token's own and the one before it, then earlier ones at random
        score = torch.rand(cu[-1], hkv, nb, generator=g, device=dev)
        score = torch.where(b == 0, 4.0, torch.where(b == qb, 3.0, torch.where(b == qb - 1, 2.0, score)))
        score = torch.where(b <= qb, score, -1.0)
        top = torch.topk(score, min(topk, nb), dim=-1)
        idx = torch.where(top.values >= 0, top.indices, -1).to(torch.int32)
        s["block_idx"] = torch.nn.functional.pad(idx, (0, topk - idx.shape[-1]), value=-1).contiguous()
    return s


# ---------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plan, "write": _write, "attend": _attend, "select": _select}[s["op"]](s)


def _run_own(s):
    import block_sparse_attention_selected_b200 as nsa

    if s["op"] == "plan":
        cu, kv_lens, slots, positions, used = nsa.nsa_sel_paged_plan(
            s["new_lens"], s["cached_lens"], s["free_pages"], s["block_table"], s["page"], s["total_tokens"])
        return dict(cu_seqlens=cu, kv_lens=kv_lens, slots=slots, positions=positions, pages_used=used,
                    block_table=s["block_table"])
    if s["op"] == "write":
        nsa.nsa_sel_paged_write_kv(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if s["op"] == "attend":
        out, lse = nsa.nsa_sel_paged_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["cu_seqlens"], s["kv_lens"],
                                              s["block_table"], scale=s["scale"], window_size=s["window"])
    else:
        out, lse = nsa.nsa_sel_paged_sel_fwd(s["q"], s["k_cache"], s["v_cache"], s["cu_seqlens"], s["kv_lens"],
                                             s["block_table"], s["block_idx"], s["block"], scale=s["scale"],
                                             window_size=s["window"])
    return dict(out=out, lse=lse)


def _plan(s):
    new, old, page, table = s["new_lens"], s["cached_lens"], s["page"], s["block_table"]
    dev = table.device
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    cu = torch.cat([zero, torch.cumsum(new, 0)])
    have, need = (old + page - 1) // page, (old + new + page - 1) // page
    ends = torch.cumsum(need - have, 0)
    first = ends - (need - have)                       # where a request's new pages start
    col = torch.arange(table.shape[1], device=dev)[None, :]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - have[:, None]).clamp(0, max(s["free_pages"].numel() - 1, 0))
    table.copy_(torch.where(fresh, s["free_pages"][at.long()], table))
    t = torch.arange(s["total_tokens"], device=dev)
    req = torch.searchsorted(cu[1:], t, right=True)
    real = req < new.numel()
    r = req.clamp(max=new.numel() - 1)
    pos = torch.where(real, old[r] + t - cu[r], 0)
    slots = torch.where(real, table[r, (pos // page)].long() * page + pos % page, -1)
    return dict(cu_seqlens=cu.to(torch.int32), kv_lens=old + new, slots=slots, positions=pos.to(torch.int32),
                pages_used=ends[-1:].to(torch.int32), block_table=table)


def _write(s):
    n = s["valid"]
    for_k = s["k_cache"].view(-1, s["hkv"], s["d"])
    for_v = s["v_cache"].view(-1, s["hkv"], s["d"])
    for_k[s["slots"][:n]] = s["k"][:n]
    for_v[s["slots"][:n]] = s["v"][:n]
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])


def _softmax_pv(scores, keep, v):
    """(out, natural log-sum-exp) of rows of scores over the kept keys; nothing kept: 0, -inf."""
    scores = scores.masked_fill_(~keep, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(torch.where(torch.isfinite(m), m, 0.0)))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return out, (m + torch.log(total)).squeeze(-1)


def _attend(s):
    q, cu, kv = s["q"], s["cu_seqlens"], s["kv_lens"]
    T, hq, d = q.shape
    hkv, page, window = s["hkv"], s["page"], s["window"]
    G, R, M, L = hq // hkv, kv.numel(), s["max_q"], s["max_kv"]
    npages = _pages(L, page)
    table = s["block_table"][:, :npages].clamp(min=0).long()
    q_lens = cu[1:] - cu[:-1]
    key = torch.arange(npages * page, device=q.device)
    held = (key[None, :] < kv[:, None])[:, None, :, None]
    k = s["k_cache"][table].reshape(R, -1, hkv, d).permute(0, 2, 1, 3).float()
    v = s["v_cache"][table].reshape(R, -1, hkv, d).permute(0, 2, 1, 3).float().masked_fill_(~held, 0.0)
    i = torch.arange(M, device=q.device)
    row = (cu[:-1, None] + i[None, :]).clamp(max=T - 1).long()
    qp = q[row].float().reshape(R, M, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(R, hkv, G * M, d)
    pos = (kv - q_lens)[:, None] + i[None, :]
    keep = key[None, None, :] <= pos[:, :, None]
    if window:
        keep = keep & (key[None, None, :] > pos[:, :, None] - window)
    keep = keep[:, None].expand(R, G, M, -1).reshape(R, 1, G * M, -1)
    out, lse = _softmax_pv(torch.matmul(qp, k.transpose(-1, -2)).mul_(s["scale"]), keep, v)
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(cu[1:].long(), t, right=True)
    at = t - cu[r]
    out = out.view(R, hkv, G, M, d).permute(0, 3, 1, 2, 4)[r, at].reshape(T, hq, d)
    lse = lse.view(R, hkv, G, M).permute(0, 3, 1, 2)[r, at].reshape(T, hq).t().contiguous()
    return dict(out=out.to(q.dtype), lse=lse)


def _select(s):
    q, cu, kv, idx = s["q"], s["cu_seqlens"], s["kv_lens"], s["block_idx"]
    T, hq, d = q.shape
    hkv, page, bs = s["hkv"], s["page"], s["block"]
    G = hq // hkv
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(cu[1:].long(), t, right=True)
    pos = ((kv - (cu[1:] - cu[:-1]))[r] + t - cu[r])[:, None, None, None]
    key = idx[..., None].long() * bs + torch.arange(bs, device=q.device)
    keep = (idx[..., None] >= 0) & (key <= pos)
    if s["window"]:
        keep = keep & (key > pos - s["window"])
    keep, key = keep.reshape(T, hkv, -1), torch.where(keep, key, 0).reshape(T, hkv, -1)
    phys = s["block_table"][r[:, None, None], key // page].long()
    head = torch.arange(hkv, device=q.device)[None, :, None]
    k = s["k_cache"][phys, key % page, head].float()
    v = s["v_cache"][phys, key % page, head].float()
    scores = torch.matmul(q.float().view(T, hkv, G, d), k.transpose(-1, -2)).mul_(s["scale"])
    out, lse = _softmax_pv(scores, keep[:, :, None, :], v)
    return dict(out=out.reshape(T, hq, d).to(q.dtype), lse=lse.reshape(T, hq).t().contiguous())


# -------------------------------------------------------------------- what it cannot save

def work(case):
    op = case["op"]
    if op == "plan":
        new, kv = _lengths(case)
        r, fresh = len(new), sum(_pages(b, case["page"]) - _pages(b - a, case["page"]) for a, b in zip(new, kv))
        # lengths in, cumulative and total lengths out; free pages in, table entries out;
        # slot and position per row; the table entry of each request's last held page
        return {"bytes": 8 * r + 8 * r + 8 * fresh + 12 * (sum(new) + case["pad"]) + 4 * r,
                "flops": 0}
    if op == "write":
        return {"bytes": case["tokens"] * (case["hkv"] * case["d"] * 2 * 2 * 2 + 8), "flops": 0}
    q, kv = _lengths(case)
    hq, hkv, d, w = case["hq"], case["hkv"], case["d"], case["window"]
    T = sum(q)
    rows = pairs = 0
    for n, m in zip(q, kv):
        seen = [min(p + 1, w) if w else p + 1 for p in range(m - n, m)]
        if op == "select":
            most = case["topk"] * case["block"]
            seen = [min(c, most) for c in seen]
            rows += min(m, sum(seen))
        else:
            rows += min(m, n - 1 + w) if w else m
        pairs += sum(seen)
    io = T * hq * (2 * d * 2 + 4)
    index = 4 * T * hkv * case["topk"] if op == "select" else 0
    return {"bytes": io + rows * hkv * d * 2 * 2 + index + 4 * rows // case["page"] + 8 * len(q),
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the definition, 64 bits

def exact(case, seed):
    def plan(s):
        new, old = s["new_lens"].tolist(), s["cached_lens"].tolist()
        free, table, page = s["free_pages"].tolist(), s["block_table"].cpu().numpy().copy(), s["page"]
        cu, slots, positions, taken = [0], [], [], 0
        for r, (a, b) in enumerate(zip(new, old)):
            for i in range(_pages(b, page), _pages(a + b, page)):
                table[r, i] = free[taken]
                taken += 1
            cu.append(cu[-1] + a)
            positions += range(b, b + a)
            slots += [int(table[r, p // page]) * page + p % page for p in range(b, b + a)]
        pad = s["total_tokens"] - len(slots)
        return dict(cu_seqlens=np.array(cu, np.int32), kv_lens=np.array([a + b for a, b in zip(new, old)], np.int32),
                    slots=np.array(slots + [-1] * pad, np.int64), positions=np.array(positions + [0] * pad, np.int32),
                    pages_used=np.array([taken], np.int32), block_table=table)

    def write(s):
        got = {}
        for name in ("k", "v"):
            cache = s[name + "_cache"]
            flat = cache.double().reshape(-1, s["hkv"] * s["d"])
            rows = s[name].double().reshape(s["k"].shape[0], -1)
            flat.index_copy_(0, s["slots"][:s["valid"]], rows[:s["valid"]])
            got[name + "_cache"] = flat.reshape(cache.shape)
        return got

    def attention(s):
        cu, kv, page = s["cu_seqlens"].tolist(), s["kv_lens"].tolist(), s["page"]
        T, hq, d = s["q"].shape
        hkv = s["hkv"]
        G = hq // hkv
        out = torch.zeros(T, hq, d, dtype=torch.float64, device=s["q"].device)
        lse = torch.full((hq, T), -math.inf, dtype=torch.float64, device=s["q"].device)
        for r, n in enumerate(kv):
            a, b = cu[r], cu[r + 1]
            key = torch.arange(n, device=out.device)
            where = s["block_table"][r].long()[key // page] * page + key % page
            place = torch.arange(n - (b - a), n, device=out.device)
            seen = place[:, None] >= key[None, :]
            if s["window"]:
                seen &= place[:, None] - key[None, :] < s["window"]
            for g in range(hkv):
                mine = seen
                if s["op"] == "select":
                    chosen = torch.zeros(b - a, _pages(n, s["block"]) + 1, dtype=torch.bool, device=out.device)
                    pick = s["block_idx"][a:b, g].long()
                    chosen.scatter_(1, torch.where(pick < 0, chosen.shape[1] - 1, pick), True)
                    chosen[:, -1] = False
                    mine = seen & chosen[:, key // s["block"]]
                kk = s["k_cache"].reshape(-1, hkv, d)[where, g].double()
                vv = s["v_cache"].reshape(-1, hkv, d)[where, g].double()
                for h in range(g * G, (g + 1) * G):
                    z = s["scale"] * (s["q"][a:b, h].double() @ kk.T)
                    z[~mine] = -math.inf
                    total = torch.logsumexp(z, 1)
                    lse[h, a:b] = total
                    out[a:b, h] = torch.exp(z - total[:, None]).nan_to_num(0.0) @ vv
        return dict(out=out, lse=lse)

    return {"plan": plan, "write": write}.get(case["op"], attention)(prepare(case, seed))
