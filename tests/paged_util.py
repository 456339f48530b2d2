"""Inputs and error bounds shared by the tests of the paged K/V cache."""
from __future__ import annotations

import numpy as np
import torch

import nsa_inputs as ni
from oracle import paged as po

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def rounded(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(DTYPES[dtype])


def make_case(q_lens, kv_lens, hq, hkv, d, ps, dtype="bf16", seed=0, gain=1.0, pad=0, topk=0, bs=64,
              poison=True, window=0, extra_pages=3):
    """A cache whose pages are scattered.  With poison, every row that no query may see is
    NaN or infinite, table entries of pages without a visible key are garbage, and so are
    the rows of q behind the last request."""
    rng = np.random.default_rng(seed)
    R = len(q_lens)
    need = [-(-n // ps) for n in kv_lens]
    pages = sum(need) + extra_pages
    width = max(max(need), 1) + 2
    perm = rng.permutation(pages)
    table = np.full((R, width), -7, np.int32)
    table[:, -1] = 2 ** 30
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    cu = ni.cu_seqlens_from_lengths(q_lens)
    T = int(cu[-1]) + pad
    q = rounded(rng.standard_normal((T, hq, d)) * gain, dtype)
    k = rounded(rng.standard_normal((pages, ps, hkv, d)), dtype)
    v = rounded(rng.standard_normal((pages, ps, hkv, d)) + 0.25, dtype)
    if poison:
        if pad:
            q[int(cu[-1]):] = float("nan")
        dead = np.ones((pages, ps), bool)
        for r, (n, m) in enumerate(zip(q_lens, kv_lens)):
            lo = max(0, m - n - window + 1) if window > 0 else 0
            j = np.arange(lo, m if n else 0)
            dead[table[r, j // ps], j % ps] = False
            first, last = lo // ps, (m - 1) // ps
            for c in range(width):
                if n == 0 or c < first or c > last:
                    table[r, c] = (-7, 2 ** 30, pages)[c % 3]
        bad = torch.from_numpy(dead)
        k[bad] = float("nan")
        v[bad] = float("inf")
        v[bad.logical_and(torch.arange(ps)[None, :] % 2 == 0)] = float("nan")
    idx = None
    if topk:
        idx = np.full((T, hkv, topk), -1, np.int32)
        for r, (n, m) in enumerate(zip(q_lens, kv_lens)):
            for t in range(n):
                i = m - n + t
                if i < 0:
                    continue
                qb = i // bs
                for g in range(hkv):
                    c = rng.permutation(qb + 1)[:topk]
                    if rng.random() < 0.7 and qb not in c:
                        c[0] = qb
                    row = np.full(topk, -1)
                    row[rng.permutation(topk)[:len(c)]] = c   # pads in any slot
                    if rng.random() < 0.2:                    # a block of the future selects nothing
                        row[row == -1] = qb + 1 + int(rng.integers(0, 9))
                        if (row > qb).sum() > 1:
                            row[row > qb] = -1
                    idx[cu[r] + t, g] = row
    return dict(q=q, k=k, v=v, cu=cu, kv=np.array(kv_lens, np.int32), table=table, idx=idx, bs=bs, T=T,
                ps=ps, window=window, scale=float(d) ** -0.5, dtype=dtype)


def oracle_table(c):
    """The table with the garbage entries made harmless for numpy's indexing."""
    return np.clip(c["table"], 0, c["k"].shape[0] - 1)


def oracle_of(c):
    with np.errstate(invalid="ignore"):
        return po.attend(c["q"].double().numpy(), c["k"].double().numpy(), c["v"].double().numpy(), c["cu"],
                         c["kv"], oracle_table(c), c["scale"], c["window"], c["idx"], c["bs"])


def score_error(c):
    """Bound on the error of one scaled score in fp32: d products (exact) added in fp32 with
    at most one step 2^-23 of the running magnitude lost per addition, which is below
    sum |q||k| <= |q|_2 |k|_2; then one multiply-add in the exponent (2^-23 of the score,
    below the same product)."""
    q = torch.nan_to_num(c["q"].double(), 0.0, 0.0, 0.0)
    k = torch.nan_to_num(c["k"].double(), 0.0, 0.0, 0.0)
    most = float(q.norm(dim=-1).max() * k.norm(dim=-1).max()) * c["scale"]
    return (q.shape[-1] + 2) * 2.0 ** -23 * most


def tolerances(c, ref):
    """(elementwise bound for out, bound for lse).  out: one rounding of the result and one
    of each weight to the 16-bit type (half a step, eps / 2, each), the weights' relative
    error from the scores (numerator and denominator), and 2^-16 for sums in fp32, the
    exponential instruction (2 units of 2^-22) and rescaling.  In fp16 a weight below 2^-14
    of the row's largest is subnormal: up to 2^-25 absolute per key instead.  lse: the
    score's error, the logarithm's relative error of the sum."""
    out, lse, bound = ref
    half = torch.finfo(DTYPES[c["dtype"]]).eps / 2
    es = score_error(c)
    tol = half * np.abs(out) + (half + 2 * es + 2.0 ** -16) * bound * (1 + half)
    if c["dtype"] == "fp16":
        vmax = float(torch.nan_to_num(c["v"].float(), 0.0, 0.0, 0.0).abs().max())
        tol = tol + 2.0 ** -25 * vmax * max(int(c["kv"].max(initial=1)), 1) + 2.0 ** -25
    fin = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return tol, es + 2.0 ** -16 + 2.0 ** -22 * fin
