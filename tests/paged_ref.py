"""64-bit plain implementations of the paged cache's operators, and the bounds their GPU results
are held to.

Bounds.  With u the half step of the 16-bit type (fp16 2^-11, bf16 2^-8) and everything else in
fp32 (half step 2^-24):
  * a score's error: the fp32 dot product of D exact 16-bit products is off by at most
    (D + 1) 2^-24 sum|q_d k_d|, its scaling, cap, bias and the subtraction of the reference by a
    few 2^-24 of the magnitudes involved; a tanh computed to 2^-22 absolute moves the score by
    cap 2^-22.  `score_error` is the largest of these over the row's visible keys.
  * lse: the score error, plus the relative error of a sum of n fp32 terms (n 2^-24) and of the
    hardware exp2 and log2 (2^-21 together, and 2^-22 of the value).
  * O: each p carries twice the score error (its own and the sum's), u from its rounding to 16
    bits, and for fp16 at most 2^-25 absolute where it is subnormal (the largest p of a row's tile is
    of order 1, so relative to the sum this is 2^-25); each moves O by that share of A = sum p |v| / l (or of
    sum |v|).  The sums are fp32 (n 2^-24), and the result is rounded once (u |O|).
  * mass: every term e^(s - lse) carries the score error and the exp2's; the sum n 2^-24.
"""
import numpy as np
import torch

import oracle
from exact_causal_attention_gb300 import inputs

HALF = {"fp16": torch.finfo(torch.float16).eps / 2, "bf16": torch.finfo(torch.bfloat16).eps / 2}
F32 = torch.finfo(torch.float32).eps / 2


def f64(t, dtype):
    """A CPU 16-bit tensor's values in float64 numpy, by the oracle's own decoder."""
    return oracle.decode(inputs.bits(t), dtype).reshape(t.shape)


def gather(cache64, table, b, length, T):
    """K and V [length, Hkv, D] of request b; tokens of pages out of range are marked in the mask."""
    P = cache64.shape[0]
    j = np.arange(length)
    page = table[b, j // T].astype(np.int64) if length else np.zeros(0, np.int64)
    ok = (page >= 0) & (page < P)
    page = np.where(ok, page, 0)
    return cache64[page, 0, j % T], cache64[page, 1, j % T], ok


def visible(pos, length, window, prefix):
    """[rows, length]: which keys the rows at these positions see."""
    j = np.arange(length)[None, :]
    p = np.asarray(pos)[:, None]
    seen = j <= p
    if window:
        seen &= j > p - window
    return seen | (j < prefix)


def scores(q, k, pos, scale, softcap, slope):
    """Scores [rows, keys] of one head and a bound on their fp32 error."""
    dot = q @ k.T
    s = dot * scale
    err = (q.shape[1] + 4) * F32 * (np.abs(q) @ np.abs(k).T) * scale
    if softcap:
        s = softcap * np.tanh(s / softcap)
        err = err + softcap * 4 * F32
    if slope:
        away = slope * np.abs(np.asarray(pos)[:, None] - np.arange(len(k))[None, :])
        s = s - away
        err = err + 4 * F32 * away
    return s, err + 4 * F32 * np.abs(s)


def attention(q, cache, table, lengths, offsets, T, dtype, scale, softcap=0.0, slopes=None, window=0, prefix=None):
    """(O [total,Hq,D], lse [total,Hq], bound on O, bound on lse), rows of no request NaN."""
    q, cache = f64(q, dtype), np.nan_to_num(f64(cache, dtype))
    table, lengths, offsets = table.numpy(), lengths.tolist(), offsets.tolist()
    total, Hq, D = q.shape
    Hkv = cache.shape[3]
    u = HALF[dtype]
    o, tol_o = np.full((total, Hq, D), np.nan), np.full((total, Hq, D), np.nan)
    lse, tol_l = np.full((total, Hq), np.nan), np.full((total, Hq), np.nan)
    for b, L in enumerate(lengths):
        r0, r1 = offsets[b], offsets[b + 1]
        if r1 == r0:
            continue
        pos = np.arange(L - (r1 - r0), L)
        k, v, ok = gather(cache, table, b, L, T)
        seen = visible(pos, L, window, int(prefix[b]) if prefix is not None else 0) & ok[None, :]
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            s, err = scores(q[r0:r1, h], k[:, kv], pos, scale, softcap, float(slopes[h]) if slopes is not None else 0.0)
            s = np.where(seen, s, -np.inf)
            top = s.max(1, initial=-np.inf)
            live = top > -np.inf
            p = np.exp(s - np.where(live, top, 0.0)[:, None])
            l = p.sum(1)
            w = p / np.where(live, l, 1.0)[:, None]
            vh = v[:, kv]
            n = seen.sum(1)
            e = np.where(seen, err, 0.0).max(1, initial=0.0)
            o[r0:r1, h] = w @ vh
            with np.errstate(divide="ignore"):
                lse[r0:r1, h] = np.where(live, top + np.log(np.where(live, l, 1.0)), -np.inf)
            mag = np.abs(np.where(live, lse[r0:r1, h], 0.0))
            tol_l[r0:r1, h] = e + n * F32 + 8 * F32 + 4 * F32 * mag + 1e-30
            A = w @ np.abs(vh)
            sub = 2.0 ** -25 * (seen @ np.abs(vh)) if dtype == "fp16" else 0.0
            tol_o[r0:r1, h] = (2 * e + n * F32 + u + 16 * F32)[:, None] * A + sub + u * np.abs(o[r0:r1, h]) + 1e-7
    return o, lse, tol_o, tol_l


def mass(q, lse, cache, table, lengths, offsets, T, dtype, scale, softcap=0.0, slopes=None, window=0, prefix=None):
    """(mass [B,Hkv,max_pages T], bound), from the given float32 lse."""
    q, cache = f64(q, dtype), np.nan_to_num(f64(cache, dtype))
    table, lengths, offsets, lse = table.numpy(), lengths.tolist(), offsets.tolist(), lse.double().numpy()
    Hq, Hkv = q.shape[1], cache.shape[3]
    out = np.zeros((len(lengths), Hkv, table.shape[1] * T))
    tol = np.zeros_like(out)
    for b, L in enumerate(lengths):
        r0, r1 = offsets[b], offsets[b + 1]
        pos = np.arange(L - (r1 - r0), L)
        k, _, ok = gather(cache, table, b, L, T)
        seen = visible(pos, L, window, int(prefix[b]) if prefix is not None else 0) & ok[None, :]
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            s, err = scores(q[r0:r1, h], k[:, kv], pos, scale, softcap, float(slopes[h]) if slopes is not None else 0.0)
            z = lse[r0:r1, h][:, None]
            z = np.where(z == -np.inf, np.inf, z)
            term = np.where(seen, np.exp(s - z), 0.0)
            out[b, kv, :L] += term.sum(0)
            # the difference s - lse is rounded at the magnitude of either
            per = err + 4 * F32 * np.where(np.isfinite(z), np.abs(z), 0.0) + 16 * F32 + (r1 - r0) * (Hq // Hkv) * F32
            tol[b, kv, :L] += (term * per).sum(0)
    return out, tol * 1.01 + 1e-30


def evict(cache, table, lengths, mass, budget, recent, T):
    """(cache, kept, new lengths, mass out) after the eviction: exact, in any type."""
    cache, m = cache.clone(), mass.clone()
    B, Hkv, most = m.shape
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    out = torch.zeros_like(m)
    lens = []
    for b in range(B):
        L = int(lengths[b])
        n = min(L, budget)
        lens.append(n)
        tail = min(recent, n)
        for h in range(Hkv):
            vals = m[b, h, :L - tail].tolist()
            order = sorted(range(len(vals)), key=lambda j: (vals[j] != vals[j], -vals[j] if vals[j] == vals[j] else 0.0, j))
            src = torch.tensor(sorted(order[:n - tail]) + list(range(L - tail, L)), dtype=torch.int64)
            dst = torch.arange(n)
            kept[b, h, :n] = src.to(torch.int32)
            out[b, h, :n] = m[b, h][src]
            rows = cache[table[b].long()[src // T], :, src % T, h].clone()
            cache[table[b].long()[dst // T], :, dst % T, h] = rows
    return cache, kept, torch.tensor(lens, dtype=torch.int32), out


def poison(cache, table, lengths, T):
    """NaN in every slot of the cache that no request's tokens cover."""
    used = torch.zeros(cache.shape[0], T, dtype=torch.bool)
    for b, L in enumerate(lengths.tolist()):
        t = torch.arange(L)
        used[table[b].long()[t // T], t % T] = True
    c = cache.clone()
    c.transpose(1, 2)[~used] = float("nan")
    return c


def chunk(B, Hq, Hkv, D, T, sizes, dtype, seed, q_std=1.0, spare_rows=0):
    """CPU inputs of a ragged chunk: sizes = [(new tokens, context), ...].  q [total + spare,Hq,D],
    the cache with its unused slots NaN, block_table (-1 past each request's pages), lengths, q_offsets."""
    _, cache, table, lens = inputs.paged_decode_inputs(B, Hq, Hkv, D, T, [c for _, c in sizes], dtype, seed)
    offsets = torch.tensor([0] + [n for n, _ in sizes]).cumsum(0).to(torch.int32)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(int(offsets[-1]) + spare_rows, Hq, D, generator=g, dtype=torch.float64) * q_std
    return q.to(torch.float32).to(inputs.TORCH_DTYPES[dtype]), poison(cache, table, lens, T), table, lens, offsets
