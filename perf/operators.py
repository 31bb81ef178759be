"""The measured cases of the paged-cache operators: attention of a chunk of new tokens over a
paged cache, one-token decode with capped, biased and windowed scores, the append of a chunk,
the attention weight that every cached token has received, and the eviction that goes by it.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits over a
padded batch), or, with ``own`` set, by the package's own entry point.  Sizes follow the paged
benchmark geometry (32 query heads, 8 key/value heads, head size 128, pages of 16 tokens, contexts
up to 32K) and the head layouts, page sizes and head sizes of the paged tests.
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------------ cases

def listed():
    base = dict(Hq=32, Hkv=8, D=128, T=16, dtype="fp16", cap=0.0, alibi=False, window=0, prefix=0)
    return [
        # Short follow-up turns of four chats, their history in the cache: latency counts.
        dict(base, name="prefill_turns", op="prefill", B=4, n=16, ctx=1000, spread=0.5, dtype="bf16"),
        # A serving step that mixes decoding requests with prompt chunks; capped, windowed layers.
        dict(base, name="prefill_mixed", op="prefill", B=8, n=700, ctx=16000, spread=1.0, dtype="bf16", cap=30.0,
             window=4096),
        # The last chunk of one long prompt.
        dict(base, name="prefill_long", op="prefill", B=1, n=4096, ctx=32768, spread=0.0),
        # Whole prompts in one chunk, a head per key/value head, distance bias, a visible prefix.
        dict(base, name="prefill_prompts", op="prefill", B=3, n=2500, ctx=2500, spread=0.6, Hq=16, Hkv=16, D=64, T=32,
             dtype="bf16", alibi=True, prefix=100),
        # One decode step at a long context: a capped layer with a sliding window and a few sink tokens.
        dict(base, name="decode_window", op="decode", B=8, ctx=32768, spread=0.5, dtype="bf16", cap=50.0, window=4096,
             prefix=4),
        # One decode step with a distance bias, ragged contexts, all tokens visible.
        dict(base, name="decode_bias", op="decode", B=16, ctx=8192, spread=0.9, alibi=True),
        # New tokens of a mixed step into the cache: small, and the chunk of a long prompt.
        dict(base, name="append_turns", op="append", B=8, n=16, ctx=2000, spread=0.5),
        dict(base, name="append_prompts", op="append", B=5, n=3500, ctx=8000, spread=0.7),
        # The weight that one decode step gives to each cached token.
        dict(base, name="mass_decode", op="mass", B=8, n=1, ctx=32768, spread=0.3, dtype="bf16"),
        # The weight that the last tokens of a prompt give to it, with capped scores.
        dict(base, name="mass_chunk", op="mass", B=2, n=500, ctx=12000, spread=0.4, cap=50.0),
        # Caches that have outgrown their budget: many short ones, and a long one.
        dict(base, name="evict_batch", op="evict", B=8, ctx=8192, spread=0.4, budget=2048, recent=256),
        dict(base, name="evict_long", op="evict", B=1, ctx=32768, spread=0.0, budget=4096, recent=64, D=64, T=64,
             dtype="bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["prefill", "prefill", "decode", "append", "mass", "evict"])
    Hq, Hkv = rng.choice([(32, 8), (16, 16), (8, 2), (16, 1), (12, 4), (28, 4), (6, 2)])
    c = dict(op=op, B=spread(1, 12), ctx=spread(40, 16000), spread=round(rng.uniform(0.0, 1.0), 2), Hq=Hq, Hkv=Hkv,
             D=rng.choice([64, 128]), T=rng.choice([8, 16, 32, 64]), dtype=rng.choice(["fp16", "bf16"]), cap=0.0,
             alibi=False, window=0, prefix=0)
    if op in ("prefill", "append", "mass"):
        c["n"] = min(c["ctx"], spread(1, 1500))
    if op in ("prefill", "decode", "mass"):
        c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
        c["alibi"] = rng.random() < 0.3
        c["window"] = rng.choice([0, 0, spread(16, 5000)])
        c["prefix"] = rng.choice([0, 0, spread(1, 300)])
    if op == "evict":
        c["budget"] = max(1, int(c["ctx"] * rng.uniform(0.1, 0.9)))
        c["recent"] = rng.choice([0, min(c["budget"], spread(1, 200))])
    return c


def _sizes(case):
    """(new tokens, context) of every request: the first has the case's sizes, the others shrink by
    up to `spread` (a spread of 1 leaves single tokens and short contexts among them)."""
    out = []
    for b in range(case["B"]):
        f = 1.0 - case["spread"] * ((b * 0.6180339887) % 1.0) if b else 1.0
        f2 = 1.0 - case["spread"] * ((b * 0.7548776662) % 1.0) if b else 1.0
        n = case.get("n", 1)
        n = n if b == 0 else max(1, int(n * f ** 3))
        ctx = max(n, int(case["ctx"] * f2)) if case["ctx"] > case.get("n", 1) else n
        out.append((n, ctx))
    return out


def _visible(case):
    """Visible (query, key) pairs and the distinct visible keys, summed over the requests."""
    pairs = keys = 0
    for n, ctx in _sizes(case):
        w, pre = case["window"], min(case["prefix"], ctx)
        seen = 0
        for p in range(ctx - n, ctx):
            lo = max(0, p - w + 1) if w else 0
            pairs += p + 1 - lo + min(pre, lo) + max(0, pre - (p + 1))
        lo = max(0, ctx - n - w + 1) if w else 0
        seen = ctx - lo + min(pre, lo)
        keys += seen
    return pairs, keys


def work(case):
    op, Hq, Hkv, D = case["op"], case["Hq"], case["Hkv"], case["D"]
    sizes = _sizes(case)
    tokens = sum(n for n, _ in sizes)
    if op == "append":
        return {"bytes": tokens * 2 * Hkv * D * 2 * 2, "flops": 0}
    if op == "evict":
        kept = sum(min(ctx, case["budget"]) for _, ctx in sizes)
        moved = sum(case["budget"] for _, ctx in sizes if ctx > case["budget"])
        return {"bytes": Hkv * (sum(ctx for _, ctx in sizes) * 4 + moved * 2 * D * 2 * 2 + kept * 8), "flops": 0}
    pairs, keys = _visible(case)
    if op == "mass":
        size = -(-max(ctx for _, ctx in sizes) // case["T"]) * case["T"]
        return {"bytes": tokens * Hq * (D * 2 + 4) + keys * Hkv * D * 2 + case["B"] * Hkv * size * 4,
                "flops": 2 * D * Hq * pairs}
    return {"bytes": tokens * Hq * (2 * D * 2 + 4) + keys * Hkv * 2 * D * 2, "flops": 4 * D * Hq * pairs}


# ----------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    B, Hq, Hkv, D, T = case["B"], case["Hq"], case["Hkv"], case["D"], case["T"]
    dev = torch.device("cuda")
    dt = torch.float16 if case["dtype"] == "fp16" else torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 11)
    host = torch.Generator().manual_seed(seed * 7919 + 12)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    sizes = _sizes(case)
    n_max, ctx_max = max(n for n, _ in sizes), max(ctx for _, ctx in sizes)
    max_pages = -(-ctx_max // T)
    used = [-(-ctx // T) for _, ctx in sizes]
    pool = sum(used) + 3
    perm = torch.randperm(pool, generator=host)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u].to(torch.int32)
        at += u
    offsets = torch.tensor([0] + [n for n, _ in sizes]).cumsum(0).to(torch.int32)
    lengths = torch.tensor([ctx for _, ctx in sizes], dtype=torch.int32)
    total = int(offsets[-1])
    st = dict(op=case["op"], B=B, Hq=Hq, Hkv=Hkv, D=D, T=T, n_max=n_max, max_pages=max_pages,
              scale=1.0 / math.sqrt(D), cap=case["cap"], window=case["window"], table=table.to(dev),
              lengths=lengths.to(dev), offsets=offsets.to(dev), total=total, slopes=None, prefix=None)
    st["cache"] = torch.empty(pool, 2, T, Hkv, D, device=dev, dtype=dt)
    for kind in range(2):
        st["cache"][:, kind] = normal(pool, T, Hkv, D)
    if case["op"] == "append":
        st["new"] = normal(total, 2, Hkv, D).to(dt)
        return st
    if case["op"] == "evict":
        # Accumulated weights are heavy-tailed, and some tokens never got any.
        m = (2.0 * normal(B, Hkv, max_pages * T)).exp_()
        st["mass"] = m * (torch.rand(B, Hkv, max_pages * T, generator=g, device=dev) > 0.05)
        st["budget"], st["recent"] = case["budget"], case["recent"]
        return st
    # Capped layers see large scores: that is what the cap is for.
    q = normal(total, Hq, D)
    st["q"] = (q * 8.0 if case["cap"] else q * 1.5).to(dt)
    if case["alibi"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, dtype=torch.float32) / Hq).to(dev)
    if case["prefix"]:
        st["prefix"] = torch.tensor([min(case["prefix"], ctx) for _, ctx in sizes], dtype=torch.int32, device=dev)
    if case["op"] == "mass":
        st["lse"] = _plain_attention(st, False)[1]
        return st
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(total, Hq, dtype=torch.float32, device=dev)
    # A serving program keeps one workspace for its steps.
    st["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device=dev)
    return st


# ----------------------------------------------------------------------------- plain forms

def _gathered(st, kind):
    """K (0) or V (1) of every request in token order, [B, Hkv, max_pages T, D] fp32."""
    rows = st["cache"][st["table"].clamp(min=0).long(), kind]
    return rows.reshape(st["B"], st["max_pages"] * st["T"], st["Hkv"], st["D"]).permute(0, 2, 1, 3).float()


def _plain_scores(st):
    """Masked scores [B, Hkv, g, n_max, max_pages T] of the padded chunks (-inf: not visible)."""
    B, Hkv, D = st["B"], st["Hkv"], st["D"]
    group, n = st["Hq"] // Hkv, st["n_max"]
    dev = st["q"].device
    first, last = st["offsets"][:-1, None].long(), st["offsets"][1:, None].long()
    i = torch.arange(n, device=dev)[None, :]
    row = (first + i).clamp(max=st["total"] - 1)
    q = st["q"][row].float().reshape(B, n, Hkv, group, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, group * n, D)
    s = torch.matmul(q, _gathered(st, 0).transpose(2, 3)).reshape(B, Hkv, group, n, -1)
    s.mul_(st["scale"])
    if st["cap"]:
        s.div_(st["cap"]).tanh_().mul_(st["cap"])
    length = st["lengths"][:, None].long()
    pos = (length - (last - first) + i)[:, :, None]  # [B, n, 1]
    key = torch.arange(s.shape[-1], device=dev)[None, None, :]
    if st["slopes"] is not None:
        away = (pos - key).abs().float()[:, None, None]
        s.sub_(st["slopes"].reshape(1, Hkv, group, 1, 1) * away)
    seen = key <= pos
    if st["window"]:
        seen = seen & (key > pos - st["window"])
    if st["prefix"] is not None:
        seen = seen | (key < st["prefix"][:, None, None])
    seen = seen & (key < length[:, :, None]) & (i < last - first)[:, :, None]
    return s.masked_fill_(~seen[:, None, None], -math.inf)


def _packed(st, x):
    """[B, Hkv, g, n_max, ...] of the padded chunks to [total, Hq, ...]."""
    t = torch.arange(st["total"], device=x.device)
    b = torch.searchsorted(st["offsets"][1:].long(), t, right=True)
    i = t - st["offsets"].long()[b]
    return x[b, :, :, i].reshape(st["total"], st["Hq"], *x.shape[4:])


def _plain_attention(st, output=True):
    s = _plain_scores(st)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = _packed(st, (top + total.log()).squeeze(-1))
    if not output:
        return None, lse
    B, Hkv, group, n, keys = p.shape
    o = torch.matmul(p.reshape(B, Hkv, group * n, keys), _gathered(st, 1)).reshape(B, Hkv, group, n, -1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return _packed(st, o).to(st["q"].dtype), lse


def _plain_mass(st):
    s = _plain_scores(st)
    B, Hkv, group, n, keys = s.shape
    lse = st["lse"].new_zeros(B, n, st["Hq"])
    t = torch.arange(st["total"], device=s.device)
    b = torch.searchsorted(st["offsets"][1:].long(), t, right=True)
    lse[b, t - st["offsets"].long()[b]] = st["lse"]
    lse = lse.reshape(B, n, Hkv, group).permute(0, 2, 3, 1)[..., None]
    return s.sub_(lse).exp_().sum((2, 3))


def _plain_append(st):
    t = torch.arange(st["total"], device=st["new"].device)
    b = torch.searchsorted(st["offsets"][1:].long(), t, right=True)
    n = (st["offsets"][1:] - st["offsets"][:-1]).long()
    pos = st["lengths"].long()[b] - n[b] + t - st["offsets"].long()[b]
    st["cache"][st["table"].long()[b, pos // st["T"]], :, pos % st["T"]] = st["new"]
    return st["cache"]


def _plain_evict(st):
    B, Hkv, T, D, budget = st["B"], st["Hkv"], st["T"], st["D"], st["budget"]
    mass = st["mass"]
    tokens = mass.shape[-1]
    length = st["lengths"].long()[:, None, None]
    key = torch.arange(tokens, device=mass.device)[None, None, :]
    # Rank: the last `recent` tokens first, then by weight, then by index; tokens past the length last.
    rank = torch.where(key >= length, -1.0, torch.where(key >= length - st["recent"], math.inf, mass.double()))
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :min(budget, tokens)]
    new = length.clamp(max=budget)
    slot = torch.arange(order.shape[-1], device=mass.device)[None, None, :]
    kept = torch.where(slot < new, order, tokens).sort(dim=-1).values  # in token order, unused slots last
    held = slot.expand_as(kept) < new
    src = torch.where(held, kept, 0)
    b = torch.arange(B, device=mass.device)[:, None, None].expand_as(kept)
    h = torch.arange(Hkv, device=mass.device)[None, :, None].expand_as(kept)
    table, cache = st["table"].long(), st["cache"]
    rows = cache[table[b, src // T].clamp(min=0), :, src % T, h]
    to = slot.expand_as(kept)
    cache[table[b, to // T][held], :, (to % T)[held], h[held]] = rows[held]
    moved = torch.where(held, mass.gather(2, src), 0.0)
    out_mass = torch.zeros_like(mass)
    out_mass[..., :kept.shape[-1]] = moved
    pad = torch.full((B, Hkv, budget - kept.shape[-1]), -1, dtype=torch.int32, device=mass.device)
    kept = torch.cat([torch.where(held, kept, -1).to(torch.int32), pad], -1)
    return kept, st["lengths"].clamp(max=budget), out_mass, cache


def run(state):
    st = state
    op = st["op"]
    if own:
        import exact_causal_attention_gb300 as eca

        if op == "append":
            eca.paged_append_chunk(st["new"], st["cache"], st["table"], st["lengths"], st["offsets"])
            return st["cache"]
        if op == "evict":
            kept, lengths, mass = eca.paged_evict(st["cache"], st["table"], st["lengths"], st["mass"], st["budget"],
                                                  recent=st["recent"])
            return kept, lengths, mass, st["cache"]
        form = dict(scale=st["scale"], softcap=st["cap"], alibi_slopes=st["slopes"], window=st["window"],
                    prefix_lens=st["prefix"])
        if op == "mass":
            return eca.paged_attn_mass(st["q"], st["lse"], st["cache"], st["table"], st["lengths"], st["offsets"], **form)
        if op == "decode":
            return eca.decode_paged(st["q"], st["cache"], st["table"], st["lengths"], out=st["out"], lse=st["lse"],
                                    workspace=st["workspace"], **form)
        return eca.prefill_paged(st["q"], st["cache"], st["table"], st["lengths"], st["offsets"], out=st["out"],
                                 lse=st["lse"], workspace=st["workspace"], **form)
    if op == "append":
        return _plain_append(st)
    if op == "evict":
        return _plain_evict(st)
    if op == "mass":
        return _plain_mass(st)
    return _plain_attention(st)


# ------------------------------------------------------------------- 64-bit definitions

def _exact_head(q, k, case, pos, slope, prefix):
    """Scores of one head's rows at positions `pos` against keys 0 .. len(k) - 1, 64 bits."""
    s = (q @ k.T) / math.sqrt(case["D"])
    if case["cap"]:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    j = torch.arange(len(k), device=q.device)
    if slope:
        s -= slope * (pos[:, None] - j).abs()
    hidden = j > pos[:, None]
    if case["window"]:
        hidden |= j <= pos[:, None] - case["window"]
    hidden &= j >= prefix
    s[hidden] = -math.inf
    return s


def exact(case, seed):
    st = prepare(case, seed)
    B, Hq, Hkv, D, T = case["B"], case["Hq"], case["Hkv"], case["D"], case["T"]
    table, sizes = st["table"].tolist(), _sizes(case)
    cache = st["cache"]
    if case["op"] == "append":
        new, at = st["new"].cpu(), 0
        got = cache.cpu()
        for b, (n, ctx) in enumerate(sizes):
            for i in range(n):
                p = ctx - n + i
                got[table[b][p // T], :, p % T] = new[at + i]
            at += n
        return got.double()
    if case["op"] == "evict":
        got, mass = cache.cpu(), st["mass"].cpu()
        out_mass = torch.zeros_like(mass, dtype=torch.float64)
        kept = torch.full((B, Hkv, case["budget"]), -1, dtype=torch.int32)
        lengths = torch.tensor([min(ctx, case["budget"]) for _, ctx in sizes], dtype=torch.int32)
        for b, (_, ctx) in enumerate(sizes):
            pages = torch.tensor(table[b])
            for h in range(Hkv):
                m = mass[b, h, :ctx].tolist()
                m_new = min(ctx, case["budget"])
                tail = min(case["recent"], m_new)
                best = sorted(range(ctx - tail), key=lambda j: (-m[j], j))[:m_new - tail]
                src = torch.tensor(sorted(best) + list(range(ctx - tail, ctx)))
                dst = torch.arange(m_new)
                kept[b, h, :m_new] = src.to(torch.int32)
                out_mass[b, h, :m_new] = mass[b, h][src].double()
                rows = got[pages[src // T], :, src % T, h].clone()
                got[pages[dst // T], :, dst % T, h] = rows
        return kept, lengths, out_mass, got.double()
    dev = cache.device
    out = torch.zeros(st["total"], Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((st["total"], Hq), -math.inf, dtype=torch.float64, device=dev)
    mass = torch.zeros(B, Hkv, st["max_pages"] * T, dtype=torch.float64, device=dev)
    at = 0
    for b, (n, ctx) in enumerate(sizes):
        j = torch.arange(ctx, device=dev)
        page = torch.tensor(table[b], device=dev)[j // T]
        pos = torch.arange(ctx - n, ctx, device=dev)
        prefix = min(case["prefix"], ctx)
        for kv in range(Hkv):
            k = cache[page, 0, j % T, kv].double()
            v = cache[page, 1, j % T, kv].double()
            for h in range(kv * (Hq // Hkv), (kv + 1) * (Hq // Hkv)):
                slope = float(st["slopes"][h]) if case["alibi"] else 0.0
                s = _exact_head(st["q"][at:at + n, h].double(), k, case, pos, slope, prefix)
                if case["op"] == "mass":
                    mass[b, kv, :ctx] += torch.exp(s - st["lse"][at:at + n, h].double()[:, None]).sum(0)
                    continue
                z = torch.logsumexp(s, 1)
                lse[at:at + n, h] = z
                out[at:at + n, h] = torch.exp(s - z[:, None]) @ v
        at += n
    return mass if case["op"] == "mass" else (out, lse)
