"""Append of a chunk, attention weight per cached token and eviction by it, against plain
implementations (paged_ref.py): copies and whole numbers exactly, the weights within their
derived bound; and the whole life of a cache run together."""
import math

import numpy as np
import pytest
import torch

import paged_ref as ref
from exact_causal_attention_gb300 import inputs
from test_prefill_paged import A, CASES, SZ, case_inputs, lib, near, to_call  # noqa: F401

T16 = inputs.TORCH_DTYPES


# ------------------------------------------------------------------------- append of a chunk

APPEND = [
    # Hkv, D, T, [(new, context)], dtype
    (2, 64, 16, [(1, 1)], "fp16"),
    (2, 128, 8, [(3, 20), (17, 17), (0, 9), (1, 64)], "bf16"),
    (1, 64, 64, [(130, 300), (64, 128)], "fp16"),
    (7, 128, 32, [(33, 65), (0, 0), (2, 33)], "bf16"),
    (8, 128, 16, [(1 + b % 4, 5 + 3 * b) for b in range(100)], "fp16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,D,T,sizes,dtype", APPEND)
def test_append_chunk_writes_exactly_the_new_rows(cuda_lib, Hkv, D, T, sizes, dtype):
    eca = cuda_lib
    _, cache, table, lens, offsets = ref.chunk(len(sizes), Hkv, Hkv, D, T, sizes, dtype, 31 + D + T)
    spare = 3  # packed rows behind the last request: neither read nor written
    total = int(offsets[-1])
    new = torch.randn(total + spare, 2, Hkv, D, generator=torch.Generator().manual_seed(3)).to(T16[dtype])
    want = cache.clone()
    for b, (n, L) in enumerate(sizes):
        for i in range(n):
            t = L - n + i
            want[int(table[b, t // T]), :, t % T] = new[int(offsets[b]) + i]
    got = cache.cuda()
    eca.paged_append_chunk(new.cuda(), got, table.cuda(), lens.cuda(), offsets.cuda())
    torch.cuda.synchronize()
    assert eca.device_status() == 0
    assert np.array_equal(inputs.bits(got.cpu()), inputs.bits(want))


@pytest.mark.gpu
def test_append_chunk_of_single_rows_is_append(cuda_lib):
    eca = cuda_lib
    sizes = [(1, L) for L in (1, 16, 17, 400)]
    _, cache, table, lens, offsets = ref.chunk(4, 2, 2, 128, 16, sizes, "fp16", 8)
    new = torch.randn(4, 2, 2, 128, dtype=torch.float32).half().cuda()
    a, b = cache.cuda(), cache.cuda()
    eca.paged_append(new, a, table.cuda(), lens.cuda())
    eca.paged_append_chunk(new, b, table.cuda(), lens.cuda(), offsets.cuda())
    torch.cuda.synchronize()
    assert np.array_equal(inputs.bits(a.cpu()), inputs.bits(b.cpu()))


@pytest.mark.gpu
def test_append_chunk_skips_and_reports_bad_places(cuda_lib):
    eca = cuda_lib
    sizes = [(20, 40), (4, 50)]
    _, cache, table, lens, offsets = ref.chunk(2, 2, 2, 64, 16, sizes, "fp16", 9)
    new = torch.randn(24, 2, 2, 64).half()
    bad = table.clone()
    bad[0, 1] = cache.shape[0]
    got = cache.cuda()
    eca.paged_append_chunk(new.cuda(), got, bad.cuda(), lens.cuda(), offsets.cuda())
    assert eca.device_status() == -9
    want = cache.clone()
    for b, (n, L) in enumerate(sizes):
        for i in range(n):
            t = L - n + i
            if b == 0 and t // 16 == 1:
                continue
            want[int(table[b, t // 16]), :, t % 16] = new[int(offsets[b]) + i]
    assert np.array_equal(inputs.bits(got.cpu()), inputs.bits(want))
    assert eca.device_status() == 0


# ------------------------------------------------------------------------- attention weight

def plain_lse(name):
    q, cache, table, lens, offsets, dtype, T, form = case_inputs(name)
    _, l, _, _ = ref.attention(q, cache, table, lens, offsets, T, dtype, 1.0 / math.sqrt(q.shape[2]), **form)
    return q, cache, table, lens, offsets, dtype, T, form, torch.from_numpy(l).float()


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_mass_matches_the_definition(cuda_lib, name):
    eca = cuda_lib
    q, cache, table, lens, offsets, dtype, T, form, lse = plain_lse(name)
    scale = 1.0 / math.sqrt(q.shape[2])
    want, tol = ref.mass(q, lse, cache, table, lens, offsets, T, dtype, scale, **form)
    args = (q.cuda(), lse.cuda(), cache.cuda(), table.cuda(), lens.cuda(), offsets.cuda())
    got = eca.paged_attn_mass(*args, **to_call(form))
    torch.cuda.synchronize()
    assert eca.device_status() == 0
    near(got, want, tol)
    # Added to what is there, and every row's weight comes to 1 over the keys.
    had = torch.rand(got.shape, generator=torch.Generator().manual_seed(4)).cuda()
    more = eca.paged_attn_mass(*args, mass=had.clone(), **to_call(form))
    assert torch.equal(more, had + got)
    Hq, Hkv = q.shape[1], cache.shape[3]
    rows = (offsets[1:] - offsets[:-1]).double() * (Hq // Hkv)
    assert np.allclose(got.double().sum(2).cpu().numpy(), rows[:, None].numpy(), rtol=1e-3)


@pytest.mark.gpu
def test_mass_of_a_decode_step(cuda_lib):
    eca = cuda_lib
    Hq, Hkv, D, T = 16, 4, 128, 16
    lengths = [1, 1000, 0, 129, 2500]
    q, cache, table, lens = inputs.paged_decode_inputs(5, Hq, Hkv, D, T, lengths, "bf16", 12)
    cache = ref.poison(cache, table, lens, T)
    d = [x.cuda() for x in (q, cache, table, lens)]
    o, lse = eca.decode_paged(*d)
    got = eca.paged_attn_mass(d[0], lse, *d[1:])
    assert eca.device_status() == 0
    rows = [b for b, L in enumerate(lengths) if L]
    offsets = torch.tensor([0, 1, 2, 2, 3, 4], dtype=torch.int32)
    want, tol = ref.mass(q[rows], lse.cpu()[rows], cache, table, lens, offsets, T, "bf16", 1.0 / math.sqrt(D))
    near(got, want, tol)


@pytest.mark.gpu
def test_mass_with_bad_pages_and_rows_without_keys(cuda_lib):
    eca = cuda_lib
    q, cache, table, lens, offsets, dtype, T, form, lse = plain_lse("chunk_ends_in_tile")
    scale = 1.0 / math.sqrt(q.shape[2])
    bad = table.clone()
    bad[0, 2] = -3
    lse[5:9] = -math.inf  # rows that saw nothing add nothing
    got = eca.paged_attn_mass(q.cuda(), lse.cuda(), cache.cuda(), bad.cuda(), lens.cuda(), offsets.cuda())
    assert eca.device_status() == -9
    want, tol = ref.mass(q, lse, cache, bad, lens, offsets, T, dtype, scale)
    near(got, want, tol)


@pytest.mark.gpu
def test_mass_repeats_and_replays_bit_identically(cuda_lib):
    eca = cuda_lib
    q, cache, table, lens, offsets, dtype, T, form, lse = plain_lse("long_context")
    args = [x.cuda() for x in (q, lse, cache, table, lens, offsets)]
    want = eca.paged_attn_mass(*args)
    mass = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mass.zero_()
        eca.paged_attn_mass(*args, mass=mass)
    side = torch.cuda.Stream()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(mass, want)
        with torch.cuda.stream(side):
            again = eca.paged_attn_mass(*args)
        torch.cuda.synchronize()
        assert torch.equal(again, want)
    assert eca.device_status() == 0


# ------------------------------------------------------------------------------- eviction

EVICT = {
    # Hkv, D, T, lengths, dtype, budget, recent, masses
    "shrinks": (2, 64, 16, [100, 30, 64], "fp16", 40, 8, "spread"),
    "one_token": (2, 128, 16, [1, 50], "bf16", 1, 0, "spread"),
    "only_recent": (1, 64, 8, [90, 24], "fp16", 16, 16, "spread"),
    "nothing_to_do": (2, 64, 32, [20, 0, 33], "bf16", 64, 10, "spread"),
    "all_equal": (3, 64, 16, [200, 77], "fp16", 50, 7, "equal"),
    "ties_at_the_border": (2, 128, 16, [300, 150], "bf16", 101, 3, "few_values"),
    "odd_values": (2, 64, 16, [400], "fp16", 200, 0, "odd"),
    "long": (2, 128, 64, [9000, 5000], "fp16", 2049, 100, "spread"),
    "past_shared_memory": (1, 64, 64, [40000, 33000], "fp16", 5000, 64, "spread"),
    "past_shared_memory_ties": (2, 64, 64, [36000], "bf16", 20000, 5, "few_values"),
    "most_stays": (2, 64, 16, [3000], "fp16", 2990, 100, "few_values"),
    "just_over": (4, 64, 16, [1025, 1024], "bf16", 1024, 1, "spread"),
}


def evict_inputs(name):
    Hkv, D, T, lengths, dtype, budget, recent, kind = EVICT[name]
    B = len(lengths)
    _, cache, table, lens = inputs.paged_decode_inputs(B, Hkv, Hkv, D, T, lengths, dtype, 50 + len(name))
    shape = (B, Hkv, max(table.shape[1], -(-budget // T)) * T)
    if table.shape[1] * T < shape[2]:
        table = torch.cat([table, torch.full((B, shape[2] // T - table.shape[1]), -1, dtype=torch.int32)], 1)
    g = torch.Generator().manual_seed(len(name))
    if kind == "spread":
        mass = torch.exp(2 * torch.randn(shape, generator=g))
    elif kind == "equal":
        mass = torch.full(shape, 0.25)
    elif kind == "few_values":
        mass = torch.randint(0, 4, shape, generator=g).float() / 8
    else:
        pool = torch.tensor([0.0, -0.0, math.nan, math.inf, -math.inf, -1.5, 1e-42, -1e-42, 3e38, 1.0])
        mass = pool[torch.randint(0, len(pool), shape, generator=g)]
    return cache, table, lens, mass, budget, recent, T


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", EVICT)
def test_evict_keeps_what_it_should(cuda_lib, name, in_place):
    eca = cuda_lib
    cache, table, lens, mass, budget, recent, T = evict_inputs(name)
    want = ref.evict(cache, table, lens, mass, budget, recent, T)
    dc, dt, dl, dm = cache.cuda(), table.cuda(), lens.cuda(), mass.cuda()
    kw = dict(new_lengths=dl, mass_out=dm) if in_place else {}
    kept, lengths, out = eca.paged_evict(dc, dt, dl, dm, budget, recent, **kw)
    torch.cuda.synchronize()
    assert eca.device_status() == 0
    assert torch.equal(kept.cpu(), want[1])
    assert torch.equal(lengths.cpu(), want[2])
    assert torch.equal(torch.nan_to_num(out.cpu(), nan=9e9), torch.nan_to_num(want[3], nan=9e9))
    assert np.array_equal(inputs.bits(dc.cpu()), inputs.bits(want[0]))
    if not in_place:
        assert torch.equal(dl.cpu(), lens)
        assert np.array_equal(dm.cpu().numpy(), mass.numpy(), equal_nan=True)


@pytest.mark.gpu
def test_evict_skips_and_reports_bad_pages(cuda_lib):
    eca = cuda_lib
    cache, table, lens, mass, budget, recent, T = evict_inputs("shrinks")
    bad = table.clone()
    bad[0, 5] = cache.shape[0] + 1  # positions 80 .. 95 of request 0
    dc = cache.cuda()
    kept, lengths, _ = eca.paged_evict(dc, bad.cuda(), lens.cuda(), mass.cuda(), budget, recent)
    assert eca.device_status() == -9
    want = ref.evict(cache, table, lens, mass, budget, recent, T)
    assert torch.equal(kept.cpu(), want[1]) and torch.equal(lengths.cpu(), want[2])
    got, moved = dc.cpu(), want[0]
    for h in range(2):
        for slot, src in enumerate(want[1][0, h].tolist()):
            page, off = int(table[0, slot // T]), slot % T
            if 80 <= src < 96:  # not read: the place keeps what it had
                assert torch.equal(got[page, :, off, h], cache[page, :, off, h])
            else:
                assert torch.equal(got[page, :, off, h], moved[page, :, off, h])
    for b in (1, 2):
        pages = table[b][table[b] >= 0].long()
        assert torch.equal(got[pages], moved[pages])
    assert eca.device_status() == 0


# ---------------------------------------------------------------------- the life of a cache

@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_append_attend_weigh_evict_and_go_on(cuda_lib, captured):
    """Two prompts go in by chunks, a decode step follows, the weights of all of it pick the tokens
    that stay, and the next steps run on the shrunken cache; every step against the plain 64-bit form.
    Run eagerly, and once more with the step's calls captured in one graph."""
    eca = cuda_lib
    Hq, Hkv, D, T, dtype = 8, 2, 128, 16, "fp16"
    B, pages = 2, 20
    scale = 1.0 / math.sqrt(D)
    g = torch.Generator().manual_seed(99)
    perm = torch.randperm(B * pages + 2, generator=g)[:B * pages].to(torch.int32).reshape(B, pages)
    cache = torch.full((B * pages + 2, 2, T, Hkv, D), float("nan"), dtype=torch.float16)
    lengths = torch.zeros(B, dtype=torch.int32)
    dc, dt = cache.cuda(), perm.cuda()
    mass = torch.zeros(B, Hkv, pages * T, device="cuda")
    total_mass = np.zeros(mass.shape)
    steps = [[100, 7], [90, 60], [1, 1], None, [1, 1], [30, 2]]
    for n in steps:
        if n is None:
            budget, recent = 64, 16
            want = ref.evict(dc.cpu(), perm, lengths, mass.cpu(), budget, recent, T)
            dl = lengths.cuda()
            kept, _, _ = eca.paged_evict(dc, dt, dl, mass, budget, recent, new_lengths=dl, mass_out=mass)
            torch.cuda.synchronize()
            assert eca.device_status() == 0
            assert torch.equal(kept.cpu(), want[1])
            assert np.array_equal(inputs.bits(dc.cpu()), inputs.bits(want[0]))
            assert torch.equal(mass.cpu(), want[3])
            lengths, total_mass = want[2], want[3].double().numpy()
            assert torch.equal(dl.cpu(), lengths)
            continue
        lengths = lengths + torch.tensor(n, dtype=torch.int32)
        offsets = torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32)
        total = int(offsets[-1])
        new = torch.randn(total, 2, Hkv, D, generator=g).half()
        q = (2 * torch.randn(total, Hq, D, generator=g)).half()
        dl, do, dq, dn = lengths.cuda(), offsets.cuda(), q.cuda(), new.cuda()
        out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
        lse = torch.full(q.shape[:2], float("nan"), device="cuda")

        def step():
            eca.paged_append_chunk(dn, dc, dt, dl, do)
            eca.prefill_paged(dq, dc, dt, dl, do, out=out, lse=lse)
            eca.paged_attn_mass(dq, lse, dc, dt, dl, do, mass=mass)

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert eca.device_status() == 0
        now = dc.cpu()
        for b in range(B):
            for i in range(n[b]):
                t = int(lengths[b]) - n[b] + i
                assert torch.equal(now[int(perm[b, t // T]), :, t % T], new[int(offsets[b]) + i])
        o, l, tol_o, tol_l = ref.attention(q, now, perm, lengths, offsets, T, dtype, scale)
        near(lse, l, tol_l)
        near(out, o, tol_o)
        m, tol_m = ref.mass(q, lse.cpu(), now, perm, lengths, offsets, T, dtype, scale)
        near(mass, total_mass + m, tol_m + 4 * ref.F32 * (total_mass + m))
        total_mass = mass.double().cpu().numpy()
        if max(n) == 1:
            o2, l2 = eca.decode_paged(dq, dc, dt, dl)
            near(l2, l, tol_l)
            near(o2, o, tol_o)


# ---------------------------------------------------------------- refusals, without a GPU

@pytest.mark.gpu
@pytest.mark.parametrize("op", ["prefill", "decode", "decode_form", "mass", "evict"])
def test_results_allocated_for_another_stream(cuda_lib, op):
    """With stream= given, results and workspaces belong to that stream: a write still queued on the
    current stream, to a block that was freed since, does not reach them."""
    eca = cuda_lib
    B, Hq, Hkv, D, T, pages = 2, 8, 2, 64, 16, 64
    g = torch.Generator().manual_seed(5)
    lens = torch.tensor([900, 700], dtype=torch.int32).cuda()
    cache = torch.randn((B * pages, 2, T, Hkv, D), generator=g).half().cuda()
    table = torch.randperm(B * pages, generator=g).int().reshape(B, pages).cuda()
    q = torch.randn((B, Hq, D), generator=g).half().cuda()
    lse = torch.full((B, Hq), 5.0, device="cuda")
    offsets = torch.arange(B + 1, dtype=torch.int32).cuda()
    weights = torch.rand((B, Hkv, pages * T), generator=g).cuda()

    def call(stream):
        if op == "prefill":
            return eca.prefill_paged(q, cache, table, lens, offsets, stream=stream)
        if op == "decode":
            return eca.decode_paged(q, cache, table, lens, stream=stream)
        if op == "decode_form":
            return eca.decode_paged(q, cache, table, lens, stream=stream, window=500)
        if op == "mass":
            return (eca.paged_attn_mass(q, lse, cache, table, lens, stream=stream),)
        return eca.paged_evict(cache, table, lens, weights, 1000, 10, stream=stream)

    want = [x.clone() for x in call(None)]  # (the eviction moves nothing: every request fits its budget)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        held = [torch.empty_like(x) for x in want for _ in range(3)]
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        for x in held:
            x.fill_(7)
        del held, x
        got = call(stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert eca.device_status() == 0


def test_append_chunk_refusals_without_a_gpu(lib):
    f = lib.attn_paged_append_chunk

    def c(new=A, cache=A + SZ, table=A + 3 * SZ, lengths=A + 4 * SZ, offsets=A + 5 * SZ, total=8, B=2, Hkv=2, D=128,
          T=16, mp=4, P=40):
        return f(new, cache, table, lengths, offsets, total, B, Hkv, D, T, mp, P, None)

    for name in ("new", "cache", "table", "lengths", "offsets"):
        assert c(**{name: None}) == -1, name
    assert c(total=-1) == -1
    assert c(T=12) == -1
    assert c(D=80) == -3
    assert c(new=A + 8) == -2
    assert c(offsets=A + 2) == -2
    assert c(new=A + SZ) == -1  # over the cache
    assert c(total=0, new=None) == 0


def test_mass_refusals_without_a_gpu(lib):
    for fn in ("attn_paged_mass", "attn_paged_mass_bf16"):
        f = getattr(lib, fn)

        def c(q=A, lse=A + SZ, cache=A + 2 * SZ, table=A + 4 * SZ, lengths=A + 5 * SZ, offsets=A + 6 * SZ,
              mass=A + 8 * SZ, acc=0, total=8, B=2, Hq=8, Hkv=2, D=128, T=16, mp=4, P=40, scale=0.1, cap=0.0,
              window=0, slopes=None, prefix=None):
            return f(q, lse, cache, table, lengths, offsets, mass, acc, total, B, Hq, Hkv, D, T, mp, P, scale, cap,
                     window, slopes, prefix, None)

        for name in ("q", "lse", "cache", "table", "lengths", "mass"):
            assert c(**{name: None}) == -1, name
        assert c(offsets=None) == -1  # then total must be B
        assert c(Hkv=3) == -1
        assert c(D=72) == -3
        assert c(cap=-1.0) == -1
        assert c(window=-1) == -1
        assert c(scale=math.inf) == -1
        assert c(B=4097, total=4097, offsets=None) == -1
        assert c(mp=(1 << 27) - 8, B=1) == -1  # positions up to 2^31 - 128
        assert c(mass=A + 2) == -2
        assert c(lse=A + SZ + 2) == -2
        assert c(q=A + 8) == -2
        assert c(mass=A + 16) == -1      # over q
        assert c(mass=A + 2 * SZ) == -1  # over the cache


def test_evict_refusals_without_a_gpu(lib):
    f = lib.attn_paged_evict

    def c(cache=A, table=A + 3 * SZ, lengths=A + 4 * SZ, mass=A + 5 * SZ, kept=A + 6 * SZ, new=A + 7 * SZ,
          out=A + 8 * SZ, B=2, Hkv=2, D=128, T=16, mp=4, P=40, budget=32, recent=4):
        return f(cache, table, lengths, mass, kept, new, out, B, Hkv, D, T, mp, P, budget, recent, None)

    for name in ("cache", "table", "lengths", "mass", "kept", "new"):
        assert c(**{name: None}) == -1, name
    assert c(budget=0) == -1
    assert c(budget=65) == -1  # past max_pages * page_size
    assert c(mp=(1 << 27) - 8, B=1) == -1  # positions up to 2^31 - 128
    assert c(recent=-1) == -1
    assert c(recent=33) == -1
    assert c(D=96) == -3
    assert c(T=48) == -1
    assert c(mass=A + 5 * SZ + 2) == -2
    assert c(kept=A + 5 * SZ) == -1          # kept over mass
    assert c(out=A + 5 * SZ + 64) == -1      # mass_out partly over mass
    assert c(out=A + 64) == -1               # mass_out over the cache
