"""Attention of a ragged chunk over the paged cache and the one-token decode with score forms,
against the plain 64-bit implementation (paged_ref.py, where the bounds are derived).  Cache slots
past each length are NaN, block-table entries past each request's pages are -1."""
import math

import numpy as np
import pytest
import torch

import paged_ref as ref

ALIBI = "alibi"  # slopes 2^(-8 (h + 1) / Hq)

# B is len(sizes); sizes: (new tokens, context)
CASES = {
    "one_token": (4, 4, 64, 16, [(1, 1)], "fp16", {}),
    "decode_like": (8, 2, 128, 16, [(1, 100), (1, 1), (1, 257)], "bf16", {}),
    "whole_prompts": (4, 4, 128, 16, [(130, 130), (5, 5), (64, 64)], "fp16", {}),
    "chunk_ends_in_tile": (8, 2, 128, 16, [(70, 333), (33, 128), (1, 129)], "fp16", {}),
    "grouped_7": (14, 2, 64, 32, [(40, 200), (3, 77)], "bf16", {}),
    "grouped_3_page_8": (6, 2, 128, 8, [(90, 250)], "fp16", {}),
    "mqa_16": (16, 1, 64, 64, [(37, 190), (20, 20)], "fp16", {}),
    "mqa_200_heads": (200, 1, 64, 16, [(5, 40)], "bf16", {}),
    "empty_requests": (4, 2, 64, 16, [(0, 0), (3, 50), (0, 70), (2, 2), (0, 0)], "fp16", {}),
    "long_context": (8, 2, 128, 16, [(9, 3001), (150, 2100)], "bf16", {}),
    "many_requests": (4, 2, 64, 8, [(1 + b % 3, 1 + (37 * b) % 90 + b % 3) for b in range(70)], "fp16", {}),
    "cap": (8, 2, 128, 16, [(60, 300), (1, 90)], "bf16", dict(softcap=20.0, q_std=10.0)),
    "small_cap": (4, 4, 64, 16, [(20, 150)], "fp16", dict(softcap=2.0, q_std=3.0)),
    "alibi": (8, 8, 64, 16, [(140, 300), (1, 200)], "fp16", dict(slopes=ALIBI)),
    "alibi_grouped_prefix": (8, 2, 128, 16, [(40, 170), (64, 64)], "bf16", dict(slopes=ALIBI, prefix=[30, 64])),
    "alibi_negative": (4, 2, 64, 16, [(40, 700), (300, 300)], "fp16", dict(slopes="away")),
    "cap_fp16_long": (8, 2, 128, 16, [(40, 1200)], "fp16", dict(softcap=30.0, q_std=8.0)),
    "cap_bf16_long": (8, 2, 128, 16, [(40, 1200), (130, 600)], "bf16", dict(softcap=50.0, q_std=8.0)),
    "cap_vast": (4, 2, 64, 16, [(40, 300)], "fp16", dict(softcap=5000.0, q_std=8.0)),
    "cap_tiny": (4, 2, 64, 16, [(40, 300)], "fp16", dict(softcap=1e-5)),
    "cap_bf16_low_start": (4, 2, 64, 16, [(150, 900)], "bf16", dict(softcap=70.0, q_std=20.0)),
    "window": (8, 2, 128, 16, [(50, 700), (1, 500), (129, 129)], "fp16", dict(window=100)),
    "window_1": (4, 2, 64, 16, [(5, 40), (130, 130)], "fp16", dict(window=1)),
    "window_tile_edge": (4, 1, 64, 32, [(256, 640)], "bf16", dict(window=128)),
    "window_sinks": (8, 2, 128, 16, [(20, 900), (1, 400), (7, 7)], "fp16", dict(window=64, prefix=[4, 200, 3])),
    "prefix": (4, 4, 64, 16, [(200, 200), (10, 100), (3, 9)], "fp16", dict(prefix=[150, 20, 1000])),
    "everything": (8, 2, 128, 16, [(70, 600), (1, 333)], "bf16",
                   dict(softcap=30.0, slopes=ALIBI, window=200, prefix=[5, 0], q_std=8.0)),
}


def slopes_of(kind, Hq):
    """ALIBI: 2^(-8 (h + 1) / Hq); "away": negative, weight that grows with the distance."""
    h = torch.arange(1, Hq + 1, dtype=torch.float32)
    return torch.exp2(-8.0 * h / Hq) if kind == ALIBI else -0.05 * h


def case_inputs(name, spare_rows=0):
    Hq, Hkv, D, T, sizes, dtype, form = CASES[name]
    form = dict(form)
    q, cache, table, lens, offsets = ref.chunk(len(sizes), Hq, Hkv, D, T, sizes, dtype, 1000 + len(name) * 7 + D,
                                               form.pop("q_std", 1.0), spare_rows)
    if "slopes" in form:
        form["slopes"] = slopes_of(form["slopes"], Hq)
    if "prefix" in form:
        form["prefix"] = torch.tensor(form["prefix"], dtype=torch.int32)
    return q, cache, table, lens, offsets, dtype, T, form


def to_call(form):
    """The reference's names to the binding's, tensors on the GPU."""
    names = {"slopes": "alibi_slopes", "prefix": "prefix_lens"}
    return {names.get(k, k): v.cuda() if isinstance(v, torch.Tensor) else v for k, v in form.items()}


def near(got, want, tol):
    got = got.double().cpu().numpy()
    assert not np.isnan(got).any()
    inf = ~np.isfinite(want)
    assert np.array_equal(got[inf], want[inf])
    bad = np.abs(got[~inf] - want[~inf]) > tol[~inf]
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.max(np.abs(got[~inf] - want[~inf]) / tol[~inf]):.2f} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_prefill_matches_the_definition(cuda_lib, name):
    eca = cuda_lib
    q, cache, table, lens, offsets, dtype, T, form = case_inputs(name)
    scale = 1.0 / math.sqrt(q.shape[2])
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    eca.prefill_paged(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), offsets.cuda(), out=out, lse=lse,
                      **to_call(form))
    torch.cuda.synchronize()
    assert eca.device_status() == 0
    o, l, tol_o, tol_l = ref.attention(q, cache, table, lens, offsets, T, dtype, scale, **form)
    near(lse, l, tol_l)
    near(out, o, tol_o)


DECODE = [name for name, c in CASES.items() if c[6] and not (c[0] // c[1] > 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [1, 3, None])
@pytest.mark.parametrize("name", DECODE)
def test_decode_with_score_forms_matches_the_definition(cuda_lib, name, splits):
    eca = cuda_lib
    Hq, Hkv, D, T, sizes, dtype, form = CASES[name]
    form = dict(form)
    lengths = [c for _, c in sizes] + [0, 1, 1500]
    sizes = [(min(1, c), c) for c in lengths]
    q, cache, table, lens, offsets = ref.chunk(len(sizes), Hq, Hkv, D, T, sizes, dtype, 77 + len(name),
                                               form.pop("q_std", 1.0))
    if "slopes" in form:
        form["slopes"] = slopes_of(form["slopes"], Hq)
    if "prefix" in form:
        form["prefix"] = torch.tensor([*form["prefix"], 3, 1, 40], dtype=torch.int32)
    o, l, tol_o, tol_l = ref.attention(q, cache, table, lens, offsets, T, dtype, 1.0 / math.sqrt(D), **form)
    empty = lengths.index(0)
    at = int(offsets[empty])
    dq = torch.cat([q[:at], torch.zeros_like(q[:1]), q[at:]]).cuda()  # decode takes a row for the empty request too
    out = torch.full(dq.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(dq.shape[:2], float("nan"), device="cuda")
    eca.decode_paged(dq, cache.cuda(), table.cuda(), lens.cuda(), kv_splits=splits, out=out, lse=lse, **to_call(form))
    torch.cuda.synchronize()
    assert eca.device_status() == 0
    assert torch.all(out[empty] == 0) and torch.all(lse[empty] == -math.inf)
    rows = [b for b in range(len(lengths)) if b != empty]
    near(lse[rows], l, tol_l)
    near(out[rows], o, tol_o)


@pytest.mark.gpu
def test_rows_behind_the_last_sequence_are_left_alone(cuda_lib):
    eca = cuda_lib
    q, cache, table, lens, offsets, dtype, T, form = case_inputs("chunk_ends_in_tile", spare_rows=9)
    q[int(offsets[-1]):] = float("nan")
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    eca.prefill_paged(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), offsets.cuda(), out=out, lse=lse)
    torch.cuda.synchronize()
    assert eca.device_status() == 0
    n = int(offsets[-1])
    assert torch.all(out[n:] == 7.0) and torch.all(lse[n:] == 7.0)
    o, l, tol_o, tol_l = ref.attention(q[:n], cache, table, lens, offsets, T, dtype, 1.0 / math.sqrt(q.shape[2]))
    near(lse[:n], l, tol_l)
    near(out[:n], o, tol_o)


@pytest.mark.gpu
def test_pages_outside_the_window_are_not_followed(cuda_lib):
    """With a window, the table's entries before it may be freed (-1) or name any page."""
    eca = cuda_lib
    q, cache, table, lens, offsets, dtype, T, form = case_inputs("window_sinks")
    free = table.clone()
    for b, (n, L) in enumerate(CASES["window_sinks"][4]):
        first = max(0, L - n - form["window"] + 1) // T       # first page any row's window reaches
        keep = -(-min(int(form["prefix"][b]), L) // T)        # pages of the prefix
        free[b, keep:max(keep, first)] = -5
    scale = 1.0 / math.sqrt(q.shape[2])
    o, l, tol_o, tol_l = ref.attention(q, cache, table, lens, offsets, T, dtype, scale, **form)
    out, lse = eca.prefill_paged(q.cuda(), cache.cuda(), free.cuda(), lens.cuda(), offsets.cuda(), **to_call(form))
    assert eca.device_status() == 0
    near(lse, l, tol_l)
    near(out, o, tol_o)


@pytest.mark.gpu
def test_bad_table_entries_and_offsets_are_reported_not_followed(cuda_lib):
    eca = cuda_lib
    q, cache, table, lens, offsets, dtype, T, _ = case_inputs("chunk_ends_in_tile")
    scale = 1.0 / math.sqrt(q.shape[2])
    bad = table.clone()
    bad[0, 1] = cache.shape[0] + 3
    bad[0, 20] = -7
    out, lse = eca.prefill_paged(q.cuda(), cache.cuda(), bad.cuda(), lens.cuda(), offsets.cuda())
    assert eca.device_status() == -9
    # the tokens of those pages count as not visible
    o, l, tol_o, tol_l = ref.attention(q, cache, bad, lens, offsets, T, dtype, scale)
    near(lse, l, tol_l)
    near(out, o, tol_o)
    # offsets that decrease: the requests on both sides have no valid rows, the last is fine
    wrong = offsets.clone()
    wrong[1] = int(offsets[2]) + 1000
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    eca.prefill_paged(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), wrong.cuda(), out=out, lse=lse)
    assert eca.device_status() == -9
    # a length past the table, and a chunk longer than its context
    long = lens.clone()
    long[1] = table.shape[1] * T + 1
    eca.prefill_paged(q.cuda(), cache.cuda(), table.cuda(), long.cuda(), offsets.cuda(), out=out, lse=lse)
    assert eca.device_status() == -9
    short = lens.clone()
    short[0] = 10  # 70 rows, 10 tokens: rows 0 .. 59 stand before the context and see nothing
    out, lse = eca.prefill_paged(q.cuda(), cache.cuda(), table.cuda(), short.cuda(), offsets.cuda())
    assert eca.device_status() == -9
    assert torch.all(out[:60] == 0) and torch.all(lse[:60] == -math.inf)
    o, l, tol_o, tol_l = ref.attention(q, cache, table, short, offsets, T, dtype, scale)
    near(lse, l, tol_l)
    near(out, o, tol_o)
    assert eca.device_status() == 0


@pytest.mark.gpu
def test_one_row_a_request_is_the_decode(cuda_lib):
    """A chunk of one token per request and decode_paged compute the same thing."""
    eca = cuda_lib
    sizes = [(1, L) for L in (1, 64, 65, 1000, 4097)]
    q, cache, table, lens, offsets = ref.chunk(5, 16, 4, 128, 16, sizes, "fp16", 5)
    args = (q.cuda(), cache.cuda(), table.cuda(), lens.cuda())
    o1, l1 = eca.prefill_paged(*args, offsets.cuda())
    o2, l2 = eca.decode_paged(*args)
    assert eca.device_status() == 0
    o, l, tol_o, tol_l = ref.attention(q, cache, table, lens, offsets, 16, "fp16", 1.0 / math.sqrt(128))
    for got_o, got_l in ((o1, l1), (o2, l2)):
        near(got_l, l, tol_l)
        near(got_o, o, tol_o)


@pytest.mark.gpu
def test_graph_streams_and_repeats(cuda_lib):
    """The same bits eagerly, repeated, on another stream and replayed from a graph whose lengths and
    offsets changed in place between replays."""
    eca = cuda_lib
    q, cache, table, lens, offsets, dtype, T, form = case_inputs("window_sinks")
    g = [x.cuda() for x in (q, cache, table, lens, offsets)]
    kw = to_call(form)
    first = eca.prefill_paged(*g, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = eca.prefill_paged(*g, **kw)
    torch.cuda.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    need = eca.prefill_workspace_bytes(q.shape[0], lens.shape[0], q.shape[1], cache.shape[3], q.shape[2], T, table.shape[1])
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eca.prefill_paged(*g, out=out, lse=lse, workspace=ws, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)
    shorter = lens.clone()
    shorter[0] = 650
    g[3].copy_(shorter)
    graph.replay()
    torch.cuda.synchronize()
    assert eca.device_status() == 0
    o, l, tol_o, tol_l = ref.attention(q, cache, table, shorter, offsets, T, dtype, 1.0 / math.sqrt(q.shape[2]), **form)
    near(lse, l, tol_l)
    near(out, o, tol_o)


@pytest.mark.gpu
def test_calls_at_once_on_two_streams(cuda_lib):
    eca = cuda_lib
    work = []
    for name in ("long_context", "window"):
        q, cache, table, lens, offsets, dtype, T, form = case_inputs(name)
        work.append(([x.cuda() for x in (q, cache, table, lens, offsets)], to_call(form)))
    want = [eca.prefill_paged(*a, **kw) for a, kw in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [[], []]
    for _ in range(5):
        for i, (a, kw) in enumerate(work):
            with torch.cuda.stream(streams[i]):
                got[i].append(eca.prefill_paged(*a, **kw))
    torch.cuda.synchronize()
    assert eca.device_status() == 0
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


@pytest.mark.gpu
@pytest.mark.parametrize("B,splits", [(40, None), (40, 6), (520, 10)])
def test_decode_form_of_many_requests(cuda_lib, B, splits):
    """More than 32 requests (the segments' size is then the even share), and more groups than the
    in-kernel merge has counters for (520 x 8), merged by the second kernel."""
    eca = cuda_lib
    Hq, Hkv, D, T = 8, 8, 64, 64
    rng = np.random.default_rng(6)
    lengths = [int(x) for x in rng.integers(1, 641, size=B)]
    lengths[0] = 640
    q, cache, table, lens, offsets = ref.chunk(B, Hq, Hkv, D, T, [(1, L) for L in lengths], "fp16", 93)
    form = dict(slopes=torch.exp2(-torch.arange(1, Hq + 1, dtype=torch.float32)), window=300,
                prefix=torch.from_numpy(rng.integers(0, 40, size=B).astype(np.int32)))
    out, lse = eca.decode_paged(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), kv_splits=splits, **to_call(form))
    assert eca.device_status() == 0
    o, l, tol_o, tol_l = ref.attention(q, cache, table, lens, offsets, T, "fp16", 1.0 / math.sqrt(D), **form)
    near(lse, l, tol_l)
    near(out, o, tol_o)


@pytest.mark.gpu
@pytest.mark.parametrize("q_std,cap", [(300.0, 5.0), (0.01, 50.0), (40.0, 30.0)])
def test_cap_of_scores_far_beyond_and_far_below_it(cuda_lib, q_std, cap):
    eca = cuda_lib
    q, cache, table, lens, offsets = ref.chunk(2, 8, 2, 128, 16, [(50, 260), (1, 300)], "bf16", 17, q_std)
    o, l, tol_o, tol_l = ref.attention(q, cache, table, lens, offsets, 16, "bf16", 1.0 / math.sqrt(128), softcap=cap)
    out, lse = eca.prefill_paged(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), offsets.cuda(), softcap=cap)
    assert eca.device_status() == 0
    near(lse, l, tol_l)
    near(out, o, tol_o)


@pytest.mark.gpu
def test_workspace_contents_do_not_matter(cuda_lib):
    eca = cuda_lib
    for name in ("long_context", "window_sinks", "everything"):
        q, cache, table, lens, offsets, dtype, T, form = case_inputs(name)
        g = [x.cuda() for x in (q, cache, table, lens, offsets)]
        want = eca.prefill_paged(*g, **to_call(form))
        need = eca.prefill_workspace_bytes(q.shape[0], lens.shape[0], q.shape[1], cache.shape[3], q.shape[2], T, table.shape[1])
        for fill in (0, 255):  # 255: NaN as fp32, -1 as int32
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            got = eca.prefill_paged(*g, workspace=ws, **to_call(form))
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_two_graphs_at_once(cuda_lib):
    """Graphs captured with workspaces of their own, replayed side by side."""
    eca = cuda_lib
    graphs, outs, want = [], [], []
    for name in ("long_context", "chunk_ends_in_tile"):
        q, cache, table, lens, offsets, dtype, T, form = case_inputs(name)
        g = [x.cuda() for x in (q, cache, table, lens, offsets)]
        want.append(eca.prefill_paged(*g))
        out, lse = torch.empty_like(want[-1][0]), torch.empty_like(want[-1][1])
        need = eca.prefill_workspace_bytes(q.shape[0], lens.shape[0], q.shape[1], cache.shape[3], q.shape[2], T, table.shape[1])
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                eca.prefill_paged(*g, out=out, lse=lse, workspace=ws)
        graphs.append((graph, g, ws))
        outs.append((out, lse))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for stream, (graph, _, _) in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert eca.device_status() == 0
    for (o, l), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.gpu
def test_whole_prompt_is_the_dense_forward(cuda_lib):
    """A prompt in one chunk, long enough that every CTA takes parts of several units, against the
    dense kernel on the same values (whose own error against 64 bits the parity tests bound)."""
    eca = cuda_lib
    N, Hq, Hkv, D, T = 3000, 16, 4, 128, 16
    g = torch.Generator(device="cuda").manual_seed(21)
    q, k, v = (torch.randn(N, h, D, generator=g, device="cuda").half() for h in (Hq, Hkv, Hkv))
    pages = -(-N // T)
    table = torch.randperm(pages + 5, generator=torch.Generator().manual_seed(3))[:pages].to(torch.int32).cuda()[None]
    cache = torch.full((pages + 5, 2, T, Hkv, D), float("nan"), dtype=torch.float16, device="cuda")
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    eca.paged_append_chunk(torch.stack([k, v], 1).contiguous(), cache, table, lens, offsets)
    out, lse = eca.prefill_paged(q, cache, table, lens, offsets)
    do, dl = eca.attn_fwd_gqa(*(x.permute(1, 0, 2)[None].contiguous() for x in (q, k, v)))
    assert eca.device_status() == 0
    do, dl = do[0].permute(1, 0, 2), dl[0].permute(1, 0)
    # Both sides' lse within 1e-4 of the exact one; both round P and O to fp16: u (A + |O|) each, and
    # A = sum p |v| / l is at most the largest |v| of the head.
    assert (lse - dl).abs().max() <= 2e-4
    bound = 2 * (ref.HALF["fp16"] * (v.abs().amax().float() + do.abs().float()) + 2.0 ** -25 * v.abs().float().sum(0).amax())
    assert ((out.float() - do.float()).abs() <= bound).all()
    assert (out.float() - do.float()).abs().mean() <= 2 * ref.HALF["fp16"] * do.abs().float().mean() + 1e-5


@pytest.mark.gpu
def test_nothing_to_do(cuda_lib):
    """No rows at all, and requests that bring none."""
    eca = cuda_lib
    cache = torch.zeros(4, 2, 16, 2, 64, dtype=torch.float16, device="cuda")
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 0], dtype=torch.int32, device="cuda")
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    out, lse = eca.prefill_paged(q, cache, table, lens, none)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    eca.paged_append_chunk(torch.empty(0, 2, 2, 64, dtype=torch.float16, device="cuda"), cache, table, lens, none)
    mass = eca.paged_attn_mass(q, lse, cache, table, lens, none)
    assert torch.all(mass == 0)
    spare = torch.full((5, 4, 64), 3.0, dtype=torch.float16, device="cuda")  # rows of no request
    out, lse = torch.full_like(spare, 7.0), torch.full((5, 4), 7.0, device="cuda")
    eca.prefill_paged(spare, cache, table, lens, none, out=out, lse=lse)
    mass = eca.paged_attn_mass(spare, lse, cache, table, lens, none, mass=mass + 1.0)
    assert eca.device_status() == 0
    assert torch.all(out == 7.0) and torch.all(lse == 7.0) and torch.all(mass == 1.0)


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^31 elements (4 GiB and more), the pages in use at its far end."""
    eca = cuda_lib
    Hq, Hkv, D, T = 8, 8, 128, 64
    pages = (1 << 31) // (2 * T * Hkv * D) + 40
    sizes = [(50, 500), (1, 700)]
    q, small, table, lens, offsets = ref.chunk(2, Hq, Hkv, D, T, sizes, "fp16", 9)
    big = torch.empty(pages, 2, T, Hkv, D, dtype=torch.float16, device="cuda")
    shift = pages - small.shape[0]
    big[shift:] = small.cuda()
    far = torch.where(table >= 0, table + shift, table)
    out, lse = eca.prefill_paged(q.cuda(), big, far.cuda(), lens.cuda(), offsets.cuda())
    assert eca.device_status() == 0
    o, l, tol_o, tol_l = ref.attention(q, small, table, lens, offsets, T, "fp16", 1.0 / math.sqrt(D))
    near(lse, l, tol_l)
    near(out, o, tol_o)


# ---------------------------------------------------------------- refusals, without a GPU

A, SZ = 0x10000000, 1 << 24


def c_call(lib, fn="attn_prefill_paged", **kw):
    a = dict(q=A, cache=A + SZ, table=A + 3 * SZ, lengths=A + 4 * SZ, offsets=A + 5 * SZ, out=A + 6 * SZ,
             lse=A + 7 * SZ, total=64, B=2, Hq=8, Hkv=2, D=128, T=16, mp=16, P=40, scale=0.1, cap=0.0, window=0,
             slopes=None, prefix=None, ws=A + 64 * SZ, wsb=1 << 30)
    a.update(kw)
    return getattr(lib, fn)(a["q"], a["cache"], a["table"], a["lengths"], a["offsets"], a["out"], a["lse"], a["total"],
                            a["B"], a["Hq"], a["Hkv"], a["D"], a["T"], a["mp"], a["P"], a["scale"], a["cap"],
                            a["window"], a["slopes"], a["prefix"], a["ws"], a["wsb"], None)


@pytest.fixture(scope="module")
def lib():
    import exact_causal_attention_gb300 as eca
    from exact_causal_attention_gb300 import build

    build.build()
    return eca.load_library()


@pytest.mark.parametrize("fn", ["attn_prefill_paged", "attn_prefill_paged_bf16"])
def test_refusals_without_a_gpu(lib, fn):
    def refused(code, **kw):
        assert c_call(lib, fn, **kw) == code, kw

    for name in ("q", "cache", "table", "lengths", "offsets", "out"):
        refused(-1, **{name: None})
    refused(-1, total=-1)
    refused(-1, B=0)
    refused(-1, Hkv=3)
    refused(-1, Hq=0)
    refused(-3, D=96)
    refused(-1, T=24)
    refused(-1, scale=0.0)
    refused(-1, scale=math.nan)
    refused(-1, cap=-1.0)
    refused(-1, cap=math.inf)
    refused(-1, cap=math.nan)
    refused(-1, window=-1)
    refused(-2, q=A + 2)
    refused(-2, out=A + 6 * SZ + 8)
    refused(-2, lse=A + 2)
    refused(-2, offsets=A + 5 * SZ + 1)
    refused(-2, slopes=A + 1)
    refused(-2, prefix=A + 2)
    refused(-1, out=A + 16)           # over q
    refused(-1, out=A + SZ + 64)      # over the cache
    refused(-1, P=1 << 27)            # 2^32 token rows
    refused(-1, mp=(1 << 27) - 8, T=16, B=1)  # positions up to 2^31 - 128
    refused(-1, B=4097)
    refused(-1, total=1 << 30)        # (row, head) pairs past an int
    assert c_call(lib, fn, total=0, q=None, out=None, lse=None) == 0
    need = lib.attn_prefill_workspace_bytes(64, 2, 8, 2, 128, 16, 16)
    if need:
        refused(-1, ws=None)
        refused(-1, wsb=need - 1)
        refused(-2, ws=A + 64 * SZ + 16)
        refused(-1, ws=A)
    assert lib.attn_prefill_workspace_bytes(64, 2, 8, 2, 96, 16, 16) == 0
    assert lib.attn_prefill_workspace_bytes(64, 2, 8, 3, 128, 16, 16) == 0


@pytest.mark.parametrize("fn", ["attn_decode_paged_form", "attn_decode_paged_form_bf16"])
def test_decode_form_refusals_without_a_gpu(lib, fn):
    def c(cap=0.0, window=0, slopes=None, prefix=None, Hkv=2, splits=1):
        return getattr(lib, fn)(A, A + SZ, A + 3 * SZ, A + 4 * SZ, A + 6 * SZ, None, 2, 8, Hkv, 128, 16, 16, 40, 0.1,
                                cap, window, slopes, prefix, splits, None, 0, None)

    assert c(cap=-0.5) == -1
    assert c(cap=math.nan) == -1
    assert c(window=-2) == -1
    assert c(slopes=A + 1) == -2
    assert c(prefix=A + 3) == -2
    assert c(Hkv=3) == -1
    assert c(splits=2) == -1


def test_header_declares_what_the_binding_loads(lib):
    import os
    import re

    import exact_causal_attention_gb300 as eca
    from exact_causal_attention_gb300 import build

    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(build.INCLUDE, "attn_cache.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(attn_\w+)\s*\(", text, flags=re.M))
    assert names == set(eca.CACHE_SIGNATURES)
    for name in names:
        assert hasattr(lib, name), name


def test_cache_header_compiles_as_c(tmp_path):
    import shutil
    import subprocess

    from exact_causal_attention_gb300 import build

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use.c"
    src.write_text('#include "attn_cache.h"\nint main(void) { return attn_prefill_paged == 0; }\n')
    subprocess.run([cc, "-std=c11", "-Wall", "-Wextra", "-pedantic", "-c", "-I", build.INCLUDE, "-o",
                    str(tmp_path / "use.o"), str(src)], check=True)


def test_binding_refuses_what_it_cannot_pass():
    import exact_causal_attention_gb300 as eca

    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    cache = torch.zeros(4, 2, 16, 2, 64, dtype=torch.float16)
    table, lens, off = (torch.zeros(s, dtype=torch.int32) for s in ((2, 3), (2,), (3,)))
    for bad in (dict(), dict(cache=cache.float()), dict(lens=lens.long()), dict(table=table[:1])):
        a = {"cache": cache, "table": table, "lens": lens, **bad}
        with pytest.raises((TypeError, ValueError)):
            eca.prefill_paged(q, a["cache"], a["table"], a["lens"], off)
        with pytest.raises((TypeError, ValueError)):
            eca.paged_attn_mass(q, torch.zeros(3, 4), a["cache"], a["table"], a["lens"], off)
        with pytest.raises((TypeError, ValueError)):
            eca.paged_append_chunk(torch.zeros(3, 2, 2, 64, dtype=torch.float16), a["cache"], a["table"], a["lens"], off)
        with pytest.raises((TypeError, ValueError)):
            eca.paged_evict(a["cache"], a["table"], a["lens"], torch.zeros(2, 2, 48), 8)
