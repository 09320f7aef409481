"""Attention over the paged cache against the fp64 form (needs a GB300).

Tolerance of an output: its bf16 rounding (2^-8 of it), the bf16 rounding of each probability before P V (2^-8 of
sum_j p_j |v_j|, "reach"; the row sum takes the unrounded ones), and what the fp32 scores lose: a score is off by at
most 2^-18 sum_c |q_c k_c| scale (d <= 128 products, accumulated in fp32 by the tensor core with truncation), at most
80 for N(0, 1) inputs of these sizes, so each probability by 2^-11 of itself; eight times that for the wide rows.
lse: the forward tests' 1e-3 covers the same score error (2^-18 * 80 = 3e-4).
"""

import random

import numpy as np
import pytest
import torch

import exact_io_aware_31_gb300 as fa
from oracle import serve
from tests.gpu_util import TOL_LSE, f64, require_gpu
from tests.test_gpu_norm_rope import pool, ragged, status

pytestmark = pytest.mark.gpu

BF, SCORE = 2.0 ** -8, 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def check(o, lse, ref, wide=1.0, rows=slice(None)):
    ro, rl, reach = ref
    live = ~np.isnan(rl)
    assert np.isfinite(f64(o)[live]).all()
    err = np.abs(f64(o)[live] - ro[live]) - (BF * np.abs(ro[live]) + (BF + wide * SCORE) * reach[live])
    assert err.max() <= 2.0 ** -126, float(err.max())
    got, want = f64(lse)[live], rl[live]
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fine = np.isfinite(want)
    assert (np.abs(got[fine] - want[fine]) <= wide * TOL_LSE).all()


CASES = [
    # q_lens, kv_lens, Hq, Hk, d, page, token_major, causal
    ([1], [1], 1, 1, 64, 16, False, True),
    ([1], [130], 16, 16, 64, 16, False, True),
    ([1], [128], 8, 1, 128, 128, False, True),
    ([1, 1, 1, 1], [5, 127, 129, 1000], 8, 2, 128, 16, True, True),
    ([1] * 9, [16 * i + 1 for i in range(9)], 6, 2, 64, 64, False, True),        # groups of three
    ([0, 3, 0, 1, 8, 0], [0, 3, 50, 0, 300, 700], 4, 4, 128, 32, False, True),   # empty sequences, kv 0
    ([2, 5, 7], [1, 3, 7], 4, 2, 64, 16, False, True),                           # rows that see no key
    ([8, 8], [777, 1024], 16, 16, 64, 32, True, True),
    ([5], [3000], 64, 1, 128, 64, False, False),                                 # 64 heads share keys
    ([3, 1], [400, 260], 128, 1, 64, 256, False, True),                          # 128 heads: a tile a token
    ([9, 2], [500, 64], 70, 1, 128, 16, True, True),
    ([33], [33], 4, 1, 128, 16, False, True),                                    # 132 rows
    ([64, 65], [64, 200], 2, 1, 64, 128, False, True),
    ([128], [128], 1, 1, 128, 128, False, True),
    ([129], [129], 2, 2, 128, 32, False, True),
    ([300, 1, 40, 0, 257], [300, 900, 41, 10, 2049], 4, 2, 128, 64, False, True),
    ([300, 1, 40, 0, 257], [300, 900, 41, 10, 2049], 4, 2, 64, 16, True, True),
    ([200, 130], [90, 135], 3, 1, 128, 32, False, True),                         # chunks longer than their keys
    ([150, 270], [600, 0], 5, 1, 64, 16, False, False),
    ([700], [1500], 4, 1, 128, 512, False, True),                                # a page over several key tiles
    ([257], [1000], 7, 1, 128, 64, True, False),
]
IDS = [f"s{len(c[0])}q{max(c[0])}k{max(c[1])}h{c[2]}_{c[3]}d{c[4]}p{c[5]}{'c' if c[7] else ''}" for c in CASES]


def batch(case, seed=17, wide=False):
    q_lens, kv_lens, Hq, Hk, d, page, token_major, causal = case
    pages, table = pool(kv_lens, Hk, d, page, token_major, seed)
    cu = ragged(q_lens)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(int(cu[-1]), Hq, d, generator=g) * (8.0 if wide else 1.0)
    return q.bfloat16().cuda(), pages, table, cu, torch.tensor(kv_lens, dtype=torch.int32)


def reference(q, pages, table, cu, lens, scale, causal):
    kp, vp = (np.nan_to_num(f64(p)) for p in pages)
    return serve.paged_attention(f64(q), kp, vp, table.numpy(), cu.numpy(), lens.numpy(), scale, causal)


@pytest.mark.parametrize("hint", [None, 0, 1, 10 ** 6])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_against_the_oracle(case, hint):
    """Each hint selects a kernel variant of its own; all must give the same attention."""
    q, pages, table, cu, lens = batch(case)
    ref = reference(q, pages, table, cu, lens, 0.11, case[7])
    o, lse = fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), scale=0.11, causal=case[7],
                              max_q=max(case[0]) if hint is None else hint)
    assert status() == fa.FA_OK
    check(o, lse, ref)


@pytest.mark.parametrize("case", [CASES[3], CASES[7], CASES[15], CASES[16], CASES[20]], ids=lambda c: f"d{c[4]}p{c[5]}")
def test_wide_rows(case):
    q, pages, table, cu, lens = batch(case, seed=23, wide=True)
    ref = reference(q, pages, table, cu, lens, case[4] ** -0.5, case[7])
    o, lse = fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), causal=case[7], max_q=max(case[0]))
    assert status() == fa.FA_OK
    check(o, lse, ref, wide=8.0)


@pytest.mark.parametrize("scale", [-0.1, 0.0])
@pytest.mark.parametrize("case", [CASES[3], CASES[15]], ids=["q1", "chunks"])
def test_scales(case, scale):
    q, pages, table, cu, lens = batch(case)
    ref = reference(q, pages, table, cu, lens, scale, True)
    o, lse = fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), scale=scale, max_q=max(case[0]))
    check(o, lse, ref)


@pytest.mark.parametrize("hint", [None, 0, 1])
@pytest.mark.parametrize("case", CASES[1:9] + CASES[11:17], ids=IDS[1:9] + IDS[11:17])
def test_a_query_of_nan_is_seen(case, hint):
    """Rows whose query is NaN are NaN (not zero, as rows without a key are), the others as before."""
    q, pages, table, cu, lens = batch(case)
    o, lse, reach = reference(q, pages, table, cu, lens, 0.11, case[7])
    poisoned = torch.zeros(q.shape[:2], dtype=torch.bool)
    poisoned[::3, ::2] = True
    q.masked_fill_(poisoned[..., None].cuda(), float("nan"))
    lse = np.where(poisoned.numpy() & np.isfinite(lse), np.nan, lse)
    got, got_lse = fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), scale=0.11, causal=case[7],
                                    max_q=max(case[0]) if hint is None else hint)
    assert status() == fa.FA_OK
    check(got, got_lse, (o, lse, reach))
    assert np.isnan(f64(got)[np.isnan(lse)]).all() and np.isnan(f64(got_lse)[np.isnan(lse)]).all()


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", CASES[3:8] + CASES[15:19], ids=IDS[3:8] + IDS[15:19])
def test_what_lies_behind_a_sequence_does_not_matter(case, fill):
    """Every key and value that no sequence owns is NaN or infinite."""
    q, pages, table, cu, lens = batch(case)
    ref = reference(q, pages, table, cu, lens, 0.11, case[7])
    page = case[5]
    owned = torch.zeros(pages[0].shape[0], page, dtype=torch.bool)
    for s, n in enumerate(case[1]):
        for j in range(n):
            owned[table[s, j // page], j % page] = True
    for p in pages:
        p.masked_fill_(~owned[:, None, :, None].cuda(), fill)
    o, lse = fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), scale=0.11, causal=case[7],
                              max_q=max(case[0]))
    assert status() == fa.FA_OK
    check(o, lse, ref)


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d,hint", [
    ([1], [40000], 2, 1, 128, 1),            # one unit cut into more parts than a warp has lanes
    ([1], [20000], 4, 4, 64, 1),
    ([5, 1], [9000, 12000], 8, 1, 128, 5),
    ([140], [6000], 2, 1, 128, 140),         # two-tile units, cut
    ([1, 260, 1], [8000, 4000, 3], 2, 1, 64, 260),
])
def test_long_caches_are_cut(q_lens, kv_lens, Hq, Hk, d, hint):
    case = (q_lens, kv_lens, Hq, Hk, d, 64, False, True)
    q, pages, table, cu, lens = batch(case)
    ref = reference(q, pages, table, cu, lens, d ** -0.5, True)
    args = (q, *pages, table.cuda(), cu.cuda(), lens.cuda())
    o, lse = fa.paged_forward(*args, max_q=hint)
    assert status() == fa.FA_OK
    check(o, lse, ref)
    for _ in range(3):  # the same bits on every run, whatever the workspace held
        ws = torch.full((fa.fa_fwd_paged_workspace_size(d),), 255, dtype=torch.uint8, device="cuda")
        o2, lse2 = fa.paged_forward(*args, max_q=hint, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("hint", [0, 200])
@pytest.mark.parametrize("q,kv,Hq,Hk,d,long", [
    (6, 110, 64, 8, 64, 1),      # every unit one query tile, most of one key tile
    (7, 300, 64, 8, 128, 1),     # 1 to 3 key tiles
    (82, 200, 4, 4, 128, 7),     # among single tokens
    (120, 128, 2, 2, 64, 3),
])
def test_rows_of_small_units(q, kv, Hq, Hk, d, long, hint):
    """Runs of units of one query tile and one key tile or a few: the half of a CTA that has no key tile must not get
    ahead of the other."""
    g = torch.Generator().manual_seed(5)
    q_lens = [int(torch.randint(max(1, q - 30), q + 1, (1,), generator=g)) if s % long == 0 else 1 for s in range(72)]
    kv_lens = [max(n, int(torch.randint(n, kv + 1, (1,), generator=g))) for n in q_lens]
    case = (q_lens, kv_lens, Hq, Hk, d, 32, False, True)
    q, pages, table, cu, lens = batch(case)
    ref = reference(q, pages, table, cu, lens, 0.11, True)
    args = (q, *pages, table.cuda(), cu.cuda(), lens.cuda())
    for _ in range(3):
        o, lse = fa.paged_forward(*args, scale=0.11, max_q=hint)
        assert status() == fa.FA_OK
        check(o, lse, ref)


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d", [
    ([267], [5885], 1, 1, 64),                   # a row group's rows in two tiles, 46 parts
    ([31, 57], [9001, 3000], 5, 1, 128),         # units of each form
    ([3, 300, 2], [70, 2500, 5000], 6, 2, 64),
    ([7], [30000], 4, 1, 128),
])
def test_parts_shared_by_warps(q_lens, kv_lens, Hq, Hk, d, hint):
    """Units cut into many parts, some rows of NaN among the others; the same bits on every run."""
    case = (q_lens, kv_lens, Hq, Hk, d, 32, True, True)
    q, pages, table, cu, lens = batch(case, seed=29)
    o, lse, reach = reference(q, pages, table, cu, lens, 0.09, True)
    q[1::5, 0] = float("nan")
    lse[1::5, 0] = np.nan
    args = (q, *pages, table.cuda(), cu.cuda(), lens.cuda())
    got, got_lse = fa.paged_forward(*args, scale=0.09, max_q=hint)
    assert status() == fa.FA_OK
    check(got, got_lse, (o, lse, reach))
    assert np.isnan(f64(got)[1::5, 0]).all() and np.isnan(f64(got_lse)[1::5, 0]).all()
    again, again_lse = fa.paged_forward(*args, scale=0.09, max_q=hint)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    assert torch.equal(got_lse.view(torch.int32), again_lse.view(torch.int32))


@pytest.mark.parametrize("d,page,q,hint", [(128, 16, 1, 1), (64, 32, 5, 5), (128, 64, 1, 200), (64, 128, 40, 200)])
def test_runs_of_many_tiles_and_units(d, page, q, hint):
    """Several units of several key tiles in each CTA's run, sequences that end inside a tile among them."""
    n = 48
    q_lens = [q if i % 3 else 1 for i in range(n)]
    kv_lens = [600 + (i * 397) % 1500 for i in range(n)]
    case = (q_lens, kv_lens, 16, 8, d, page, False, True)
    q, pages, table, cu, lens = batch(case)
    ref = reference(q, pages, table, cu, lens, d ** -0.5, True)
    o, lse = fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), max_q=hint)
    assert status() == fa.FA_OK
    check(o, lse, ref)


def test_more_sequences_than_threads():
    n = 1000
    q_lens = [(i * 7) % 3 for i in range(n)]
    kv_lens = [q + (i * 13) % 90 for i, q in enumerate(q_lens)]
    case = (q_lens, kv_lens, 2, 1, 64, 16, False, True)
    q, pages, table, cu, lens = batch(case)
    ref = reference(q, pages, table, cu, lens, 0.125, True)
    for hint in (2, 500):
        o, lse = fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), max_q=hint)
        assert status() == fa.FA_OK
        check(o, lse, ref)


def test_strided_queries_and_rows_behind_the_last_sequence():
    case = CASES[15]
    q, pages, table, cu, lens = batch(case)
    T, Hq, d = q.shape
    wide = torch.full((T + 3, Hq + 5, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:T, 2:2 + Hq] = q
    o = torch.full((T + 3, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 3, Hq), 4.0, device="cuda")
    for hint in (1, 300):
        fa.paged_forward(wide[:, 2:2 + Hq], *pages, table.cuda(), cu.cuda(), lens.cuda(), scale=0.11, max_q=hint,
                         out=o, lse=lse)
        assert status() == fa.FA_OK
        check(o[:T], lse[:T], reference(q, pages, table, cu, lens, 0.11, True))
        assert bool((o[T:] == 3.0).all()) and bool((lse[T:] == 4.0).all())


def test_pages_shared_between_sequences_and_no_lse():
    case = ([2, 1], [70, 70], 4, 2, 128, 32, False, True)
    q, pages, table, cu, lens = batch(case)
    table[1, :2] = table[0, :2]            # a common prefix
    ref = reference(q, pages, table, cu, lens, 0.1, True)
    o, lse = fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), scale=0.1)
    check(o, lse, ref)
    o2 = torch.empty_like(o)
    ws = torch.empty(fa.fa_fwd_paged_workspace_size(128), dtype=torch.uint8, device="cuda")
    t, c, n = table.cuda(), cu.cuda(), lens.cuda()
    k, v = pages
    st = fa.fa_fwd_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), o2.data_ptr(), None, t.data_ptr(), c.data_ptr(),
                         n.data_ptr(), 3, 2, 4, 2, 128, k.shape[0], 32, t.shape[1], *q.stride()[:2], *k.stride()[:3],
                         *v.stride()[:3], 0.1, 1, 0, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == fa.FA_OK and status() == fa.FA_OK
    check(o2, lse, ref)


@pytest.mark.parametrize("hint", [2, 400])
@pytest.mark.parametrize("page", [16, 128])
def test_bad_pages_and_lengths(hint, page):
    """Pages outside the pool are keys of zeros; lengths are cut to the table; the others are untouched."""
    kv_lens = [page + 3, 2 * page, 40, 2 * page]
    case = ([2, 2, 2, 2], kv_lens, 2, 1, 64, page, False, True)
    q, pages, table, cu, lens = batch(case)
    good = table.clone()
    table[1, 0], table[3, 1] = 10 ** 9, -1
    zero = pages[0].shape[0]                # the oracle's page of zeros
    ref_pages = [torch.cat([p, torch.zeros_like(p[:1])]) for p in pages]
    good[1, 0], good[3, 1] = zero, zero
    good[good < 0] = zero                   # (what lies behind a sequence's own pages in the table is outside too)
    long = lens.clone()
    long[1] = 2 * page + 99                 # behind the table: cut to its width
    cut = torch.clamp(long, max=table.shape[1] * page)
    ref = reference(q, ref_pages, good, cu, cut, 0.1, True)
    o, lse = fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), long.cuda(), scale=0.1, max_q=hint)
    assert status() == fa.FA_ERR_DEVICE_INDEX and status() == fa.FA_OK
    check(o, lse, ref)
    bad_cu = cu.clone()
    bad_cu[4] = 10 ** 6                     # past T: cut to it
    o, lse = fa.paged_forward(q, *pages, table.cuda(), bad_cu.cuda(), lens.cuda(), scale=0.1, max_q=hint)
    assert status() == fa.FA_ERR_DEVICE_INDEX
    check(o, lse, reference(q, ref_pages, good, cu, lens, 0.1, True))


def test_a_cache_past_32_bits():
    page, Hk, d = 64, 1, 128
    P = (1 << 31) // (page * 256) + 8                       # keys and values side by side in a row
    both = torch.zeros((P, Hk, page, 2 * d), dtype=torch.bfloat16, device="cuda")
    kp, vp = both[..., :d], both[..., d:]
    lens = torch.tensor([100], dtype=torch.int32)
    table = torch.tensor([[P - 1, P - 3]], dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    for p in (P - 1, P - 3):
        both[p] = torch.randn(Hk, page, 2 * d, generator=g).bfloat16().cuda()
    q = torch.randn(3, 2, d, generator=g).bfloat16().cuda()
    small = [torch.cat([x[P - 1:], x[P - 3:P - 2]]) for x in (kp, vp)]
    ref = reference(q, small, torch.tensor([[0, 1]]), ragged([3]), lens, 0.09, True)
    o, lse = fa.paged_forward(q, kp, vp, table.cuda(), ragged([3]).cuda(), lens.cuda(), scale=0.09)
    assert status() == fa.FA_OK
    check(o, lse, ref)


def test_graph_serves_changing_lengths_and_streams():
    """One captured step, replayed with other lengths, page tables and inputs; two graphs with a workspace each."""
    base = ([1, 6, 3], [90, 400, 3], 4, 2, 64, 16, False, True)
    other = ([4, 0, 6], [300, 77, 6], 4, 2, 64, 16, False, True)
    a, b = batch(base), batch(other, seed=40)
    rows = max(a[2].shape[1], b[2].shape[1])
    pad = lambda t: torch.nn.functional.pad(t, (0, rows - t.shape[1]))  # noqa: E731
    P = max(a[1][0].shape[0], b[1][0].shape[0])
    live = [torch.zeros((P, *a[1][0].shape[1:]), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    q, table, cu, lens = a[0].clone(), pad(a[2]).cuda(), a[3].cuda(), a[4].cuda()

    def put(x):
        for dst, src in zip(live, x[1]):
            dst[:src.shape[0]] = src
        q.copy_(x[0])
        table.copy_(pad(x[2]))
        cu.copy_(x[3])
        lens.copy_(x[4])

    args = (q, *live, table, cu, lens)
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        ws = torch.empty(fa.fa_fwd_paged_workspace_size(64), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fa.paged_forward(*args, scale=0.2, workspace=ws)
        graphs.append((graph, out, ws))    # the workspace lives as long as the graph that writes it
    for x in (a, b, a):
        put(x)
        ref = reference(x[0], x[1], x[2], x[3], x[4], 0.2, True)
        side.wait_stream(torch.cuda.current_stream())
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()          # at the same time
        eager = fa.paged_forward(*args, scale=0.2, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for o, lse in (graphs[0][1], graphs[1][1], eager):
            check(o, lse, ref)
    assert status() == fa.FA_OK


@pytest.mark.parametrize("Hq,Hk,d,page,inter", [(4, 4, 64, 16, False), (6, 2, 128, 64, True)])
def test_a_served_sequence_equals_the_whole_attention(Hq, Hk, d, page, inter):
    """Two sequences arrive in chunks and single tokens (append, then attention): the same rows as one causal pass
    over the whole sequences."""
    g = torch.Generator().manual_seed(77)
    N = [150, 41]
    qkv = [torch.randn(n, Hq + 2 * Hk, d, generator=g).bfloat16() for n in N]
    w = [(1 + 0.2 * torch.randn(d, generator=g)).bfloat16() for _ in "qk"]
    rope = fa.rope_table(max(N), d)
    (kp, vp), table = pool(N, Hk, d, page, True, 50)
    chunks = [(100, 7), (1, 1), (0, 1), (40, 31), (1, 0), (1, 1), (7, 0)]
    at, out, lses = [0, 0], [[], []], [[], []]
    for c in chunks:
        rows = torch.cat([x[a:a + n] for x, a, n in zip(qkv, at, c)]).cuda()
        at = [a + n for a, n in zip(at, c)]
        cu, lens = ragged(c).cuda(), torch.tensor(at, dtype=torch.int32).cuda()
        qn = fa.paged_append(rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:], kp, vp, table.cuda(), cu, lens,
                             *(t.cuda() for t in w), rope=rope, interleaved=inter)
        o, lse = fa.paged_forward(qn, kp, vp, table.cuda(), cu, lens, max_q=max(c))
        for s in range(2):
            out[s].append(o[cu[s]:cu[s + 1]])
            lses[s].append(lse[cu[s]:cu[s + 1]])
    assert status() == fa.FA_OK and at == N
    for s, x in enumerate(qkv):
        xs = x.cuda()[None].transpose(1, 2)                                      # [1, heads, N, d]
        qn, kn = fa.qk_norm_rope(xs[:, :Hq], xs[:, Hq:Hq + Hk], *(t.cuda() for t in w), rope=rope, interleaved=inter)
        kn, v = (t.repeat_interleave(Hq // Hk, 1).contiguous() for t in (kn, xs[:, Hq + Hk:]))
        o, lse = fa.forward(qn, kn, v, causal=True)
        ref = serve.paged_attention(f64(qn[0].transpose(0, 1)), f64(kn), f64(v), np.array([[0]]), [0, N[s]], [N[s]],
                                    d ** -0.5, True)
        check(torch.cat(out[s]), torch.cat(lses[s]), ref)
        check(o[0].transpose(0, 1), lse[0].T, ref)


@pytest.mark.parametrize("seed", range(40))
def test_any_mix_of_lengths(seed):
    """Batches drawn at random: every form, groups that divide nothing, empty sequences, chunks longer than their keys,
    lengths at tile borders; any hint; rows behind the batch untouched."""
    r = random.Random(seed)
    while True:
        d, G, S = r.choice([64, 128]), r.choice([1, 2, 3, 5, 8, 12, 20, 33, 100]), int(2 ** r.uniform(0, 7))
        Hk = r.choice([1, 2, 4, 16]) if G < 16 else 1
        long_q, long_kv = r.choice([1, 2, 6, 40, 150, 400]), r.choice([10, 130, 300, 1500])
        if S * long_kv < 30000 and S * long_q * (long_q + long_kv) * Hk * G < 6e6:
            break
    q_lens = [r.randint(0, long_q) if r.random() < 0.6 else 1 for _ in range(S)] + [1]
    kv_lens = [n + r.randint(0, long_kv) if r.random() < 0.9 else r.randint(0, long_kv) for n in q_lens]
    kv_lens = [n // 128 * 128 if r.random() < 0.1 else n for n in kv_lens]
    case = (q_lens, kv_lens, Hk * G, Hk, d, r.choice([16, 32, 128, 256]), r.random() < 0.5, r.random() < 0.8)
    q, pages, table, cu, lens = batch(case, seed=seed)
    T = q.shape[0]
    ref = reference(q, pages, table, cu, lens, 0.1, case[7])
    q = torch.cat([q, q[:1].expand(3, -1, -1)])
    for hint in (0, max(q_lens), r.choice([1, 3, 50, 10 ** 6])):
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        fa.paged_forward(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), scale=0.1, causal=case[7], max_q=hint, out=o,
                         lse=lse)
        assert status() == fa.FA_OK
        check(o[:T], lse[:T], ref)
        assert (o[T:] == 7).all() and (lse[T:] == 7).all()


def test_strides_of_single_elements_mean_nothing():
    """A dimension of size 1 may come with any stride: one page, one key head, one token, one row."""
    g = torch.Generator().manual_seed(31)
    d, page = 64, 16
    new = lambda *n: torch.randn(n, generator=g).bfloat16().cuda()
    q, k, v, kp, vp = new(1, 4, d), new(1, 1, d), new(1, 1, d), new(1, 1, page, d), new(1, 1, page, d)
    rope = fa.rope_table(page, d)
    table, cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0]], [0, 1], [9]))
    odd = lambda t, *steps: torch.as_strided(t, t.shape, steps)
    kp2, vp2 = kp.clone(), vp.clone()
    plain = fa.paged_append(q, k, v, kp, vp, table, cu, lens, rope=rope)
    strange = fa.paged_append(odd(q, 3, d, 1), odd(k, 5, 0, 1), odd(v, 0, 1, 1), odd(kp2, 1, 3, d, 1), odd(vp2, 0, 0, d, 1),
                              table, cu, lens, rope=rope)
    assert torch.equal(plain, strange) and torch.equal(kp, kp2) and torch.equal(vp, vp2)
    for a, b in zip(fa.paged_forward(plain, kp, vp, table, cu, lens),
                    fa.paged_forward(odd(plain, 7, d, 1), odd(kp, 1, 3, d, 1), odd(vp, 0, 0, d, 1), table, cu, lens)):
        assert torch.equal(a, b)
    x, y = new(1, 2, 8, d), new(1, 1, 8, d)
    for a, b in zip(fa.qk_norm_rope(x, y), fa.qk_norm_rope(odd(x, 9, 8 * d, d, 1), odd(y, 1, 2, d, 1))):
        assert torch.equal(a, b)
    for a, b in zip(fa.qk_norm_rope_backward(x, y, x, y),
                    fa.qk_norm_rope_backward(x, y, odd(x, 9, 8 * d, d, 1), odd(y, 1, 2, d, 1))):
        assert torch.equal(a, b)
    assert status() == fa.FA_OK


def test_helpers_refuse_on_the_host():
    """What would be read or written at a wrong address is refused before any launch."""
    case = CASES[3]
    q, pages, table, cu, lens = batch(case)
    good = dict(q=q, k_pages=pages[0], v_pages=pages[1], page_table=table.cuda(), cu_seqlens=cu.cuda(), kv_lens=lens.cuda())
    fa.paged_forward(**good)
    room = torch.empty(fa.fa_fwd_paged_workspace_size(case[4]), dtype=torch.uint8)
    for bad in (dict(workspace=room), dict(page_table=table), dict(kv_lens=lens.cuda().long()), dict(kv_lens=lens.cuda()[:-1]),
                dict(cu_seqlens=cu.cuda()[:-1]), dict(page_table=table.cuda().t()), dict(q=q.float()), dict(q=q[..., :64]),
                dict(v_pages=pages[1].cpu()), dict(v_pages=pages[1][:, :1]), dict(out=torch.empty_like(q).float()),
                dict(out=torch.empty(q.shape, dtype=q.dtype)), dict(lse=torch.empty(q.shape[:2], device="cuda").t()),
                dict(q=q[0])):
        with pytest.raises(ValueError):
            fa.paged_forward(**good | bad)
    for bad in (dict(workspace=room.cuda()[:-1].clone()), dict(max_q=-1), dict(q=q[:, :3])):
        with pytest.raises(fa.FaError):
            fa.paged_forward(**good | bad)
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)), dict(q_weight=torch.ones(64)),
                dict(grads=(x.cpu(), x)), dict(positions=torch.zeros(1, 8, device="cuda")), dict(rope=torch.zeros(8, 64))):
        with pytest.raises(ValueError):
            fa.qk_norm_rope_backward(x, x, x, x, **bad)
    assert status() == fa.FA_OK
