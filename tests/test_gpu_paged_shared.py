"""Attention of a batch whose sequences share keys against the fp64 form (needs a GB300).

Tolerances are those of tests/test_gpu_paged.py (its ``check``): the output's rounding, that of the probabilities, and
the scores' error.  The parts of a row are joined in fp32: a weight 2^(m_i - m) has a relative error of a few 2^-23,
and there are at most some hundred parts, far below the 2^-11 that the scores' error is allowed.
"""

import random

import numpy as np
import pytest
import torch

import exact_io_aware_31_gb300 as fa
from tests.gpu_util import f64, require_gpu
from tests.test_gpu_norm_rope import pool, ragged, status
from tests.test_gpu_paged import check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# groups: (keys in shared pages, ((new tokens, keys behind the shared ones), ...)); a group of 0 shared keys is none
SHAPES = {
    "two": ([(1024, [(1, 1), (1, 1)])], 4, 4),
    "samples": ([(512, [(1, 5 + i) for i in range(9)])], 8, 2),
    "one tile": ([(768, [(1, 1 + 17 * i) for i in range(11)])], 12, 3),                     # 44 rows
    "two tiles": ([(1280, [(1, 200 - i) for i in range(50)])], 4, 1),                       # 200 rows
    "many rows": ([(640, [(1, 1 + i % 7) for i in range(150)])], 8, 2),                     # three units of tokens
    "groups": ([(1024, [(1, 3)] * 4), (512, [(2, 40), (3, 9), (1, 130)]), (2048, [(1, 1)] * 6)], 4, 2),
    "odd group": ([(900, [(5, 5 + i) for i in range(12)])], 10, 2),
    "loners": ([(0, [(1, 300)]), (1024, [(1, 3)] * 5), (0, [(4, 40)]), (0, [(1, 1)])], 4, 2),
    "empty": ([(1024, [(0, 0), (1, 3), (0, 50), (2, 2), (1, 700), (0, 0)]), (1024, []), (512, [(0, 9)] * 2)], 4, 4),
    "chunks": ([(1500, [(40, 40), (1, 9), (150, 200), (3, 3)])], 4, 1),
    "long chunks": ([(300, [(260, 260), (130, 140)])], 2, 1),
    "heads of one key head": ([(2000, [(1, 4)] * 7)], 64, 1),
    "tile a token": ([(600, [(1, 4)] * 3)], 128, 1),
    "16 rows": ([(1300, [(1, 200 + 90 * i) for i in range(7)]), (0, [(1, 1), (1, 700)])], 32, 2),
    "20 heads a key head": ([(800, [(1, 500), (1, 31), (1, 33)])], 20, 1),
    "32 heads a key head": ([(600, [(1, 450), (1, 7)] * 3)], 64, 2),
    "long": ([(9000, [(1, 20)] * 5)], 2, 1),                                                # cut into many parts
    "long, two tiles": ([(12000, [(1, 20 + i) for i in range(70)])], 4, 1),
}
FORMS = [(64, 16, False, True), (128, 32, True, True), (128, 128, False, True), (64, 256, False, False)]


def batch(groups, Hq, Hk, d, page, token_major, seed=11, wide=1.0):
    """Queries, pools, table, cu_seqlens, kv_lens, groups, prefix_lens.  Shared keys lie in shared pages as far as
    those are full; what is left over in the last one is copied."""
    q_lens, kv_lens, starts, prefix = [], [], [], []
    for keys, seqs in groups:
        starts.append(len(q_lens))
        prefix.append(keys)
        for n, own in seqs:
            q_lens.append(n)
            kv_lens.append(keys + own if n or own else 0)
    starts.append(len(q_lens))
    pages, table = pool(kv_lens, Hk, d, page, token_major, seed)
    for g, (keys, seqs) in enumerate(groups):
        live = [s for s in range(starts[g], starts[g + 1]) if kv_lens[s] >= keys]
        for s in live[1:]:
            full = keys // page
            table[s, :full] = table[live[0], :full]
            if keys % page:
                for p in pages:
                    p[table[s, full].long(), :, :keys % page] = p[table[live[0], full].long(), :, :keys % page]
    cu = ragged(q_lens)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(int(cu[-1]), Hq, d, generator=g) * wide).bfloat16().cuda()
    ints = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return q, pages, table, cu, ints(kv_lens), ints(starts), ints(prefix)


def call(x, **kw):
    q, pages, table, cu, lens, groups, prefix = x
    return fa.paged_forward_shared(q, *pages, table.cuda(), cu.cuda(), lens.cuda(), groups.cuda(), prefix.cuda(), **kw)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"d{f[0]}p{f[1]}{'t' if f[2] else ''}{'c' if f[3] else ''}")
@pytest.mark.parametrize("shape", SHAPES)
def test_against_the_oracle(shape, form):
    d, page, token_major, causal = form
    x = batch(*SHAPES[shape], d, page, token_major)
    ref = reference(*x[:5], 0.11, causal)
    o, lse = call(x, scale=0.11, causal=causal)
    assert status() == fa.FA_OK
    check(o, lse, ref)


@pytest.mark.parametrize("hint", [1, 2, 5, 10 ** 6])
@pytest.mark.parametrize("shape", ["groups", "odd group", "16 rows", "empty", "loners"])
def test_hints(shape, hint):
    """The hint moves entries from one kernel to the other; all give the same attention."""
    x = batch(*SHAPES[shape], 128, 32, False)
    o, lse = call(x, scale=0.11, max_q=hint)
    assert status() == fa.FA_OK
    check(o, lse, reference(*x[:5], 0.11, True))


@pytest.mark.parametrize("Hq,Hk,d", [(32, 8, 128), (16, 16, 64), (16, 1, 128), (24, 1, 64)])
def test_more_units_than_ctas(Hq, Hk, d):
    """Every CTA takes several units, of one stage to a dozen, from the counter; the longest entries come in parts."""
    lens = [1 + 37 * i % 401 for i in range(180)]
    x = batch([(256, [(1, n) for n in lens[:90]]), (0, [(1, n) for n in lens[90:]] + [(1, 5000)])], Hq, Hk, d, 16, True)
    want = call(x, scale=0.2, max_q=1)
    assert status() == fa.FA_OK
    check(*want, reference(*x[:5], 0.2, True))
    for _ in range(3):                     # whichever CTA takes which unit
        assert all(torch.equal(a, b) for a, b in zip(call(x, scale=0.2, max_q=1), want))


@pytest.mark.parametrize("Hq,Hk,d,most", [(20, 4, 128, 5), (20, 4, 64, 5), (8, 2, 128, 8), (8, 2, 64, 8), (16, 1, 128, 2),
                                          (17, 1, 64, 1)])
def test_units_of_one_and_of_two_row_tiles(Hq, Hk, d, most):
    """Entries of 1 to 32 rows side by side, more than CTAs, whose second tile has rows or none; NaN in one token's
    query reaches no other one's rows."""
    seqs = [(1 + i % most, most + 53 * i % 611) for i in range(190)]
    x = batch([(256, seqs[:80]), (0, seqs[80:] + [(most, 4000)])], Hq, Hk, d, 32, False)
    want = call(x, scale=0.2, max_q=most)
    assert status() == fa.FA_OK
    check(*want, reference(*x[:5], 0.2, True))
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(call(x, scale=0.2, max_q=most), want))
    x[0][int(x[3][100])] = float("nan")    # the first token of sequence 100
    o, lse = call(x, scale=0.2, max_q=most)
    bad = torch.isnan(o.float()).any(-1).any(-1)
    assert bad.nonzero().flatten().tolist() == [int(x[3][100])]


@pytest.mark.parametrize("scale", [-0.1, 0.0])
@pytest.mark.parametrize("shape", ["samples", "chunks"])
def test_scales(shape, scale):
    x = batch(*SHAPES[shape], 64, 32, False)
    o, lse = call(x, scale=scale)
    check(o, lse, reference(*x[:5], scale, True))


@pytest.mark.parametrize("shape", ["one tile", "groups", "long, two tiles"])
def test_wide_rows(shape):
    x = batch(*SHAPES[shape], 128, 32, False, wide=8.0)
    o, lse = call(x)
    check(o, lse, reference(*x[:5], 128 ** -0.5, True), wide=8.0)


@pytest.mark.parametrize("shape,shared", [("samples", 512), ("two tiles", 1280), ("long", 8960)])
def test_the_shared_keys_are_the_first_sequences(shape, shared):
    """Where the sequences' own copies differ (which the contract forbids), the first one's keys and values count: so
    they are read once.  What is shared is the keys in whole tiles."""
    groups, Hq, Hk = SHAPES[shape]
    q, pages, table, cu, lens, starts, prefix = batch(groups, Hq, Hk, 64, 16, False)
    apart, at = table.clone(), pages[0].shape[0]
    n = shared // 16
    extra = [torch.randn(n * (len(lens) - 1), *p.shape[1:], device="cuda").bfloat16() for p in pages]
    for s in range(1, len(lens)):
        apart[s, :n] = torch.arange(at, at + n)
        at += n
    pages = [torch.cat([p, e]) for p, e in zip(pages, extra)]
    o, lse = call((q, pages, apart, cu, lens, starts, prefix), scale=0.11)
    assert status() == fa.FA_OK
    check(o, lse, reference(q, pages, table, cu, lens, 0.11, True))


@pytest.mark.parametrize("claim", [0, 1, 127, 128, 500, 10 ** 9])
def test_any_true_length_is_right(claim):
    """From none of the shared keys to more than a sequence has in front of its new tokens (the same pages serve all)."""
    q, pages, table, cu, lens, starts, prefix = batch([(1024, [(1, 1), (3, 3), (1, 90), (20, 20)])], 4, 2, 64, 16, False)
    ref = reference(q, pages, table, cu, lens, 0.11, True)
    for causal in (True, False):
        prefix[0] = min(claim, table.shape[1] * 16) if claim < 10 ** 9 else 1024
        o, lse = call((q, pages, table, cu, lens, starts, prefix), scale=0.11, causal=causal)
        assert status() == fa.FA_OK
        check(o, lse, ref if causal else reference(q, pages, table, cu, lens, 0.11, False))


def test_a_prefix_longer_than_a_sequence():
    """Two sequences of the group hold 1024 of the keys, one 300 and one 0: what is shared is cut to what all hold."""
    for kv in ([1025, 301, 1025], [1025, 1, 1025], [1025, 0, 1025]):
        q, pages, table, cu, lens, starts, _ = batch([(0, [(1, n) for n in (1025, 1025, 1025)])], 8, 1, 64, 32, False)
        table[1:, :32] = table[0, :32]
        lens = torch.tensor(kv, dtype=torch.int32)
        x = (q, pages, table, cu, lens, starts, torch.tensor([1024], dtype=torch.int32))
        o, lse = call(x, scale=0.2)
        assert status() == fa.FA_OK
        check(o, lse, reference(*x[:5], 0.2, True))


@pytest.mark.parametrize("n", [0, 1])
def test_no_groups(n):
    q, pages, table, cu, lens, _, _ = batch(*SHAPES["loners"], 128, 16, False)
    x = (q, pages, table, cu, lens, torch.tensor([len(lens)] * (n + 1), dtype=torch.int32),
         torch.zeros(n, dtype=torch.int32))
    o, lse = call(x, scale=0.11)
    assert status() == fa.FA_OK
    check(o, lse, reference(*x[:5], 0.11, True))


def test_many_sequences_and_groups():
    """More of both than the plan's block has threads; every group of two to four, some that are not worth it."""
    rng = random.Random(4)
    groups = [(rng.choice([0, 130, 520, 1100]), [(1, rng.randint(1, 9))] * rng.randint(2, 4)) for _ in range(1100)]
    x = batch(groups, 1, 1, 64, 16, False)
    assert len(x[4]) > 2048
    o, lse = call(x, scale=0.2)
    assert status() == fa.FA_OK
    check(o, lse, reference(*x[:5], 0.2, True))


@pytest.mark.parametrize("groups", [4096, 4097])
def test_limit_of_groups(groups):
    x = list(batch([(0, [(1, 9)])] * 3, 1, 1, 64, 16, False))
    x[5] = torch.cat([x[5][:3], torch.full((groups - 2,), 3, dtype=torch.int32)])
    x[6] = torch.zeros(groups, dtype=torch.int32)
    if groups > 4096:
        with pytest.raises(fa.FaError) as e:
            call(x, workspace=torch.empty(1 << 27, dtype=torch.uint8, device="cuda"))
        assert e.value.status == fa.FA_ERR_UNSUPPORTED
    else:
        check(*call(x), reference(*x[:5], 0.125, True))


@pytest.mark.parametrize("shape", ["samples", "one tile", "groups", "long, two tiles", "chunks"])
def test_a_query_of_nan_is_seen(shape):
    x = batch(*SHAPES[shape], 64, 32, False)
    o, lse, reach = reference(*x[:5], 0.11, True)
    poisoned = torch.zeros(x[0].shape[:2], dtype=torch.bool)
    poisoned[::3, ::2] = True
    x[0].masked_fill_(poisoned[..., None].cuda(), float("nan"))
    lse = np.where(poisoned.numpy() & np.isfinite(lse), np.nan, lse)
    got, got_lse = call(x, scale=0.11)
    assert status() == fa.FA_OK
    check(got, got_lse, (o, lse, reach))
    assert np.isnan(f64(got)[np.isnan(lse)]).all() and np.isnan(f64(got_lse)[np.isnan(lse)]).all()


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape", ["samples", "groups", "empty", "chunks"])
def test_what_lies_behind_a_sequence_does_not_matter(shape, fill):
    groups, Hq, Hk = SHAPES[shape]
    q, pages, table, cu, lens, starts, prefix = x = batch(groups, Hq, Hk, 64, 32, False)
    ref = reference(*x[:5], 0.11, True)
    owned = torch.zeros(pages[0].shape[0], 32, dtype=torch.bool)
    for s, n in enumerate(lens.tolist()):
        for j in range(n):
            owned[table[s, j // 32], j % 32] = True
    for p in pages:
        p.masked_fill_(~owned[:, None, :, None].cuda(), fill)
    o, lse = call(x, scale=0.11)
    assert status() == fa.FA_OK
    check(o, lse, ref)


@pytest.mark.parametrize("shape", ["groups", "many rows", "long, two tiles", "loners"])
def test_any_workspace_and_the_same_bits(shape):
    """Whatever the workspace holds, and whoever used it before."""
    x = batch(*SHAPES[shape], 128, 16, False)
    T, Hq = x[0].shape[:2]
    need = fa.fa_fwd_paged_shared_workspace_size(T, len(x[4]), len(x[6]), Hq, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    want = call(x, workspace=ws)
    check(*want, reference(*x[:5], 128 ** -0.5, True))
    for fill in (0, 0x80, 0x7f, None):
        if fill is None:                          # leftovers of other work
            call(batch(*SHAPES["two"], 128, 16, False), workspace=ws)
        else:
            ws.fill_(fill)
        got = call(x, workspace=ws)
        assert status() == fa.FA_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(fa.FaError) as e:
        call(x, workspace=ws[:-256])
    assert e.value.status == fa.FA_ERR_WORKSPACE


def test_strided_queries_rows_of_no_sequence_and_no_lse():
    groups, Hq, Hk = SHAPES["groups"]
    q, pages, table, cu, lens, starts, prefix = batch(groups, Hq, Hk, 64, 32, False)
    T = q.shape[0]
    wide = torch.full((T + 5, 3 * Hq, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = wide[:, Hq:2 * Hq]
    view[2:T + 2] = q
    ref = reference(q, pages, table, cu, lens, 0.11, True)
    o = torch.full((T + 5, Hq, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 5, Hq), 4.0, device="cuda")
    call((view, pages, table, cu + 2, lens, starts, prefix), scale=0.11, out=o, lse=lse)
    assert status() == fa.FA_OK
    check(o[2:T + 2], lse[2:T + 2], ref)
    for rows in (slice(0, 2), slice(T + 2, None)):
        assert bool((o[rows] == 3.0).all()) and bool((lse[rows] == 4.0).all())
    need = fa.fa_fwd_paged_shared_workspace_size(T, len(lens), len(prefix), Hq, 64)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    t, c, n, g, x = (v.cuda() for v in (table, cu, lens, starts, prefix))
    o2 = torch.empty_like(q)
    k, v = pages
    st = fa.fa_fwd_paged_shared(q.data_ptr(), k.data_ptr(), v.data_ptr(), o2.data_ptr(), None, t.data_ptr(),
                                c.data_ptr(), n.data_ptr(), g.data_ptr(), x.data_ptr(), T, len(lens), len(prefix), Hq,
                                Hk, 64, k.shape[0], 32, t.shape[1], *q.stride()[:2], *k.stride()[:3], *v.stride()[:3],
                                0.11, 1, 0, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == fa.FA_OK and status() == fa.FA_OK
    check(o2, lse[2:T + 2], ref)


def test_bad_groups_prefixes_and_pages():
    """What is out of range is cut to it and said; the sequences that it does not touch are right."""
    groups, Hq, Hk = [(1024, [(1, 3)] * 4), (512, [(2, 40)] * 6)], 4, 2
    q, pages, table, cu, lens, starts, prefix = x = batch(groups, Hq, Hk, 64, 32, False)
    ref = reference(*x[:5], 0.11, True)
    for st, pre in ((torch.tensor([-5, 4, 99]), prefix), (starts, torch.tensor([-3, 512])),
                    (starts, torch.tensor([10 ** 9, 512])), (torch.tensor([0, 4, 2]), prefix)):
        o, lse = call((q, pages, table, cu, lens, st.to(torch.int32), pre.to(torch.int32)), scale=0.11)
        assert status() == fa.FA_ERR_DEVICE_INDEX and status() == fa.FA_OK
        check(o, lse, ref)                        # (each of these still says nothing untrue of these pages)
    good = table.clone()
    table[4:, 2] = pages[0].shape[0]              # a shared page outside the pool is keys of zeros
    good[4:, 2] = pages[0].shape[0]
    zeros = [torch.cat([p, torch.zeros_like(p[:1])]) for p in pages]
    o, lse = call((q, pages, table, cu, lens, starts, prefix), scale=0.11)
    assert status() == fa.FA_ERR_DEVICE_INDEX
    check(o, lse, reference(q, zeros, good, cu, lens, 0.11, True))


def test_graph_serves_changing_groups_and_streams():
    """One captured step, replayed with other groups, lengths and pages; two graphs at once with a workspace each."""
    steps = [batch([(512, [(1, 4)] * 5), (0, [(3, 9)])], 4, 2, 64, 16, False),
             batch([(0, [(2, 90)]), (1024, [(1, 7)] * 3 + [(3, 3)])], 4, 2, 64, 16, False, seed=40)]
    steps.append(batch([(256, [(1, 1)] * 2), (700, [(2, 30)] * 3)], 4, 2, 64, 16, False, seed=50))
    cols = max(x[2].shape[1] for x in steps)
    P = max(x[1][0].shape[0] for x in steps)
    live = [torch.zeros((P, *steps[0][1][0].shape[1:]), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    S, T = 6, 8
    q, table = torch.zeros(T, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(S, cols, dtype=torch.int32).cuda()
    cu, lens = torch.zeros(S + 1, dtype=torch.int32).cuda(), torch.zeros(S, dtype=torch.int32).cuda()
    groups, prefix = torch.zeros(3, dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()

    def put(x):
        for dst, src in zip(live, x[1]):
            dst[:src.shape[0]] = src
        n, t = len(x[4]), x[0].shape[0]
        q[:t] = x[0]
        table[:n, :x[2].shape[1]] = x[2].cuda()
        cu[:n + 1] = x[3].cuda()
        cu[n + 1:] = t                             # places without a sequence
        lens.zero_()
        lens[:n] = x[4].cuda()
        groups.copy_(x[5])
        prefix.copy_(x[6])
        return t

    args = (q, *live, table, cu, lens, groups, prefix)
    side, graphs = torch.cuda.Stream(), []
    for _ in range(2):
        ws = torch.empty(fa.fa_fwd_paged_shared_workspace_size(T, S, 2, 4, 64), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fa.paged_forward_shared(*args, scale=0.2, workspace=ws)
        graphs.append((graph, out, ws))
    for x in (*steps, steps[0]):
        t = put(x)
        ref = reference(*x[:5], 0.2, True)
        side.wait_stream(torch.cuda.current_stream())
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        eager = fa.paged_forward_shared(*args, scale=0.2, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert status() == fa.FA_OK
        for o, lse in (graphs[0][1], graphs[1][1], eager):
            check(o[:t], lse[:t], ref)


@pytest.mark.parametrize("seed", range(24))
def test_any_mix_of_groups(seed):
    rng = random.Random(100 + seed)
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256])
    Hk = rng.choice([1, 2, 3])
    Hq = Hk * rng.choice([1, 2, 3, 4, 7, 16])
    groups = []
    for _ in range(rng.randint(1, 5)):
        n = rng.choice([1, 1, rng.randint(2, 5), rng.randint(6, 60)])
        most = rng.choice([1, 1, 1, 4, 60])
        seqs = [(q, q + rng.randint(0, 150)) for q in (rng.randint(0, most) for _ in range(rng.randint(0, 30)))]
        groups.append((rng.choice([0, rng.randint(1, 400), rng.randint(400, 4000)]) * (n > 0), seqs))
    if not any(q for _, seqs in groups for q, _ in seqs):
        groups.append((300, [(1, 1)] * 3))
    causal = rng.random() < 0.8
    x = batch(groups, Hq, Hk, d, page, rng.random() < 0.5, seed=seed)
    o, lse = call(x, scale=0.13, causal=causal, max_q=rng.choice([0, 1, 60]))
    assert status() == fa.FA_OK
    check(o, lse, reference(*x[:5], 0.13, causal))


def test_helpers_refuse_on_the_host():
    q, pages, table, cu, lens, groups, prefix = (
        x if isinstance(x, list) else x.cuda() for x in batch(*SHAPES["two"], 64, 16, False))
    good = (q, *pages, table, cu, lens, groups, prefix)
    for i, bad in ((6, groups[:1]), (6, groups.long()), (6, groups.cpu()), (7, prefix.float()), (7, prefix[None]),
                   (3, table.long()), (0, q.float())):
        with pytest.raises(ValueError):
            fa.paged_forward_shared(*good[:i], bad, *good[i + 1:])
    assert status() == fa.FA_OK
