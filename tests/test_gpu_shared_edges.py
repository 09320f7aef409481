"""Shared keys and the cache's tables at the edges of what their calls allow (needs a GB300).

Tolerances are those of tests/test_gpu_paged.py (its ``check``); tables are whole numbers and equal the plain form's.
"""

import random

import numpy as np
import pytest
import torch

import exact_io_aware_31_gb300 as fa
from tests.gpu_util import require_gpu
from tests.test_gpu_norm_rope import status
from tests.test_gpu_paged import check, reference
from tests.test_gpu_paged_shared import batch, call
from tests.test_gpu_paged_tables import OLD, State, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("groups", [0, 1])
@pytest.mark.parametrize("what", ["keys", "rows"])
@pytest.mark.parametrize("S,at", [(3, 2), (300, 299), (600, 511), (600, 512), (600, 599), (1300, 1024)])
def test_lengths_of_every_sequence_are_checked(S, at, what, groups):
    """More sequences than the plan's block has threads, with groups and without: a length out of range is said
    wherever it stands, and the other sequences are right."""
    q, pages, table, cu, lens, _, _ = batch([(0, [(1, 1 + i % 40) for i in range(S)])], 2, 1, 64, 16, False)
    if what == "keys":
        lens[at] = -1                             # no keys, then: a row of zeros
    else:
        cu[at + 1:] += 3                          # three rows more, the last ones behind the batch
        q = torch.cat([q, q[:3]])
        cu[-1] += 7                               # (cut to the batch's rows)
    x = (q, pages, table, cu, lens, torch.tensor([S] * (groups + 1), dtype=torch.int32),
         torch.zeros(groups, dtype=torch.int32))
    o, lse = call(x, scale=0.2)
    assert status() == fa.FA_ERR_DEVICE_INDEX and status() == fa.FA_OK
    good = lens.clamp_min(0), cu.clamp_max(q.shape[0])
    check(o, lse, reference(q, pages, table, good[1], good[0], 0.2, True))


@pytest.mark.parametrize("page", [-1, 9, 2 ** 31 - 1])
def test_a_page_outside_of_the_pool_has_no_slots(page):
    """In a request's row, or come back to the pool from there: tokens in it have the slot -1, and every call that
    meets it says so."""
    s = State([40], 4, 16, 9)
    s.table[0, 2] = s.plain.table[0, 2] = page    # the page that the next tokens go to
    _, _, _, _, slots = s.extend([0], [12])
    assert (slots < 0).tolist() == [True] * 8 + [False] * 4
    s.table[0, 1] = s.plain.table[0, 1] = page    # one that no new token goes to
    s.extend([0], [3])
    s.release([0])
    s = State([40, 0, 0], 4, 16, 9)
    s.table[0, 1] = s.plain.table[0, 1] = page
    s.release([0])
    got = s.extend([2, 1], [16, 40])              # takes all that came back
    assert (got[4] >= 0).sum() == 16 + 40 - 16
    s.extend([-1, 1], [0, 0])
    s.release([1, 2], [33, 16])
    s.extend([0], [5])


def test_pages_outside_of_the_pool_among_many():
    """More sequences than a block looks at: whichever block meets the page says so."""
    s = State([300] * 700, 40, 16, 700 * 19 + 700 * 2 + 5)
    s.table[650, 3] = s.plain.table[650, 3] = -4
    s.extend(list(range(700)), [1 + i % 9 for i in range(700)])
    s.extend([650], [1])
    s.extend([r for r in range(700) if r != 650], [20] * 699)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hk,d,dead,seqs", [
    (8, 2, 64, (3,), [(1, 5 + i) for i in range(9)]),
    (8, 2, 128, (0, 4, 8), [(1, 5 + i) for i in range(9)]),                            # the first and the last one
    (4, 1, 64, (0, 1, 30, 31, 32, 69), [(1, 200 - i) for i in range(70)]),             # 280 rows, two units of them
    (8, 2, 64, (0, 4, 9), [(40, 40), (1, 3), (3, 3), (1, 9), (9, 9), (2, 2)] + [(1, 4)] * 3 + [(150, 150)]),  # chunks
    (32, 1, 64, (1,), [(1, 40), (1, 2), (1, 30)]),
    (64, 1, 128, (1,), [(1, 4)] * 7),
])
def test_a_sequence_that_was_left_out_keeps_no_group_from_sharing(Hq, Hk, d, dead, seqs, causal):
    """Tokens of a sequence without keys (its pages were not there) see nothing, and the keys of the others are
    shared all the same: those of the first that has some count, as each has copies of its own that differ."""
    q, pages, table, cu, lens, starts, prefix = batch([(1280, seqs), (0, [(1, 70)])], Hq, Hk, d, 16, False)
    live = [s for s in range(len(seqs)) if s not in dead]
    for s in dead:
        lens[s] = 0
        table[s] = -7
    apart, at, n = table.clone(), pages[0].shape[0], 1280 // 16
    extra = [torch.randn(n * (len(live) - 1), *p.shape[1:], device="cuda").bfloat16() for p in pages]
    for s in live[1:]:
        apart[s, :n] = torch.arange(at, at + n)
        at += n
    pages = [torch.cat([p, e]) for p, e in zip(pages, extra)]
    o, lse = call((q, pages, apart, cu, lens, starts, prefix), scale=0.11, causal=causal)
    assert status() == fa.FA_OK
    check(o, lse, reference(q, pages, table, cu, lens, 0.11, causal))


def test_a_pool_that_runs_out_keeps_no_group_from_sharing():
    """Six requests behind a prompt, pages for five of them: the sixth is left out of the step, the others share."""
    page, max_pages, n, P = 16, 100, 64, 6 * 100
    lens, table = ints([0] + [n * page] * 6), torch.full((7, max_pages), -5, dtype=torch.int32, device="cuda")
    pool = fa.paged_pool(P)
    free = ints(list(range(P - 1, n + 6 * n - 1, -1)))
    pool[0] = 5                                   # five pages are left
    pool[2:7] = free[:5]
    for r in range(1, 7):                         # each with a copy that differs: the first one's counts
        table[r, :n] = torch.arange((r - 1) * n, r * n, dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    pages = [torch.randn(P, 2, page, 64, generator=g).bfloat16().cuda() for _ in "kv"]
    q = torch.randn(6, 8, 64, generator=g).bfloat16().cuda()
    cu, kv, pt, _, slots = fa.paged_extend(ints([1, 2, 3, 4, 5, 6]), ints([1] * 6), lens, table, pool, page, 6)
    assert status() == fa.FA_ERR_DEVICE_INDEX
    assert kv.tolist() == [n * page + 1] * 5 + [0] and slots.tolist()[5] == -1
    o, lse = fa.paged_forward_shared(q, *pages, pt, cu, kv, ints([0, 6]), ints([n * page]), scale=0.2)
    assert status() == fa.FA_OK
    want = pt.cpu()
    want[:5, :n] = want[0, :n]
    want[5] = -7
    check(o, lse, reference(q, pages, want, cu.cpu(), kv.cpu(), 0.2, True))


@pytest.mark.parametrize("tokens", [0, 1, 300])
def test_a_step_without_sequences(tokens):
    """Its rows are all behind the last sequence."""
    s = State([20, 0], 4, 16, 9)
    got = s.extend([], [], tokens=tokens)         # (into tensors that hold the step before's values)
    assert got[0].tolist() == [0] and (got[3] == 0).all() and (got[4] == -1).all()
    s.extend([], [], tokens=tokens, wanted=(False, True))
    s.extend([], [], tokens=tokens, wanted=(True, False))
    torch.full((4096,), OLD, dtype=torch.int64, device="cuda")   # what the next tensors may be made of
    cu, kv, table, positions, slots = fa.paged_extend(ints([]), ints([]), s.lens, s.table, s.pool, 16, tokens)
    assert cu.tolist() == [0] and kv.shape == (0,) and table.shape == (0, 4)
    assert positions.tolist() == [0] * tokens and slots.tolist() == [-1] * tokens
    out = (ints([OLD]), ints([]), ints(np.zeros((0, 4))), ints([OLD] * tokens),
           torch.full((tokens,), OLD, dtype=torch.int64, device="cuda"))
    none = ints([])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.paged_extend(none, none, s.lens, s.table, s.pool, 16, tokens, out=out, stream=torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    assert out[0].tolist() == [0] and (out[3] == 0).all() and (out[4] == -1).all()
    s.release([])


@pytest.mark.parametrize("tokens", [2 ** 31 - 1, 2 ** 31 - 127, 2 ** 31 - 128])
def test_the_most_rows(tokens):
    """A count of rows next to 2^31, maps not wanted: the tables are written."""
    s = State([20, 0, 64, 33], 8, 16, 24)
    batch, new = [2, -1, 0, 3], [3, 0, 20, 1]
    out = (ints([OLD] * 5), ints([OLD] * 4), ints(np.full((4, 8), OLD)), None, None)
    fa.paged_extend(ints(batch), ints(new), s.lens, s.table, s.pool, 16, tokens, out=out)
    want = s.plain.extend(batch, new, 24, np.full((4, 8), OLD))
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(out[:3], want[:3]))
    s.same()


@pytest.mark.parametrize("tokens", [-1, 2 ** 31])
def test_rows_that_cannot_be_are_refused_before_anything_is_made(tokens):
    s = State([20], 4, 16, 9)
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    with pytest.raises(ValueError):
        fa.paged_extend(s.lens, s.lens, s.lens, s.table, s.pool, 16, tokens)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    s.same()


@pytest.mark.parametrize("kept", [-1, 5, 2 ** 31 - 1, -2 ** 31])
def test_counts_of_shared_pages_that_cannot_be(kept):
    """A request whose count is outside of its row stays as it was; the others give their pages back."""
    s = State([20, 0, 64, 33], 4, 16, 16)
    s.release([0, 2, 3], [5, 0, 40], [0, 0, kept, 1])          # keeps more than it has, besides
    s.release([2, 0, 3, 1], [16, 0, 1, 0], [0, kept, kept, 4])
    s.release([0, 3], None, [kept, 0, 0, 1])
    s.release([0, 3], None, [4, 0, 0, 0])                       # as many as a row may have: none is its own
    s.release([0, 1])


def test_a_count_of_shared_pages_of_no_sequence_has_no_part():
    s = State([20, 0, 64, 33], 4, 16, 16)
    s.release([0, -1], [5, 0], [0, -3, 99, 1])


def test_a_captured_call_keeps_its_workspace():
    """Calls without a workspace in two captured graphs, replayed among each other's and other memory's use."""
    xs = [batch([(1280, [(1, 5 + i) for i in range(9)])], 8, 2, 128, 16, False),
          batch([(1024, [(1, 3)] * 4), (512, [(2, 40), (3, 9), (1, 130)])], 4, 2, 64, 16, False, seed=20)]
    xs = [tuple([p.cuda() for p in t] if isinstance(t, list) else t.cuda() for t in x) for x in xs]
    refs = [reference(x[0], x[1], *(t.cpu() for t in x[2:5]), 0.11, True) for x in xs]
    outs, graphs = [], []
    for order in ((0, 1, 0), (1, 0, 1)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            made = []
            for i in order:
                made.append((i, call(xs[i], scale=0.11)))
                torch.full((1 << 22,), 3, dtype=torch.uint8, device="cuda")   # takes what was given back
        graphs.append(graph)
        outs.append(made)
    side = torch.cuda.Stream()
    for _ in range(5):
        for made in outs:
            for _, (o, lse) in made:
                o.zero_(), lse.zero_()
        torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(255)     # another pool's memory
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        eager = call(xs[0], scale=0.11)
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.current_stream().wait_stream(side)
        assert status() == fa.FA_OK
        for i, (o, lse) in (*outs[0], *outs[1], (0, eager)):
            check(o, lse, refs[i])


def test_partial_rows_past_2_31_floats():
    """140000 single tokens of 64 heads behind one prompt: places of partial rows, and bytes of the workspace, that 32
    bits do not hold; sequences from both ends and between are compared."""
    S, Hq, Hk, d, page, prompt = 140000, 64, 2, 128, 16, 256
    assert 2 * S * Hq * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(6)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    n = prompt // page
    pages = [rand(S + n, Hk, page, d) for _ in "kv"]
    q = rand(S, Hq, d)
    table = torch.cat([torch.arange(n, device="cuda").expand(S, n), n + torch.randperm(S, generator=g, device="cuda")[:, None]],
                      1).int().contiguous()
    lens = (prompt + 1 + torch.arange(S, device="cuda") % page).int()
    cu = torch.arange(S + 1, device="cuda").int()
    o, lse = fa.paged_forward_shared(q, *pages, table, cu, lens, ints([0, S]), ints([prompt]), scale=0.2, max_q=1)
    assert status() == fa.FA_OK
    some = torch.tensor([0, 1, S - 1, S - 2, *range(5, S, S // 40)], device="cuda")
    used = torch.cat([torch.arange(n, device="cuda"), table[some, n].long()])
    own = torch.cat([torch.arange(n).expand(len(some), n), n + torch.arange(len(some))[:, None]], 1).int()
    check(o[some], lse[some], reference(q[some], [p[used] for p in pages], own, torch.arange(len(some) + 1).int(),
                                        lens[some].cpu(), 0.2, True))


@pytest.mark.parametrize("seed", range(12))
def test_any_mix_of_groups_with_sequences_left_out(seed):
    rng = random.Random(700 + seed)
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 128])
    Hk = rng.choice([1, 2, 3])
    Hq = Hk * rng.choice([1, 4, 7, 16, 40])
    groups = []
    for _ in range(rng.randint(1, 4)):
        most = rng.choice([1, 1, 5, 60])
        seqs = [(q, q + rng.randint(0, 150)) for q in (rng.randint(0, most) for _ in range(rng.randint(2, 50)))]
        groups.append((rng.choice([0, rng.randint(200, 4000)]), seqs))
    groups.append((0, [(1, 30)]))
    causal = rng.random() < 0.8
    x = batch(groups, Hq, Hk, d, page, rng.random() < 0.5, seed=seed)
    for s in range(len(x[4]) - 1):
        if rng.random() < 0.25:
            x[4][s] = 0
    o, lse = call(x, scale=0.13, causal=causal, max_q=rng.choice([0, 1, 60]))
    assert status() == fa.FA_OK
    check(o, lse, reference(*x[:5], 0.13, causal))
