"""A paged cache's tables kept on the device, against plain loops over whole numbers (needs a GB300): all are equal."""

import random

import numpy as np
import pytest
import torch

import exact_io_aware_31_gb300 as fa
from oracle import serve
from tests.gpu_util import f64, require_gpu
from tests.test_gpu_norm_rope import status
from tests.test_gpu_paged import check

pytestmark = pytest.mark.gpu

OLD = 77  # what the step's tables hold before


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class State:
    """The requests on the device beside the plain form's."""

    def __init__(self, lens, max_pages, page, num_pages, seed=1):
        rng = np.random.default_rng(seed)
        order = rng.permutation(num_pages)
        table = np.full((len(lens), max_pages), -5)
        at = 0
        for r, n in enumerate(lens):
            used = -(-n // page)
            table[r, :used] = order[at:at + used]
            at += used
        self.page, self.num_pages = page, num_pages
        self.plain = serve.Tables(lens, table, order[at:].tolist(), num_pages, page)
        self.lens, self.table = ints(lens), ints(table)
        self.pool = ints([num_pages - at, 0] + order[at:].tolist() + [-9] * at)

    def same(self):
        free = self.plain.free
        assert self.pool[:2].tolist() == [len(free), 0]
        assert self.pool[2:2 + len(free)].tolist() == free
        assert self.lens.tolist() == self.plain.lens
        assert np.array_equal(self.table.cpu().numpy(), self.plain.table)
        want, self.plain.bad = self.plain.bad, False
        assert status() == (fa.FA_ERR_DEVICE_INDEX if want else fa.FA_OK)

    def extend(self, requests, new, tokens=None, wanted=(True, True)):
        S, T = len(requests), sum(max(0, n) for r, n in zip(requests, new) if r >= 0) if tokens is None else tokens
        out = (ints([OLD] * (S + 1)), ints([OLD] * S), ints(np.full((S, self.table.shape[1]), OLD)),
               ints([OLD] * T) if wanted[0] else None,
               torch.full((T,), OLD, dtype=torch.int64, device="cuda") if wanted[1] else None)
        got = fa.paged_extend(ints(requests), ints(new), self.lens, self.table, self.pool, self.page, T, out=out)
        want = self.plain.extend(requests, new, T, np.full((S, self.table.shape[1]), OLD))
        for name, g, w in zip(("cu_seqlens", "kv_lens", "page_table", "positions", "slots"), got, want):
            assert g is None or np.array_equal(g.cpu().numpy(), w), name
        self.same()
        return got

    def release(self, requests, keep=None, kept=None):
        fa.paged_release(ints(requests), self.lens, self.table, self.pool, self.page,
                         None if keep is None else ints(keep), None if kept is None else ints(kept))
        self.plain.release(requests, keep, kept)
        self.same()


def test_one_token():
    s = State([130], 16, 16, 20)
    for _ in range(40):
        s.extend([0], [1])


@pytest.mark.parametrize("page", [16, 64, 65536])
def test_lengths_around_a_page(page):
    lens = [0, 1, page - 1, page, page + 1, 2 * page, 0]
    for new in (0, 1, page - 1, page, page + 1):
        s = State(lens, 8, page, 60)
        s.extend(list(range(7)), [new] * 7)
        s.extend([6, 0, -1, 3], [0, 1, 5, page])
        s.release([3, 0, -2, 5])
        s.extend([0, 3], [3, 5])


@pytest.mark.parametrize("seed", range(12))
def test_steps_of_a_server(seed):
    """Requests arrive, grow, take speculated tokens back and end, in steps of changing batches with empty places."""
    rng = random.Random(seed)
    page, R = rng.choice([16, 32, 128]), rng.choice([3, 40, 700])
    s = State([0] * R, rng.choice([5, 300]), page, rng.choice([R * 2 + 3, R * 40]), seed)
    for step in range(12):
        live = rng.sample(range(R), rng.randint(1, R))
        batch = live + [-1] * rng.choice([0, 0, 5])
        rng.shuffle(batch)
        new = [rng.choice([0, 1, 1, rng.randint(1, 9), rng.randint(1, 400)]) for _ in batch]
        s.extend(batch, new, tokens=rng.choice([None, sum(new) + 100, max(1, sum(new) - 50)]))
        some = rng.sample(range(R), rng.randint(0, R))
        s.release(some, [rng.randint(0, s.plain.lens[r]) for r in some] if rng.random() < 0.6 else None)


def test_what_is_refused_leaves_its_request():
    def fresh():
        return State([20, 0, 64, 33], 4, 16, 16)
    for batch, new in (([0, 4, 1], [1, 1, 1]), ([0, 10 ** 9, 1], [3, 0, 40]),           # no such request
                       ([0, 1, 0, 1], [1, 5, 9, 0]),                                     # the same one twice
                       ([2, 1, 3], [1, 64, 32]), ([3, 1], [31, 65]),                     # past the end of its row
                       ([1, 0, 3], [-4, 2, -1])):
        fresh().extend(batch, new)
    fresh().extend([1, 0, 3], [2 ** 31 - 1, 2 ** 31 - 1, 1], tokens=9)                  # sums past 32 bits
    for T in (0, 1, 4, 5, 6):
        fresh().extend([0, 1, 2, 3], [1, 4, 0, 1], tokens=T)
    s = State([0, 0, 0, 30], 8, 16, 7)                                                   # 5 pages are free
    s.extend([0, 1, 2, 3], [40, 49, 16, 1])       # three, four too many, one behind them, none
    s.extend([1, 2], [17, 1])                     # two: fits now; one more does not
    s.release([0])
    s.extend([2], [1])
    for n in (-3, 99):                            # a count that cannot be is cut to the pool
        s = State([0, 5], 4, 16, 6)
        s.pool[0] = n
        fa.paged_extend(ints([1]), ints([1]), s.lens, s.table, s.pool, 16, 1)
        assert status() == fa.FA_ERR_DEVICE_INDEX
        assert s.pool[0].item() == (0 if n < 0 else 6) and s.lens.tolist() == [0, 6]


def test_what_cannot_be_given_back():
    s = State([20, 0, 64, 33], 4, 16, 16)
    s.release([0, 4, 0, -1, 2], [5, 0, 0, 0, 64])             # no such request, the same one twice
    s.release([2, 3], [65, -1])                               # keeps what it does not have
    s.release([3, 2], [3, 17], [0, 0, 3, 1])                  # pages that are not its own
    s.release([2], None, [0, 0, 2, 0])
    s = State([64, 64, 33], 4, 16, 11)
    s.plain.lens[0] = s.plain.lens[1] = 64
    s.release([0])
    s.lens[0] = s.plain.lens[0] = 64                          # the caller's mistake: its pages are back already
    s.release([0, 1, 2])                                      # more than there is room for: nothing happens
    s = State([40], 4, 16, 9)
    s.table[0, 1] = s.plain.table[0, 1] = 9                   # no page of the pool: said
    s.release([0])


@pytest.mark.parametrize("wanted", [(True, False), (False, True), (False, False)])
def test_maps_that_are_not_wanted(wanted):
    State([3, 0], 40, 16, 100).extend([0, 1], [300, 5], tokens=400, wanted=wanted)


def test_largest_batch():
    """4096 sequences of 16384 requests in any order, rows of 300 pages, and 4097 that are refused."""
    rng = random.Random(3)
    R = 16384
    lens = [rng.choice([0, 15, 16, rng.randint(0, 4000)]) for _ in range(R)]
    s = State(lens, 300, 16, sum(-(-n // 16) for n in lens) + 9000)
    batch = rng.sample(range(R), 4096)
    s.extend(batch, [rng.choice([1, 1, 20]) for _ in batch])
    s.release(batch, [s.plain.lens[r] // 2 for r in batch])
    with pytest.raises(fa.FaError) as e:
        fa.paged_release(ints(batch + [1]), s.lens, s.table, s.pool, 16)
    assert e.value.status == fa.FA_ERR_UNSUPPORTED


def test_long_rows():
    """Rows of many pieces, a chunk of 70000 tokens among them."""
    s = State([0, 500000, 16 * 8000 - 1], 40000, 16, 90000)
    s.extend([1, 0, 2], [3, 70000, 2])
    s.release([0, 2, 1], [69999, 5, 16])


def test_a_turn_leaves_the_pool_as_it_was():
    s = State([9, 100, 31, 0], 64, 16, 90)
    before = s.pool.clone()
    first = [x.clone() for x in s.extend([3, 1, 0, 2], [400, 30, 9, 1])]
    s.release([3, 1, 0, 2], [0, 100, 9, 31])
    assert torch.equal(before, s.pool)
    assert all(torch.equal(a, b) for a, b in zip(first, s.extend([3, 1, 0, 2], [400, 30, 9, 1])))


def test_graph_and_stream():
    """A captured turn, replayed: tokens come and one of each is taken back."""
    s = State([5, 0, 33], 64, 16, 150)
    batch, new, keep = ints([2, -1, 0, 1]), ints([3, 0, 2, 17]), ints([0] * 4)
    out = tuple(x.clone() for x in s.extend([2, -1, 0, 1], [3, 0, 2, 17]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.paged_extend(batch, new, s.lens, s.table, s.pool, 16, 22, out=out)
        fa.paged_release(batch, s.lens, s.table, s.pool, 16, keep_lens=keep)
    for _ in range(4):
        lens = [s.plain.lens[r] for r in (2, 0, 1)]
        keep.copy_(ints([lens[0] + 2, 0, lens[1] + 1, lens[2] + 16]))
        graph.replay()
        want = s.plain.extend([2, -1, 0, 1], [3, 0, 2, 17], 22, out[2].cpu().numpy())
        s.plain.release([2, -1, 0, 1], [lens[0] + 2, 0, lens[1] + 1, lens[2] + 16])
        s.same()
        assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(out, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.paged_extend(batch, new, s.lens, s.table, s.pool, 16, 22, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = s.plain.extend([2, -1, 0, 1], [3, 0, 2, 17], 22, got[2].cpu().numpy())
    s.same()
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want))
    with pytest.raises(ValueError):
        fa.paged_extend(batch, new.long(), s.lens, s.table, s.pool, 16, 22)
    with pytest.raises(ValueError):
        fa.paged_release(batch, s.lens[:2], s.table, s.pool, 16)


@pytest.mark.parametrize("Hq,Hk,d,page", [(8, 2, 64, 16), (4, 4, 128, 32)])
def test_a_server_with_a_shared_prompt(Hq, Hk, d, page):
    """Tables, append, attention and release as a server calls them: five requests share a prompt's full pages, take
    speculated tokens, and some of those are taken back; every step's attention is compared."""
    g = torch.Generator().manual_seed(8)
    R, max_pages, num_pages, n = 7, 1200 // page, 3 * 1200 // page, 5
    rand = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    kp, vp = (torch.zeros(num_pages, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    lens, table = ints([0] * R), ints(np.zeros((R, max_pages)))
    pool, turn = fa.paged_pool(num_pages), fa.rope_table(1200, d)
    prompt = 1000 // page * page
    keys = {r: [] for r in range(R)}             # (key, value) of each token, as projected

    def step(batch, new, groups, prefix):
        T = sum(new)
        q, k, v = rand(T, Hq, d), rand(T, Hk, d), rand(T, Hk, d)
        cu, kv, pages, pos, _ = fa.paged_extend(ints(batch), ints(new), lens, table, pool, page, T)
        for i, r in enumerate(batch):
            a, b = cu[i].item(), cu[i + 1].item()
            keys[r] = keys[r] + list(zip(k[a:b], v[a:b]))
        qr = fa.paged_append(q, k, v, kp, vp, pages, cu, kv, rope=turn, norm=False)
        o, lse = fa.paged_forward_shared(qr, kp, vp, pages, cu, kv, ints(groups), ints(prefix), scale=0.1)
        assert status() == fa.FA_OK
        # a cache of its own for every sequence, of the rotated keys
        own, at = [], []
        for r in batch:
            kk, vv = (torch.stack(x) for x in zip(*keys[r]))
            pos32 = torch.arange(len(kk), dtype=torch.int32, device="cuda")[None]
            kk = fa.qk_norm_rope(kk.transpose(0, 1)[None], kk.transpose(0, 1)[None], rope=turn, positions=pos32,
                                 norm=False)[1][0]
            own.append((f64(kk), f64(vv.transpose(0, 1))))
            at.append(len(keys[r]))
        most = max(at)
        flat = [np.stack([np.pad(x[i], ((0, 0), (0, most - x[i].shape[1]), (0, 0))) for x in own]) for i in (0, 1)]
        ref = serve.paged_attention(f64(qr), *flat, np.arange(len(batch))[:, None], cu.cpu().numpy(), np.array(at), 0.1,
                                    True)
        check(o, lse, ref)

    step([6], [prompt], [0, 1], [0])             # the prompt is a request of its own
    members = [2, 0, 5, 3, 1]
    table[members, :prompt // page] = table[6, :prompt // page]
    lens[members] = prompt
    kept = ints([prompt // page] * R)
    kept[6] = 0
    for r in members:
        keys[r] = list(keys[6])
    free = pool[0].item()
    for accepted in (3, 1, 2, 0, 3):
        step([6, *members], [2] + [3] * n, [1, 6], [prompt])
        end = {r: len(keys[r]) - (3 - accepted if r != 6 else 0) for r in (6, *members)}
        fa.paged_release(ints([6, *members]), lens, table, pool, page, ints([end[r] for r in (6, *members)]), kept)
        for r, x in end.items():
            keys[r] = keys[r][:x]
        assert lens.tolist()[0] == end[0] and status() == fa.FA_OK
    fa.paged_release(ints(members), lens, table, pool, page, kept_pages=kept)
    assert status() == fa.FA_OK and pool[0].item() == free - (-(-len(keys[6]) // page) - prompt // page)
    used = set(table[6, :-(-len(keys[6]) // page)].tolist())
    stack = pool[2:2 + pool[0].item()].tolist()
    assert len(set(stack)) == len(stack) and not used & set(stack) and len(stack) + len(used) == num_pages
