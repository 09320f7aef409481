"""Norm, rotation and paged cache at the edges of what their calls allow (needs a GB300).

Tolerances are those of the tests of each operator (tests/test_gpu_norm_rope.py, tests/test_gpu_paged.py).
"""

import numpy as np
import pytest
import torch

import exact_io_aware_31_gb300 as fa
from oracle import serve
from tests.gpu_util import f64, require_gpu
from tests.test_gpu_norm_rope import F32, pool, ragged, status
from tests.test_gpu_paged import CASES, IDS, batch, check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def aside(t, behind=16):
    """A contiguous copy of ``t`` that starts ``behind`` bytes past a 256-byte border (and no nearer to one)."""
    n = behind // t.element_size()
    room = torch.zeros(t.numel() + 2 * n, dtype=t.dtype, device="cuda")
    assert room.data_ptr() % 256 == 0
    out = room[n:n + t.numel()].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("hint", [None, 0, 1, 10 ** 6])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_attention_at_16_byte_addresses(case, hint):
    """16 bytes are the alignment that every tensor is promised to need; each form of a unit writes rows of its own."""
    q, pages, table, cu, lens = batch(case)
    if case[6]:
        pages = [aside(p.transpose(1, 2)).transpose(1, 2) for p in pages]
    else:
        pages = [aside(p) for p in pages]
    ref = reference(q, pages, table, cu, lens, 0.11, case[7])
    room = torch.full((q.numel() + 16,), 3.0, dtype=torch.bfloat16, device="cuda")
    stats = torch.full((q.shape[0] * q.shape[1] + 2,), 4.0, device="cuda")
    o, lse = room[8:-8].view(q.shape), stats[1:-1].view(q.shape[:2])
    assert o.data_ptr() % 32 == 16
    fa.paged_forward(aside(q), *pages, *(aside(t, 4) for t in (table, cu, lens)), scale=0.11, causal=case[7],
                     max_q=max(case[0]) if hint is None else hint, out=o, lse=lse)
    assert status() == fa.FA_OK
    check(o, lse, ref)
    assert bool((room[:8] == 3).all()) and bool((room[-8:] == 3).all()) and stats[0] == 4 and stats[-1] == 4


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d", [
    ([267], [5885], 1, 1, 64),
    ([1, 140], [9000, 6000], 2, 1, 128),
])
def test_merged_rows_at_16_byte_addresses(q_lens, kv_lens, Hq, Hk, d):
    """Units that were cut: the merge writes them."""
    q, pages, table, cu, lens = batch((q_lens, kv_lens, Hq, Hk, d, 64, False, True))
    args = (*pages, table.cuda(), cu.cuda(), lens.cuda())
    want = fa.paged_forward(q, *args)
    out = aside(torch.zeros_like(q))
    got = fa.paged_forward(aside(q), *args, out=out)
    assert status() == fa.FA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("Hq,Hk,N,d", [(1, 1, 37, 64), (5, 2, 70, 128), (17, 9, 33, 64)])
def test_norm_and_append_at_16_byte_addresses(Hq, Hk, N, d):
    g = torch.Generator().manual_seed(8)
    new = lambda *n: torch.randn(n, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v = new(1, Hq, N, d), new(1, Hk, N, d), new(N, Hk, d)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in "qk"]
    rope = fa.rope_table(N, d)
    dz = [torch.randn_like(x) for x in (q, k)]
    want = *fa.qk_norm_rope(q, k, *w, rope=rope), *fa.qk_norm_rope_backward(*dz, q, k, *w, rope=rope)
    w2, rope2 = [aside(t) for t in w], aside(rope)
    outs, grads = ([aside(torch.zeros_like(x)) for x in (q, k)] for _ in range(2))
    got = (*fa.qk_norm_rope(aside(q), aside(k), *w2, rope=rope2, out=outs),
           *fa.qk_norm_rope_backward(*(aside(x) for x in dz), aside(q), aside(k), *w2, rope=rope2, grads=grads))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    (kp, vp), table = pool([N], Hk, d, 16, False, 3)
    meta = table.cuda(), ragged([N]).cuda(), torch.tensor([N], dtype=torch.int32).cuda()
    rows = [x[0].transpose(0, 1).contiguous() for x in (q, k)]
    kp2, vp2 = aside(kp), aside(vp)
    out = fa.paged_append(*rows, v, kp, vp, *meta, *w, rope=rope)
    out2 = fa.paged_append(*(aside(x) for x in (*rows, v)), kp2, vp2, *(aside(t, 4) for t in meta), *w2, rope=rope2,
                           out=aside(torch.zeros_like(out)))
    assert status() == fa.FA_OK
    assert torch.equal(out, out2) and torch.equal(kp, kp2) and torch.equal(vp, vp2)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [1e-5, 0.0])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq,Hk,d", [(17, 9, 64), (9, 16, 128), (8, 8, 64), (4, 2, 128), (1, 1, 64), (1, 2, 128)])
def test_rows_without_a_position_are_in_no_gradient(Hq, Hk, d, fill, eps, interleaved):
    """Padding rows (position -1, or past the table) hold NaN or infinities, in x, in dz or in both: their dq and dk
    are zero, and the weights' gradients are those of the other rows.  Each kernel variant of the gradient."""
    B, N = 2, 41
    g = torch.Generator().manual_seed(13)
    x = [torch.randn(B, h, N, d, generator=g).bfloat16().cuda() for h in (Hq, Hk)]
    dz = [torch.randn(t.shape, generator=g).bfloat16().cuda() for t in x]
    w = [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in "qk"]
    pos = torch.arange(N, dtype=torch.int32).repeat(B, 1)
    pos[0, 5:9], pos[1, ::7], pos[1, 40] = -1, N, 2 ** 31 - 1
    gone = ((pos < 0) | (pos >= N))
    at = torch.where(gone, 0, pos).numpy()
    kw = dict(rope=fa.rope_table(N, d), positions=pos.cuda(), eps=eps, interleaved=interleaved)
    refs = []
    for t, z, wi in zip(x, dz, w):
        z = f64(z) * ~gone.numpy()[:, None, :, None]
        size = np.abs(z).max(-1, keepdims=True) * 2 * np.abs(f64(t)) / np.sqrt((f64(t) ** 2).mean(-1, keepdims=True) + eps)
        bound = ((size[..., 0].size + 16) * 2.0 ** -24 + F32) * size.reshape(-1, d).sum(0)
        refs.append((serve.norm_rope_grad(z, f64(t), f64(wi), eps, f64(kw["rope"]), at, interleaved)[1], bound))
    clean = fa.qk_norm_rope_backward(*dz, *x, *w, **kw)
    for in_x, in_dz in ((True, True), (True, False), (False, True)):
        mask = gone.cuda()[:, None, :, None]
        x2 = [t.masked_fill(mask, fill) if in_x else t for t in x]
        dz2 = [t.masked_fill(mask, fill) if in_dz else t for t in dz]
        got = fa.qk_norm_rope_backward(*dz2, *x2, *w, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, clean))
        for dx, dw, (ref, bound) in zip(got[:2], got[2:], refs):
            assert bool((dx.masked_select(mask) == 0).all())
            assert (np.abs(f64(dw) - ref) <= bound).all()
    assert status() == fa.FA_ERR_DEVICE_INDEX


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hk,d", [
    ([40, 70, 9], [700, 900, 800], 1, 1, 64),        # one query tile, partly filled
    ([14, 3, 25], [1000, 600, 1500], 15, 3, 128),    # groups of 5: rows that no copy fills
    ([150, 200, 1], [900, 1100, 500], 3, 1, 128),    # two tiles, the second partly filled
    ([60, 12, 7], [700, 2000, 640], 20, 1, 64),
    ([5, 2, 9], [640, 1000, 1300], 12, 1, 64),       # four copies
])
def test_a_sequence_is_the_same_bits_whatever_others_hold(q_lens, kv_lens, Hq, Hk, d, hint):
    """Queries, keys and values of another sequence, or queries behind the last one, change no bit of a sequence's
    rows: tiles hold rows of neighbours and leftovers, which must have no part in when a row is rescaled."""
    q, pages, table, cu, lens = batch((q_lens, kv_lens, Hq, Hk, d, 32, False, True))
    T = q.shape[0]
    rows = torch.cat([q, torch.zeros(140, Hq, d, dtype=q.dtype, device="cuda")])
    args = table.cuda(), cu.cuda(), lens.cuda()
    run = lambda x, p: [t[:T] for t in fa.paged_forward(x, *p, *args, scale=0.11, max_q=hint)]  # noqa: E731
    want = run(rows, pages)
    g = torch.Generator().manual_seed(6)
    noise = lambda *n: (100 * torch.randn(n, generator=g)).bfloat16().cuda()  # noqa: E731
    for s in (*range(len(q_lens)), None):
        x, p = rows.clone(), [t.clone() for t in pages]
        x[T:] = noise(140, Hq, d)
        keep = torch.ones(T, dtype=torch.bool)
        if s is not None:
            keep[cu[s]:cu[s + 1]] = False
            x[cu[s]:cu[s + 1]] = noise(q_lens[s], Hq, d)
            used = table[s, :-(-kv_lens[s] // 32)].long()
            for t in p:
                t[used.cuda()] = noise(len(used), *t.shape[1:])
        for a, b in zip(run(x, p), want):
            assert torch.equal(a[keep.cuda()], b[keep.cuda()])
    assert status() == fa.FA_OK


def test_helpers_refuse_what_is_no_tensor():
    """With the ValueError of a CPU tensor, whichever argument it is."""
    Hq, Hk, d, page = 2, 1, 64, 16
    (kp, vp), table = pool([20], Hk, d, page, False, 1)
    x = torch.randn(3, Hq + 2 * Hk, d, device="cuda").bfloat16()
    meta = dict(page_table=table.cuda(), cu_seqlens=ragged([3]).cuda(), kv_lens=torch.tensor([20]).int().cuda())
    append = dict(q=x[:, :Hq], k=x[:, Hq:Hq + Hk], v=x[:, Hq + Hk:], k_pages=kp, v_pages=vp, **meta)
    attend = dict(q=fa.paged_append(**append), k_pages=kp, v_pages=vp, **meta)
    turn = dict(q=x[None, :, :Hq].transpose(1, 2), k=x[None, :, Hq:Hq + Hk].transpose(1, 2))
    z = fa.qk_norm_rope(**turn)
    back = dict(dq_out=z[0], dk_out=z[1], **turn)
    extra = dict(q_weight=None, k_weight=None, rope=None)
    room = dict(workspace=None)
    for f, args, more in ((fa.paged_append, append, dict(extra, out=None)), (fa.paged_forward, attend, dict(room, out=None, lse=None)),
                          (fa.qk_norm_rope, turn, dict(extra, positions=None)),
                          (fa.qk_norm_rope_backward, back, dict(extra, positions=None, **room))):
        f(**args)
        for name in (*args, *more):
            for bad in ([1.0] * 64, np.zeros((3, 2, 64), dtype=np.float32)):
                with pytest.raises(ValueError):
                    f(**args | {name: bad})
    for f, args, names in ((fa.paged_append, append, ("q", "k", "v", "k_pages", "v_pages", "page_table")),
                           (fa.paged_forward, attend, ("q", "k_pages", "v_pages", "page_table")),
                           (fa.qk_norm_rope, turn, ("q", "k")), (fa.qk_norm_rope_backward, back, ("q", "k", "dq_out"))):
        for name in names:
            with pytest.raises(ValueError):
                f(**args | {name: None})
    assert status() == fa.FA_OK


def test_nothing_to_do():
    """No token, no sequence, sequences without a token: nothing is written and nothing recorded."""
    Hq, Hk, d, page = 4, 2, 64, 16
    (kp, vp), table = pool([20, 40], Hk, d, page, False, 1)
    kept = kp.clone(), vp.clone()
    lens = torch.tensor([20, 40], dtype=torch.int32).cuda()
    rope = fa.rope_table(64, d)
    for T, meta in ((0, (table.cuda(), ragged([0, 0]).cuda(), lens)), (5, (table.cuda(), ragged([0, 0]).cuda(), lens)),
                    (5, (table[:0].cuda(), ragged([]).cuda(), lens[:0])), (0, (table[:0, :0].cuda(), ragged([]).cuda(), lens[:0]))):
        x = torch.randn(T, Hq + 2 * Hk, d, device="cuda").bfloat16()
        out = torch.full((T, Hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
        o, lse = torch.full_like(out, 6.0), torch.full((T, Hq), 7.0, device="cuda")
        fa.paged_append(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], kp, vp, *meta, rope=rope, out=out)
        for hint in (0, 1):
            fa.paged_forward(x[:, :Hq], kp, vp, *meta, max_q=hint, out=o, lse=lse)
        assert status() == fa.FA_OK
        assert bool((out == 5).all()) and bool((o == 6).all()) and bool((lse == 7).all())
    assert torch.equal(kp, kept[0]) and torch.equal(vp, kept[1])
