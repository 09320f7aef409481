"""Norm with rotation, its gradient and the cache write against the fp64 forms (needs a GB300).

Tolerances, from the number of fp32 roundings (2^-24 each) and the one bf16 rounding of a stored value (2^-8 of it,
``finfo(bfloat16).eps / 2``):

* z: r = 1 / rms is within 2^-21 (a sum of d <= 128 squares in a tree at most 12 additions deep, the division, the
  addition of eps and a reciprocal root good to 2^-22), the products add three roundings, the rotation two: the fp32
  value is within 2^-20 (|y_a| + |y_b|) of z, with |y_a| + |y_b| <= sqrt(2) * 2 max|y| of the row.
* dx = r (g w - x k): k = r^2 mean(x w g) is within 2^-19 of r^2 mean|x w g|, the rest as above.
* dw: n terms of relative error 2^-20 summed in fp32, any order: (n + 16) 2^-24 of the sum of magnitudes.
"""

import numpy as np
import pytest
import torch

import exact_io_aware_31_gb300 as fa
from oracle import serve
from tests.gpu_util import f64, require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = 2.0 ** -8, 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def status():
    return fa.fa_get_device_status(torch.cuda.current_stream().cuda_stream)


def draw(B, Hq, Hk, N, d, layout, seed):
    g = torch.Generator().manual_seed(seed)
    if layout == "packed":      # a slice of the projection's rows, token-major, with values behind
        x = torch.randn(B, N, Hq + 2 * Hk + 1, d, generator=g).bfloat16().cuda()
        return x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    if layout == "broadcast":   # one key head's row for every head and batch
        q = torch.randn(B, Hq, N, d, generator=g).bfloat16().cuda()
        return q, torch.randn(1, 1, N, d, generator=g).bfloat16().cuda().expand(B, Hk, N, d)
    return tuple(torch.randn(B, h, N, d, generator=g).bfloat16().cuda() for h in (Hq, Hk))


CASES = [
    # B, Hq, Hk, N, d, rope, interleaved, positions, weights, layout
    (1, 1, 1, 1, 64, 64, False, False, "f32", "heads"),
    (1, 1, 1, 1, 128, 128, True, True, "bf16", "packed"),
    (2, 5, 1, 37, 64, 32, False, True, "bf16", "packed"),
    (3, 12, 4, 65, 128, 128, False, False, "f32", "heads"),
    (2, 17, 9, 33, 128, 64, True, False, "f32", "packed"),
    (1, 33, 7, 19, 64, 16, False, True, None, "broadcast"),
    (2, 16, 16, 129, 64, 64, True, False, "bf16", "broadcast"),
    (1, 8, 2, 50, 128, 0, False, False, "f32", "packed"),       # norm alone
    (2, 4, 4, 21, 128, 96, False, True, "nonorm", "packed"),    # rotation alone
    (1, 3, 3, 40, 64, 48, True, False, "nonorm", "heads"),
]
IDS = [f"b{c[0]}h{c[1]}_{c[2]}n{c[3]}d{c[4]}r{c[5]}{'i' if c[6] else ''}{c[8] or ''}{c[9]}" for c in CASES]


def setup(case):
    B, Hq, Hk, N, d, rope, inter, positions, weights, layout = case
    q, k = draw(B, Hq, Hk, N, d, layout, 11 + N + d)
    g = torch.Generator().manual_seed(3)
    wt = torch.float32 if weights == "f32" else torch.bfloat16
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(wt).cuda() if weights in ("f32", "bf16") else None for _ in "qk"]
    table = fa.rope_table(3 * N + 5, rope, device="cuda") if rope else None
    pos = torch.randint(0, 3 * N + 5, (B, N), generator=g).to(torch.int32) if positions else None
    kw = dict(rope=table, positions=pos.cuda() if positions else None, eps=1e-5, interleaved=inter,
              norm=weights != "nonorm")
    at = pos.numpy() if positions else np.tile(np.arange(N), (B, 1))
    ref = dict(eps=1e-5, table=f64(table) if rope else None, positions=at, interleaved=inter, norm=kw["norm"])
    return q, k, w, kw, ref


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    q, k, w, kw, ref = setup(case)
    outs = fa.qk_norm_rope(q, k, *w, **kw)
    assert status() == fa.FA_OK
    for z, x, wi in zip(outs, (q, k), w):
        assert z.is_contiguous() and z.shape == x.shape
        r = serve.norm_rope(f64(x), None if wi is None else f64(wi), **ref)
        err = np.abs(f64(z) - r) - BF * np.abs(r)
        assert (err <= 3 * F32 * np.abs(r).max(-1, keepdims=True)).all(), float(err.max())


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    q, k, w, kw, ref = setup(case)
    g = torch.Generator().manual_seed(9)
    dz = [torch.randn(x.shape, generator=g).bfloat16().cuda() for x in (q, k)]
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw)
    assert status() == fa.FA_OK
    again = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw)
    for dx, dw, x, z, wi, dw2 in zip((dq, dk), (dqw, dkw), (q, k), dz, w, again[2:]):
        wr = None if wi is None else f64(wi)
        rx, rw = serve.norm_rope_grad(f64(z), f64(x), wr, **ref)
        big = np.abs(rx).max(-1, keepdims=True)
        if kw["norm"]:  # cancelled terms: r (|g w| + |x| r^2 mean|x w g|)
            xn = np.asarray(f64(x))
            r = 1 / np.sqrt((xn ** 2).mean(-1, keepdims=True) + kw["eps"])
            gw = np.abs(f64(z)).max(-1, keepdims=True) * 2 * (1 if wr is None else np.abs(wr).max())
            big = r * gw * (1 + (np.abs(xn) * r).max(-1, keepdims=True) ** 2)
        err = np.abs(f64(dx) - rx) - BF * np.abs(rx)
        assert (err <= 4 * F32 * big).all(), float(err.max())
        if kw["norm"]:
            size = np.abs(f64(z)).max(-1, keepdims=True) * 2 * np.abs(f64(x)) * r
            n = size[..., 0].size
            bound = ((n + 16) * 2.0 ** -24 + F32) * size.reshape(-1, x.shape[-1]).sum(0)
            assert (np.abs(f64(dw) - rw) <= bound).all()
            assert torch.equal(dw, dw2)
        else:
            assert dw is None


def test_backward_into_a_packed_buffer_and_without_weight_gradients():
    q, k, w, kw, ref = setup(CASES[4])
    B, Hq, N, d = q.shape
    Hk = k.shape[1]
    dz = [torch.randn(x.shape, device="cuda").bfloat16() for x in (q, k)]
    buf = torch.full((B, N, Hq + 2 * Hk, d), 7.0, dtype=torch.bfloat16, device="cuda")
    dq, dk = buf[:, :, :Hq].transpose(1, 2), buf[:, :, Hq:Hq + Hk].transpose(1, 2)
    want = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw)
    got = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw, grads=(dq, dk), weight_grads=False)
    assert got[2] is None and got[3] is None
    assert torch.equal(dq, want[0]) and torch.equal(dk, want[1])
    assert bool((buf[:, :, Hq + Hk:] == 7.0).all())


@pytest.mark.parametrize("H", [(3, 1), (17, 9)])
def test_no_eps(H):
    """eps = 0: rows of a warp that belong to no head must not reach the weights' gradients."""
    g = torch.Generator().manual_seed(12)
    q, k = (torch.randn(2, h, 7, 64, generator=g).bfloat16().cuda() for h in H)
    dz = [torch.randn(x.shape, generator=g).bfloat16().cuda() for x in (q, k)]
    grads = fa.qk_norm_rope_backward(*dz, q, k, eps=0.0)
    for dx, dw, x, z in zip(grads[:2], grads[2:], (q, k), dz):
        rx, rw = serve.norm_rope_grad(f64(z), f64(x), None, 0.0, None, None, False)
        assert np.abs(f64(dx) - rx).max() <= 2 * BF * np.abs(rx).max()
        assert np.abs(f64(dw) - rw).max() <= 1e-4 * np.abs(rw).max()
    assert all(bool(t.isfinite().all()) for t in fa.qk_norm_rope(q, k, eps=0.0))


def test_positions_outside_the_table():
    q, k, w, kw, ref = setup((1, 4, 2, 6, 64, 64, False, True, "f32", "packed"))
    good = fa.qk_norm_rope(q, k, *w, **kw)
    kw["positions"][0, 2], kw["positions"][0, 4] = -1, kw["rope"].shape[0]
    bad = fa.qk_norm_rope(q, k, *w, **kw)
    assert status() == fa.FA_ERR_DEVICE_INDEX and status() == fa.FA_OK
    for b, g in zip(bad, good):
        assert bool((b[:, :, [2, 4]] == 0).all()) and torch.equal(b[:, :, [0, 1, 3, 5]], g[:, :, [0, 1, 3, 5]])
    grads = fa.qk_norm_rope_backward(*bad, q, k, *w, **kw)
    assert status() == fa.FA_ERR_DEVICE_INDEX
    assert all(bool((x[:, :, [2, 4]] == 0).all()) and bool(x.isfinite().all()) for x in grads[:2])
    assert all(bool(x.isfinite().all()) for x in grads[2:])


def test_training_step_through_the_attention():
    """norm + rotation -> attention -> its backward -> their backward, against autograd in fp64 on the CPU."""
    B, H, N, d = 1, 2, 200, 64
    g = torch.Generator().manual_seed(21)
    qkv = torch.randn(B, N, 3 * H, d, generator=g).bfloat16()
    do = torch.randn(B, H, N, d, generator=g).bfloat16()
    w = [1 + 0.2 * torch.randn(d, generator=g) for _ in "qk"]
    table = fa.rope_table(N, d, device="cpu")
    x = [t.double().requires_grad_() for t in (qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:2 * H].transpose(1, 2),
                                               qkv[:, :, 2 * H:].transpose(1, 2), *w)]
    c, s = table[:, :d // 2].double(), table[:, d // 2:].double()

    def turn(t, wt):
        y = t / (t.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * wt
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    p = (turn(x[0], x[3]) @ turn(x[1], x[4]).transpose(2, 3) * d ** -0.5)
    p = p.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), float("-inf")).softmax(-1)
    ((p @ x[2]) * do.double()).sum().backward()

    qkv_g = qkv.cuda()
    q, k = qkv_g[:, :, :H].transpose(1, 2), qkv_g[:, :, H:2 * H].transpose(1, 2)
    v = qkv_g[:, :, 2 * H:].transpose(1, 2).contiguous()
    wg = [t.cuda() for t in w]
    qn, kn = fa.qk_norm_rope(q, k, *wg, rope=table.cuda())
    o, lse = fa.forward(qn, kn, v, causal=True)
    dqn, dkn, dv = fa.backward(qn, kn, v, o, lse, do.cuda(), causal=True)
    got = (*fa.qk_norm_rope_backward(dqn, dkn, q, k, *wg, rope=table.cuda()), dv)
    assert status() == fa.FA_OK
    for name, t, r in zip(("dq", "dk", "dqw", "dkw", "dv"), got, (x[0], x[1], x[3], x[4], x[2])):
        r = r.grad.numpy()
        assert np.abs(f64(t) - r).max() <= 2e-2 * np.abs(r).max(), name   # the gradient tolerance of the attention tests


def test_other_stream_and_graph():
    q, k, w, kw, ref = setup(CASES[3])
    want = fa.qk_norm_rope(q, k, *w, **kw)
    dz = [torch.randn_like(t) for t in want]
    want_g = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.qk_norm_rope(q, k, *w, **kw, stream=side)
    got_g = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip((*got, *got_g), (*want, *want_g)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = fa.qk_norm_rope(q, k, *w, **kw)
        dx = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw)
    for _ in range(2):
        for t in (*z, *dx):
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((*z, *dx), (*want, *want_g)))


# ------------------------------------------------------------------- cache ----
APPENDS = [
    # q_lens, kv_lens, Hq, Hk, d, page, token_major, rope, interleaved, weights
    ([1], [1], 1, 1, 64, 16, False, 64, False, "f32"),
    ([1, 1, 1], [17, 32, 33], 8, 2, 128, 16, True, 128, True, "bf16"),
    ([0, 5, 0, 0, 3, 0], [0, 70, 9, 0, 3, 40], 5, 1, 64, 32, False, 32, False, "f32"),
    ([40, 1, 7], [40, 300, 130], 12, 4, 128, 64, True, 64, False, None),
    ([2] * 40, list(range(2, 42)), 4, 4, 64, 16, False, 16, True, "bf16"),
    ([9, 4], [9, 20], 3, 3, 128, 256, False, 0, False, "nonorm"),
    ([3] * 1100, [3 + i % 29 for i in range(1100)], 2, 1, 64, 16, False, 64, False, "f32"),
]


def pool(kv_lens, Hk, d, page, token_major, seed, extra=3):
    """A cache of random (stale) contents and a page table of scattered pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in kv_lens]
    total = sum(need) + extra
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(kv_lens), max(max(need), 1)), -7, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    shape = (total, page, Hk, d) if token_major else (total, Hk, page, d)
    pages = [torch.randn(shape, generator=g).bfloat16().cuda() for _ in "kv"]
    return [p.transpose(1, 2) if token_major else p for p in pages], table


def ragged(q_lens):
    return torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32)


@pytest.mark.parametrize("case", APPENDS, ids=[f"s{len(c[0])}h{c[2]}_{c[3]}d{c[4]}p{c[5]}{c[9] or ''}" for c in APPENDS])
def test_append(case):
    q_lens, kv_lens, Hq, Hk, d, page, token_major, rope, inter, weights = case
    (kp, vp), table = pool(kv_lens, Hk, d, page, token_major, 31)
    before = kp.clone(), vp.clone()
    cu = ragged(q_lens)
    T = int(cu[-1])
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T + 2, Hq + 2 * Hk, d, generator=g).bfloat16().cuda()   # two rows behind the last sequence
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    wt = torch.float32 if weights == "f32" else torch.bfloat16
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(wt).cuda() if weights in ("f32", "bf16") else None for _ in "qk"]
    rt = fa.rope_table(max(kv_lens), rope) if rope else None
    out = torch.full((T + 2, Hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    fa.paged_append(q, k, v, kp, vp, table.cuda(), cu.cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(), *w,
                    rope=rt, eps=1e-5, interleaved=inter, norm=weights != "nonorm", out=out)
    assert status() == fa.FA_OK
    wr = [None if t is None else f64(t) for t in w]
    rq, rk, rv = serve.paged_append(f64(q[:T]), f64(k[:T]), f64(v[:T]), f64(before[0]), f64(before[1]), table.numpy(),
                                    cu.numpy(), kv_lens, *wr, 1e-5, f64(rt) if rope else None, inter,
                                    weights != "nonorm")
    assert bool((out[T:] == 5.0).all())
    assert np.array_equal(f64(vp), rv)
    same = rk == f64(before[0])
    assert np.array_equal(f64(kp)[same], rk[same])                     # slots of no new token: bit for bit
    for got, r in ((f64(out[:T]), rq), (f64(kp), rk)):
        err = np.abs(got - r) - BF * np.abs(r)
        assert (err <= 3 * F32 * np.abs(r).max(-1, keepdims=True)).all(), float(err.max())


def test_append_tokens_without_a_slot():
    """A length shorter than the chunk, one past the table, and a page outside the pool."""
    Hq, Hk, d, page = 2, 1, 64, 16
    (kp, vp), _ = pool([48] * 3, Hk, d, page, False, 5)
    table = torch.tensor([[0, 1], [2, 3], [4, kp.shape[0]]], dtype=torch.int32).cuda()
    cu, lens = ragged([3, 2, 2]).cuda(), torch.tensor([1, 33, 18], dtype=torch.int32).cuda()
    x = torch.randn(7, Hq + 2 * Hk, d, device="cuda").bfloat16()
    before = kp.clone(), vp.clone()
    out = fa.paged_append(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], kp, vp, table, cu, lens,
                          rope=fa.rope_table(64, 64))
    assert status() == fa.FA_ERR_DEVICE_INDEX
    zero = (out == 0).all(-1).all(-1).tolist()
    assert zero == [True, True, False, False, True, False, False]   # -2, -1 | 32 (past the table)
    changed = (kp != before[0]).any(-1).any(1).nonzero().tolist()
    assert changed == [[0, 0], [3, 15]]                             # position 0 of the first, 31 of the second
    assert (vp != before[1]).any(-1).any(1).nonzero().tolist() == changed


def test_append_past_32_bits():
    """A slot more than 2^31 elements into a pool (strides of a wide pool; only the touched rows are written)."""
    page, Hk, d = 16, 1, 64
    P = (1 << 31) // (page * 128) + 8                                # keys and values side by side in a row
    both = torch.zeros((P, Hk, page, 2 * d), dtype=torch.bfloat16, device="cuda")
    kp, vp = both[..., :d], both[..., d:]
    table = torch.tensor([[P - 1]], dtype=torch.int32).cuda()
    x = torch.randn(1, 3, d, device="cuda").bfloat16()
    fa.paged_append(x[:, :1], x[:, 1:2], x[:, 2:], kp, vp, table, ragged([1]).cuda(),
                    torch.tensor([6], dtype=torch.int32).cuda(), norm=False)
    assert status() == fa.FA_OK
    assert torch.equal(kp[P - 1, 0, 5], x[0, 1]) and torch.equal(vp[P - 1, 0, 5], x[0, 2])
    assert int(torch.count_nonzero(both[-16:])) == 2 * d and int(torch.count_nonzero(both[:16])) == 0
