"""Norm with rotation, its gradient and the cache write at sizes where a warp takes several tokens (needs a GB300).

What the launches choose at 152 SMs (csrc/fa_norm_rope.cu): the forward gives a warp 2 tokens from 1824 CTAs of one
token a warp on and 4 from 3648, its row kernels (few heads) 2 turns above 912 CTAs and 4 above 1824; the gradient has
2048 CTAs at most, each with a row of partial sums, and goes on in more tokens a warp; the append gives a warp all
heads of a token from 608 groups of 8 tokens on.

Tolerances: of z and dx as in tests/test_gpu_norm_rope.py.  Of dw: a term is within 2^-20 of itself, and passes at most
``depth`` fp32 additions of 2^-24 each (the tokens and steps of a thread, 2 of lanes, 8 of warps, and 16 + 2 + 32 in
the kernel that adds the partial sums): (2^-20 + depth 2^-24) sum |dy x r|.  The gradients that come in are made of the
rows themselves and noise, so that dw grows like its number of terms and a row that is missing shows.
"""

import numpy as np
import pytest
import torch

import exact_io_aware_31_gb300 as fa
from oracle import serve
from tests.gpu_util import f64, require_gpu
from tests.test_gpu_norm_rope import BF, F32, ragged, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def packed(B, Hq, Hk, N, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, N, Hq + Hk + 1, d, generator=g, device="cuda", dtype=torch.bfloat16)
    return x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2), g


def inputs(B, Hq, Hk, N, d, rope, interleaved, seed=3):
    q, k, g = packed(B, Hq, Hk, N, d, seed)
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in "qk"]
    pos = torch.randint(0, 512, (B, N), generator=g, device="cuda", dtype=torch.int32)
    kw = dict(rope=fa.rope_table(512, rope), positions=pos, eps=1e-5, interleaved=interleaved)
    ref = dict(eps=1e-5, table=f64(kw["rope"]), positions=pos.cpu().numpy(), interleaved=interleaved)
    return q, k, w, kw, ref, g


def outgoing(q, k, g, kw):
    """Gradients of the outputs: the turned rows (so dy is about x) and noise."""
    return [(z.float() + torch.randn(z.shape, generator=g, device="cuda")).bfloat16()
            for z in fa.qk_norm_rope(q, k, rope=kw["rope"], positions=kw["positions"], interleaved=kw["interleaved"],
                                     norm=False)]


@pytest.mark.parametrize("Hq,Hk,d,B,N,rope,interleaved", [
    (17, 17, 64, 3, 1234, 64, False),     # 4 chunks a token x 463 groups: 2 tokens a warp
    (17, 17, 64, 3, 2435, 32, True),      # x 914: 4 tokens
    (9, 5, 128, 1, 10003, 128, False),    # 3 x 1251
    (8, 8, 64, 5, 2921, 64, True),        # chunks of two steps, 2 x 1826
    (4, 3, 128, 1, 14603, 96, False),     # the same
    (1, 1, 64, 2, 15013, 64, False),      # row by row, 940 CTAs: 2 turns
    (1, 1, 64, 7, 8581, 64, True),        # 1878: 4 turns
    (1, 2, 128, 1, 19991, 64, False),     # 1875: 4 turns
])
def test_forward(Hq, Hk, d, B, N, rope, interleaved):
    q, k, w, kw, ref, _ = inputs(B, Hq, Hk, N, d, rope, interleaved)
    outs = fa.qk_norm_rope(q, k, *w, **kw)
    assert status() == fa.FA_OK
    for z, x, wi in zip(outs, (q, k), w):
        r = serve.norm_rope(f64(x), f64(wi), **ref)
        err = np.abs(f64(z) - r) - BF * np.abs(r)
        assert (err <= 3 * F32 * np.abs(r).max(-1, keepdims=True)).all(), float(err.max())


@pytest.mark.parametrize("Hq,Hk,d,B,N,rope,interleaved", [
    (16, 16, 64, 3, 3001, 64, False),     # four steps: 1126 groups on 1024 runs of tokens, 2 tokens a warp
    (9, 9, 128, 1, 9001, 64, True),       # 1126 on 512: 3 tokens
    (8, 8, 64, 7, 1287, 64, False),       # two steps: 1127 on 1024
    (4, 4, 128, 1, 9003, 128, True),      # the same
    (8, 4, 64, 2, 5471, 48, False),       # one step: 1368 on 682: 3 tokens
    (4, 2, 128, 1, 6005, 128, True),      # 751 on 682
    (2, 1, 64, 1, 999, 64, False),        # (the one-step and row kernels without a second token)
    (4, 2, 128, 1, 333, 128, False),
    (1, 1, 64, 3, 22003, 64, False),      # row by row: 2064 CTAs of one turn, so 2 turns
    (1, 1, 128, 1, 70001, 128, True),     # 4376: 4 turns
])
def test_backward(Hq, Hk, d, B, N, rope, interleaved):
    q, k, w, kw, ref, g = inputs(B, Hq, Hk, N, d, rope, interleaved)
    dz = outgoing(q, k, g, kw)
    got = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw)
    again = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw)
    assert status() == fa.FA_OK and all(torch.equal(a, b) for a, b in zip(got, again))
    depth = 4 * 4 + 60
    for dx, dw, x, z, wi in zip(got[:2], got[2:], (q, k), dz, w):
        x, z = f64(x), f64(z)
        rx, rw = serve.norm_rope_grad(z, x, f64(wi), **ref)
        r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-5)
        gw = np.abs(z).max(-1, keepdims=True) * 2 * np.abs(f64(wi)).max()
        big = r * gw * (1 + (np.abs(x) * r).max(-1, keepdims=True) ** 2)
        err = np.abs(f64(dx) - rx) - BF * np.abs(rx)
        assert (err <= 4 * F32 * big).all(), float(err.max())
        size = np.abs(z).max(-1, keepdims=True) * 2 * np.abs(x) * r   # |dy| <= |z_a| + |z_b|
        bound = (F32 + depth * 2.0 ** -24) * size.reshape(-1, d).sum(0)
        assert (np.abs(f64(dw) - rw) <= bound).all()
        assert (bound < 1e-3 * np.abs(rw)).all()   # (a sixteenth of a warp's tokens missing would show)


@pytest.mark.parametrize("Hq,Hk,d,page,rope,interleaved", [
    (20, 4, 128, 64, 128, False),   # four steps, 5 chunks a token, walked by one warp
    (17, 5, 64, 16, 32, True),      # the same
    (8, 4, 64, 32, 64, False),      # two steps
    (4, 2, 128, 16, 64, True),
    (2, 1, 64, 16, 64, False),      # one step
    (1, 2, 128, 128, 128, True),
])
def test_append(Hq, Hk, d, page, rope, interleaved):
    g = torch.Generator().manual_seed(Hq)
    S = 61
    q_lens = [0 if i % 7 == 3 else int(n) for i, n in enumerate(torch.randint(1, 250, (S,), generator=g))]
    q_lens[5] = 1007
    kv_lens = [n + int(e) for n, e in zip(q_lens, torch.randint(0, 40, (S,), generator=g))]
    cu = ragged(q_lens)
    T = int(cu[-1])
    assert T > 4864 and T % 8 != 0
    need = [-(-n // page) for n in kv_lens]
    order = torch.randperm(sum(need) + 3, generator=g).to(torch.int32)
    table = torch.full((S, max(need)), -7, dtype=torch.int32)
    for s, n in enumerate(need):
        table[s, :n] = order[sum(need[:s]):sum(need[:s]) + n]
    x = torch.randn(T + 2, Hq + 2 * Hk, d, generator=g).bfloat16().cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    w = [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in "qk"]
    rt = fa.rope_table(max(kv_lens), rope)
    kp, vp = (torch.full((len(order), page, Hk, d), 9.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in "kv")
    out = torch.full((T + 2, Hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    fa.paged_append(q, k, v, kp, vp, table.cuda(), cu.cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(), *w,
                    rope=rt, eps=1e-5, interleaved=interleaved, out=out)
    assert status() == fa.FA_OK and bool((out[T:] == 5).all())
    seq = np.repeat(np.arange(S), q_lens)
    pos = np.arange(T) - cu.numpy()[seq] + (np.array(kv_lens) - np.array(q_lens))[seq]
    slot = table.numpy()[seq, pos // page], pos % page
    turn = lambda t, wi: serve.norm_rope(f64(t[:T]).transpose(1, 0, 2)[None], f64(wi), 1e-5, f64(rt), pos[None],  # noqa: E731
                                         interleaved)[0].transpose(1, 0, 2)
    kg = f64(kp).transpose(0, 2, 1, 3)
    for got, r in ((f64(out[:T]), turn(q, w[0])), (kg[slot], turn(k, w[1]))):
        err = np.abs(got - r) - BF * np.abs(r)
        assert (err <= 3 * F32 * np.abs(r).max(-1, keepdims=True)).all(), float(err.max())
    vg = f64(vp).transpose(0, 2, 1, 3)
    assert np.array_equal(vg[slot], f64(v[:T]))
    kg[slot], vg[slot] = 9.0, 9.0
    assert (kg == 9).all() and (vg == 9).all()     # no other slot was written


@pytest.mark.parametrize("Hq,Hk", [(16, 1), (1, 1)])
def test_past_32_bits(Hq, Hk):
    """Every tensor of the queries passes 2^31 elements, by chunks and row by row; sampled rows, and all of dw."""
    d, P = 64, 4096
    N = (1 << 31) // (Hq * d) + 77
    q, k, g = packed(1, Hq, Hk, N, d, 7)
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in "qk"]
    kw = dict(rope=fa.rope_table(P, d), positions=(torch.arange(N, device="cuda", dtype=torch.int32) % P)[None], eps=1e-5)
    z = fa.qk_norm_rope(q, k, *w, **kw)
    dz = fa.qk_norm_rope(q, k, rope=kw["rope"], positions=kw["positions"], norm=False)
    got = fa.qk_norm_rope_backward(*dz, q, k, *w, **kw)
    assert status() == fa.FA_OK
    at = torch.tensor([0, 1, N // 2, (1 << 31) // (Hq * d) - 1, (1 << 31) // (Hq * d), N - 70, N - 2, N - 1])
    ref = dict(eps=1e-5, table=f64(kw["rope"]), positions=(at.numpy() % P)[None], interleaved=False)
    pick = lambda t: f64(t[:, :, at.cuda()])  # noqa: E731
    for zi, dzi, dx, dw, x, wi in zip(z, dz, got[:2], got[2:], (q, k), w):
        assert zi.numel() > 1 << 31 or x.shape[1] < Hq
        r = serve.norm_rope(pick(x), f64(wi), **ref)
        assert (np.abs(pick(zi) - r) <= BF * np.abs(r) + 3 * F32 * np.abs(r).max(-1, keepdims=True)).all()
        xs, dzs = pick(x), pick(dzi)
        rx, _ = serve.norm_rope_grad(dzs, xs, f64(wi), **ref)
        inv = 1 / np.sqrt((xs ** 2).mean(-1, keepdims=True) + 1e-5)
        big = inv * np.abs(dzs).max(-1, keepdims=True) * 2 * np.abs(f64(wi)).max()
        big *= 1 + (np.abs(xs) * inv).max(-1, keepdims=True) ** 2
        assert (np.abs(pick(dx) - rx) <= BF * np.abs(rx) + 4 * F32 * big).all()
        want = torch.zeros(d, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        c, s = kw["rope"][:, :d // 2].double(), kw["rope"][:, d // 2:].double()
        for n0 in range(0, N, 1 << 18):
            n = slice(n0, min(n0 + (1 << 18), N))
            xs, dzs, p = x[:, :, n].double(), dzi[:, :, n].double(), kw["positions"][0, n].long()
            a, b = dzs[..., :d // 2], dzs[..., d // 2:]
            dy = torch.cat([a * c[p] + b * s[p], b * c[p] - a * s[p]], -1)
            term = dy * xs * (xs.pow(2).mean(-1, keepdim=True) + 1e-5).rsqrt()
            want += term.sum((0, 1, 2))
            size += term.abs().sum((0, 1, 2))
        # 512 tokens of two rows, or 257 of four, a thread
        assert bool(((dw.double() - want).abs() <= (4 * F32 + 1100 * 2.0 ** -24) * size).all())
