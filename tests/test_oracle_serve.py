"""The fp64 forms in oracle/serve.py, pinned: differences, invariants, and the rectangular attention oracle (CPU only)."""

import numpy as np
import pytest

from oracle import serve
from oracle.decode import attention_forward_rect


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rope", [0, 16, 32])
@pytest.mark.parametrize("norm", [False, True])
def test_gradient_against_differences(interleaved, rope, norm):
    rng = np.random.default_rng(5)
    B, H, N, d, eps = 2, 2, 3, 32, 1e-3
    x, dz, w = rng.normal(size=(B, H, N, d)), rng.normal(size=(B, H, N, d)), 1 + 0.3 * rng.normal(size=d)
    table = serve.rope_table(9, rope) if rope else None
    pos = rng.integers(0, 9, size=(B, N))

    def f(x, w):
        return float((serve.norm_rope(x, w, eps, table, pos, interleaved, norm) * dz).sum())

    dx, dw = serve.norm_rope_grad(dz, x, w, eps, table, pos, interleaved, norm)
    step = 1e-5  # central differences: error O(step^2) + 1e-16 / step
    for _ in range(12):
        i = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = step
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * step) - dx[i]) < 1e-7
    if norm:
        for c in (0, 7, 31):
            e = np.zeros(d)
            e[c] = step
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * step) - dw[c]) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(6)
    q, k = rng.normal(size=(1, 1, 1, 64)), rng.normal(size=(1, 1, 1, 64))
    table = serve.rope_table(100, 64)
    turn = lambda x, p: serve.norm_rope(x, None, 0.0, table, np.array([[p]]), interleaved, norm=False)[0, 0, 0]  # noqa: E731
    assert abs(np.linalg.norm(turn(q, 77)) - np.linalg.norm(q)) < 1e-12
    assert abs(turn(q, 30) @ turn(k, 20) - turn(q, 75) @ turn(k, 65)) < 1e-11
    assert np.array_equal(turn(q, 0), q[0, 0, 0])


def test_paged_attention_equals_the_rectangular_oracle():
    rng = np.random.default_rng(7)
    Hq, Hk, d, page, n, m = 4, 2, 8, 16, 37, 5
    k, v = rng.normal(size=(Hk, 48, d)), rng.normal(size=(Hk, 48, d))
    table = np.array([[3, 0, 2]])
    kp, vp = np.zeros((5, Hk, page, d)), np.zeros((5, Hk, page, d))
    for i, p in enumerate(table[0]):
        kp[p], vp[p] = k[:, i * page:(i + 1) * page], v[:, i * page:(i + 1) * page]
    q = rng.normal(size=(m, Hq, d))
    for causal in (False, True):
        o, lse, _ = serve.paged_attention(q, kp, vp, table, [0, m], [n], 0.3, causal)
        ref_o, ref_lse = attention_forward_rect(q.transpose(1, 0, 2)[None], np.repeat(k[None, :, :n], 2, 1),
                                                np.repeat(v[None, :, :n], 2, 1), 0.3, causal)
        assert np.abs(o - ref_o[0].transpose(1, 0, 2)).max() < 1e-13
        assert np.abs(lse - ref_lse[0].T).max() < 1e-13


def test_rows_without_keys():
    kp = np.ones((1, 1, 16, 4))
    o, lse, _ = serve.paged_attention(np.ones((3, 1, 4)), kp, kp, np.array([[0]]), [0, 3], [1], 1.0, True)
    assert np.array_equal(o[:2], np.zeros((2, 1, 4))) and np.all(np.isneginf(lse[:2])) and np.all(o[2] == 1.0)


def test_append_then_read_back():
    rng = np.random.default_rng(8)
    kp = rng.normal(size=(3, 2, 16, 16))
    k, v = rng.normal(size=(2, 2, 16)), rng.normal(size=(2, 2, 16))
    table = serve.rope_table(32, 16)
    q_out, kn, vn = serve.paged_append(k, k, v, kp, kp, np.array([[2, 1]]), [0, 2], [17], None, None, 1e-6, table, False)
    assert np.array_equal(vn[2, :, 15], v[0]) and np.array_equal(vn[1, :, 0], v[1])
    assert np.array_equal(kn[2, :, 15], q_out[0]) and np.array_equal(kn[1, :, 0], q_out[1])
    kn[2, :, 15], kn[1, :, 0] = kp[2, :, 15], kp[1, :, 0]
    assert np.array_equal(kn, kp)
