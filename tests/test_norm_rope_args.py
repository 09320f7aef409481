"""What the norm, rotation and cache calls refuse (CPU only: validation fails before any device work)."""

import pytest
import torch

import exact_io_aware_31_gb300 as fa
from exact_io_aware_31_gb300 import build

A = 1 << 20  # a 16-byte aligned fake address; validation fails before it is used
INVALID, UNSUPPORTED, WORKSPACE = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load_library()


TURN = dict(norm=1, q_weight=A, k_weight=A, weights_f32=0, eps=1e-6, rope=A, rope_len=64, rope_dim=64, interleaved=0)
COMMON = [
    (dict(d=96), UNSUPPORTED), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(Hq=1 << 15), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(norm=2), INVALID),
    (dict(weights_f32=-1), INVALID), (dict(interleaved=3), INVALID), (dict(rope_dim=24), INVALID),
    (dict(rope_dim=-16), INVALID), (dict(rope_dim=128), INVALID), (dict(rope=None), INVALID),
    (dict(rope=A + 4), INVALID), (dict(rope_len=0), INVALID), (dict(q_weight=A + 2), INVALID),
    (dict(q=None), INVALID), (dict(k=A + 8), INVALID),
]
FWD = dict(q=A, k=A, q_out=A, k_out=A, B=2, Hq=4, Hk=2, N=64, d=64, q_stride_b=1 << 14, q_stride_h=64, q_stride_n=256,
           k_stride_b=1 << 14, k_stride_h=64, k_stride_n=256, **TURN, positions=None, stream=None)
BWD = dict(dq_out=A, dk_out=A, q=A, k=A, dq=A, dk=A, dq_weight=A, dk_weight=A,
           **{n: FWD[n] for n in list(FWD)[4:15]}, **{"d" + n: FWD[n] for n in list(FWD)[9:15]}, **TURN,
           positions=None, workspace=A, workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(N=65), INVALID), (dict(B=1 << 20, N=1 << 12), INVALID),
    (dict(k_out=None), INVALID), (dict(q_stride_n=12), INVALID), (dict(k_stride_h=-64), INVALID),
    (dict(positions=A + 2), INVALID),
])
def test_norm_rope_refusals(kw, code):
    assert fa.fa_qk_norm_rope(**(FWD | kw)) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(B=0), INVALID), (dict(N=65), INVALID), (dict(dq_out=None), INVALID), (dict(dk=A + 8), INVALID),
    (dict(dq_stride_h=0), INVALID), (dict(dk_stride_n=32), INVALID), (dict(dq_weight=A + 2), INVALID),
    (dict(norm=0), INVALID), (dict(workspace=None), WORKSPACE), (dict(workspace=A + 16), WORKSPACE),
    (dict(workspace_bytes=1024 * 2 * 64 * 4 - 1), WORKSPACE),
])
def test_norm_rope_bwd_refusals(kw, code):
    assert fa.fa_qk_norm_rope_bwd(**(BWD | kw)) == code


CACHE = dict(page_table=A, cu_seqlens=A, kv_lens=A)
APPEND = dict(q=A, k=A, v=A, q_out=A, k_pages=A, v_pages=A, **CACHE, T=5, S=2, Hq=4, Hk=2, d=64, num_pages=8,
              page_size=16, max_pages=4, q_stride_t=256, q_stride_h=64, k_stride_t=128, k_stride_h=64, v_stride_t=128,
              v_stride_h=64, kp_stride_p=2048, kp_stride_h=1024, kp_stride_r=64, vp_stride_p=2048, vp_stride_h=1024,
              vp_stride_r=64, **TURN, stream=None)
POOL = [
    (dict(T=-1), INVALID), (dict(S=-1), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(page_size=8), INVALID), (dict(page_size=48), INVALID), (dict(page_size=1 << 17), INVALID),
    (dict(max_pages=1 << 27), INVALID), (dict(k_pages=A + 8), INVALID), (dict(v_pages=None), INVALID),
    (dict(page_table=None), INVALID), (dict(cu_seqlens=None), INVALID), (dict(kv_lens=A + 2), INVALID),
    (dict(kp_stride_p=2044), INVALID), (dict(vp_stride_r=32), INVALID), (dict(kp_stride_h=0), INVALID),
]


@pytest.mark.parametrize("kw,code", COMMON + POOL + [
    (dict(v=None), INVALID), (dict(q_out=A + 8), INVALID), (dict(k_stride_t=100), INVALID), (dict(Hk=1 << 14), INVALID),
    (dict(T=0), fa.FA_OK), (dict(S=0), fa.FA_OK), (dict(T=0, q=None, k=None, v=None, q_out=None), fa.FA_OK),
])
def test_append_refusals(kw, code):
    assert fa.fa_paged_append(**(APPEND | kw)) == code


def test_workspace_size():
    assert fa.fa_qk_norm_rope_bwd_workspace_size(64) == 1024 * 2 * 64 * 4
    assert fa.fa_qk_norm_rope_bwd_workspace_size(128) == 1024 * 2 * 128 * 4
    assert fa.fa_qk_norm_rope_bwd_workspace_size(96) == 0


def test_status_string():
    assert fa.fa_status_string(fa.FA_ERR_DEVICE_INDEX).startswith("FA_ERR_DEVICE_INDEX")


def test_helpers_reject_cpu_tensors():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_backward(x, x, x, x)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.paged_append(x[0], x[0], x[0], x, x, i[None], i, i[:1])


def test_rope_table_layout():
    t = fa.rope_table(5, 4, base=100.0, device="cpu")
    angle = torch.arange(5, dtype=torch.float64)[:, None] * torch.tensor([1.0, 0.1], dtype=torch.float64)
    assert t.dtype == torch.float32 and torch.equal(t, torch.cat([angle.cos(), angle.sin()], 1).float())
    for bad in ((0, 4), (5, 3), (5, 0)):
        with pytest.raises(ValueError):
            fa.rope_table(*bad, device="cpu")


FWD_PAGED = dict(q=A, k_pages=A, v_pages=A, o=A, lse=A, **CACHE, T=5, S=2, Hq=4, Hk=2, d=64, num_pages=8, page_size=16,
                 max_pages=4, q_stride_t=256, q_stride_h=64, **{n: v for n, v in APPEND.items() if n[1:9] == "p_stride"},
                 scale=0.1, causal=1, max_q=0, workspace=A, workspace_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,code", POOL + [
    (dict(d=96), UNSUPPORTED), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(Hq=5), INVALID),
    (dict(Hq=258), UNSUPPORTED), (dict(Hq=1 << 15, Hk=1 << 14), INVALID), (dict(T=1 << 30), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(causal=2), INVALID), (dict(max_q=-1), INVALID), (dict(q=A + 8), INVALID),
    (dict(o=None), INVALID), (dict(lse=A + 2), INVALID), (dict(q_stride_t=0), INVALID), (dict(q_stride_h=68), INVALID),
    (dict(q_stride_t=1 << 31), INVALID), (dict(workspace=None), WORKSPACE), (dict(workspace=A + 64), WORKSPACE),
    (dict(T=0), fa.FA_OK), (dict(S=0, q=None, o=None, workspace=None), fa.FA_OK),
])
def test_paged_forward_refusals(kw, code):
    assert fa.fa_fwd_paged(**(FWD_PAGED | kw)) == code
