"""Work lists of the serving and training operators around the attention kernels.

Four operators: the norm of queries and keys for each head with the position
rotation in the same pass (``norm_rope``), its gradient (``norm_rope_bwd``),
the same pass on a ragged batch of new tokens that also writes keys and values
into a paged cache (``append``), and attention of those tokens over the paged
cache (``attention``).  ``run`` computes each in elementary torch operations
in 32 bits, or, where ``own`` is true, by the package's entry points.
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
ROPE_BASE = 10000.0


def listed():
    """The shapes named in workloads.py, and grouped key heads as such layers have them."""
    return [
        # training: queries and keys of the GPT-2 medium batch, rotated over the whole head
        {"name": "norm_rope_b64_h16_n1024_d64", "op": "norm_rope", "B": 64, "N": 1024, "Hq": 16, "Hk": 16, "d": 64,
         "rope": 64, "interleaved": False, "positions": False, "w32": True},
        # training: one odd-length sequence with grouped key heads, half of the head rotated in neighbouring pairs
        {"name": "norm_rope_b1_h32_8_n4093_d128", "op": "norm_rope", "B": 1, "N": 4093, "Hq": 32, "Hk": 8, "d": 128,
         "rope": 64, "interleaved": True, "positions": True, "w32": False},
        # the gradients of the first, what its backward pass hands to the projections
        {"name": "norm_rope_bwd_b64_h16_n1024_d64", "op": "norm_rope_bwd", "B": 64, "N": 1024, "Hq": 16, "Hk": 16,
         "d": 64, "rope": 64, "interleaved": False, "positions": False, "w32": True},
        # a small, odd training batch with packed positions
        {"name": "norm_rope_bwd_b2_h12_4_n777_d128", "op": "norm_rope_bwd", "B": 2, "N": 777, "Hq": 12, "Hk": 4,
         "d": 128, "rope": 128, "interleaved": False, "positions": True, "w32": False},
        # serving: one new token of each of 64 sequences goes into the cache
        {"name": "append_s64_q1_h32_8_d128_p64", "op": "append", "S": 64, "q": 1, "long": 64, "kv": 4096, "ragged": True,
         "Hq": 32, "Hk": 8, "d": 128, "page": 64, "token_major": False, "rope": 128, "interleaved": False, "w32": False},
        # serving: two long prompts arrive beside 14 running sequences, small pages, token-major cache
        {"name": "append_s16_q4096_h32_8_d128_p16", "op": "append", "S": 16, "q": 4096, "long": 2, "kv": 4500,
         "ragged": True, "Hq": 32, "Hk": 8, "d": 128, "page": 16, "token_major": True, "rope": 64,
         "interleaved": True, "w32": True},
        # the smallest call: one short sequence, one token
        {"name": "attention_s1_q1_kv130_h16_d64_p16", "op": "attention", "S": 1, "q": 1, "long": 1, "kv": 130,
         "ragged": False, "Hq": 16, "Hk": 16, "d": 64, "page": 16, "token_major": False, "causal": True},
        # one token against the long-sequence shape's whole cache
        {"name": "attention_s1_q1_kv16384_h16_d128_p64", "op": "attention", "S": 1, "q": 1, "long": 1, "kv": 16384,
         "ragged": False, "Hq": 16, "Hk": 16, "d": 128, "page": 64, "token_major": False, "causal": True},
        # a decoding batch of ragged lengths, grouped heads, token-major pages
        {"name": "attention_s64_q1_kv8192_h32_8_d128_p16", "op": "attention", "S": 64, "q": 1, "long": 64, "kv": 8192,
         "ragged": True, "Hq": 32, "Hk": 8, "d": 128, "page": 16, "token_major": True, "causal": True},
        # eight speculated tokens of the GPT-2 medium batch against its 1024-key cache
        {"name": "attention_s64_q8_kv1024_h16_d64_p32", "op": "attention", "S": 64, "q": 8, "long": 64, "kv": 1024,
         "ragged": True, "Hq": 16, "Hk": 16, "d": 64, "page": 32, "token_major": False, "causal": True},
        # chunked prefill: 2048 new tokens of two long prompts
        {"name": "attention_s2_q2048_kv16384_h32_8_d128_p128", "op": "attention", "S": 2, "q": 2048, "long": 2,
         "kv": 16384, "ragged": True, "Hq": 32, "Hk": 8, "d": 128, "page": 128, "token_major": False, "causal": True},
        # a mixed serving step: two chunks beside 14 single tokens, odd group size
        {"name": "attention_s16_q509_kv4096_h20_4_d128_p64", "op": "attention", "S": 16, "q": 509, "long": 2,
         "kv": 4096, "ragged": True, "Hq": 20, "Hk": 4, "d": 128, "page": 64, "token_major": False, "causal": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    """One more case: head layouts, page sizes and lengths of the same ranges, odd ones among them."""
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "attention", "attention", "attention"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 5, 8, 16])
    Hq = Hk * rng.choice([1, 1, 2, 3, 4, 5, 8])
    case = {"op": op, "Hq": Hq, "Hk": Hk, "d": d}
    if op != "attention":
        case["rope"] = rng.choice([d, d, d // 2, 16])
        case["interleaved"] = rng.random() < 0.4
        case["w32"] = rng.random() < 0.5
    if op in ("norm_rope", "norm_rope_bwd"):
        rows = _log(rng, 40, 65536 * 2048 // ((Hq + Hk) * d))   # tokens: no more bytes than the largest listed case
        B = min(rows, _log(rng, 1, 64))
        return case | {"B": B, "N": max(1, rows // B), "positions": rng.random() < 0.5}
    case |= {"page": rng.choice([16, 32, 64, 128, 256]), "token_major": rng.random() < 0.5, "ragged": rng.random() < 0.8}
    S = _log(rng, 1, 64)
    if op == "append":
        q = _log(rng, 1, max(1, min(4096, 8192 * 40 * 128 // (S * (Hq + 2 * Hk) * d))))
        return case | {"S": S, "q": q, "long": rng.randint(1, S), "kv": q + _log(rng, 1, 512)}
    # attention: single tokens, a few, or chunks; bounded by the largest listed case's pairs and cache
    q = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 2048)])
    long = S if q <= 8 else rng.randint(1, min(S, 4))
    kv = _log(rng, 100, 32768)
    kv = min(kv, 64 * 8192 * 8 * 128 // (S * Hk * d), (1 << 41) // (4 * d * Hq * q * S))
    return case | {"S": S, "q": q, "long": long, "kv": max(kv, q), "causal": rng.random() < 0.85}


def _lengths(case):
    """New tokens and cache lengths (new tokens included) of each sequence: by the case alone."""
    qs, kvs = [], []
    for i in range(case["S"]):
        q = case["q"] if i * case["long"] // case["S"] != (i + 1) * case["long"] // case["S"] else 1
        part = 1.0 - 0.75 * math.modf(i * 0.6180339887)[0] if case["ragged"] else 1.0
        qs.append(q)
        kvs.append(max(q, round(case["kv"] * part)))
    return qs, kvs


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rope_table(length, dim):
    """[length, dim] fp32: cosines, then sines, of p * base^(-2 i / dim); angles in 64 bits."""
    i = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * ROPE_BASE ** (-2.0 * i / dim)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    st = {"case": case}
    if case["op"] != "attention":
        wt = torch.float32 if case["w32"] else torch.bfloat16
        st["q_weight"], st["k_weight"] = ((1.0 + 0.2 * _randn(g, d, dtype=torch.float32)).to(wt) for _ in range(2))
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        B, N = case["B"], case["N"]
        # the projection's output: queries and keys side by side in one row per token
        qk = _randn(g, B, N, Hq + Hk, d)
        st["q"], st["k"] = qk[:, :, :Hq].transpose(1, 2), qk[:, :, Hq:].transpose(1, 2)
        st["rope"] = _rope_table(2 * N, case["rope"])
        st["positions"] = None
        if case["positions"]:  # every sequence starts somewhere in the table
            start = torch.randint(0, N + 1, (B, 1), generator=g, device="cuda")
            st["positions"] = (start + torch.arange(N, device="cuda")).to(torch.int32)
        if case["op"] == "norm_rope_bwd":
            st["dq_out"], st["dk_out"] = _randn(g, B, Hq, N, d), _randn(g, B, Hk, N, d)
        return st
    qs, kvs = _lengths(case)
    page, S = case["page"], case["S"]
    T = sum(qs)
    need = [-(-n // page) for n in kvs]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)  # pages are anywhere in the pool
    table = torch.zeros((S, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for s in range(S):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    st["page_table"] = table
    st["cu_seqlens"] = torch.tensor([0] + [sum(qs[:i + 1]) for i in range(S)], dtype=torch.int32, device="cuda")
    st["kv_lens"] = torch.tensor(kvs, dtype=torch.int32, device="cuda")
    shape = (pool, page, Hk, d) if case["token_major"] else (pool, Hk, page, d)
    st["k_pages"], st["v_pages"] = _randn(g, *shape), _randn(g, *shape)
    if case["token_major"]:
        st["k_pages"], st["v_pages"] = st["k_pages"].transpose(1, 2), st["v_pages"].transpose(1, 2)
    if case["op"] == "append":
        qkv = _randn(g, T, Hq + 2 * Hk, d)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        st["rope"] = _rope_table(max(kvs), case["rope"])
    else:
        st["q"] = _randn(g, T, Hq, d)
    return st


def _turn(x, cos, sin, interleaved):
    """Rotate the first 2 * cos.shape[-1] columns of the rows of x, in x's type."""
    half = cos.shape[-1]
    r = x[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _norm_rope(x, w, cos, sin, interleaved):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return _turn(y, cos, sin, interleaved).to(torch.bfloat16)


def _norm_rope_bwd(dz, x, w, cos, sin, interleaved):
    x, dy = x.float(), _turn(dz.float(), cos, -sin, interleaved)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat = x * r
    g = dy * w.float()
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    dw = (dy * xhat).double().sum((0, 1, 2)).float()
    return dx.to(torch.bfloat16), dw


def _angles(st, positions):
    """Cosines and sines at the given positions, the table's row split in two."""
    rows = st["rope"][positions.long()]
    half = rows.shape[-1] // 2
    return rows[..., :half], rows[..., half:]


def _slots(st):
    """For every new token: its sequence, its position there, and its page and row in the pool."""
    cu, lens, table = st["cu_seqlens"].long(), st["kv_lens"].long(), st["page_table"].long()
    t = torch.arange(st["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[seq] - cu[seq + 1] + t
    page = st["k_pages"].shape[2]
    return seq, pos, table[seq, pos // page], pos % page


def _gathered(st, pages):
    """The pages of every sequence side by side, padded: [S, Hk, longest, d] in 32 bits, zero behind each end."""
    table = st["page_table"].long()
    x = pages[table].transpose(2, 3).flatten(1, 2).transpose(1, 2).float()
    live = torch.arange(x.shape[2], device="cuda") < st["kv_lens"].long()[:, None]
    return torch.where(live[:, None, :, None], x, 0.0), live


def _attention(st):
    case = st["case"]
    G, Hk, d = case["Hq"] // case["Hk"], case["Hk"], case["d"]
    cu, lens = st["cu_seqlens"].long(), st["kv_lens"].long()
    T, S = st["q"].shape[0], cu.shape[0] - 1
    keys, live = _gathered(st, st["k_pages"])
    values, _ = _gathered(st, st["v_pages"])
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    at = t - cu[seq]
    q = torch.zeros((S, case["q"], Hk, G, d), device="cuda")
    q[seq, at] = st["q"].float().view(T, Hk, G, d)
    rows = q.permute(0, 2, 1, 3, 4).flatten(2, 3)                       # [S, Hk, tokens * G, d]
    s = rows @ keys.transpose(2, 3) * d ** -0.5                         # [S, Hk, tokens * G, longest]
    see = live[:, None, :]
    if case["causal"]:
        last = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(case["q"], device="cuda")
        see = see & (torch.arange(live.shape[1], device="cuda") <= last[:, :, None])
    else:
        see = see.expand(S, case["q"], live.shape[1])
    s = s.view(S, Hk, case["q"], G, -1).masked_fill_(~see[:, None, :, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ values).view(S, Hk, case["q"], G, d) / l
    lse = (m + l.log()).squeeze(-1)
    o, lse = (x.transpose(1, 2)[seq, at] for x in (o, lse))             # back to one row per token
    return o.reshape(T, -1, d).to(torch.bfloat16), lse.reshape(T, -1)


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if own:
        import exact_io_aware_31_gb300 as fa
        if op == "attention":
            return fa.paged_forward(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["cu_seqlens"],
                                    st["kv_lens"], causal=case["causal"], max_q=case["q"])
        how = dict(eps=EPS, interleaved=case["interleaved"])
        weights = (st["q_weight"], st["k_weight"], st["rope"])
        if op == "norm_rope":
            return fa.qk_norm_rope(st["q"], st["k"], *weights, positions=st["positions"], **how)
        if op == "norm_rope_bwd":
            return fa.qk_norm_rope_backward(st["dq_out"], st["dk_out"], st["q"], st["k"], *weights,
                                            positions=st["positions"], **how)
        q_out = fa.paged_append(st["q"], st["k"], st["v"], st["k_pages"], st["v_pages"], st["page_table"],
                                st["cu_seqlens"], st["kv_lens"], *weights, **how)
        return q_out, st["k_pages"], st["v_pages"]
    if op == "attention":
        return _attention(st)
    if op == "append":
        _, pos, page, row = _slots(st)
        cos, sin = (x[:, None] for x in _angles(st, pos))
        q_out = _norm_rope(st["q"], st["q_weight"], cos, sin, case["interleaved"])
        st["k_pages"][page, :, row] = _norm_rope(st["k"], st["k_weight"], cos, sin, case["interleaved"])
        st["v_pages"][page, :, row] = st["v"]
        return q_out, st["k_pages"], st["v_pages"]
    B, N = case["B"], case["N"]
    positions = st["positions"] if case["positions"] else torch.arange(N, device="cuda").expand(B, N)
    cos, sin = (x[:, None] for x in _angles(st, positions))
    if op == "norm_rope":
        return (_norm_rope(st["q"], st["q_weight"], cos, sin, case["interleaved"]),
                _norm_rope(st["k"], st["k_weight"], cos, sin, case["interleaved"]))
    dq, dqw = _norm_rope_bwd(st["dq_out"], st["q"], st["q_weight"], cos, sin, case["interleaved"])
    dk, dkw = _norm_rope_bwd(st["dk_out"], st["k"], st["k_weight"], cos, sin, case["interleaved"])
    return dq, dk, dqw, dkw


def work(case):
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    if case["op"] == "attention":
        qs, kvs = _lengths(case)
        T = sum(qs)
        pairs = sum(q * n - (q * (q - 1) // 2 if case["causal"] else 0) for q, n in zip(qs, kvs))
        table = sum(-(-n // case["page"]) for n in kvs)
        return {"bytes": 4 * T * Hq * d + 4 * T * Hq + 4 * sum(kvs) * Hk * d + 4 * table + 4 * (2 * case["S"] + 1),
                "flops": 4 * pairs * Hq * d}
    if case["op"] == "append":
        qs, _ = _lengths(case)
        T = sum(qs)
        return {"bytes": 4 * T * (Hq + 2 * Hk) * d + 4 * T * case["rope"] + 4 * T,
                "flops": T * (Hq + Hk) * (4 * d + 3 * case["rope"])}
    tokens = case["B"] * case["N"]
    rows = (tokens if case["positions"] else case["N"]) * case["rope"]
    back = case["op"] == "norm_rope_bwd"
    return {"bytes": (6 if back else 4) * tokens * (Hq + Hk) * d + 4 * rows + 4 * tokens * case["positions"],
            "flops": tokens * (Hq + Hk) * ((10 if back else 4) * d + 3 * case["rope"])}


# ---------------------------------------------------------------- 64 bits ----
def _exact_rotation(table, positions, interleaved, d):
    """The rotation as d x d matrices, one per position: y = R x."""
    half = table.shape[1] // 2
    c, s = table[positions, :half].double(), table[positions, half:].double()
    R = torch.zeros(positions.shape[0], d, d, dtype=torch.float64, device="cuda")
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    R[:, a, a], R[:, b, b], R[:, a, b], R[:, b, a] = c, c, -s, s
    rest = torch.arange(2 * half, d, device="cuda")
    R[:, rest, rest] = 1.0
    return R


def _exact_rows(x, w, R):
    """z = R (w * x / rms(x)) for x [tokens, heads, d], R [tokens, d, d]."""
    x = x.double()
    y = w.double() * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return torch.einsum("tij,thj->thi", R, y)


def _exact_rows_grad(dz, x, w, R):
    """dx and dw of sum(z * dz), by the derivative of x / rms(x)."""
    x, w = x.double(), w.double()
    dy = torch.einsum("tij,thi->thj", R, dz.double())
    ms = x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS
    dw = (dy * x / ms.sqrt()).sum((0, 1))
    v = dy * w
    dx = v / ms.sqrt() - x * (v * x).sum(-1, keepdim=True) / (x.shape[-1] * ms * ms.sqrt())
    return dx, dw


def exact(case, seed):
    st = prepare(case, seed)
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        B, N = case["B"], case["N"]
        outs = []
        dws = [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2)]
        for x, w, dz, dw in ((st["q"], st["q_weight"], st.get("dq_out"), dws[0]),
                             (st["k"], st["k_weight"], st.get("dk_out"), dws[1])):
            out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for b in range(B):
                for n in range(0, N, 4096):
                    m = min(N, n + 4096)
                    pos = st["positions"][b, n:m].long() if case["positions"] else torch.arange(n, m, device="cuda")
                    R = _exact_rotation(st["rope"], pos, case["interleaved"], d)
                    rows = x[b, :, n:m].transpose(0, 1)
                    if dz is None:
                        z = _exact_rows(rows, w, R)
                    else:
                        z, part = _exact_rows_grad(dz[b, :, n:m].transpose(0, 1), rows, w, R)
                        dw += part
                    out[b, :, n:m] = z.transpose(0, 1)
            outs.append(out)
        return tuple(outs) if case["op"] == "norm_rope" else (*outs, *dws)
    qs, kvs = _lengths(case)
    page = case["page"]
    if case["op"] == "append":
        q_out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        kp, vp = st["k_pages"].double(), st["v_pages"].double()
        at = 0
        for s in range(case["S"]):
            for n in range(0, qs[s], 2048):
                m = min(qs[s], n + 2048)
                pos = torch.arange(n, m, device="cuda") + kvs[s] - qs[s]
                R = _exact_rotation(st["rope"], pos, case["interleaved"], d)
                q_out[at + n:at + m] = _exact_rows(st["q"][at + n:at + m], st["q_weight"], R)
                where = st["page_table"][s, torch.div(pos, page, rounding_mode="floor")].long()
                kp[where, :, pos % page] = _exact_rows(st["k"][at + n:at + m], st["k_weight"], R)
                vp[where, :, pos % page] = st["v"][at + n:at + m].double()
            at += qs[s]
        return q_out, kp, vp
    T = sum(qs)
    o = torch.empty(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(T, Hq, dtype=torch.float64, device="cuda")
    G, at = Hq // Hk, 0
    for s in range(case["S"]):
        pages = st["page_table"][s, :-(-kvs[s] // page)].long()
        keys = st["k_pages"][pages].transpose(0, 1).reshape(Hk, -1, d)[:, :kvs[s]].double()
        values = st["v_pages"][pages].transpose(0, 1).reshape(Hk, -1, d)[:, :kvs[s]].double()
        for n in range(0, qs[s], 1024):
            m = min(qs[s], n + 1024)
            rows = st["q"][at + n:at + m].double().view(m - n, Hk, G, d).permute(1, 2, 0, 3)
            score = torch.einsum("hgqd,hkd->hgqk", rows, keys) / math.sqrt(d)
            if case["causal"]:
                i = torch.arange(n, m, device="cuda")[:, None] + kvs[s] - qs[s]
                score = torch.where(torch.arange(kvs[s], device="cuda") <= i, score, -math.inf)
            z = torch.logsumexp(score, -1)
            out = torch.einsum("hgqk,hkd->hgqd", torch.exp(score - z[..., None]), values)
            o[at + n:at + m] = out.permute(2, 0, 1, 3).reshape(m - n, Hq, d)
            lse[at + n:at + m] = z.permute(2, 0, 1).reshape(m - n, Hq)
        at += qs[s]
    return o, lse
