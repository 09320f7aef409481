"""Work lists of the operators of a serving step whose batch shares prompts.

Three operators: the step's tables, lengths and slots built on the GPU from
the requests' lengths, with pages taken from a pool (``extend``), pages given
back to it (``release``), and attention of a batch whose sequences share their
first pages (``shared``).  A pass of the first two is a whole turn that leaves
the requests as it found them, so that any number of passes see the same step.
``run`` computes each in elementary torch operations, or, where ``own`` is
true, by the package's entry points.
"""

from __future__ import annotations

import math

import torch

own = False


def listed():
    """The shapes named in workloads.py and perf/operators.py as batches that share prompts have them."""
    return [
        # the smallest step: one running request, one token
        {"name": "extend_s1_q1_p16", "op": "extend", "S": 1, "R": 4, "q": 1, "long": 1, "kv": 130, "page": 16,
         "pad": 0, "ragged": False},
        # a decoding step of 256 requests among 512 places, small pages, a captured batch with empty places
        {"name": "extend_s256_q1_kv8192_p16", "op": "extend", "S": 256, "R": 512, "q": 1, "long": 256, "kv": 8192,
         "page": 16, "pad": 31, "ragged": True},
        # speculated tokens of which none is accepted
        {"name": "extend_s64_q7_kv4096_p64", "op": "extend", "S": 64, "R": 64, "q": 7, "long": 64, "kv": 4096,
         "page": 64, "pad": 0, "ragged": True},
        # a large batch of long requests: the tables are what is moved
        {"name": "extend_s1024_q1_kv32768_p16", "op": "extend", "S": 1024, "R": 1500, "q": 1, "long": 1024,
         "kv": 32768, "page": 16, "pad": 0, "ragged": True},
        # 14 short requests and two prompts of 4096 tokens arrive, and end
        {"name": "release_s16_q4096_p16", "op": "release", "S": 16, "R": 64, "q": 4096, "long": 2, "kv": 97,
         "page": 16, "pad": 0, "ragged": True},
        # a whole batch of finished requests gives its pages back
        {"name": "release_s200_q3000_p32", "op": "release", "S": 200, "R": 256, "q": 3001, "long": 200, "kv": 0,
         "page": 32, "pad": 3, "ragged": True},
        # the smallest shared call: four samples of one short prompt
        {"name": "shared_g1_s4_q1_p512_h16_d64", "op": "shared", "groups": 1, "S": 4, "alone": 0, "q": 1, "long": 4,
         "prefix": 512, "own": 60, "ragged": False, "Hq": 16, "Hk": 16, "d": 64, "page": 16, "token_major": False,
         "causal": True},
        # a decoding batch behind one system prompt
        {"name": "shared_g1_s64_q1_p8192_h32_8_d128", "op": "shared", "groups": 1, "S": 64, "alone": 0, "q": 1,
         "long": 64, "prefix": 8192, "own": 512, "ragged": True, "Hq": 32, "Hk": 8, "d": 128, "page": 16,
         "token_major": True, "causal": True},
        # many samples of a prompt of odd length, every head its own keys
        {"name": "shared_g1_s128_q1_p1021_h16_d64", "op": "shared", "groups": 1, "S": 128, "alone": 0, "q": 1,
         "long": 128, "prefix": 1021, "own": 67, "ragged": True, "Hq": 16, "Hk": 16, "d": 64, "page": 32,
         "token_major": False, "causal": True},
        # four prompts, a few speculated tokens of each sample, odd group size, three sequences of their own
        {"name": "shared_g4_s51_q5_p4093_h20_4_d128", "op": "shared", "groups": 4, "S": 48, "alone": 3, "q": 5,
         "long": 48, "prefix": 4093, "own": 301, "ragged": True, "Hq": 20, "Hk": 4, "d": 128, "page": 64,
         "token_major": False, "causal": True},
        # a large decoding batch, own parts half of the prompt
        {"name": "shared_g2_s256_q1_p2048_h32_8_d128", "op": "shared", "groups": 2, "S": 256, "alone": 0, "q": 1,
         "long": 256, "prefix": 2048, "own": 1024, "ragged": True, "Hq": 32, "Hk": 8, "d": 128, "page": 64,
         "token_major": False, "causal": True},
        # eight questions of 509 tokens about one long document
        {"name": "shared_g1_s8_q509_p16384_h32_8_d128", "op": "shared", "groups": 1, "S": 8, "alone": 0, "q": 509,
         "long": 8, "prefix": 16384, "own": 515, "ragged": False, "Hq": 32, "Hk": 8, "d": 128, "page": 128,
         "token_major": False, "causal": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    """One more case: batches, prompts, head layouts and page sizes of the same ranges, odd ones among them."""
    op = rng.choice(["extend", "release", "shared", "shared", "shared"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op != "shared":
        S = _log(rng, 1, 1024)
        q = rng.choice([1, rng.randint(2, 8), _log(rng, 9, 4096)]) if op == "extend" else _log(rng, 1, 4096)
        long = rng.randint(1, max(1, min(S, 400000 // q)))
        kv = _log(rng, 1, min(32768, 20000 * 1024 // S)) if op == "extend" else rng.choice([0, _log(rng, 1, 2048)])
        return {"op": op, "S": S, "R": S + rng.choice([0, rng.randint(1, 600)]), "q": q, "long": long, "kv": kv, "page": page,
                "pad": rng.choice([0, rng.randint(0, S - 1)]), "ragged": rng.random() < 0.8}
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 5, 8, 16])
    Hq = Hk * rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
    groups = rng.choice([1, 1, 2, _log(rng, 3, 16)])
    # single tokens, a few, or chunks; bounded by the largest listed cases' pairs and own keys
    q = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 512)])
    S = max(groups, _log(rng, 2, 256 if q <= 8 else 16))
    long = S if q <= 8 else rng.randint(1, min(S, 8))
    tokens = q * long + S - long
    prefix = max(1, min(_log(rng, 64, 32768), (1 << 40) // (4 * d * Hq * tokens), (1 << 19) // groups))
    most = 256 * 1024 * 8 * 128 // (S * Hk * d)
    mine = max(1, min(_log(rng, 1, 2048), most, (1 << 39) // (4 * d * Hq * tokens)))
    return {"op": op, "groups": groups, "S": S, "alone": rng.choice([0, 0, rng.randint(1, 4)]), "q": q, "long": long,
            "prefix": prefix, "own": mine, "ragged": rng.random() < 0.8, "Hq": Hq, "Hk": Hk, "d": d, "page": page,
            "token_major": rng.random() < 0.5, "causal": rng.random() < 0.85}


def _part(i):
    """Between 1/4 and 1, spread evenly: by the index alone."""
    return 1.0 - 0.75 * math.modf(i * 0.6180339887)[0]


def _new(case, i, S):
    """New tokens of sequence i: `long` of the S sequences bring q, the others one."""
    return case["q"] if i * case["long"] // S != (i + 1) * case["long"] // S else 1


def _steps(case):
    """New tokens and cached keys of each sequence of a step (extend, release)."""
    qs, lens = [], []
    for i in range(case["S"]):
        part = _part(i) if case["ragged"] else 1.0
        q = _new(case, i, case["S"])
        qs.append(max(1, round(q * part)) if case["op"] == "release" else q)
        lens.append(round(case["kv"] * part))
    return qs, lens


def _batch(case):
    """Of a shared batch: the groups' first sequences, their shared keys (whole pages), new tokens, lengths."""
    S, n, page = case["S"], case["groups"], case["page"]
    first = [g * S // n for g in range(n + 1)]
    shared = [max(1, round(case["prefix"] * (_part(g + 1) if case["ragged"] and g else 1.0)) // page) * page
              for g in range(n)]
    qs, kvs = [], []
    for i in range(S + case["alone"]):
        q = _new(case, i, S) if i < S else 1
        g = sum(i >= f for f in first[1:])
        mine = max(1, round(case["own"] * (_part(i) if case["ragged"] else 1.0)))
        qs.append(q)
        kvs.append((shared[g] if i < S else 0) + mine + q - 1)
    return first, shared, qs, kvs


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(qs):
    cu = [0]
    for q in qs:
        cu.append(cu[-1] + q)
    return cu


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    page, st = case["page"], {"case": case}
    if case["op"] != "shared":
        qs, lens = _steps(case)
        S, R = case["S"], case["R"]
        held = [-(-n // page) for n in lens]
        most = max(-(-(n + q) // page) for n, q in zip(lens, qs))
        taken = sum(held)
        spare = sum(-(-(n + q) // page) for n, q in zip(lens, qs)) - taken
        num_pages = taken + spare + 5
        order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)  # pages are anywhere in the pool
        place = torch.randperm(R, generator=g, device="cuda").to(torch.int32)[:S]      # requests, too
        st["requests"] = torch.cat([place, _ints([-1] * case["pad"])])
        st["new_lens"] = _ints(qs + [0] * case["pad"])
        st["request_lens"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        st["request_lens"][place.long()] = _ints(lens)
        st["lens"] = _ints(lens + [0] * case["pad"])         # what the requests keep at the end of the turn
        st["request_table"] = torch.zeros(R, most, dtype=torch.int32, device="cuda")
        row = torch.repeat_interleave(place.long(), _ints(held).long())
        col = torch.cat([torch.arange(n, device="cuda") for n in held])
        st["request_table"][row, col] = order[:taken]
        st["pool"] = torch.zeros(num_pages + 2, dtype=torch.int32, device="cuda")
        st["pool"][0] = num_pages - taken
        st["pool"][2:2 + num_pages - taken] = order[taken:]
        # the step's buffers, as a program with captured graphs keeps them
        T, S = sum(qs), S + case["pad"]
        st["out"] = (torch.zeros(S + 1, dtype=torch.int32, device="cuda"),
                     torch.zeros(S, dtype=torch.int32, device="cuda"),
                     torch.zeros(S, most, dtype=torch.int32, device="cuda"),
                     torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda"))
        return st
    first, shared, qs, kvs = _batch(case)
    n, S, Hq, Hk, d = case["groups"], case["S"], case["Hq"], case["Hk"], case["d"]
    common = [shared[sum(i >= f for f in first[1:])] // page if i < S else 0 for i in range(len(qs))]
    need = [-(-k // page) for k in kvs]
    num_pages = sum(s // page for s in shared) + sum(a - c for a, c in zip(need, common)) + 3
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(qs), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for j in range(n):
        table[first[j]:first[j + 1], :shared[j] // page] = order[at:at + shared[j] // page]
        at += shared[j] // page
    for i in range(len(qs)):
        table[i, common[i]:need[i]] = order[at:at + need[i] - common[i]]
        at += need[i] - common[i]
    st["page_table"], st["cu_seqlens"], st["kv_lens"] = table, _ints(_starts(qs)), _ints(kvs)
    st["groups"], st["prefix_lens"] = _ints(first), _ints(shared)
    shape = (num_pages, page, Hk, d) if case["token_major"] else (num_pages, Hk, page, d)
    for name in ("k_pages", "v_pages"):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
        st[name] = x.transpose(1, 2) if case["token_major"] else x
    st["q"] = torch.randn(sum(qs), Hq, d, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    return st


# ------------------------------------------------------------- plain forms ----
def _more(x, n=1):
    """x with n rows more, for what is written nowhere."""
    return torch.cat([x, x.new_zeros(n, *x.shape[1:])])


def _extend(st):
    """The step's tables in torch operations: no request is refused in these batches; empty places have none."""
    page, R = st["case"]["page"], st["case"]["R"]
    cu, kv_lens, page_table, positions, slots = st["out"]
    r = torch.where(st["requests"] >= 0, st["requests"], R).long()
    lens, table, free = _more(st["request_lens"]), _more(st["request_table"]), st["pool"][2:]
    old, new = lens[r].long(), torch.where(r < R, st["new_lens"], 0).long()
    cu.zero_()
    cu[1:] = new.cumsum(0)
    kv_lens.copy_(old + new)
    held, need = (old + page - 1) // page, (old + new + page - 1) // page
    before = (need - held).cumsum(0) - (need - held)         # pages that the sequences in front take
    at = torch.arange(page_table.shape[1], device="cuda")
    top = st["pool"][0] - 1 - (before[:, None] + at - held[:, None])
    fresh = (at >= held[:, None]) & (at < need[:, None])
    rows = torch.where(fresh, free[top.clamp(0, free.shape[0] - 1)], table[r])
    page_table.copy_(torch.where(at < need[:, None], rows, page_table))
    t = torch.arange(positions.shape[0], device="cuda")
    seq = torch.searchsorted(cu.long(), t, right=True) - 1
    pos = old[seq] + t - cu[seq]
    positions.copy_(pos)
    slots.copy_(page_table[seq, pos // page].long() * page + pos % page)
    table[r], lens[r] = rows, kv_lens
    st["request_table"].copy_(table[:R])
    st["request_lens"].copy_(lens[:R])
    st["pool"][0] -= (need - held).sum()


def _release(st):
    page, R = st["case"]["page"], st["case"]["R"]
    r = torch.where(st["requests"] >= 0, st["requests"], R).long()
    lens, table, free = _more(st["request_lens"]), _more(st["request_table"]), st["pool"][2:]
    first, last = ((x.long() + page - 1) // page for x in (st["lens"], lens[r]))
    given = last - first
    before = given.cumsum(0) - given
    at = torch.arange(table.shape[1], device="cuda")
    # on the stack so that they would be taken in the same order again; entries that stay go behind its end
    place = st["pool"][0] + given.sum() - 1 - (before[:, None] + at - first[:, None])
    goes = (at >= first[:, None]) & (at < last[:, None])
    stack = _more(free)
    stack[torch.where(goes, place, free.shape[0])] = table[r]
    free.copy_(stack[:-1])
    lens[r] = st["lens"]
    st["request_lens"].copy_(lens[:R])
    st["pool"][0] += given.sum()


def _partial(q, keys, values, see):
    """Maximum, sum and unnormalised output of rows q [.., n, d] over keys [.., m, d] where `see` allows (None: all)."""
    s = q @ keys.transpose(-1, -2) * q.shape[-1] ** -0.5
    if see is not None:
        s.masked_fill_(~see, float("-inf"))
    m = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = s.sub_(m).exp_()
    return m, p.sum(-1, keepdim=True), p @ values


def _shared(st):
    case = st["case"]
    Hk, d, page, G = case["Hk"], case["d"], case["page"], case["Hq"] // case["Hk"]
    first, shared, qs, _ = _batch(case)   # sizes of tensors: what a program knows of its batch on the host
    cu, lens, table = st["cu_seqlens"].long(), st["kv_lens"].long(), st["page_table"].long()
    T, S, q_max = st["q"].shape[0], len(qs), max(qs)
    rows = st["q"].float().view(T, Hk, G, d).permute(1, 0, 2, 3)           # [Hk, T, G, d]
    m1 = torch.full((Hk, T, G, 1), -3e38, device="cuda")
    l1, o1 = torch.zeros_like(m1), torch.zeros(Hk, T, G, d, device="cuda")
    start = _starts(qs)
    skip = torch.zeros(S, dtype=torch.int64, device="cuda")
    for j in range(case["groups"]):                                        # a prompt once for all its rows
        a, b = start[first[j]], start[first[j + 1]]
        used = table[first[j], :shared[j] // page]
        k, v = (x[used].transpose(0, 1).flatten(1, 2).float() for x in (st["k_pages"], st["v_pages"]))
        got = _partial(rows[:, a:b].flatten(1, 2), k, v, None)
        m1[:, a:b], l1[:, a:b], o1[:, a:b] = (x.view(Hk, b - a, G, -1) for x in got)
        skip[first[j]:first[j + 1]] = shared[j]
    # the rest of every sequence, side by side
    own_max = max(k - s for k, s in zip(*_own(case)))
    at = torch.arange(own_max, device="cuda") + skip[:, None]              # [S, longest]
    live = at < lens[:, None]
    where = table.gather(1, (at // page).clamp_max(table.shape[1] - 1))
    k, v = (torch.where(live[:, :, None, None], x[where, :, at % page], 0.0).float().transpose(1, 2)
            for x in (st["k_pages"], st["v_pages"]))                       # [S, Hk, longest, d]
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[seq]
    q = torch.zeros(S, Hk, q_max, G, d, device="cuda")
    q[seq, :, i] = st["q"].float().view(T, Hk, G, d)
    see = live[:, None, :].expand(S, q_max, own_max)
    if case["causal"]:
        last = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(q_max, device="cuda")
        see = see & (at[:, None, :] <= last[:, :, None])
    see = see[:, None, :, None, :].expand(S, Hk, q_max, G, own_max).flatten(2, 3)
    m2, l2, o2 = (x.view(S, Hk, q_max, G, -1)[seq, :, i].transpose(0, 1) for x in _partial(q.flatten(2, 3), k, v, see))
    m = torch.maximum(m1, m2)
    w1, w2 = (m1 - m).exp(), (m2 - m).exp()
    l = l1 * w1 + l2 * w2
    o, lse = (o1 * w1 + o2 * w2) / l, m + l.log()
    return o.transpose(0, 1).reshape(T, Hk * G, d).to(torch.bfloat16), lse.transpose(0, 1).reshape(T, Hk * G)


def _own(case):
    """Lengths and shared keys of each sequence."""
    first, shared, _, kvs = _batch(case)
    skip = [shared[sum(i >= f for f in first[1:])] if i < case["S"] else 0 for i in range(len(kvs))]
    return kvs, skip


def run(state):
    st, case = state, state["case"]
    if case["op"] == "shared":
        if not own:
            return _shared(st)
        import exact_io_aware_31_gb300 as fa
        return fa.paged_forward_shared(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["cu_seqlens"],
                                       st["kv_lens"], st["groups"], st["prefix_lens"], causal=case["causal"],
                                       max_q=case["q"])
    if own:
        import exact_io_aware_31_gb300 as fa
        state_of = (st["request_lens"], st["request_table"], st["pool"], case["page"])
        fa.paged_extend(st["requests"], st["new_lens"], *state_of, tokens=st["out"][3].shape[0], out=st["out"])
        fa.paged_release(st["requests"], *state_of, keep_lens=st["lens"])
    else:
        _extend(st)
        _release(st)
    return (*st["out"], st["request_lens"], st["request_table"], st["pool"])


def work(case):
    page = case["page"]
    if case["op"] == "shared":
        first, shared, qs, kvs = _batch(case)
        Hq, Hk, d, T = case["Hq"], case["Hk"], case["d"], sum(qs)
        pairs = sum(q * n - (q * (q - 1) // 2 if case["causal"] else 0) for q, n in zip(qs, kvs))
        _, skip = _own(case)
        keys = sum(shared) + sum(k - s for k, s in zip(kvs, skip))
        return {"bytes": 4 * T * Hq * d + 4 * T * Hq + 4 * keys * Hk * d + 4 * (-(-keys // page)) + 4 * (2 * len(qs) + 1)
                + 4 * (2 * len(shared) + 1), "flops": 4 * pairs * Hq * d}
    qs, lens = _steps(case)
    S, T = case["S"] + case["pad"], sum(qs)
    held = sum(-(-n // page) for n in lens)
    new = sum(-(-(n + q) // page) for n, q in zip(lens, qs)) - held
    # entries in use read and written, new ones written to the requests' rows too, and given back; lengths; positions, slots
    return {"bytes": 8 * held + 12 * new + 8 * new + 4 * (7 * S + 1) + 12 * T, "flops": 4 * T + 8 * S}


# ---------------------------------------------------------------- 64 bits ----
def _exact_tables(st):
    """The turn's outputs by plain loops over whole numbers on the host."""
    case, page = st["case"], st["case"]["page"]
    requests, new_lens, keep = (st[n].tolist() for n in ("requests", "new_lens", "lens"))
    lens, table, pool = (st[n].cpu().numpy().astype("int64") for n in ("request_lens", "request_table", "pool"))
    cu, kv_lens, page_table, positions, slots = (x.cpu().numpy().astype("int64") for x in st["out"])
    free = pool[2:2 + pool[0]].tolist()
    t = 0
    for s, (r, n) in enumerate(zip(requests, new_lens)):
        cu[s] = t
        if r >= 0:
            for j in range((lens[r] + page - 1) // page, (lens[r] + n + page - 1) // page):
                table[r, j] = free.pop()
            for p in range(lens[r], lens[r] + n):
                positions[t], slots[t] = p, table[r, p // page] * page + p % page
                t += 1
            lens[r] += n
            kv_lens[s] = lens[r]
            used = (lens[r] + page - 1) // page
            page_table[s, :used] = table[r, :used]
        else:
            kv_lens[s] = 0
    cu[len(requests)] = t
    back = []
    for r, k in zip(requests, keep):
        if r >= 0:
            back += table[r, (k + page - 1) // page:(lens[r] + page - 1) // page].tolist()
            lens[r] = k
    free += back[::-1]
    pool[0] = len(free)
    pool[2:2 + len(free)] = free
    return tuple(torch.from_numpy(x) for x in (cu, kv_lens, page_table, positions, slots, lens, table, pool))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] != "shared":
        return _exact_tables(st)
    page, Hq, Hk, d = case["page"], case["Hq"], case["Hk"], case["d"]
    _, _, qs, kvs = _batch(case)
    o = torch.empty(sum(qs), Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(sum(qs), Hq, dtype=torch.float64, device="cuda")
    G, at = Hq // Hk, 0
    for s, (q, n) in enumerate(zip(qs, kvs)):                # every sequence by itself, over all of its pages
        pages = st["page_table"][s, :-(-n // page)].long()
        keys, values = (x[pages].transpose(0, 1).reshape(Hk, -1, d)[:, :n].double() for x in (st["k_pages"],
                                                                                             st["v_pages"]))
        for a in range(0, q, 64):
            b = min(q, a + 64)
            rows = st["q"][at + a:at + b].double().view(b - a, Hk, G, d).permute(1, 2, 0, 3)
            score = torch.einsum("hgqd,hkd->hgqk", rows, keys) / math.sqrt(d)
            if case["causal"]:
                i = torch.arange(a, b, device="cuda")[:, None] + n - q
                score = torch.where(torch.arange(n, device="cuda") <= i, score, -math.inf)
            z = torch.logsumexp(score, -1)
            out = torch.einsum("hgqk,hkd->hgqd", torch.exp(score - z[..., None]), values)
            o[at + a:at + b] = out.permute(2, 0, 1, 3).reshape(b - a, Hq, d)
            lse[at + a:at + b] = z.permute(2, 0, 1).reshape(b - a, Hq)
        at += q
    return o, lse
