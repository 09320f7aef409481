"""Plain forms of the operators around the attention kernels: norm with rotation, paged cache and its tables, paged
attention (fp64; the tables in whole numbers).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): slow, obvious, CPU.

Conventions are those of ``include/fa.h``: a rotation table row holds the
cosines, then the sines, of one position; the pairs are ``(i, i + half)`` or,
interleaved, ``(2i, 2i + 1)`` of the first ``rope_dim`` columns; new token i of
a sequence has position ``kv_len - q_len + i``; key j is visible to it iff
``j < kv_len`` and (causal) ``j <= kv_len - q_len + i``.
"""

from __future__ import annotations

import numpy as np

__all__ = ["rope_table", "norm_rope", "norm_rope_grad", "paged_append", "paged_attention", "Tables"]


def rope_table(length, dim, base=10000.0):
    """[length, dim] fp64: cosines, then sines, of p * base^(-2 i / dim)."""
    out = np.empty((length, dim))
    for p in range(length):
        for i in range(dim // 2):
            angle = p * base ** (-2.0 * i / dim)
            out[p, i], out[p, dim // 2 + i] = np.cos(angle), np.sin(angle)
    return out


def _pairs(half, interleaved):
    return [(2 * i, 2 * i + 1) if interleaved else (i, i + half) for i in range(half)]


def _rotate(y, table, positions, interleaved, back=False):
    """Rows y [..., N, d] turned by the angles of ``positions`` ([..., N], broadcast)."""
    half = table.shape[1] // 2
    rows = table[positions]
    out = y.copy()
    for i, (a, b) in enumerate(_pairs(half, interleaved)):
        c, s = rows[..., i], rows[..., half + i] * (-1.0 if back else 1.0)
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def norm_rope(x, w, eps, table, positions, interleaved, norm=True):
    """z = R(position) (w * x / rms(x)) for x [B, H, N, d], positions [B, N]; w None is ones, table None no rotation."""
    x = np.asarray(x, dtype=np.float64)
    y = x
    if norm:
        y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
        y = y if w is None else y * np.asarray(w, dtype=np.float64)
    return y.copy() if table is None else _rotate(y, table, positions[:, None], interleaved)


def norm_rope_grad(dz, x, w, eps, table, positions, interleaved, norm=True):
    """(dx, dw) of sum(z * dz); dw is None without the norm."""
    x, dz = np.asarray(x, dtype=np.float64), np.asarray(dz, dtype=np.float64)
    dy = dz if table is None else _rotate(dz, table, positions[:, None], interleaved, back=True)
    if not norm:
        return dy.copy(), None
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    dw = (dy * x * r).reshape(-1, x.shape[-1]).sum(0)
    g = dy if w is None else dy * np.asarray(w, dtype=np.float64)
    return r * (g - x * r * (g * x * r).mean(-1, keepdims=True)), dw


def paged_append(q, k, v, k_pages, v_pages, page_table, cu, lens, qw, kw, eps, table, interleaved, norm=True):
    """(q_out, k_pages, v_pages) in fp64, the pages copied; q_out rows of no sequence are NaN."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    kp, vp = np.array(k_pages, dtype=np.float64), np.array(v_pages, dtype=np.float64)
    page = kp.shape[2]
    q_out = np.full(q.shape, np.nan)
    for s in range(len(lens)):
        for t in range(cu[s], cu[s + 1]):
            pos = lens[s] - cu[s + 1] + t
            at = np.array([[pos]])
            q_out[t] = norm_rope(q[t][None, :, None], qw, eps, table, at, interleaved, norm)[0, :, 0]
            kp[page_table[s, pos // page], :, pos % page] = norm_rope(k[t][None, :, None], kw, eps, table, at,
                                                                      interleaved, norm)[0, :, 0]
            vp[page_table[s, pos // page], :, pos % page] = v[t]
    return q_out, kp, vp


def paged_attention(q, k_pages, v_pages, page_table, cu, lens, scale, causal):
    """(o [T, Hq, d], lse [T, Hq]) in fp64; a row that sees no key is zero with lse -inf, rows of no sequence NaN.

    Also returns ``reach [T, Hq, d]`` = sum_j p_j |v_j|, what a relative error of the probabilities can move."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, d = q.shape
    Hk, page = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hk
    o, reach, lse = np.full((T, Hq, d), np.nan), np.zeros((T, Hq, d)), np.full((T, Hq), np.nan)
    for s in range(len(lens)):
        n = int(lens[s])
        used = page_table[s, :(n + page - 1) // page]
        for h in range(Hk):
            keys = np.concatenate([k_pages[p, h] for p in used] + [np.zeros((0, d))])[:n].astype(np.float64)
            vals = np.concatenate([v_pages[p, h] for p in used] + [np.zeros((0, d))])[:n].astype(np.float64)
            for t in range(cu[s], cu[s + 1]):
                see = min(n, n - cu[s + 1] + t + 1) if causal else n
                for g in range(h * G, (h + 1) * G):
                    if see <= 0:
                        o[t, g], lse[t, g] = 0.0, -np.inf
                        continue
                    sc = scale * (keys[:see] @ q[t, g])
                    m = sc.max()
                    e = np.exp(sc - m)
                    lse[t, g] = m + np.log(e.sum())
                    o[t, g] = (e / e.sum()) @ vals[:see]
                    reach[t, g] = (e / e.sum()) @ np.abs(vals[:see])
    return o, lse, reach


class Tables:
    """The requests of a paged cache: lengths [R], rows of pages [R, max_pages], the stack of free pages."""

    def __init__(self, lens, table, free, num_pages, page_size):
        self.lens, self.table, self.free = list(lens), np.array(table), list(free)
        self.num_pages, self.page = num_pages, page_size
        self.bad = False                       # something was refused

    def pages(self, n):
        return -(-n // self.page)

    def extend(self, requests, new_lens, tokens, page_table):
        """(cu_seqlens, kv_lens, page_table, positions, slots); ``page_table`` holds what is there before."""
        S, most = len(requests), self.table.shape[1]
        cu, kv, out = [0], [], np.array(page_table)
        positions, slots = np.zeros(tokens, dtype=np.int64), np.full(tokens, -1, dtype=np.int64)
        seen, row, asked, have = set(), 0, 0, len(self.free)
        for s, r in enumerate(requests):
            n = max(0, new_lens[s]) if r >= 0 else 0
            first = row
            row += n
            cu.append(min(row, tokens))
            kv.append(0)
            if r < 0:
                continue
            self.bad |= new_lens[s] < 0
            fine = r < len(self.lens) and r not in seen
            seen.add(r)
            fine = fine and 0 <= self.lens[r] and self.lens[r] + n <= most * self.page and (n == 0 or row <= tokens)
            if fine:
                held, need = self.pages(self.lens[r]), self.pages(self.lens[r] + n)
                asked += need - held
                fine = need == held or asked <= have
            if not fine:
                self.bad = True
                positions[min(first, tokens):min(row, tokens)] = -1
                continue
            for j in range(held, need):
                self.table[r, j] = self.free.pop()
            at = np.arange(self.lens[r], self.lens[r] + n)
            positions[first:row] = at
            slots[first:row] = self.table[r, at // self.page].astype(np.int64) * self.page + at % self.page
            self.lens[r] += n
            kv[s] = self.lens[r]
            out[s, :need] = self.table[r, :need]
            lost = [not 0 <= x < self.num_pages for x in out[s, :need]]  # no pages of the pool: no slots in them
            self.bad |= any(lost)
            slots[first:row] = np.where(np.array(lost, dtype=bool)[at // self.page], -1, slots[first:row])
        return np.array(cu), np.array(kv), out, positions, slots

    def release(self, requests, keep_lens=None, kept_pages=None):
        back, lens, seen = [], list(self.lens), set()
        for s, r in enumerate(requests):
            if r < 0:
                continue
            keep = 0 if keep_lens is None else keep_lens[s]
            most = self.table.shape[1]
            if (r >= len(lens) or r in seen or not 0 <= keep <= lens[r] <= most * self.page
                    or kept_pages is not None and not 0 <= kept_pages[r] <= most):
                self.bad = True
                seen.add(r)
                continue
            seen.add(r)
            first = max(self.pages(keep), 0 if kept_pages is None else kept_pages[r])
            back += [int(x) for x in self.table[r, first:self.pages(lens[r])]]
            lens[r] = keep
        self.bad |= any(not 0 <= x < self.num_pages for x in back)
        if len(self.free) + len(back) > self.num_pages:
            self.bad = True
            return
        self.lens, self.free = lens, self.free + back[::-1]
