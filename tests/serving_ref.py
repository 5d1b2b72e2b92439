"""Plain 64-bit references of the paged cache's operators, and their tolerances.

Tolerances follow from the arithmetic, for unit query, key and value rows:

  * a raw dot of 64 bf16 products in fp32 is off by at most 64 * 2^-23 (the
    tensor cores may truncate, a whole step instead of half of one);
  * a logit z = c dot is off by c times that and a few fp32 roundings, which is
    the relative error e of its weight;
  * n_eff = l^2 / l2 is then off by 4 e, and by the summation of n terms (at
    most 3 n roundings of 2^-24);
  * a weight enters the value product rounded to bf16 (half a step, 2^-8
    relative), so acc is off by (2^-8 + e) sum p |v| per column, the direction
    by that and the norm's share of it, and the output is rounded to bf16 once;
  * the magnitude moves by e and n_eff's error: far below 2^-9 |u|.
"""
from __future__ import annotations

import numpy as np
import torch

PAGE, DIM = 64, 64


def mixing_row(q, keys, values, u, s, alpha, L, beta):
    """One row against its visible keys (float64).  Returns out, neff and their
    tolerances."""
    n = keys.shape[0]
    if n == 0:
        return np.zeros(DIM), 0.0, np.zeros(DIM), 0.0
    c = s * (1 + alpha * np.log(n / L)) if n > L else s
    dot = keys @ q
    z = c * dot
    w = np.exp(z - z.max())
    acc = w @ values
    l, l2 = w.sum(), (w * w).sum()
    neff = l * l / l2
    norm = max(np.linalg.norm(acc), 1e-30)
    z0 = z.mean() + z.std() * np.sqrt(2 * np.log(n))
    gate = 1 / (1 + np.exp(-beta * (z.max() - z0)))
    count = gate * np.tanh(np.log(neff) / np.log(L)) * u
    out = acc / norm + count
    e = c * 64 * 2.0 ** -23 + 16 * 2.0 ** -24 * (1 + abs(z).max())
    off = (2.0 ** -8 + 2 * e) * (w @ abs(values))
    tol = (off + abs(acc) / norm * np.linalg.norm(off)) / norm * (1 + 2.0 ** -7)
    tol = tol + 2.0 ** -8 * abs(out) + 2.0 ** -9 * abs(u) + 1e-6
    return out, neff, tol, neff * (4 * e + 3 * n * 2.0 ** -24 + 1e-6)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def check_rows(got_out, got_neff, refs, what=""):
    """got_out [R, 64], got_neff [R] against a list of mixing_row's answers."""
    out = np.stack([r[0] for r in refs])
    neff = np.array([r[1] for r in refs])
    tol = np.stack([r[2] for r in refs])
    ntol = np.array([r[3] for r in refs])
    o, n = f64(got_out).reshape(out.shape), f64(got_neff).reshape(neff.shape)
    assert np.isfinite(o).all() and np.isfinite(n).all(), f"{what}: not finite"
    worst = (abs(o - out) / np.maximum(tol, 1e-30)).max()
    assert (abs(o - out) <= tol).all(), f"{what}: out off by {worst:.2f} of its tolerance"
    worst = (abs(n - neff) / np.maximum(ntol, 1e-30)).max()
    assert (abs(n - neff) <= ntol).all(), f"{what}: neff off by {worst:.2f} of its tolerance"


def cached(kv, table_row, head, length):
    """Keys and values of a row's first `length` positions (float64)."""
    pos = np.arange(length)
    pages = np.asarray(table_row)[pos // PAGE]
    return kv[pages, 0, head, pos % PAGE], kv[pages, 1, head, pos % PAGE]


# ------------------------------------------------------- the cache, on host ---

class HostCache:
    """The cache's operations, token by token and page by page, in numpy."""

    def __init__(self, kv, refs, bounds):
        self.kv, self.refs, self.bounds = kv.copy(), refs.copy(), bounds.copy()

    def reserve(self, table, lens, grow):
        """In place; returns granted.  Rows ask in order."""
        refs0, N = self.refs.copy(), len(lens)
        cap = table.shape[1] * PAGE
        ok = [0 <= lens[i] <= cap and grow[i] >= 0 and lens[i] + grow[i] <= cap for i in range(N)]
        tail = {}
        for i in range(N):
            if ok[i] and grow[i] > 0 and lens[i] % PAGE:
                page = table[i, lens[i] // PAGE]
                if not 0 <= page < len(refs0):
                    ok[i] = False
                else:
                    tail[i] = page
        keeper = {}
        for i, page in tail.items():
            sharers = [j for j, p in tail.items() if p == page]
            if len(sharers) == refs0[page]:
                keeper[page] = sharers[-1]
        free = [p for p in range(len(refs0)) if refs0[p] == 0]
        granted = np.zeros(N, np.int32)
        out_of_pages = False
        for i in range(N):
            if not ok[i]:
                continue
            copy = i in tail and refs0[tail[i]] > 1 and keeper.get(tail[i]) != i
            have, want = -(-lens[i] // PAGE), -(-(lens[i] + grow[i]) // PAGE)
            need = want - have + copy
            if out_of_pages or need > len(free):
                out_of_pages = True
                continue
            if copy:
                src, dst, part = tail[i], free.pop(0), lens[i] % PAGE
                self.kv[dst, :, :, :part] = self.kv[src, :, :, :part]
                self.bounds[dst] = self.bounds[src]
                self.refs[dst] = 1
                self.refs[src] -= 1
                table[i, lens[i] // PAGE] = dst
            for c in range(have, want):
                table[i, c] = free.pop(0)
                self.refs[table[i, c]] = 1
            granted[i] = grow[i]
            lens[i] += grow[i]
        return granted

    def append(self, k, v, table, lens, counts, pick=None):
        for i in range(len(lens)):
            first = lens[i] - counts[i]
            for t in range(counts[i]):
                src = t if pick is None else pick[i, t]
                page, at = table[i, (first + t) // PAGE], (first + t) % PAGE
                self.kv[page, 0, :, at] = k[i, src]
                self.kv[page, 1, :, at] = v[i, src]
            if counts[i]:
                for c in range(first // PAGE, (lens[i] - 1) // PAGE + 1):
                    rows = self.kv[table[i, c], 0, :, :min(PAGE, lens[i] - c * PAGE)]
                    self.bounds[table[i, c], :, 0] = rows.min(1)
                    self.bounds[table[i, c], :, 1] = rows.max(1)

    def fork(self, src_table, src_lens, src_rows, table, lens):
        for i, r in enumerate(src_rows):
            if r < 0:
                continue
            n = -(-src_lens[r] // PAGE)
            table[i, :n] = src_table[r, :n]
            lens[i] = src_lens[r]
            for c in range(n):
                self.refs[table[i, c]] += 1

    def free(self, table, lens, keep=None):
        for i in range(len(lens)):
            k = 0 if keep is None else keep[i]
            if k < 0 or k >= lens[i]:
                continue
            for c in range(-(-k // PAGE), -(-lens[i] // PAGE)):
                self.refs[table[i, c]] -= 1
                table[i, c] = -1
            lens[i] = k

    def compact(self, table, lens):
        live = np.flatnonzero(self.refs > 0)
        n = len(live)
        src = live[live >= n]
        dst = np.setdiff1d(np.arange(n), live)
        to = {int(s): int(d) for s, d in zip(src, dst)}
        self.kv[dst], self.bounds[dst] = self.kv[src], self.bounds[src]
        self.refs[dst] = self.refs[src]
        self.refs[src] = 0
        for i in range(len(lens)):
            for c in range(-(-lens[i] // PAGE)):
                table[i, c] = to.get(int(table[i, c]), table[i, c])
        return n


# --------------------------------------------------- keys that are alike ---

ALIKE = ["equal", "near", "outliers first", "outlier last"]


def alike_keys(kind, key, n, rng):
    """n keys along `key` (float64 unit vector), up to the kind: the spread of a
    row's products is then far below their mean, and with it the null floor."""
    a = np.ones(n)
    if kind == "near":
        a -= rng.integers(0, 3, n) / 256
    elif kind == "outliers first":
        a[:PAGE] = -1
    elif kind == "outlier last":
        a[-1] = -1
    return torch.from_numpy(a[:, None] * key).bfloat16()


def at_angle(key, dot, shape, rng):
    """Unit vectors (float64) whose product with the unit vector `key` is `dot`."""
    x = rng.standard_normal((*shape, DIM))
    x -= (x @ key)[..., None] * key
    return dot * key + np.sqrt(1 - dot ** 2) * x / np.linalg.norm(x, axis=-1, keepdims=True)
