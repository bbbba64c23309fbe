"""Plain forms for the tests of the step around the cache: block tables and slots
in Python lists, the rotation in binary64 numpy, the verification in exact
fractions.  They share nothing with the kernels."""
from fractions import Fraction

import numpy as np

from paged_kv_cache_41_gb300 import pkv


class Blocks:
    """Block tables and the stack of free ids in plain lists."""

    def __init__(self, num_blocks, p, tables, free, count):
        self.nb, self.p = num_blocks, p
        self.tables = [list(map(int, row)) for row in tables]
        self.free, self.count, self.err = list(map(int, free)), int(count), 0

    def update(self, lens, base, add, num_rows, window=0, sinks=0):
        p, nb = self.p, self.nb
        b, width = len(lens), len(self.tables[0]) if self.tables else 0
        cap = width * p
        if not 0 <= self.count <= nb:
            self.err |= pkv.DEVERR_BLOCK
            self.count = min(max(self.count, 0), nb)
        new, bad = [], []
        for r in range(b):
            x = (int(base[r]) if base is not None else 0) + int(add[r])
            wrong = not (0 <= lens[r] <= cap and 0 <= x <= cap and (base is None or base[r] >= 0))
            if wrong:
                self.err |= pkv.DEVERR_LENGTH
            new.append(int(lens[r]) if wrong else x)
            bad.append(wrong)
        for r in reversed(range(b)):
            if bad[r]:
                continue
            row = self.tables[r]
            go = list(range(-(-new[r] // p), -(-int(lens[r]) // p)))[::-1]
            lo = min(int(lens[r]), new[r]) - window
            if window > 0 and lo > 0:
                for j in reversed(range(-(-sinks // p), lo // p)):
                    if row[j] < 0:
                        break
                    go.append(j)
            for j in go:
                x, row[j] = row[j], -1
                if x >= nb:
                    self.err |= pkv.DEVERR_BLOCK
                elif x >= 0:
                    if self.count < nb:
                        self.free[self.count] = x
                        self.count += 1
                    else:
                        self.err |= pkv.DEVERR_BLOCK
        ptr, rows, asked, given = [0], 0, 0, 0
        out, slots, pos = [], [-1] * num_rows, [-1] * num_rows
        for r in range(b):
            n = 0 if bad[r] else max(0, new[r] - int(lens[r]))
            rows += n
            want, held = -(-new[r] // p), -(-int(lens[r]) // p)
            if n and rows > num_rows:
                self.err |= pkv.DEVERR_LENGTH
                out.append(int(lens[r]))
            else:
                need = 0 if bad[r] or not n else want - held
                asked += need
                if need and asked > self.count:
                    self.err |= pkv.DEVERR_POOL
                    out.append(int(lens[r]))
                else:
                    for e in range(need):
                        x = self.free[self.count - 1 - (asked - need + e)]
                        if not 0 <= x < nb:
                            self.err |= pkv.DEVERR_BLOCK
                            x = -1
                        self.tables[r][held + e] = x
                    given = asked if need else given
                    out.append(new[r])
                    for i in range(n):
                        at = int(lens[r]) + i
                        x = self.tables[r][at // p]
                        if 0 <= x < nb:
                            slots[ptr[-1] + i], pos[ptr[-1] + i] = x * p + at % p, at
            ptr.append(min(rows, num_rows))
        self.count -= given
        return out, ptr, slots, pos


# ------------------------------------------------------------------ rotation
def rotate64(x, weight, eps, cos_sin, positions, axis_of, interleaved):
    """x [n, heads, d] binary64 -> (normed and rotated, the size of the terms that
    each element is the sum of)."""
    n, _, d = x.shape
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    rot = 0 if cos_sin is None else cos_sin.shape[1]
    y, size = x.copy(), np.abs(x)
    for j in range(rot // 2):
        at = positions[axis_of[j]]
        c, s = (cos_sin[at, k].astype(np.float64)[:, None] for k in (j, rot // 2 + j))
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
        size[:, :, a] = np.abs(x[:, :, a] * c) + np.abs(x[:, :, b] * s)
        size[:, :, b] = np.abs(x[:, :, b] * c) + np.abs(x[:, :, a] * s)
    return y, size


# -------------------------------------------------------------- verification
def as_prob(x):
    x = float(x)
    return Fraction(0) if not x > 0 else Fraction(min(x, 1.0))


def verify(p, q, tokens, masks, uniforms):
    """One sequence in exact fractions: p (and q) [n][vocab], tokens, masks (None: a
    chain) and uniforms [n].  Returns (accepted rows, next token)."""
    n, vocab = len(tokens), len(p[0]) if len(p) else 0
    if n == 0:
        return [], -1
    up = []
    for i in range(n):
        older = masks[i] & ((1 << i) - 1) if masks is not None else (1 << (i - 1) if i else 0)
        up.append(older.bit_length() - 1)

    def number(u):
        u = float(u)
        return Fraction(0) if not u >= 0 else Fraction(min(u, float(np.nextafter(np.float32(1), np.float32(0)))))

    kept, at = [0], 0
    while True:
        pa = [as_prob(x) for x in p[at]]
        qa = [as_prob(x) for x in q[at]] if q is not None else None
        c, mass, out, go = Fraction(0), Fraction(1), [], None
        for x in range(1, n):
            if up[x] != at or not 0 <= tokens[x] < vocab:
                continue
            t, u = int(tokens[x]), number(uniforms[x])
            if q is not None:
                rest = max(pa[t] - c * qa[t], Fraction(0))
                yes = u * qa[t] * mass < rest
            else:
                rest = Fraction(0) if t in out else pa[t]
                yes = u * mass < rest
            if yes:
                go = x
                break
            out.append(t)
            if q is not None:
                c += mass
                mass = sum(max(a - c * b, Fraction(0)) for a, b in zip(pa, qa))
            else:
                mass -= rest
        if go is not None:
            kept.append(go)
            at = go
            continue
        if q is not None:
            r = [max(a - c * b, Fraction(0)) for a, b in zip(pa, qa)]
        else:
            r = [Fraction(0) if v in out else a for v, a in enumerate(pa)]
        if not sum(r):
            r = pa
        whole, run = sum(r), Fraction(0)
        if not whole:
            return kept, -1
        for v, x in enumerate(r):
            run += x
            if run > number(uniforms[0]) * whole:
                return kept, v
