"""Plain restatement of the paged memory: lists and loops, one entry after the
other, and the attention over a slot's rows in float64 with a bound on what
the storage type's roundings can do to it.  Test infrastructure only."""

from __future__ import annotations

import numpy as np


class Book:
    """table, start, rows, refs as the header describes them, as lists."""

    def __init__(self, n_slots, max_pages, n_pages, page_rows):
        self.table = [[-1] * max_pages for _ in range(n_slots)]
        self.start = [0] * n_slots
        self.rows = [0] * n_slots
        self.refs = [0] * n_pages
        self.P = page_rows

    @property
    def max_pages(self):
        return len(self.table[0])

    def good(self, s):
        return (0 <= s < len(self.rows) and 0 <= self.start[s] < self.P and self.rows[s] >= 0
                and self.start[s] + self.rows[s] <= self.max_pages * self.P)

    def pages(self, s):
        return -(-(self.start[s] + self.rows[s]) // self.P)

    def reserve(self, slots, cu):
        """granted, copy_src, copy_dst; refused: some entry asked and got nothing."""
        refs0 = list(self.refs)
        free = [p for p, c in enumerate(refs0) if c == 0]
        used, seen, refused, blocked = 0, set(), False, False
        granted, src, dst = [], [], []
        for i, s in enumerate(slots):
            count = cu[i + 1] - cu[i]
            fresh = s not in seen
            seen.add(s)
            g, a, z = 0, -1, -1
            if self.good(s) and count == 0 and cu[i] >= 0:
                pass
            elif not self.good(s) or count < 0 or cu[i] < 0 or not fresh:
                refused = True
            else:
                end = self.start[s] + self.rows[s]
                have, want = self.pages(s), -(-(end + count) // self.P)
                last = self.table[s][have - 1] if end % self.P else None
                bad = want > self.max_pages or (last is not None and not 0 <= last < len(refs0))
                shared = not bad and last is not None and refs0[last] > 1
                need = want - have + shared
                if bad or (need > 0 and (blocked or used + need > len(free))):
                    refused = True
                    blocked = blocked or not bad
                else:
                    new = free[used:used + need]
                    used += need
                    g = count
                    if shared:
                        a, z = last, new[0]
                        self.table[s][have - 1] = z
                        self.refs[a] -= 1
                    for j, p in enumerate(new[1:] if shared else new):
                        self.table[s][have + j] = p
                    for p in new:
                        self.refs[p] = 1
                    self.rows[s] += count
            granted.append(g)
            src.append(a)
            dst.append(z)
        return granted, src, dst, refused

    def place(self, s, j):
        """Page and row of live row j of slot s."""
        x = self.start[s] + j
        return self.table[s][x // self.P], x % self.P

    def append(self, pool, slots, cu, granted, src, dst, new):
        """pool [pages, H, P, D] (changed), new [T, H, D]."""
        for i, s in enumerate(slots):
            g = granted[i]
            if g == 0:
                continue
            old = (self.start[s] + self.rows[s] - g) % self.P
            if src[i] >= 0 and dst[i] >= 0:
                pool[dst[i]][:, :old] = pool[src[i]][:, :old]
            for t in range(g):
                p, x = self.place(s, self.rows[s] - g + t)
                pool[p][:, x] = new[cu[i] + t]

    def fork(self, src, dst):
        ok = []
        empty = [r == 0 for r in self.rows]
        for i, (a, d) in enumerate(zip(src, dst)):
            good = (self.good(a) and 0 <= d < len(self.rows) and a not in dst and d not in dst[:i] and empty[d]
                    and a != d)
            if good:
                n = self.pages(a)
                self.table[d][:n] = self.table[a][:n]
                self.start[d], self.rows[d] = self.start[a], self.rows[a]
                for p in self.table[a][:n]:
                    self.refs[p] += 1
            ok.append(int(good))
        return ok

    def free(self, slots, keep):
        refused = False
        for i, s in enumerate(slots):
            if not self.good(s) or s in slots[:i]:
                refused = True
                continue
            n, kept = self.pages(s), min(self.rows[s], max(0, keep[i]))
            begin = self.start[s] + self.rows[s] - kept
            dead = begin // self.P if kept else n
            for p in self.table[s][:dead]:
                self.refs[p] -= 1
            self.table[s] = self.table[s][dead:] + [-1] * dead
            self.start[s] = begin % self.P if kept else 0
            self.rows[s] = kept
        return refused

    def compact(self):
        """new_id, moves (src, dst)."""
        live = [p for p, c in enumerate(self.refs) if c > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] == 0]
        movers = [p for p in live if p >= n]
        new_id = [p if c > 0 else -1 for p, c in enumerate(self.refs)]
        for a, z in zip(movers, holes):
            new_id[a] = z
            self.refs[z], self.refs[a] = self.refs[a], 0
        self.table = [[new_id[p] if p >= 0 else -1 for p in row] for row in self.table]
        return new_id, movers, holes

    def gather(self, pool, s):
        """Live rows [rows, H, D] of slot s."""
        out = [pool[p][:, x] for p, x in (self.place(s, j) for j in range(self.rows[s]))]
        return np.stack(out) if out else np.zeros((0, pool.shape[1], pool.shape[3]), pool.dtype)


def attend(q, k, v, r, u, vb, scale):
    """o [n, H, D], lse [H, n] and S [H, n, rows] (the scores' sums of absolute
    products) for the n newest positions of the live rows k, v; float64."""
    q, k, v, r, u, vb = (np.asarray(x, np.float64) for x in (q, k, v, r, u, vb))
    n, H, D = q.shape
    m = len(k) - n
    o = np.zeros((n, H, D))
    lse = np.full((H, n), -np.inf)
    size = np.zeros((H, n, len(k)))
    for h in range(H):
        for t in range(n):
            seen = m + t + 1
            if seen <= 0:
                continue
            a, b = q[t, h] + u[h], q[t, h] + vb[h]
            dist = r[m + t - np.arange(seen), h]
            z = scale * (k[:seen, h] @ a + dist @ b)
            w = np.exp(z - z.max())
            lse[h, t] = z.max() + np.log(w.sum())
            o[t, h] = (w / w.sum()) @ v[:seen, h]
            size[h, t, :seen] = abs(scale) * (np.abs(k[:seen, h]) @ np.abs(a) + np.abs(dist) @ np.abs(b))
    return o, lse, size


def tolerance(q, k, v, r, u, vb, scale, step, terms, out_step):
    """o, lse and, per element of each, what roundings can do to them to first
    order.  step: the largest relative rounding of an operand; terms: how many
    such roundings a score's products and a weight's product carry; out_step:
    the output's own rounding.

    A score is a sum of products whose operands are each off by at most `step`
    (relative), so it is off by at most e_j = terms * step * S_j, S_j the sum
    of the products' absolute values.  A weight w_j = exp(z_j) is then off by
    e_j, and once more by terms * step where it is rounded and summed; o is
    the weighted mean of v, so |do| <= sum_j p_j (|v_j| + |o|) (e_j +
    terms * step) + out_step * |o|, and |dlse| <= sum_j p_j e_j + terms * step
    + step * |lse|.
    """
    o, lse, size = attend(q, k, v, r, u, vb, scale)
    va = np.abs(np.asarray(v, np.float64))
    q64, k64, r64 = (np.asarray(x, np.float64) for x in (q, k, r))
    n, H, _ = o.shape
    m = len(k) - n
    do, dl = np.zeros_like(o), np.zeros_like(lse)
    for h in range(H):
        for t in range(n):
            seen = m + t + 1
            if seen <= 0:
                continue
            z = scale * (k64[:seen, h] @ (q64[t, h] + u[h]) + r64[m + t - np.arange(seen), h] @ (q64[t, h] + vb[h]))
            p = np.exp(z - lse[h, t])
            e = terms * step * (size[h, t, :seen] + 1.0)
            do[t, h] = (p * e) @ (va[:seen, h] + np.abs(o[t, h])) + out_step * np.abs(o[t, h])
            dl[h, t] = p @ e + step * abs(lse[h, t])
    return o, lse, do, dl


def spread(q, k, v, r, u, vb, scale, step, out_step):
    """The sum over all elements of o of the variance that independent
    roundings give them to first order, an upper bound.

    A rounding to nearest moves a value x by at most step * |x|, evenly spread,
    so its variance is at most s2 x^2, s2 = step^2 / 3.  With z_j = scale
    (a . k_j + b . r_j), a = q + u, b = q + v, and o = sum_j p_j v_j,
    do = sum_j p_j (v_j - o) dz_j, so per element of o
      a rounded:            s2 sum_d (scale a_d)^2 (sum_j p_j (v_j - o) k_jd)^2
      b rounded:            the same with b and r_j
      b . r_j rounded:      s2 sum_j (p_j (v_j - o) scale b.r_j)^2
      p_j rounded (for the product with v alone):  s2 sum_j (p_j v_j)^2
      o rounded:            (out_step^2 / 3) o^2.
    """
    q, k, v, r, u, vb = (np.asarray(x, np.float64) for x in (q, k, v, r, u, vb))
    o, lse, _ = attend(q, k, v, r, u, vb, scale)
    n, H, _ = o.shape
    m = len(k) - n
    s2 = step ** 2 / 3
    total = out_step ** 2 / 3 * (o ** 2).sum()
    for h in range(H):
        for t in range(n):
            seen = m + t + 1
            if seen <= 0:
                continue
            a, b = q[t, h] + u[h], q[t, h] + vb[h]
            kk, rr, vv = k[:seen, h], r[m + t - np.arange(seen), h], v[:seen, h]
            far = rr @ b
            p = np.exp(scale * (kk @ a + far) - lse[h, t])[:, None]
            away = p * (vv - o[t, h])  # [j, element]
            total += s2 * (((scale * a) ** 2) @ (kk.T @ away) ** 2).sum()
            total += s2 * (((scale * b) ** 2) @ (rr.T @ away) ** 2).sum()
            total += s2 * ((away * (scale * far)[:, None]) ** 2).sum()
            total += s2 * ((p * vv) ** 2).sum()
    return total
