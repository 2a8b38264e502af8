"""Plain 64-bit attention and a Python page allocator for the paged-cache and
sliding-window tests, with error bounds that follow from the arithmetic."""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def visible(n_keys, pos, window, sinks):
    """Boolean [len(pos), n_keys]: key j is seen from position p."""
    j = torch.arange(n_keys)[None, :]
    p = torch.as_tensor(pos)[:, None]
    see = j <= p
    if window > 0:
        see &= (j > p - window) | (j < sinks)
    return see


def attend(q, k, v, see, scale=None):
    """Rows of q [R, D] over k, v [N, D] under see [R, N], all float64 (CPU).

    Returns (o, A, E, s1): A = sum p |v| / sum p (the scale of an error in P),
    E = the bound of a score's fp32 error, s1 = sum |v| / sum p with p relative
    to the row's maximum (the scale of an absolute error in P).
    Keys that a row does not see are left out of its sums altogether."""
    R, D = q.shape
    sc = 1.0 / D ** 0.5 if scale is None else scale
    o = torch.zeros(R, D, dtype=torch.float64)
    A = torch.zeros_like(o)
    s1 = torch.zeros_like(o)
    E = torch.zeros(R, 1, dtype=torch.float64)
    for r in range(R):
        idx = torch.nonzero(see[r])[:, 0]
        if len(idx) == 0:
            continue
        kk, vv = k[idx], v[idx]
        s = kk @ q[r] * sc
        p = torch.exp(s - s.max())
        l = p.sum()
        o[r] = (p @ vv) / l
        A[r] = (p @ vv.abs()) / l
        s1[r] = vv.abs().sum(0) / l
        # D products are added in fp32, one rounding each, then scaled
        E[r] = (D + 2) * 2.0 ** -24 * (kk.abs() @ q[r].abs()).max() * sc
    return o, A, E, s1


def bound(dt, o, A, E, s1, n, p_eps):
    """|error| <= half a step of the output type
               + A * (both scores' errors in exp, the rounding p_eps of P, the
                      fp32 roundings of n weights and sums, the exponential's)
               + f16 only: weights below 2^-14 are rounded to multiples of 2^-24."""
    out = torch.finfo(DT[dt]).eps / 2
    sub = s1 * 2.0 ** -25 if dt == "f16" and p_eps > 0 else 0.0
    return out * o.abs() + A * (2 * E + p_eps + (n + 64) * 2.0 ** -24 + 2.0 ** -20) * (1 + out) + sub + 1e-30


class Pool:
    """The allocator's rules in Python: lowest free page first."""

    def __init__(self, B, M, P, S):
        self.S, self.P = S, P
        self.table = np.full((B, M), -1, dtype=np.int32)
        self.refs = np.zeros(P, dtype=np.int32)
        self.len = np.zeros(B, dtype=np.int32)

    def reserve(self, add):
        need = [(b, i) for b in range(len(self.len)) if add[b] > 0
                for i in range(self.len[b] // self.S, (self.len[b] + add[b] - 1) // self.S + 1)
                if self.table[b, i] < 0]
        free = [p for p in range(self.P) if self.refs[p] == 0]
        if len(need) > len(free):
            return False
        for (b, i), p in zip(need, free):
            self.table[b, i] = p
            self.refs[p] = 1
        return True

    def free(self, window=0, sinks=0):
        for b, n in enumerate(self.len):
            for i in range(self.table.shape[1]):
                toks = range(i * self.S, (i + 1) * self.S)
                lo = n - window if window > 0 else 0
                if self.table[b, i] >= 0 and not any(t < n and (t >= lo or t < sinks) for t in toks):
                    self.refs[self.table[b, i]] -= 1
                    self.table[b, i] = -1

    def fork(self, src, dst):
        refs = self.refs.copy()
        for s, d in zip(src, dst):
            for p in self.table[d]:
                if p >= 0:
                    refs[p] -= 1
            for p in self.table[s, :self.len[s] // self.S]:
                if p >= 0:
                    refs[p] += 1
        tails = [s for s in src if self.len[s] % self.S and self.table[s, self.len[s] // self.S] >= 0]
        free = [p for p in range(self.P) if refs[p] == 0]
        if len(tails) > len(free):
            return None
        pairs = []
        for s, d in zip(src, dst):
            full = self.len[s] // self.S
            row = np.full(self.table.shape[1], -1, dtype=np.int32)
            row[:full] = self.table[s, :full]
            pair = (-1, -1)
            if self.len[s] % self.S and self.table[s, full] >= 0:
                row[full] = free.pop(0)
                refs[row[full]] = 1
                pair = (int(self.table[s, full]), int(row[full]))
            self.table[d] = row
            self.len[d] = self.len[s]
            pairs.append(pair)
        self.refs = refs
        return pairs

    def compact(self):
        live = [p for p in range(self.P) if self.refs[p] > 0]
        L = len(live)
        src = [p for p in live if p >= L]
        dst = [p for p in range(L) if self.refs[p] <= 0]
        to = dict(zip(src, dst))
        self.table = np.vectorize(lambda p: to.get(int(p), int(p)))(self.table).astype(np.int32)
        refs = np.zeros_like(self.refs)
        for p in live:
            refs[to.get(p, p)] = self.refs[p]
        self.refs = refs
        return list(zip(src, dst))
