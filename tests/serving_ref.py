"""Plain 64-bit forms of the serving-side operators, for the tests: token log probabilities
(numpy), attention over a paged cache (torch, float64) and the page tables (Python lists)."""
import math

import numpy as np
import torch


def token_logprobs(x, tokens, T, K):
    """x [N,V] float64.  Returns logprob, entropy, lse, ids [N,K], top logprobs [N,K]."""
    N, V = x.shape
    lp, H, lse = (np.full(N, np.nan) for _ in range(3))
    ids, top = np.full((N, K), -1, np.int64), np.full((N, K), np.nan)
    for n in range(N):
        t = int(tokens[n])
        row = x[n]
        if t < 0 or t >= V or np.isnan(row).any() or (row == np.inf).any():
            continue
        order = np.lexsort((np.arange(V), -row))[:K]
        ids[n] = order
        m = row.max()
        if m == -np.inf:
            lp[n], H[n], lse[n], top[n] = -np.inf, 0.0, -np.inf, -np.inf
            continue
        u = (row - m) / T
        e = np.exp(u)
        ln_s = math.log(math.fsum(e))
        logp = u - ln_s
        p = np.exp(logp)
        lp[n] = logp[t]
        lse[n] = m / T + ln_s
        H[n] = -np.sum(np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0))
        top[n] = logp[order]
    return lp, H, lse, ids, top


def token_logprobs_grad(x, tokens, T, gl, ge):
    N, V = x.shape
    d = np.zeros((N, V))
    for n in range(N):
        t = int(tokens[n])
        m = x[n].max()
        if t < 0 or t >= V or m == -np.inf:
            continue
        if np.isnan(x[n]).any() or m == np.inf:
            d[n] = np.nan
            continue
        u = (x[n] - m) / T
        logp = u - math.log(math.fsum(np.exp(u)))
        p = np.exp(logp)
        plogp = np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0)
        d[n] = -gl[n] * p - ge[n] * (plogp - p * plogp.sum())
        d[n, t] += gl[n]
        d[n] /= T
    return d


def attention(q, k, v, table, lens, q_start, scale, k_scale=None, v_scale=None, window=0):
    """q [T,Hq,D], pools [P,H,ps,D] as float64 tensors (already the values they hold), on one
    device.  Returns out, lse, sum_j w_j |v_j| and max_j sum_d |q_d k_jd| (for the tolerances)."""
    T, Hq, D = q.shape
    H, ps = k.shape[1], k.shape[2]
    G = Hq // H
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    dot = torch.zeros((T, Hq), dtype=torch.float64, device=q.device)
    for r, n in enumerate(lens):
        nq = q_start[r + 1] - q_start[r]
        for i in range(nq):
            last = n - nq + i
            first = max(0, last - window + 1) if window else 0
            if last < first:
                continue
            j = torch.arange(first, last + 1, device=q.device)
            page = torch.as_tensor(table[r], device=q.device).long()[j // ps]
            t = q_start[r] + i
            for h in range(H):
                kk, vv = k[page, h, j % ps], v[page, h, j % ps]
                if k_scale is not None:
                    kk, vv = kk * float(k_scale[h]), vv * float(v_scale[h])
                heads = slice(h * G, (h + 1) * G)
                s = q[t, heads] @ kk.T * scale
                lse[t, heads] = torch.logsumexp(s, 1)
                w = torch.exp(s - lse[t, heads][:, None])
                out[t, heads] = w @ vv
                mag[t, heads] = w @ vv.abs()
                dot[t, heads] = (q[t, heads].abs() @ kk.abs().T).amax(1) * abs(scale)
    return out, lse, mag, dot


class Tables:
    """The page tables as Python lists, with the calls that change them."""

    def __init__(self, table, lens, ref, page_size):
        self.table = [list(map(int, row)) for row in table]
        self.lens = list(map(int, lens))
        self.ref = list(map(int, ref))
        self.ps = page_size

    def pages(self, n):
        return -(-n // self.ps)

    def fork(self, src, dst):
        before = list(self.lens)
        for f, (s, d) in enumerate(zip(src, dst)):
            if before[d] != 0 or s in dst or d in dst[:f]:
                continue
            n = self.pages(self.lens[s])
            self.table[d] = self.table[s][:n] + [-1] * (len(self.table[s]) - n)
            for p in self.table[s][:n]:
                self.ref[p] += 1
            self.lens[d] = self.lens[s]

    def reserve(self, n_new):
        """Returns granted, copies."""
        free = [p for p, c in enumerate(self.ref) if c == 0]
        shared = list(self.ref)
        granted, copies, at = [], [], 0
        for r, n in enumerate(n_new):
            have, want = self.pages(self.lens[r]), self.pages(self.lens[r] + n)
            copy = n > 0 and self.lens[r] % self.ps != 0 and shared[self.table[r][have - 1]] > 1
            need = want - have + copy
            if n < 0 or want > len(self.table[r]):
                granted.append(0)
                copies.append((-1, -1))
                continue
            at += need
            if need > 0 and at > len(free):
                granted.append(0)
                copies.append((-1, -1))
                continue
            mine = free[at - need:at]
            pair = (-1, -1)
            if copy:
                pair = (self.table[r][have - 1], mine.pop(0))
                self.ref[pair[0]] -= 1
                self.table[r][have - 1] = pair[1]
                self.ref[pair[1]] = 1
            for i, p in enumerate(mine):
                self.table[r][have + i] = p
                self.ref[p] = 1
            self.lens[r] += n
            granted.append(n)
            copies.append(pair)
        return granted, copies

    def truncate(self, new_len):
        for r, n in enumerate(new_len):
            n = max(0, n)
            if n >= self.lens[r]:
                continue
            for j in range(self.pages(n), self.pages(self.lens[r])):
                self.ref[self.table[r][j]] -= 1
                self.table[r][j] = -1
            self.lens[r] = n

    def compact(self):
        """Returns the moves (from, to)."""
        used = sum(c > 0 for c in self.ref)
        holes = [p for p in range(used) if self.ref[p] == 0]
        movers = [p for p in range(used, len(self.ref)) if self.ref[p] > 0]
        to = dict(zip(movers, holes))
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
        return list(to.items())
