"""Plain 64-bit forms of what stands around the cache and the logits, for the tests: rotary
positions, attention of long blocks (torch, float64) and the adjustment of logits (numpy)."""
import math

import numpy as np
import torch


def angles(positions, rates):
    """Radians [T, pairs] in (-pi, pi], from rates in 2^-64 turns: position * rate modulo one turn, in
    whole numbers."""
    p = np.asarray(positions, dtype=np.int64).astype(np.uint64)[:, None]
    with np.errstate(over="ignore"):
        turns = p * np.asarray(rates, dtype=np.int64).astype(np.uint64)[None]
    return turns.astype(np.int64).astype(np.float64) * 2.0 ** -64 * math.tau


def turned(x, positions, rates, interleaved=False, magnitude=1.0, inverse=False):
    """x [T,H,D] float64 (numpy).  Returns the result, and |x_u| + |x_w| of each turned element's pair
    (0 for the others), for the tolerances."""
    a = angles(positions, rates)[:, None] * (-1.0 if inverse else 1.0)
    n = a.shape[2]
    u, w = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y, mag = x.copy(), np.zeros_like(x)
    y[..., u] = magnitude * (x[..., u] * np.cos(a) - x[..., w] * np.sin(a))
    y[..., w] = magnitude * (x[..., w] * np.cos(a) + x[..., u] * np.sin(a))
    mag[..., u] = mag[..., w] = abs(magnitude) * (np.abs(x[..., u]) + np.abs(x[..., w]))
    return y, mag


def attention(q, k, v, table, lens, q_start, scale, k_scale=None, v_scale=None, window=0):
    """As serving_ref.attention, with a request's queries at once.  What a query does not see has no part
    in its sums, whatever it holds."""
    T, Hq, D = q.shape
    H, ps = k.shape[1], k.shape[2]
    G = Hq // H
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    dot = torch.zeros((T, Hq), dtype=torch.float64, device=q.device)
    for r, n in enumerate(lens):
        t = slice(int(q_start[r]), int(q_start[r + 1]))
        nq = t.stop - t.start
        if nq == 0:
            continue
        last = torch.arange(n - nq, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)
        seen = (j <= last) if not window else (j <= last) & (j > last - window)
        some = seen.any(1)
        if not some.any():
            continue
        page = torch.as_tensor(np.asarray(table[r]), device=q.device).long()[j // ps]
        page, gone = page.clamp(min=0), page < 0  # (pages that no query sees may be gone)
        for h in range(H):
            kk, vv = k[page, h, j % ps].clone(), v[page, h, j % ps].clone()
            kk[gone], vv[gone] = 0.0, 0.0
            if k_scale is not None:
                kk, vv = kk * float(k_scale[h]), vv * float(v_scale[h])
            heads = slice(h * G, (h + 1) * G)
            s = torch.einsum("tgd,sd->tgs", q[t, heads], kk) * scale
            s = torch.where(seen[:, None], s, -math.inf)
            top = torch.logsumexp(s, 2)
            w = torch.where(some[:, None, None], torch.exp(s - top[..., None]), 0.0)
            odd = ~torch.isfinite(vv).all(1)
            fine = torch.where(odd[:, None], 0.0, vv)
            o, m = w @ fine, w @ fine.abs()
            for i in odd.nonzero()[:, 0].tolist():  # these reach the queries that see them alone
                sees = seen[:, i]
                # (the magnitude, by which weights' roundings count, is the sum of w |v| over all that is seen:
                # such a token's finite elements are in o, and so in it too)
                o[sees] += w[sees][..., i, None] * vv[i]
                m[sees] += w[sees][..., i, None] * vv[i].abs()
            lse[t, heads] = torch.where(some[:, None], top, -math.inf)
            out[t, heads], mag[t, heads] = o, m
            a = torch.einsum("tgd,sd->tgs", q[t, heads].abs(), kk.abs())
            dot[t, heads] = torch.where(seen[:, None], a, 0.0).amax(2) * abs(scale)
    return out, lse, mag, dot


def adjusted(x, tokens, q_start, history=None, history_len=None, prompt_len=None, repetition=None, frequency=None,
             presence=None, bias_ids=None, bias=None, mask=None, mask_row=None):
    """x [N,V] float64.  Rows of no slot come back as they are.  Also the largest magnitude on the way to
    each value, for the tolerances."""
    x, most = x.copy(), np.abs(x)
    V = x.shape[1]
    for r in range(len(q_start) - 1):
        L = 0 if history is None else min(max(int(history_len[r]), 0), history.shape[1])
        said = [] if history is None else list(history[r, :L])
        p = 0 if prompt_len is None else int(prompt_len[r])
        for n in range(q_start[r], q_start[r + 1]):
            seq = said + ([] if tokens is None else list(tokens[q_start[r]:n + 1]))
            known = sorted({t for t in seq if 0 <= t < V})
            if repetition is not None:
                for t in known:
                    x[n, t] = x[n, t] / repetition[r] if x[n, t] > 0 else x[n, t] * repetition[r]
            most[n] = np.fmax(most[n], np.abs(x[n]))
            count = np.zeros(V)
            for t in seq[max(p, 0):]:
                if 0 <= t < V:
                    count[t] += 1
            if frequency is not None:
                x[n] -= frequency[r] * count
                most[n] = np.fmax(most[n], np.abs(frequency[r] * count))
            if presence is not None:
                x[n] -= presence[r] * (count > 0)
                most[n] = np.fmax(most[n], np.abs(presence[r] * (count > 0)))
            if bias_ids is not None:
                for t, b in zip(bias_ids[r], bias[r]):
                    if 0 <= t < V:
                        x[n, t] += b
                        most[n, t] += abs(b)
            m = -1 if mask is None else (n if mask_row is None else int(mask_row[n]))
            if mask is not None and 0 <= m < mask.shape[0]:
                words = np.ascontiguousarray(mask[m].astype(np.int32)).view(np.uint8)
                x[n, np.unpackbits(words, bitorder="little")[:V] == 0] = -math.inf
    return x, most
