"""Cases for the operators a serving loop needs around a speculative round: the log
probabilities of the emitted tokens (with entropy, the best alternatives and, for training,
the gradient), attention of the verified block over a paged key-value cache, and the cache's
page operations (fork, reserve with copy on write, write, truncate, compact).

``run`` computes each operator in a plain form, or, where ``own`` is true, through
``speculative_decoding_draft_03_gb300.binding``.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # one small round's emitted tokens (4 requests, 4 drafts): launch latency
        dict(name="logprob_small", op="logprob", N=16, V=1024, dtype="f32", top_k=4, temperature=1.0, absent=0.3,
             masked=0.0, train=False),
        # 32 requests, 7 drafts: log probabilities and 20 alternatives of each emitted token,
        # part of the rows under a grammar's vocabulary mask
        dict(name="logprob_f32_top20", op="logprob", N=256, V=151936, dtype="f32", top_k=20, temperature=0.8,
             absent=0.3, masked=0.25, train=False),
        # 256 requests, 5 drafts, bf16 target logits: the largest serving batch
        dict(name="logprob_bf16_top5", op="logprob", N=1536, V=129280, dtype="bf16", top_k=5, temperature=1.0,
             absent=0.3, masked=0.0, train=False),
        # a training step on sampled tokens: values, entropy bonus and the logits' gradient
        dict(name="logprob_train_bf16", op="logprob", N=1024, V=151936, dtype="bf16", top_k=0, temperature=1.0,
             absent=0.1, masked=0.0, train=True),
        # the same with an odd vocabulary in 32 bits (rows that start off the 16-byte grid)
        dict(name="logprob_train_f32_odd", op="logprob", N=300, V=50257, dtype="f32", top_k=0, temperature=1.3,
             absent=0.1, masked=0.1, train=True),
        # a few short requests, one new token each: launch latency
        dict(name="attend_small", op="attend", R=4, Hq=8, Hkv=2, D=64, page=16, min_len=1, max_len=200, max_q=1,
             dtype="bf16", cache="bf16", window=0),
        # plain decoding of 32 requests: one new token each, ragged lengths
        dict(name="attend_decode", op="attend", R=32, Hq=32, Hkv=8, D=128, page=16, min_len=1000, max_len=8192,
             max_q=1, dtype="bf16", cache="bf16", window=0),
        # the verified block of 32 requests: 1 to 8 new tokens each, ragged lengths
        dict(name="attend_verify", op="attend", R=32, Hq=32, Hkv=8, D=128, page=64, min_len=1000, max_len=8192,
             max_q=8, dtype="f16", cache="f16", window=0),
        # two very long contexts in an 8-bit cache: the split over the cache's length
        dict(name="attend_long_e4m3", op="attend", R=2, Hq=64, Hkv=8, D=128, page=32, min_len=100000, max_len=131072,
             max_q=1, dtype="bf16", cache="e4m3", window=0),
        # one small round's cache work: reserve, write, truncate
        dict(name="cache_round_small", op="cache_round", R=4, forks=0, Hkv=2, D=64, page=16, layers=1, pages=256,
             min_len=1, max_len=200, max_new=5, dtype="bf16", cache="bf16"),
        # 256 requests of which 64 are forked (parallel samples of one prompt): the children
        # share pages, copy the ones they write, and the rejected drafts are dropped
        dict(name="cache_round_fork", op="cache_round", R=256, forks=64, Hkv=8, D=128, page=32, layers=4, pages=6000,
             min_len=50, max_len=800, max_new=6, dtype="bf16", cache="e4m3"),
        # a fragmented pool is moved to its lower half
        dict(name="cache_compact", op="cache_compact", R=64, Hkv=8, D=128, page=16, layers=2, pages=8192, used=4096,
             dtype="bf16", cache="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprob", "logprob", "attend", "attend", "attend", "cache_round", "cache_compact"])
    if op == "logprob":
        dtype = rng.choice(["f32", "bf16", "f16"])
        V = _log_int(rng, 500, 200000)
        cap = (600 << 20) // (V * SIZE[dtype]) // (2 if dtype == "f32" else 1)
        N = _log_int(rng, 1, max(2, min(4096, cap // 2)))
        train = rng.random() < 0.4
        return dict(op=op, N=N, V=V, dtype=dtype, top_k=0 if train else rng.randrange(0, 21),
                    temperature=round(rng.uniform(0.5, 1.5), 3), absent=rng.choice([0.0, 0.2, 0.5]),
                    masked=rng.choice([0.0, 0.0, 0.3]), train=train)
    if op == "attend":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 8])
        D = rng.choice([64, 128, 128, 256])
        dtype = rng.choice(["bf16", "f16"])
        R = _log_int(rng, 1, 128)
        most = max(64, min(60000, (400 << 20) // (R * Hkv * D * 4)))
        max_len = _log_int(rng, 32, most)
        max_q = rng.choice([1, 1, 2, 5, 8, 16])
        return dict(op=op, R=R, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([8, 16, 32, 64, 128]),
                    min_len=rng.randrange(0, max(1, max_len // 2)), max_len=max_len, max_q=max_q, dtype=dtype,
                    cache=rng.choice([dtype, dtype, "e4m3"]), window=rng.choice([0, 0, 0, 100]))
    Hkv, D = rng.choice([(1, 128), (2, 64), (8, 128), (4, 64), (4, 256)])
    page = rng.choice([8, 16, 32, 64])
    layers = rng.choice([1, 2, 4])
    dtype = rng.choice(["bf16", "f16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    most = (700 << 20) // (2 * layers * page * Hkv * D * SIZE[cache])
    if op == "cache_compact":
        pages = _log_int(rng, 64, min(20000, most))
        return dict(op=op, R=rng.randrange(1, 100), Hkv=Hkv, D=D, page=page, layers=layers, pages=pages,
                    used=rng.randrange(1, pages), dtype=dtype, cache=cache)
    max_len = _log_int(rng, 16, 2000)
    max_new = rng.choice([1, 2, 5, 8, 17])
    R = _log_int(rng, 1, 300)
    R = max(1, min(R, most // (-(-(max_len + max_new) // page) + 1)))
    forks = rng.randrange(0, R)
    pages = R * (-(-(max_len + max_new) // page) + 1) + 7
    return dict(op=op, R=R, forks=forks, Hkv=Hkv, D=D, page=page, layers=layers, pages=pages, min_len=1,
                max_len=max_len, max_new=max_new, dtype=dtype, cache=cache)


def _lengths(case):
    """Context lengths and new-token counts of the requests: a function of the case."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["R"])]
    top = case.get("max_q", case.get("max_new"))
    new = [r.randint(1, top) for _ in range(case["R"])]
    if case["op"] == "attend":
        lens = [max(n, m) for n, m in zip(lens, new)]  # the length holds the new tokens too
        lens[r.randrange(case["R"])] = max(case["max_len"], top)
    return lens, new


# ------------------------------------------------------------------------------ states


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"logprob": _prepare_logprob, "attend": _prepare_attend, "cache_round": _prepare_round,
            "cache_compact": _prepare_compact}[case["op"]](case, seed, g)


def _randn(shape, g, dtype, scale=1.0):
    x = torch.empty(shape, device="cuda", dtype=torch.bfloat16 if dtype == torch.float8_e4m3fn else dtype)
    x.normal_(generator=g)
    return (x * scale).to(dtype) if scale != 1.0 or x.dtype != dtype else x


def _prepare_logprob(case, seed, g):
    N, V, dt = case["N"], case["V"], DTYPES[case["dtype"]]
    x = torch.empty((N, V), device="cuda").normal_(generator=g).mul_(3.0)
    x -= 1.1 * torch.log(torch.arange(V, device="cuda", dtype=torch.float32) + 1.0)
    logits = x.to(dt)
    if case["masked"]:
        rows = torch.rand(N, generator=g, device="cuda") < case["masked"]
        gone = torch.rand((N, V), generator=g, device="cuda") < 0.9
        gone &= rows[:, None]
        gone[:, V // 2] = False
        logits.masked_fill_(gone, -math.inf)
        del gone
    u = torch.rand((N, V), generator=g, device="cuda").clamp_(min=1e-7)
    tokens = (logits.float() / case["temperature"] - torch.log(-torch.log(u))).argmax(1).to(torch.int32)
    del u, x
    absent = torch.rand(N, generator=g, device="cuda") < case["absent"]
    tokens = torch.where(absent, -1, tokens).to(torch.int32)
    K, f32 = case["top_k"], lambda *shape: torch.empty(shape, device="cuda")
    s = dict(case=case, logits=logits, tokens=tokens, out=dict(logprob=f32(N), entropy=f32(N), lse=f32(N)))
    if K:
        s["out"].update(top_ids=torch.empty((N, K), dtype=torch.int32, device="cuda"), top_logprobs=f32(N, K))
    if case["train"]:
        s["grad"] = torch.empty_like(logits)
        s["grad_logprob"] = torch.empty(N, device="cuda").normal_(generator=g)
        s["grad_entropy"] = torch.empty(N, device="cuda").normal_(generator=g).mul_(0.1)
    return s


def _tables(case, lens, width, pages, seed, slots=None):
    """Page table, lengths and reference counts over a shuffled pool, as int32 arrays."""
    slots = slots or len(lens)
    free = np.random.RandomState(seed & 0x7FFFFFFF).permutation(pages)
    table, at = np.full((slots, width), -1, np.int32), 0
    for r, n in enumerate(lens):
        k = -(-n // case["page"])
        table[r, :k] = free[at:at + k]
        at += k
    ref = np.zeros(pages, np.int32)
    ref[table[table >= 0]] = 1
    return table, np.array(list(lens) + [0] * (slots - len(lens)), np.int32), ref


def _prepare_attend(case, seed, g):
    lens, new = _lengths(case)
    R, H, D, ps, dt = case["R"], case["Hkv"], case["D"], case["page"], DTYPES[case["dtype"]]
    width = -(-max(lens) // ps)
    pages = sum(-(-n // ps) for n in lens) + 3
    table, length, _ = _tables(case, lens, width, pages, seed)
    cu = lambda a, t=torch.int32: torch.as_tensor(np.asarray(a), device="cuda").to(t)
    T = sum(new)
    s = dict(case=case, table=cu(table), length=cu(length), q_start=cu(np.concatenate([[0], np.cumsum(new)])),
             row=cu(np.repeat(np.arange(R), new), torch.int64),
             at=cu(np.concatenate([np.arange(n) for n in new]), torch.int64),
             q=_randn((T, case["Hq"], D), g, dt, 1.5), scale=1.0 / math.sqrt(D),
             k=_randn((pages, H, ps, D), g, DTYPES[case["cache"]]), v=_randn((pages, H, ps, D), g, DTYPES[case["cache"]]),
             k_scale=None, v_scale=None)
    if case["cache"] == "e4m3":
        s["k_scale"] = torch.rand(H, generator=g, device="cuda") * 0.5 + 0.75
        s["v_scale"] = torch.rand(H, generator=g, device="cuda") * 0.5 + 0.75
    s["out"] = dict(out=torch.empty_like(s["q"]), lse=torch.empty((T, case["Hq"]), device="cuda"))
    if own:  # the workspace that a serving loop keeps
        from speculative_decoding_draft_03_gb300 import binding as b
        s["ws"] = b.workspace(b.paged_attention_workspace_size(T, R, case["Hq"], H, D, case["max_q"]), "cuda")
    return s


def _pools(case, g):
    shape = (case["layers"], case["pages"], case["Hkv"], case["page"], case["D"])
    return _randn(shape, g, DTYPES[case["cache"]]), _randn(shape, g, DTYPES[case["cache"]])


def _flat(table, length, ref):
    """The three tables in one buffer, so that one copy puts a snapshot back."""
    flat = torch.from_numpy(np.concatenate([table.ravel(), length, ref])).cuda()
    return flat, torch.empty_like(flat)


def _views(flat, slots, width):
    n = slots * width
    return flat[:n].view(slots, width), flat[n:n + slots], flat[n + slots:]


def _prepare_round(case, seed, g):
    lens, new = _lengths(case)
    R, F, H, D, ps, L = (case[k] for k in ("R", "forks", "Hkv", "D", "page", "layers"))
    live, width = R - F, -(-(case["max_len"] + case["max_new"]) // ps) + 1
    table, length, ref = _tables(case, lens[:live], width, case["pages"], seed, R)
    rs = np.random.RandomState((seed + 1) & 0x7FFFFFFF)
    src = (np.arange(F) % live).astype(np.int32) if live else np.zeros(0, np.int32)
    dst = (live + np.arange(F)).astype(np.int32)
    after = np.concatenate([length[:live], length[src]])
    keep = after + np.array([rs.randint(1, n + 1) for n in new])
    T = sum(new)
    cu = lambda a, t=torch.int32: torch.as_tensor(np.asarray(a), device="cuda").to(t)
    start, work = _flat(table, length, ref)
    k, v = _pools(case, g)
    s = dict(case=case, start=start, work=work, width=width, src=cu(src), dst=cu(dst), n_new=cu(new), keep=cu(keep),
             q_start=cu(np.concatenate([[0], np.cumsum(new)])), row=cu(np.repeat(np.arange(R), new), torch.int64),
             at=cu(np.concatenate([np.arange(n) for n in new]), torch.int64), k=k, v=v,
             new_k=_randn((L, T, H, D), g, DTYPES[case["dtype"]], 2.0),
             new_v=_randn((L, T, H, D), g, DTYPES[case["dtype"]], 2.0), k_scale=None, v_scale=None)
    if case["cache"] == "e4m3":
        s["k_scale"] = torch.rand(H, generator=g, device="cuda") * 0.01 + 0.01
        s["v_scale"] = torch.rand(H, generator=g, device="cuda") * 0.01 + 0.01
    if own:  # the workspace, the list of pools and the plan's arrays that a serving loop keeps
        from speculative_decoding_draft_03_gb300 import binding as b
        s["ws"] = b.workspace(b.cache_workspace_size(R, case["pages"]), "cuda")
        s["pools"] = b.cache_pools([p for x in (k, v) for p in x.unbind(0)])
        s["plan"] = dict(granted=torch.empty(R, dtype=torch.int32, device="cuda"),
                         copies=torch.empty((R, 2), dtype=torch.int32, device="cuda"))
    return s


def _fragments(case):
    """Which pages are in use: a function of the case."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    return sorted(r.sample(range(case["pages"]), case["used"]))


def _prepare_compact(case, seed, g):
    R, used = case["R"], _fragments(case)
    rs = np.random.RandomState(seed & 0x7FFFFFFF)
    order = rs.permutation(used)
    per = -(-case["used"] // R)
    table, length = np.full((R, per), -1, np.int32), np.zeros(R, np.int32)
    for r in range(R):
        mine = order[r * per:(r + 1) * per]
        table[r, :len(mine)] = mine
        length[r] = max(0, len(mine) * case["page"] - int(rs.randint(0, case["page"])))
    ref = np.zeros(case["pages"], np.int32)
    ref[used] = 1
    start, work = _flat(table, length, ref)
    k, v = _pools(case, g)
    s = dict(case=case, start=start, work=work, width=per, k=k, v=v)
    if own:  # the workspace, the list of pools and the plan's arrays that a serving loop keeps
        from speculative_decoding_draft_03_gb300 import binding as b
        s["ws"] = b.workspace(b.cache_workspace_size(R, case["pages"]), "cuda")
        s["pools"] = b.cache_pools([p for x in (k, v) for p in x.unbind(0)])
        s["plan"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------- passes


def run(s):
    op = s["case"]["op"]
    if op == "logprob":
        return _own_logprob(s) if own else _plain_logprob(s)
    if op == "attend":
        return _own_attend(s) if own else _plain_attend(s)
    s["work"].copy_(s["start"])  # every pass begins from the same tables
    if op == "cache_round":
        return _own_round(s) if own else _plain_round(s)
    return _own_compact(s) if own else _plain_compact(s)


def _own_logprob(s):
    from speculative_decoding_draft_03_gb300 import binding as b
    c = s["case"]
    got = dict(b.token_logprobs(s["logits"], s["tokens"], c["temperature"], c["top_k"], out=s["out"]))
    if c["train"]:
        got["grad"] = b.token_logprobs_backward(s["logits"], s["tokens"], got["lse"], got["entropy"],
                                                s["grad_logprob"], s["grad_entropy"], c["temperature"],
                                                out=s["grad"])
    return got


def _plain_logprob(s):
    c, raw = s["case"], s["logits"]
    z = raw.float() / c["temperature"]
    tok = s["tokens"].long()
    there = tok >= 0
    at = tok.clamp(min=0)[:, None]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    logp = (z - m) - torch.log(total)
    p = e / total
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    nan = torch.full((), math.nan, device=z.device)
    got = dict(logprob=torch.where(there, logp.gather(1, at)[:, 0], nan), entropy=torch.where(there, entropy, nan),
               lse=torch.where(there, lse[:, 0], nan))
    K = c["top_k"]
    if K:
        ids = torch.sort(raw.float(), dim=1, descending=True, stable=True).indices[:, :K]
        got["top_logprobs"] = torch.where(there[:, None], logp.gather(1, ids), nan)
        got["top_ids"] = torch.where(there[:, None], ids, -1).to(torch.int32)
    if c["train"]:
        # d logprob / d z_v = 1[v = token] - p_v ;  d entropy / d z_v = -p_v (ln p_v + entropy)
        gl, ge = s["grad_logprob"][:, None], s["grad_entropy"][:, None]
        d = -gl * p - ge * torch.where(p > 0, p * (logp + entropy[:, None]), 0.0)
        d.scatter_add_(1, at, gl)
        got["grad"] = torch.where(there[:, None], d / c["temperature"], 0.0).to(raw.dtype)
    return got


def _own_attend(s):
    from speculative_decoding_draft_03_gb300 import binding as b
    c = s["case"]
    o = b.paged_attention(s["q"], s["k"], s["v"], s["table"], s["length"], s["q_start"], c["max_q"], s["scale"],
                          k_scale=s["k_scale"], v_scale=s["v_scale"], window=c["window"], out=s["out"], ws=s["ws"])
    return dict(out=o["out"], lse=o["lse"])


def _plain_attend(s):
    c = s["case"]
    R, H, D, ps, nq = c["R"], c["Hkv"], c["D"], c["page"], c["max_q"]
    G = c["Hq"] // H
    new = s["q_start"][1:] - s["q_start"][:-1]
    i = torch.arange(nq, device="cuda")
    rows = (s["q_start"][:-1, None] + torch.minimum(i, new[:, None] - 1)).long()
    q = s["q"].float()[rows].view(R, nq, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, nq * G, D)

    def gathered(pool, scale):
        at = s["table"].clamp(min=0).long()
        x = pool.view(torch.uint8)[at].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[at]
        x = x.float().permute(0, 2, 1, 3, 4).reshape(R, H, -1, D)
        return x if scale is None else x * scale[None, :, None, None]

    k = gathered(s["k"], s["k_scale"])
    scores = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    pos = torch.arange(scores.shape[3], device="cuda")
    last = s["length"][:, None] - new[:, None] + i  # the query's own position
    seen = (pos <= last[:, :, None]) & (pos < s["length"][:, None, None])
    if c["window"]:
        seen &= pos > last[:, :, None] - c["window"]
    seen = seen[:, None].repeat_interleave(G, dim=2)
    scores = scores.masked_fill(~seen, -math.inf)
    m = scores.amax(3, keepdim=True).clamp(min=-1e30)
    p = torch.exp(scores - m)
    total = p.sum(3, keepdim=True)
    v = gathered(s["v"], s["v_scale"])
    v = torch.where((pos < s["length"][:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p, v) / total
    lse = (m + torch.log(total))[..., 0]
    o = o.view(R, H, nq, G, D).permute(0, 2, 1, 3, 4)[s["row"], s["at"]]
    lse = lse.view(R, H, nq, G).permute(0, 2, 1, 3)[s["row"], s["at"]]
    return dict(out=o.reshape(-1, c["Hq"], D).to(s["q"].dtype), lse=lse.reshape(-1, c["Hq"]).contiguous())


def _own_round(s):
    from speculative_decoding_draft_03_gb300 import binding as b
    c = s["case"]
    table, length, ref = _views(s["work"], c["R"], s["width"])
    if c["forks"]:
        b.cache_fork(table, length, ref, s["src"], s["dst"], c["page"], ws=s["ws"])
    plan = b.cache_reserve(table, length, ref, s["n_new"], c["page"], s["pools"], out=s["plan"], ws=s["ws"])
    for n in range(c["layers"]):
        b.cache_write(s["new_k"][n], s["new_v"][n], s["k"][n], s["v"][n], table, length, s["q_start"],
                      granted=plan["granted"], k_scale=s["k_scale"], v_scale=s["v_scale"], ws=s["ws"])
    b.cache_truncate(table, length, ref, s["keep"], c["page"], ws=s["ws"])
    return dict(table=table, length=length, ref=ref, granted=plan["granted"], copies=plan["copies"], k=s["k"], v=s["v"])


def _bytes(pool):
    return pool.view(torch.uint8) if pool.element_size() == 1 else pool.view(torch.int16)


def _plain_round(s):
    c = s["case"]
    R, ps, W = c["R"], c["page"], s["width"]
    table, length, ref = _views(s["work"], R, W)
    one = torch.ones((), dtype=torch.int32, device="cuda")
    if c["forks"]:
        src, dst = s["src"].long(), s["dst"].long()
        table[dst] = table[src]
        length[dst] = length[src]
        shared = table[dst]
        ref.index_add_(0, shared.clamp(min=0).reshape(-1).long(), (shared >= 0).int().reshape(-1))
    # reserve: pages for the new tokens, and a fresh copy of a shared page about to be written
    n = s["n_new"]
    have, want = (length + ps - 1) // ps, (length + n + ps - 1) // ps
    tail = (have - 1).clamp(min=0).long()
    last = table.gather(1, tail[:, None])[:, 0]
    copy = (length % ps != 0) & (n > 0) & (ref[last.clamp(min=0).long()] > 1)
    need = want - have + copy
    end = torch.cumsum(need, 0)
    is_free = ref == 0
    ok = (end <= is_free.sum()) | (need == 0)
    granted = torch.where(ok, n, 0).to(torch.int32)
    copy &= ok
    rank = torch.cumsum(is_free, 0) - 1
    by_rank = torch.full((ref.numel() + 1,), -1, dtype=torch.int32, device="cuda")
    pages = torch.arange(ref.numel(), device="cuda", dtype=torch.int32)
    by_rank[torch.where(is_free, rank, ref.numel())] = pages
    first = end - need
    j = torch.arange(W, device="cuda")
    fresh = (j >= have[:, None]) & (j < want[:, None]) & ok[:, None]
    order = first[:, None] + copy[:, None].long() + j - have[:, None]
    swap = copy[:, None] & (j == tail[:, None])
    order = torch.where(swap, first[:, None], order)
    taken = fresh | swap
    got = by_rank[order.clamp(min=0, max=ref.numel() - 1)]
    ref.index_add_(0, last.clamp(min=0).long(), -copy.int())
    ref.index_add_(0, got.clamp(min=0).reshape(-1).long(), (taken & (got >= 0)).int().reshape(-1))
    copies = torch.stack([torch.where(copy, last, -1), torch.where(copy, got.gather(1, tail[:, None])[:, 0], -1)], 1)
    table.copy_(torch.where(taken, got, table))
    length += granted
    fromto = copies[copy].long()
    for_k, for_v = _bytes(s["k"]), _bytes(s["v"])
    for_k[:, fromto[:, 1]] = for_k[:, fromto[:, 0]]
    for_v[:, fromto[:, 1]] = for_v[:, fromto[:, 0]]
    # write the new rows
    pos = length[s["row"]] - n[s["row"]] + s["at"]
    there = granted[s["row"]] > 0
    page = table[s["row"], (pos // ps).clamp(min=0, max=W - 1)].long()[there]
    slot = (pos % ps).long()[there]

    def rows(x, scale, pool):
        x = x.float()[:, there]
        x = x if scale is None else (x / scale[None, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        return _bytes(x.to(pool.dtype))

    for_k[:, page, :, slot] = rows(s["new_k"], s["k_scale"], s["k"]).transpose(0, 1)
    for_v[:, page, :, slot] = rows(s["new_v"], s["v_scale"], s["v"]).transpose(0, 1)
    # truncate: drop what lies past the kept tokens
    keep = torch.minimum(length, s["keep"])
    drop = (j >= ((keep + ps - 1) // ps)[:, None]) & (table >= 0)
    ref.index_add_(0, table.clamp(min=0).reshape(-1).long(), -drop.int().reshape(-1))
    table.masked_fill_(drop, -1)
    length.copy_(keep)
    return dict(table=table, length=length, ref=ref, granted=granted, copies=copies.to(torch.int32), k=s["k"], v=s["v"])


def _own_compact(s):
    from speculative_decoding_draft_03_gb300 import binding as b
    c = s["case"]
    table, length, ref = _views(s["work"], c["R"], s["width"])
    moves = b.cache_compact(table, length, ref, c["page"], s["pools"], out=s["plan"], ws=s["ws"])
    return dict(table=table, length=length, ref=ref, moves=moves, k=s["k"], v=s["v"])


def _plain_compact(s):
    table, length, ref = _views(s["work"], s["case"]["R"], s["width"])
    page = torch.arange(ref.numel(), device="cuda")
    in_use = ref > 0
    total = in_use.sum()
    holes = page[~in_use & (page < total)]
    movers = page[in_use & (page >= total)]
    to = page.clone()
    to[movers] = holes
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    ref[holes] = ref[movers]
    ref[movers] = 0
    for_k, for_v = _bytes(s["k"]), _bytes(s["v"])
    for_k[:, holes] = for_k[:, movers]
    for_v[:, holes] = for_v[:, movers]
    moves = torch.full((1,), movers.numel(), dtype=torch.int32, device="cuda")
    return dict(table=table, length=length, ref=ref, moves=moves, k=s["k"], v=s["v"])


# ------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "logprob":
        rows = case["N"] * (1.0 - case["absent"])
        size = case["V"] * SIZE[case["dtype"]]
        if case["train"]:  # the logits once, their gradient once
            return {"bytes": rows * size + case["N"] * size, "flops": 8.0 * rows * case["V"]}
        return {"bytes": rows * size + case["N"] * (16 + 8 * case["top_k"]), "flops": 4.0 * rows * case["V"]}
    if op == "attend":
        lens, new = _lengths(case)
        seen = [min(n, case["window"] + m - 1) if case["window"] else n for n, m in zip(lens, new)]
        H, D, size = case["Hkv"], case["D"], SIZE[case["dtype"]]
        cache = 2.0 * sum(seen) * H * D * SIZE[case["cache"]]
        io = sum(new) * case["Hq"] * (2 * D * size + 4)
        return {"bytes": cache + io, "flops": 4.0 * case["Hq"] * D * sum(n * m for n, m in zip(seen, new))}
    row = 2.0 * case["layers"] * case["Hkv"] * case["D"]
    page = row * case["page"] * SIZE[case["cache"]]
    if op == "cache_compact":
        used = _fragments(case)
        moved = sum(p >= len(used) for p in used)
        return {"bytes": 2.0 * moved * page + 8.0 * case["used"] + 8.0 * case["pages"], "flops": 0.0}
    lens, new = _lengths(case)
    R, F = case["R"], case["forks"]
    live = R - F
    tokens = sum(new)
    parents = {f % live for f in range(F)} if live else set()
    copies = sum(lens[p] % case["page"] != 0 for p in parents) + sum(lens[f % live] % case["page"] != 0 for f in range(F))
    rows = tokens * row * (SIZE[case["dtype"]] + SIZE[case["cache"]])
    tables = 4.0 * (sum(lens[:live]) / case["page"] + 4 * R + case["pages"])
    return {"bytes": rows + 2.0 * copies * page + tables, "flops": 0.0}


# ------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprob":
        return _exact_logprob(s)
    if case["op"] == "attend":
        return _exact_attend(s)
    return None  # whole numbers and copies


def _exact_logprob(s):
    c = s["case"]
    N, V, K = c["N"], c["V"], c["top_k"]
    f64 = lambda *shape: torch.full(shape, math.nan, dtype=torch.float64, device="cuda")
    o = dict(logprob=f64(N), entropy=f64(N), lse=f64(N))
    if K:
        o.update(top_ids=None, top_logprobs=f64(N, K))
    if c["train"]:
        o["grad"] = torch.zeros((N, V), dtype=torch.float64, device="cuda")
    tokens = s["tokens"].tolist()
    for n, t in enumerate(tokens):
        if t < 0:
            continue
        z = s["logits"][n].double() / c["temperature"]
        lp = torch.log_softmax(z, 0)
        p = torch.exp(lp)
        plogp = torch.xlogy(p, p)
        o["logprob"][n] = lp[t]
        o["entropy"][n] = -plogp.sum()
        o["lse"][n] = torch.logsumexp(z, 0)
        if K:
            o["top_logprobs"][n] = torch.topk(lp, K).values
        if c["train"]:
            gl, ge = s["grad_logprob"][n].double(), s["grad_entropy"][n].double()
            row = -gl * p - ge * (plogp - p * plogp.sum())
            row[t] += gl
            o["grad"][n] = row / c["temperature"]
    return o


def _exact_attend(s):
    c = s["case"]
    H, D, ps = c["Hkv"], c["D"], c["page"]
    G = c["Hq"] // H
    starts, lens = s["q_start"].tolist(), s["length"].tolist()
    out = torch.zeros((starts[-1], c["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((starts[-1], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")

    def context(pool, scale, pages, n, h):
        x = pool[:, h]
        x = x.view(torch.uint8)[pages].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else x[pages]
        x = x.double().reshape(-1, D)[:n]
        return x if scale is None else x * scale[h].double()

    for r, n in enumerate(lens):
        pages = s["table"][r, :-(-n // ps)].long()
        for h in range(H):
            k, v = context(s["k"], s["k_scale"], pages, n, h), context(s["v"], s["v_scale"], pages, n, h)
            for t in range(starts[r], starts[r + 1]):
                end = n - (starts[r + 1] - 1 - t)  # keys up to the query's own position
                begin = max(0, end - c["window"]) if c["window"] else 0
                heads = slice(h * G, (h + 1) * G)
                a = s["q"][t, heads].double() @ k[begin:end].T * s["scale"]
                top = torch.logsumexp(a, 1)
                lse[t, heads] = top
                out[t, heads] = torch.exp(a - top[:, None]) @ v[begin:end]
    return dict(out=out, lse=lse)
