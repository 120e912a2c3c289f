"""Cases for the operators that stand between a model's projections and the paged cache, and
between its logits and verification: rotary positions (with their gradient), appending rotated
keys with their values to a paged cache, attention of a long chunk of new tokens over it, and the
adjustment of logits by penalties for repeated tokens, biases and grammar masks.

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
        # one decoded token of 32 requests, queries and keys side by side: launch latency
        dict(name="rotary_decode", op="rotary", T=32, H=40, D=128, rot=128, dtype="bf16", interleaved=False,
             scaling="none", far=8192, train=False),
        # a prompt of 8192 tokens far into a long context, rates stretched by bands
        dict(name="rotary_prompt", op="rotary", T=8192, H=40, D=128, rot=128, dtype="bf16", interleaved=False,
             scaling="bands", far=131072, train=False),
        # a training step's forward and backward pass in 32 bits, neighbouring pairs, half of the head
        dict(name="rotary_train_f32", op="rotary", T=4096, H=32, D=128, rot=64, dtype="f32", interleaved=True,
             scaling="none", far=4096, train=True),
        # the verified block of 32 requests: 1 to 8 tokens each
        dict(name="append_verify", op="append", R=32, Hq=32, Hkv=8, D=128, rot=128, page=16, min_len=1000, max_len=8192,
             max_new=8, dtype="bf16", cache="bf16", interleaved=False, scaling="none"),
        # 16 prompts in chunks of up to 1024 tokens into an 8-bit cache
        dict(name="append_prompt_e4m3", op="append", R=16, Hq=32, Hkv=8, D=128, rot=128, page=32, min_len=0, max_len=4096,
             max_new=1024, dtype="bf16", cache="e4m3", interleaved=False, scaling="yarn"),
        # two short prompts, one chunk each: launch latency
        dict(name="chunk_small", op="chunk", R=2, Hq=8, Hkv=2, D=64, page=16, min_len=0, max_len=400, min_new=130,
             max_new=200, dtype="bf16", cache="bf16", window=0),
        # a mixed batch: some requests decode, others bring a chunk of their prompt
        dict(name="chunk_ragged", op="chunk", R=16, Hq=32, Hkv=8, D=128, page=16, min_len=1000, max_len=8192, min_new=1,
             max_new=1024, dtype="bf16", cache="bf16", window=0),
        # one whole prompt at once
        dict(name="chunk_prompt", op="chunk", R=1, Hq=32, Hkv=8, D=128, page=64, min_len=8192, max_len=8192, min_new=8192,
             max_new=8192, dtype="bf16", cache="bf16", window=0),
        # a short chunk at the end of a very long context in an 8-bit cache
        dict(name="chunk_long_e4m3", op="chunk", R=1, Hq=32, Hkv=8, D=128, page=32, min_len=65536, max_len=65536,
             min_new=512, max_new=512, dtype="f16", cache="e4m3", window=0),
        # one small round (4 requests, 4 drafts): launch latency
        dict(name="adjust_small", op="adjust", R=4, min_rows=5, max_rows=5, V=1024, dtype="f32", min_hist=1, max_hist=200,
             biases=4, masked=0.0),
        # the verified rows of 32 requests with long histories, a quarter of them under a grammar
        dict(name="adjust_verify_bf16", op="adjust", R=32, min_rows=1, max_rows=8, V=151936, dtype="bf16", min_hist=1000,
             max_hist=8192, biases=16, masked=0.25),
        # many requests with an odd vocabulary in 32 bits, very long histories
        dict(name="adjust_decode_f32_odd", op="adjust", R=128, min_rows=1, max_rows=2, V=50257, dtype="f32", min_hist=1,
             max_hist=32768, biases=300, masked=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "chunk", "chunk", "chunk", "adjust", "adjust"])
    if op == "rotary":
        D = rng.choice([64, 96, 128, 256])
        H, dtype, train = rng.choice([1, 2, 5, 8, 40, 72]), rng.choice(["f32", "bf16", "f16"]), rng.random() < 0.4
        most = (200 << 20) // (H * D * SIZE[dtype] * (2 if train else 1))
        return dict(op=op, T=_log_int(rng, 1, min(40000, most)), H=H, D=D, rot=rng.choice([D, D, D // 2, 20, 2]), dtype=dtype,
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]),
                    far=_log_int(rng, 64, 1 << 20), train=train)
    dtype = rng.choice(["bf16", "f16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    if op == "append":
        Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 80, 128, 256])
        page, max_new, max_len = rng.choice([8, 16, 20, 64]), _log_int(rng, 1, 2000), _log_int(rng, 16, 8000)
        most = (300 << 20) // (Hkv * D * 2 * SIZE[cache] * (max_new + max_len + 2 * page))
        most = min(most, (150 << 20) // (Hkv * (G + 2) * D * 2 * max_new))
        return dict(op=op, R=_log_int(rng, 1, max(1, min(200, most))), Hq=Hkv * G, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, 16]), page=page, min_len=0, max_len=max_len, max_new=max_new, dtype=dtype,
                    cache=cache, interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]))
    if op == "chunk":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        D, R, max_new = rng.choice([64, 80, 128, 128, 128]), _log_int(rng, 1, 64), _log_int(rng, 129, 4000)
        # products of at most a quarter of the whole prompt's, and a bounded cache
        most = min((1 << 28) // (R * Hkv * G * max_new // 2 + 1), (600 << 20) // (R * Hkv * D * 4))
        max_len = max(max_new, _log_int(rng, 129, max(130, min(100000, most))))
        if R * Hkv * G * max_new * max_len > 1 << 30:
            R = max(1, (1 << 30) // (Hkv * G * max_new * max_len))
        return dict(op=op, R=R, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([8, 16, 32, 64, 128]), min_len=0, max_len=max_len,
                    min_new=rng.choice([0, 1, 100]), max_new=max_new, dtype=dtype, cache=cache,
                    window=rng.choice([0, 0, 0, 500]))
    V, dtype = _log_int(rng, 500, 200000), rng.choice(["f32", "bf16", "f16"])
    max_rows = rng.choice([1, 2, 5, 9, 17])
    R = _log_int(rng, 1, max(1, min(256, (60 << 20) // (V * max_rows))))
    return dict(op=op, R=R, min_rows=rng.choice([0, 1, max_rows]), max_rows=max_rows, V=V, dtype=dtype, min_hist=0,
                max_hist=_log_int(rng, 1, 40000), biases=rng.choice([0, 1, 30, 300]), masked=rng.choice([0.0, 0.3, 1.0]))


def _lengths(case):
    """Lengths before the call and counts of new tokens (rows) of the requests: a function of the case."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    op, R = case["op"], case["R"]
    if op == "adjust":
        lens = [r.randint(case["min_hist"], case["max_hist"]) for _ in range(R)]
        new = [r.randint(case["min_rows"], case["max_rows"]) for _ in range(R)]
        new[r.randrange(R)] = case["max_rows"]
        return lens, new
    lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(R)]
    new = [r.randint(case.get("min_new", 1), case["max_new"]) for _ in range(R)]
    one = r.randrange(R)
    new[one] = case["max_new"]
    if op == "chunk":  # the lengths hold the new tokens too
        lens = [max(n, m) for n, m in zip(lens, new)]
        lens[one] = max(case["max_len"], case["max_new"])
    else:
        lens = [n + m for n, m in zip(lens, new)]
    return lens, new


# ------------------------------------------------------------------------------ states

BASE, FACTOR, ORIGINAL, LOW, HIGH = 10000.0, 8.0, 4096, 1.0, 32.0


def _frequencies(rot, scaling):
    """Radians per position of each pair, in 64 bits, and the magnitude of the rotated pairs."""
    i = np.arange(rot // 2, dtype=np.float64)
    base = BASE * FACTOR ** (rot / (rot - 2.0)) if scaling == "ntk" and rot > 2 else BASE
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / FACTOR
    if scaling == "bands":  # fast pairs as they are, slow ones stretched, a blend by their turns between
        kept = np.clip((ORIGINAL * f / (2.0 * np.pi) - LOW) / (HIGH - LOW), 0.0, 1.0)
        f = f * (kept + (1.0 - kept) / FACTOR)
    if scaling == "yarn":  # the same with a blend by the pair's index
        index = lambda turns: rot * math.log(ORIGINAL / (2.0 * math.pi * turns)) / (2.0 * math.log(BASE))
        lo, hi = max(0, math.floor(index(HIGH))), min(rot - 1, math.ceil(index(LOW)))
        r = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        f = f * (1.0 - r + r / FACTOR)
    return torch.from_numpy(f).cuda(), 0.1 * math.log(FACTOR) + 1.0 if scaling == "yarn" else 1.0


def _own_rates(case):
    from speculative_decoding_draft_03_gb300 import binding as b
    return b.rotary_rates(case["rot"], BASE, scaling=case["scaling"], factor=FACTOR, original_len=ORIGINAL, low=LOW,
                          high=HIGH, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"rotary": _prepare_rotary, "append": _prepare_append, "chunk": _prepare_chunk,
            "adjust": _prepare_adjust}[case["op"]](case, seed, g)


def _randn(shape, g, dtype, scale=1.0):
    x = torch.empty(shape, device="cuda", dtype=torch.bfloat16 if dtype == torch.float8_e4m3fn else dtype)
    x.normal_(generator=g)
    return (x * scale).to(dtype) if scale != 1.0 or x.dtype != dtype else x


def _cu(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), device="cuda").to(dtype)


def _prepare_rotary(case, seed, g):
    T, H, D, dt = case["T"], case["H"], case["D"], DTYPES[case["dtype"]]
    first = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device="cuda")
    pos = (first + torch.arange(T, device="cuda")).to(torch.int32)
    if T <= 256:  # decoded tokens of as many requests
        pos = torch.randint(0, case["far"], (T,), generator=g, device="cuda").to(torch.int32)
    f, magnitude = _frequencies(case["rot"], case["scaling"])
    s = dict(case=case, x=_randn((T, H, D), g, dt), positions=pos, frequencies=f, magnitude=magnitude)
    s["out"] = torch.empty_like(s["x"])
    if case["train"]:
        s["grad"] = _randn((T, H, D), g, dt)
        s["grad_x"] = torch.empty_like(s["x"])
    if own:
        s["rates"] = _own_rates(case)
    return s


def _tables(case, lens, seed):
    """Page table over a shuffled pool, lengths, and the number of pages."""
    ps = case["page"]
    pages, width = sum(-(-n // ps) for n in lens) + 3, max(1, -(-max(lens) // ps))
    free = np.random.RandomState(seed & 0x7FFFFFFF).permutation(pages)
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for r, n in enumerate(lens):
        k = -(-n // ps)
        table[r, :k] = free[at:at + k]
        at += k
    return _cu(table), _cu(lens), pages


def _rows_of(new):
    """First row of each request, and each row's request and place in it."""
    at = [np.arange(n) for n in new]
    return dict(q_start=_cu(np.concatenate([[0], np.cumsum(new)])), row=_cu(np.repeat(np.arange(len(new)), new), torch.int64),
                at=_cu(np.concatenate(at), torch.int64))


def _scales(case, g, low, span):
    if case["cache"] != "e4m3":
        return dict(k_scale=None, v_scale=None)
    f = lambda: torch.rand(case["Hkv"], generator=g, device="cuda") * span + low
    return dict(k_scale=f(), v_scale=f())


def _prepare_append(case, seed, g):
    lens, new = _lengths(case)
    H, D, dt = case["Hkv"], case["D"], DTYPES[case["dtype"]]
    table, length, pages = _tables(case, lens, seed)
    shape, T = (pages, H, case["page"], D), sum(new)
    f, magnitude = _frequencies(case["rot"], case["scaling"])
    s = dict(case=case, table=table, length=length, frequencies=f, magnitude=magnitude,
             k_pool=_randn(shape, g, DTYPES[case["cache"]]), v_pool=_randn(shape, g, DTYPES[case["cache"]]),
             q=_randn((T, case["Hq"], D), g, dt), k=_randn((T, H, D), g, dt, 2.0), v=_randn((T, H, D), g, dt, 2.0),
             **_rows_of(new), **_scales(case, g, 0.01, 0.01))
    s["q_out"] = torch.empty_like(s["q"])
    if own:  # the rates and the workspace that a serving loop keeps
        from speculative_decoding_draft_03_gb300 import binding as b
        s["rates"], s["ws"] = _own_rates(case), b.workspace(256, "cuda")
    return s


def _prepare_chunk(case, seed, g):
    lens, new = _lengths(case)
    H, D, dt = case["Hkv"], case["D"], DTYPES[case["dtype"]]
    table, length, pages = _tables(case, lens, seed)
    shape, T = (pages, H, case["page"], D), sum(new)
    s = dict(case=case, table=table, length=length, q=_randn((T, case["Hq"], D), g, dt, 1.5), scale=1.0 / math.sqrt(D),
             k=_randn(shape, g, DTYPES[case["cache"]]), v=_randn(shape, g, DTYPES[case["cache"]]), **_rows_of(new),
             **_scales(case, g, 0.75, 0.5))
    s["out"] = dict(out=torch.empty_like(s["q"]), lse=torch.empty((T, case["Hq"]), device="cuda"))
    if own:  # the workspace that a serving loop keeps
        from speculative_decoding_draft_03_gb300 import binding as b
        s["ws"] = b.workspace(b.chunk_attention_workspace_size(T, case["R"], case["Hq"], H, D), "cuda")
    return s


def _prepare_adjust(case, seed, g):
    lens, new = _lengths(case)
    R, V, N, dt = case["R"], case["V"], sum(new), DTYPES[case["dtype"]]
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")
    x = torch.empty((N, V), device="cuda").normal_(generator=g).mul_(3.0)
    x -= 1.1 * torch.log(torch.arange(V, device="cuda", dtype=torch.float32) + 1.0)
    words = lambda *shape: (V * rand(*shape) ** 4).to(torch.int32).clamp_(max=V - 1)  # frequent ids are low
    length = _cu(lens)
    B, W = case["biases"], -(-V // 32)
    s = dict(case=case, logits=x.to(dt), tokens=words(N), history=words(R, max(1, max(lens))), history_len=length,
             prompt_len=(length * rand(R)).to(torch.int32), repetition=1.0 + 0.4 * rand(R), frequency=rand(R) - 0.2,
             presence=rand(R) - 0.2, bias_ids=None, bias=None, mask=None, mask_row=None, **_rows_of(new))
    if B:
        ids = torch.argsort(rand(R, max(V, B)), dim=1)[:, :B] if R * V < 1 << 24 else torch.randint(
            0, V // B, (R, B), generator=g, device="cuda") + torch.arange(B, device="cuda") * (V // B)
        s.update(bias_ids=torch.where(rand(R, B) < 0.2, -1, ids).to(torch.int32), bias=4.0 * rand(R, B) - 2.0)
    if case["masked"]:
        under = max(1, round(case["masked"] * N))
        pick = torch.argsort(rand(N))[:under]
        s["mask_row"] = torch.full((N,), -1, dtype=torch.int32, device="cuda")
        s["mask_row"][pick] = torch.arange(under, dtype=torch.int32, device="cuda")
        # a grammar allows ranges of ids and some others
        bits = torch.randint(-(1 << 31), 1 << 31, (under, W), generator=g, device="cuda", dtype=torch.int64)
        some = torch.randint(-(1 << 31), 1 << 31, (under, W), generator=g, device="cuda", dtype=torch.int64)
        kind = rand(under, W)
        s["mask"] = torch.where(kind < 0.6, 0, torch.where(kind < 0.8, -1, bits & some)).to(torch.int32)
    s["out"] = torch.empty_like(s["logits"])
    return s


# ------------------------------------------------------------------------------- passes


def run(s):
    op = s["case"]["op"]
    if op == "rotary":
        return _own_rotary(s) if own else _plain_rotary(s)
    if op == "append":
        return _own_append(s) if own else _plain_append(s)
    if op == "chunk":
        return _own_chunk(s) if own else _plain_chunk(s)
    return _own_adjust(s) if own else _plain_adjust(s)


def _own_rotary(s):
    from speculative_decoding_draft_03_gb300 import binding as b
    c = s["case"]
    how = dict(interleaved=c["interleaved"], magnitude=s["magnitude"])
    got = dict(out=b.rotary(s["x"], s["positions"], s["rates"], out=s["out"], **how))
    if c["train"]:
        got["grad_x"] = b.rotary(s["grad"], s["positions"], s["rates"], inverse=True, out=s["grad_x"], **how)
    return got


def _turned(x, angle, magnitude, interleaved):
    """x [..., T, H, D] in 32 bits, its first pairs turned by angle [T, pairs] (64 bits)."""
    n = angle.shape[1]
    cos, sin = (magnitude * torch.cos(angle)).float()[:, None], (magnitude * torch.sin(angle)).float()[:, None]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    else:
        a, b = x[..., :n], x[..., n:2 * n]
    pair = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if interleaved else -2)
    return torch.cat([pair.flatten(-2), x[..., 2 * n:]], -1)


def _plain_rotary(s):
    c, dt = s["case"], s["x"].dtype
    angle = s["positions"].double()[:, None] * s["frequencies"]
    got = dict(out=_turned(s["x"].float(), angle, s["magnitude"], c["interleaved"]).to(dt))
    if c["train"]:
        got["grad_x"] = _turned(s["grad"].float(), -angle, s["magnitude"], c["interleaved"]).to(dt)
    return got


def _own_append(s):
    from speculative_decoding_draft_03_gb300 import binding as b
    q = b.cache_append(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["length"], s["q_start"], s["rates"],
                       interleaved=s["case"]["interleaved"], magnitude=s["magnitude"], k_scale=s["k_scale"],
                       v_scale=s["v_scale"], q_out=s["q_out"], ws=s["ws"])
    return dict(q=q, k_pool=s["k_pool"], v_pool=s["v_pool"])


def _plain_append(s):
    c = s["case"]
    new = s["q_start"][1:] - s["q_start"][:-1]
    pos = (s["length"] - new)[s["row"]].long() + s["at"]
    angle = pos.double()[:, None] * s["frequencies"]
    turn = lambda x: _turned(x.float(), angle, s["magnitude"], c["interleaved"])
    page, slot = s["table"][s["row"], pos // c["page"]].long(), pos % c["page"]

    def store(pool, x, scale):
        x = x if scale is None else (x / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        bits = torch.uint8 if pool.element_size() == 1 else torch.int16
        pool.view(bits)[page, :, slot] = x.to(pool.dtype).view(bits)

    store(s["k_pool"], turn(s["k"]), s["k_scale"])
    store(s["v_pool"], s["v"].float(), s["v_scale"])
    return dict(q=turn(s["q"]).to(s["q"].dtype), k_pool=s["k_pool"], v_pool=s["v_pool"])


def _own_chunk(s):
    from speculative_decoding_draft_03_gb300 import binding as b
    c = s["case"]
    o = b.chunk_attention(s["q"], s["k"], s["v"], s["table"], s["length"], s["q_start"], s["scale"], k_scale=s["k_scale"],
                          v_scale=s["v_scale"], window=c["window"], out=s["out"], ws=s["ws"])
    return dict(out=o["out"], lse=o["lse"])


def _plain_chunk(s):
    c = s["case"]
    R, H, D, nq = c["R"], c["Hkv"], c["D"], c["max_new"]
    G = c["Hq"] // H
    new = s["q_start"][1:] - s["q_start"][:-1]
    i = torch.arange(nq, device="cuda")
    rows = (s["q_start"][:-1, None] + torch.minimum(i, (new[:, None] - 1).clamp(min=0))).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"].float()[rows].view(R, nq, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, nq * G, D)

    def gathered(pool, scale):
        at = s["table"].clamp(min=0).long()
        x = pool.view(torch.uint8)[at].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[at]
        x = x.float().permute(0, 2, 1, 3, 4).reshape(R, H, -1, D)
        return x if scale is None else x * scale[None, :, None, None]

    scores = torch.matmul(q, gathered(s["k"], s["k_scale"]).transpose(2, 3)).mul_(s["scale"])
    pos = torch.arange(scores.shape[3], device="cuda")
    last = s["length"][:, None] - new[:, None] + i  # the query's own position
    unseen = (pos > last[:, :, None]) | (pos >= s["length"][:, None, None])
    if c["window"]:
        unseen |= pos <= last[:, :, None] - c["window"]
    scores.view(R, H, nq, G, -1).masked_fill_(unseen[:, None, :, None], -math.inf)
    m = scores.amax(3, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    v = gathered(s["v"], s["v_scale"])
    v = torch.where((pos < s["length"][:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p, v).div_(total)
    lse = (m + torch.log(total))[..., 0]
    o = o.view(R, H, nq, G, D).permute(0, 2, 1, 3, 4)[s["row"], s["at"]]
    lse = lse.view(R, H, nq, G).permute(0, 2, 1, 3)[s["row"], s["at"]]
    return dict(out=o.reshape(-1, c["Hq"], D).to(s["q"].dtype), lse=lse.reshape(-1, c["Hq"]).contiguous())


def _own_adjust(s):
    from speculative_decoding_draft_03_gb300 import binding as b
    return b.adjust_logits(s["logits"], s["tokens"], s["q_start"], s["history"], s["history_len"], s["prompt_len"],
                           repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                           bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"], mask_row=s["mask_row"], out=s["out"])


def _plain_adjust(s):
    c = s["case"]
    N, V, R = s["logits"].shape[0], c["V"], c["R"]
    # what each request has seen, and what it has answered, before this call
    i = torch.arange(s["history"].shape[1], device="cuda")
    there = (i < s["history_len"][:, None]).int()
    answered = there * (i >= s["prompt_len"][:, None])
    zeros = lambda n: torch.zeros((n, V), dtype=torch.int32, device="cuda")
    ids = s["history"].long()
    seen, count = zeros(R).scatter_add_(1, ids, there)[s["row"]], zeros(R).scatter_add_(1, ids, answered)[s["row"]]
    # and the row's own block, up to the token fed in for it
    j = torch.arange(c["max_rows"], device="cuda")
    ids = s["tokens"][(s["q_start"][s["row"]][:, None] + j).clamp(max=N - 1).long()].long()
    there = (j <= s["at"][:, None]).int()
    place = s["history_len"][s["row"]][:, None] + j
    seen.scatter_add_(1, ids, there)
    count.scatter_add_(1, ids, there * (place >= s["prompt_len"][s["row"]][:, None]))
    x = s["logits"].float()
    r = s["repetition"][s["row"]][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][s["row"]][:, None] * count - s["presence"][s["row"]][:, None] * (count > 0)
    if s["bias"] is not None:
        b = torch.zeros((R, V + 1), device="cuda").scatter_add_(1, s["bias_ids"].long() % (V + 1), s["bias"])
        x = x + b[s["row"], :V]
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        word = s["mask"][s["mask_row"].clamp(min=0).long()][:, v // 32]
        allowed = ((word >> (v % 32)) & 1).bool() | (s["mask_row"] < 0)[:, None]
        x = torch.where(allowed, x, -math.inf)
    return x.to(s["logits"].dtype)


# ------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "rotary":
        n = case["T"] * case["H"] * case["D"] * (2 if case["train"] else 1)
        return {"bytes": 2.0 * n * SIZE[case["dtype"]] + 4.0 * case["T"], "flops": 3.0 * n * case["rot"] / case["D"]}
    lens, new = _lengths(case)
    T = sum(new)
    if op == "append":
        D, size = case["D"], SIZE[case["dtype"]]
        rows = T * D * (2.0 * case["Hq"] * size + 2.0 * case["Hkv"] * (size + SIZE[case["cache"]]))
        return {"bytes": rows + 4.0 * sum(-(-n // case["page"]) for n in new) + 8.0 * case["R"],
                "flops": 3.0 * T * (case["Hq"] + case["Hkv"]) * case["rot"]}
    if op == "chunk":
        H, D, size, w = case["Hkv"], case["D"], SIZE[case["dtype"]], case["window"] or 1 << 40
        seen = [min(n, w + m - 1) if m else 0 for n, m in zip(lens, new)]
        pairs = sum(min(n - m + i + 1, w) for n, m in zip(lens, new) for i in range(m))
        return {"bytes": 2.0 * sum(seen) * H * D * SIZE[case["cache"]] + T * case["Hq"] * (2.0 * D * size + 4),
                "flops": 4.0 * case["Hq"] * D * pairs}
    V = case["V"]
    masks = max(1, round(case["masked"] * T)) if case["masked"] else 0
    return {"bytes": 2.0 * T * V * SIZE[case["dtype"]] + masks * V / 8.0 + 4.0 * sum(lens) + 8.0 * case["R"] * case["biases"],
            "flops": 4.0 * T * V}


# ------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "chunk": _exact_chunk, "adjust": _exact_adjust}[case["op"]](s)


def _exact_rates(rot, scaling):
    """Radians per position of each pair."""
    rates = []
    for i in range(rot // 2):
        grown = FACTOR ** (rot / (rot - 2)) if scaling == "ntk" and rot > 2 else 1.0
        f = math.exp(-2.0 * i / rot * math.log(BASE * grown))
        if scaling == "linear":
            f /= FACTOR
        elif scaling == "bands":
            turns = ORIGINAL * f / math.tau
            kept = min(1.0, max(0.0, (turns - LOW) / (HIGH - LOW)))
            f = kept * f + (1.0 - kept) * f / FACTOR
        elif scaling == "yarn":
            at = lambda turns: rot / 2.0 * math.log(ORIGINAL / (math.tau * turns), BASE)
            first, last = max(0, math.floor(at(HIGH))), min(rot - 1, math.ceil(at(LOW)))
            r = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            f = (1.0 - r) * f + r * f / FACTOR
        rates.append(f)
    return rates


def _exact_turned(x, pos, case, magnitude, sign=1.0):
    """x [T, H, D], each pair as a complex number times its own turn."""
    y = x.double().clone()
    for i, f in enumerate(_exact_rates(case["rot"], case["scaling"])):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
        turn = torch.polar(torch.full_like(pos, magnitude, dtype=torch.float64), sign * f * pos.double())[:, None]
        z = torch.complex(x[..., a].double(), x[..., b].double()) * turn
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_rotary(s):
    c = s["case"]
    o = dict(out=_exact_turned(s["x"], s["positions"], c, s["magnitude"]))
    if c["train"]:
        o["grad_x"] = _exact_turned(s["grad"], s["positions"], c, s["magnitude"], -1.0)
    return o


def _exact_append(s):
    c = s["case"]
    starts, lens = s["q_start"].tolist(), s["length"].tolist()
    k_pool, v_pool = (s[n].to(torch.float32).double() for n in ("k_pool", "v_pool"))
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for r, n in enumerate(lens):
        rows = slice(starts[r], starts[r + 1])
        pos = torch.arange(n - (starts[r + 1] - starts[r]), n, device="cuda")
        if not pos.numel():
            continue
        q[rows] = _exact_turned(s["q"][rows], pos, c, s["magnitude"])
        k, v = _exact_turned(s["k"][rows], pos, c, s["magnitude"]), s["v"][rows].double()
        if s["k_scale"] is not None:
            k, v = k / s["k_scale"].double()[:, None], v / s["v_scale"].double()[:, None]
            k, v = k.clamp(-E4M3_MAX, E4M3_MAX), v.clamp(-E4M3_MAX, E4M3_MAX)
        page = s["table"][r].long()[pos // c["page"]]
        k_pool[page, :, pos % c["page"]] = k
        v_pool[page, :, pos % c["page"]] = v
    return dict(q=q, k_pool=k_pool, v_pool=v_pool)


def _exact_chunk(s):
    c = s["case"]
    H, D, ps, w = c["Hkv"], c["D"], c["page"], c["window"] or 1 << 40
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
        pages, m = s["table"][r, :-(-n // ps)].long(), starts[r + 1] - starts[r]
        for h in range(H):
            k, v = context(s["k"], s["k_scale"], pages, n, h), context(s["v"], s["v_scale"], pages, n, h)
            heads = slice(h * G, (h + 1) * G)
            for i in range(0, m, 512):  # 512 queries at a time
                t = slice(starts[r] + i, starts[r] + min(i + 512, m))
                last = torch.arange(n - m + i, n - m + min(i + 512, m), device="cuda")[:, None]
                begin, end = max(0, n - m + i - w + 1), n - m + min(i + 512, m)
                j = torch.arange(begin, end, device="cuda")
                a = torch.einsum("tgd,sd->tgs", s["q"][t, heads].double(), k[begin:end]) * s["scale"]
                a = a.masked_fill(((j > last) | (j <= last - w))[:, None], -math.inf)
                top = torch.logsumexp(a, 2)
                lse[t, heads] = top
                out[t, heads] = torch.einsum("tgs,sd->tgd", torch.exp(a - top[..., None]), v[begin:end])
    return dict(out=out, lse=lse)


def _exact_adjust(s):
    c = s["case"]
    V, starts = c["V"], s["q_start"].tolist()
    out = s["logits"].double()
    for r in range(c["R"]):
        n, p = int(s["history_len"][r]), int(s["prompt_len"][r])
        rho, f, a = (float(s[k][r]) for k in ("repetition", "frequency", "presence"))
        for t in range(starts[r], starts[r + 1]):
            said = torch.cat([s["history"][r, :n], s["tokens"][starts[r]:t + 1]]).long()
            known, spoken = torch.bincount(said, minlength=V) > 0, torch.bincount(said[p:], minlength=V)
            x = out[t]
            x[known] = torch.where(x > 0, x / rho, x * rho)[known]
            x -= f * spoken + a * (spoken > 0).double()
            if s["bias"] is not None:
                ok = s["bias_ids"][r] >= 0
                x.index_add_(0, s["bias_ids"][r][ok].long(), s["bias"][r][ok].double())
            if s["mask"] is not None and s["mask_row"][t] >= 0:
                word = s["mask"][s["mask_row"][t].long()].cpu().numpy()
                allowed = np.unpackbits(word.view(np.uint8), bitorder="little")[:V]
                x[torch.from_numpy(allowed == 0).cuda()] = -math.inf
    return out
