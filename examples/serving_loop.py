"""A serving loop over speculative rounds: draft -> schedule -> the target's forward pass over a
paged cache -> exact verification -> the cache's rejected tail dropped -> log probabilities of
what is answered.

The target is a small random transformer (embedding, layers of grouped-query attention with a
residual, unembedding): it stands for a real one, whose calls of the cache and of the attention
would be the same.  Everything of a round runs on the device without a host read: lengths, page
choices, verify lengths and accepted counts stay there, and the block of verified rows is ragged
inside buffers of fixed size.  A request that the pool has no room for emits nothing that round, and
goes on once pages are given back.

With ``rotary`` the target's queries and keys are turned by their positions as they are appended to
the cache, and with ``adjust`` the verified logits are penalised, biased and masked first.

    python examples/serving_loop.py --rounds 8
    python examples/serving_loop.py --rounds 8 --rotary --repetition 1.2 --prompt 2000
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_draft_03_gb300 import binding as b  # noqa: E402
from speculative_decoding_draft_03_gb300 import workloads as wl  # noqa: E402


MAX_BLOCK = 512  # tokens of a prompt that go through the target at once


class ToyTarget:
    """layers x (grouped-query attention + residual) between an embedding and an unembedding."""

    def __init__(self, V, dim=128, layers=2, Hq=8, Hkv=2, D=64, seed=0, device="cuda", rates=None):
        """rates (binding.rotary_rates): queries and keys are turned by their positions."""
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)
        self.rates = rates
        self.V, self.dim, self.layers, self.Hq, self.Hkv, self.D = V, dim, layers, Hq, Hkv, D
        self.embed = rnd(V, dim)
        self.wq = rnd(layers, dim, Hq * D) / math.sqrt(dim) * 2
        self.wk = rnd(layers, dim, Hkv * D) / math.sqrt(dim)
        self.wv = rnd(layers, dim, Hkv * D) / math.sqrt(dim)
        self.wo = rnd(layers, Hq * D, dim) / math.sqrt(Hq * D)
        self.unembed = rnd(dim, V) / math.sqrt(dim) * 2

    def qkv(self, layer, x):
        T = x.shape[0]
        q = (x @ self.wq[layer]).view(T, self.Hq, self.D)
        k = (x @ self.wk[layer]).view(T, self.Hkv, self.D)
        v = (x @ self.wv[layer]).view(T, self.Hkv, self.D)
        return q.bfloat16(), k.bfloat16(), v.bfloat16()

    def out(self, layer, o):
        return o.float().reshape(o.shape[0], -1) @ self.wo[layer]

    def forward(self, tokens, cache, q_start, max_q):
        """Logits of the slots' last tokens (rows q_start[r] ..), whose room is reserved: their
        keys and values go into the cache, and they attend over it."""
        x = self.embed[tokens.long()]
        for layer in range(self.layers):
            q, k, v = self.qkv(layer, x)
            if self.rates is None:
                cache.write(layer, k, v, q_start)
            else:
                cache.append(layer, q, k, v, q_start, self.rates, q_out=q)
            o = cache.attend(layer, q, q_start, max_q, self.D ** -0.5)["out"]
            x = x + self.out(layer, torch.nan_to_num(o))  # (rows of no request hold anything)
        return x @ self.unembed

    def turned(self, x):
        """x [T,H,D] float64 turned by the positions 0 .. T-1, rounded to bfloat16."""
        if self.rates is None:
            return x
        turns = torch.arange(x.shape[0], device=x.device)[:, None] * self.rates  # (past 64 bits: whole turns)
        a = (turns.double() * 2.0 ** -63 * math.pi)[:, None]
        u, w = x.chunk(2, 2)
        return torch.cat([u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()], 2).bfloat16().double()

    def dense(self, tokens):
        """The same for one whole sequence, without a cache, in float64 (its 16-bit roundings of
        queries, keys and values kept)."""
        T = tokens.numel()
        x = self.embed[tokens.long()].double()
        mask = torch.ones((T, T), dtype=torch.bool, device=x.device).tril()
        for layer in range(self.layers):
            q, k, v = (t.double() for t in self.qkv(layer, x.float()))
            q, k = self.turned(q), self.turned(k)
            k, v = (t.repeat_interleave(self.Hq // self.Hkv, 1) for t in (k, v))
            s = torch.einsum("thd,shd->hts", q, k) * self.D ** -0.5
            p = torch.softmax(s.masked_fill(~mask, -math.inf), 2)
            x = x + torch.einsum("hts,shd->thd", p, v).reshape(T, -1) @ self.wo[layer].double()
        return x @ self.unembed.double()


class ServingLoop:
    """R requests in R slots of a paged cache, advanced by speculative rounds."""

    def __init__(self, prompts, gamma=4, page_size=16, num_pages=256, top_k=3, seed=0, cache_dtype=torch.bfloat16,
                 rotary=False, adjust=None, block=MAX_BLOCK):
        """rotary: with rotary positions.  adjust: dict of what adjust_logits takes for all requests alike,
        repetition, frequency, presence (floats), bias (dict of id: what is added), mask (bool [V],
        the ids that are allowed).  block: tokens of a prompt that go through the target at once."""
        dev = "cuda"
        self.R, self.gamma, self.top_k = len(prompts), gamma, top_k
        # sizes, step-rate table and request keys of the smallest workload; as the draft's Markov head
        # the target without its attention, W1 = embedding, W2 = unembedding, so that it is often right
        self.w = wl.make("tiny", device=dev, R=self.R, gamma=gamma)
        self.target = ToyTarget(self.w["V"], seed=seed, rates=b.rotary_rates(64) if rotary else None)
        rank, d = self.target.dim, self.w["d"]
        self.w.update(U=torch.zeros_like(self.w["U"]), W1=self.target.embed.contiguous(),
                      W2=self.target.unembed.contiguous(), rank=rank, conf_w=torch.zeros(d + rank, device=dev), conf_b=1.0)
        scales = dict(k_scale=torch.full((self.target.Hkv,), 0.02, device=dev),
                      v_scale=torch.full((self.target.Hkv,), 0.02, device=dev)) if cache_dtype.itemsize == 1 else {}
        self.cache = b.PagedCache(self.R, num_pages, page_size, num_pages // self.R, self.target.layers, self.target.Hkv,
                                  self.target.D, dtype=cache_dtype, device=dev, **scales)
        self.T = self.R * (gamma + 1)  # rows of the largest verified block
        i = torch.arange(self.T, device=dev)
        self.row_index = i
        self.prefill(prompts, block)
        self.adjust = None if adjust is None else self.adjustment(prompts, **adjust)
        self.rounds = 0

    def adjustment(self, prompts, repetition=None, frequency=None, presence=None, bias=None, mask=None):
        """What adjust_logits takes beside the logits and the block: the requests' tokens so far are kept
        on the device, one row each, as long as the cache's contexts."""
        R, V, dev = self.R, self.w["V"], "cuda"
        i32 = dict(dtype=torch.int32, device=dev)
        width = self.cache.page_table.shape[1] * self.cache.page_size + self.gamma + 1
        history = torch.full((R, width), -1, **i32)
        for r, p in enumerate(prompts):
            history[r, :len(p)] = torch.tensor(p, **i32)
        o = dict(history=history, prompt_len=torch.tensor([len(p) for p in prompts], **i32))
        for name, x in (("repetition", repetition), ("frequency", frequency), ("presence", presence)):
            if x is not None:
                o[name] = torch.full((R,), float(x), device=dev)
        if bias:
            o["bias_ids"] = torch.tensor([list(bias)] * R, **i32)
            o["bias"] = torch.tensor([list(bias.values())] * R, dtype=torch.float32, device=dev)
        if mask is not None:
            bits = torch.zeros((V + 31) // 32 * 32, dtype=torch.int64)
            bits[:V] = mask.cpu()
            words = (bits.view(-1, 32) << torch.arange(32)).sum(1)
            o["mask"] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(**i32)[None]
            o["mask_row"] = torch.zeros(self.T, **i32)
        return o

    def prefill(self, prompts, block):
        """Every token but the last goes into the cache, a block at a time; the last is the first anchor."""
        dev = "cuda"
        for at in range(0, max(len(p) - 1 for p in prompts), block):
            blocks = [p[at:min(at + block, len(p) - 1)] for p in prompts]
            n = [len(x) for x in blocks]
            q_start = torch.tensor([sum(n[:r]) for r in range(self.R + 1)], dtype=torch.int32, device=dev)
            want = torch.tensor(n, dtype=torch.int32, device=dev)
            if not torch.equal(self.cache.reserve(want)["granted"], want):
                raise RuntimeError("the pool has no room for the prompts")
            tokens = torch.tensor([t for x in blocks for t in x], dtype=torch.int32, device=dev)
            self.target.forward(tokens, self.cache, q_start, max(n))
        self.x0 = torch.tensor([p[-1] for p in prompts], dtype=torch.int32, device=dev)

    def step(self):
        """One round.  Returns dict tokens [R,gamma+1] (-1 past n_out), n_out, n_acc, ell, and of the
        emitted tokens logprob, entropy [R,gamma+1], top_ids, top_logprobs [R,gamma+1,top_k].  n_out
        is 0 for a request whose block found no room."""
        w, c, R, G1 = self.w, self.cache, self.R, self.gamma + 1
        d = b.markov_draft(w["U"], w["W1"], w["W2"], w["h"], w["conf_w"], w["conf_b"], w["conf_logit_scale"],
                           w["conf_temp"], w["temperature"], self.x0, w["req_id"], w["seed"], self.rounds)
        ell = b.schedule(d["conf"], w["sps"], w["mode"])["ell"]
        # the verified rows: each request's anchor and its first ell drafts, one after the other
        n_new = ell + 1
        q_start = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
        q_start[1:] = torch.cumsum(n_new, 0)
        r = (torch.searchsorted(q_start, self.row_index.to(torch.int32), right=True) - 1).clamp(max=R - 1)
        i = (self.row_index - q_start[r]).clamp(max=self.gamma)
        block = torch.cat([self.x0[:, None], d["x"]], 1)
        before = c.seq_len.clone()
        room = c.reserve(n_new)["granted"] > 0
        fed = block[r, i]
        logits = self.target.forward(fed, c, q_start, G1)
        if self.adjust is not None:  # (a request's tokens so far: its context's)
            b.adjust_logits(logits, fed, q_start, history_len=before, out=logits, **self.adjust)
        v = b.verify_ragged(logits, q_start[:-1].contiguous(), w["U"], w["W1"], w["W2"], self.x0, d["x"], d["logq"],
                            d["lse"], ell, w["temperature"], w["req_id"], w["seed"], self.rounds)
        c.truncate(before + 1 + v["n_acc"])  # the anchor and the accepted drafts stay
        n_out, n_acc = v["n_out"] * room, v["n_acc"] * room
        if self.adjust is not None:  # the block's tokens after the context's: as many of them as stay count
            self.adjust["history"].scatter_(1, before.long()[:, None] + torch.arange(G1, device="cuda"), block)
        answer = torch.where(room[:, None], v["tokens"], -1)
        # row i of a request gave its token i: what was emitted keeps its row's log probability
        mine = (self.row_index < q_start[-1]) & (i < n_out[r])
        emitted = torch.where(mine, answer[r, i], -1).to(torch.int32)
        lp = b.token_logprobs(logits, emitted, w["temperature"], self.top_k)
        row = (q_start[:-1, None] + torch.arange(G1, device="cuda")).clamp(max=self.T - 1).long()
        there = torch.arange(G1, device="cuda") < n_out[:, None]
        pick = lambda t, none: torch.where(there.view(R, G1, *[1] * (t.dim() - 1)), t[row], none)
        last = (n_out - 1).clamp(min=0).long()
        self.x0 = torch.where(room, answer.gather(1, last[:, None])[:, 0], self.x0)
        self.rounds += 1
        return dict(tokens=answer, n_out=n_out, n_acc=n_acc, ell=ell,
                    logprob=pick(lp["logprob"], math.nan), entropy=pick(lp["entropy"], math.nan),
                    top_ids=pick(lp["top_ids"], -1), top_logprobs=pick(lp["top_logprobs"], math.nan))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=60, help="tokens of the longest prompt, about")
    ap.add_argument("--rotary", action="store_true")
    ap.add_argument("--repetition", type=float, default=None)
    a = ap.parse_args()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1024, (int(n),), generator=g).tolist()
               for n in torch.randint(2, max(a.prompt, 3), (a.requests,), generator=g)]
    pages = -(-(a.prompt + a.rounds * 5 + 5) // 16) * a.requests
    loop = ServingLoop(prompts, num_pages=max(256, pages), rotary=a.rotary,
                       adjust=None if a.repetition is None else dict(repetition=a.repetition))
    answers = [[] for _ in prompts]
    for _ in range(a.rounds):
        o = loop.step()
        for r, n in enumerate(o["n_out"].tolist()):
            answers[r] += list(zip(o["tokens"][r, :n].tolist(), o["logprob"][r, :n].tolist()))
    for r, ans in enumerate(answers):
        print(f"request {r}: prompt of {len(prompts[r])}, {len(ans)} tokens: "
              + " ".join(f"{t}({lp:.2f})" for t, lp in ans[:12]) + (" ..." if len(ans) > 12 else ""))
    moved = loop.cache.compact().item()
    used = int((loop.cache.ref_count > 0).sum())
    print(f"{used} pages in use, {moved} moved by compaction; status {loop.cache.status()}")


if __name__ == "__main__":
    main()
