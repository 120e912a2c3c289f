"""The serving loop of examples/: what its rounds answer is checked against a dense forward pass
over each request's whole sequence, in float64.

Tolerance: the loop's fp32 products and 16-bit roundings of queries, keys, values, weights and
attention outputs (half steps of 2^-8 relative each) against the dense form, which keeps only the
roundings of queries, keys and values.  Two layers whose outputs are of order 1 or 2 add about
2 x 2 x 3 x 2^-8 to a hidden state of order 1..3, and the unembedding (columns of norm 2) carries a
hidden state's error of 0.05 (in norm, over 128 dimensions, averaging) to about 0.1 in a logit.
(With an e4m3 cache the stored keys depend on roundings of 2^-4 that a second computation does
not repeat; that attention is checked on given caches elsewhere, and here for its bookkeeping.)"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _loop(cache_dtype, prompts, **kw):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serving_loop
    return serving_loop.ServingLoop(prompts, cache_dtype=cache_dtype, **kw)


def _prompts(lens, seed=3):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 1024, (n,), generator=g).tolist() for n in lens]


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_rounds_answer_what_the_dense_model_says(cache_dtype):
    tol = 0.15
    prompts = _prompts([2, 33, 17, 58])
    loop = _loop(cache_dtype, prompts)
    seqs, lps, ents, tops = [list(p) for p in prompts], [[] for _ in prompts], [[] for _ in prompts], [[] for _ in prompts]
    for _ in range(12):
        o = loop.step()
        for r, n in enumerate(o["n_out"].tolist()):
            assert n == o["n_acc"][r] + 1
            seqs[r] += o["tokens"][r, :n].tolist()
            lps[r] += o["logprob"][r, :n].tolist()
            ents[r] += o["entropy"][r, :n].tolist()
            tops[r] += o["top_logprobs"][r, :n].tolist()
            assert torch.isnan(o["logprob"][r, n:]).all() and (o["top_ids"][r, n:] == -1).all()
    assert loop.cache.status() == 0
    assert sum(map(len, lps)) > 12 * len(prompts)  # some drafts were accepted
    assert loop.cache.seq_len.tolist() == [len(s) - 1 for s in seqs]  # all but the next anchor
    # pages: what the contexts need, no more, once each
    used = sum(-(-(len(s) - 1) // loop.cache.page_size) for s in seqs)
    assert int((loop.cache.ref_count > 0).sum()) == used and int(loop.cache.ref_count.sum()) == used
    for lp, top in zip(lps, tops):
        assert all(x <= t[0] <= 0 for x, t in zip(lp, top))
    if cache_dtype != torch.bfloat16:
        return
    for r, seq in enumerate(seqs):
        dense = torch.log_softmax(loop.target.dense(torch.tensor(seq, device="cuda")), 1)
        at = len(prompts[r]) - 1
        want = dense[torch.arange(at, len(seq) - 1), torch.tensor(seq[at + 1:], device="cuda")]
        got = torch.tensor(lps[r], device="cuda")
        assert (got - want).abs().max() < tol, (r, (got - want).abs().max())
        ent = -(dense.exp() * dense).sum(1)[at:-1]
        assert (torch.tensor(ents[r], device="cuda") - ent).abs().max() < tol
        best = dense[at:-1].topk(3, 1).values
        assert (torch.tensor(tops[r], device="cuda") - best).abs().max() < tol


def test_compaction_and_layout_change_nothing():
    """The same rounds with the pages moved between them, and with other page sizes, answer the
    same tokens."""
    prompts = _prompts([40, 9, 25])
    answers = []
    for page_size, num_pages, compact in ((16, 96, False), (16, 96, True), (8, 120, False), (64, 30, True)):
        loop = _loop(torch.bfloat16, prompts, page_size=page_size, num_pages=num_pages)
        got = []
        for k in range(8):
            o = loop.step()
            got.append((o["tokens"].tolist(), o["n_out"].tolist()))
            if compact and k == 3:
                # free the middle request's pages and give them back elsewhere: a hole to fill
                loop.cache.compact()
        assert loop.cache.status() == 0
        answers.append(got)
    assert answers[0] == answers[1]
    # (other page sizes cut the sums elsewhere: the same distribution, compared by its tokens)
    assert answers[0] == answers[2] == answers[3]
