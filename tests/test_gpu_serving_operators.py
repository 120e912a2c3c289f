"""The serving loop's rotary positions, rotated appends, attention of long blocks and adjusted logits
together: what its rounds answer against a dense forward pass over each whole sequence in float64, with
the plain form of the adjustment on its logits.

Tolerance: that of the loop without them (0.15 in a log probability: test_gpu_serving_loop.py) for hidden
states, queries and keys that differ by roundings of 16 bits.  Turned queries and keys are rounded once
more on both sides, of values that differ by 2^-23 relative: only where that crosses a tie do they differ,
by one step.  The repetition penalty multiplies or divides a logit, and so its error, by 1.25 at most, the
others add what is exact beside it: 0.15 x 1.25 < 0.2."""
import math

import numpy as np
import pytest
import torch

from tests import position_ref as ref
from tests.test_gpu_serving_loop import _loop, _prompts

pytestmark = pytest.mark.gpu

PENALTIES = dict(repetition=1.25, frequency=0.5, presence=0.25, bias={7: 2.0, 1000: -1.5, 7000: 9.0, 8: -math.inf})


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _mask(V):
    m = torch.ones(V, dtype=torch.bool)
    m[3::5] = False
    return m


def _answers(loop, prompts, rounds):
    seqs, lps = [list(p) for p in prompts], [[] for _ in prompts]
    for _ in range(rounds):
        o = loop.step()
        for r, n in enumerate(o["n_out"].tolist()):
            seqs[r] += o["tokens"][r, :n].tolist()
            lps[r] += o["logprob"][r, :n].tolist()
    assert loop.cache.status() == 0
    assert loop.cache.seq_len.tolist() == [len(s) - 1 for s in seqs]
    return seqs, lps


def _check(loop, prompts, seqs, lps, mask, tol=0.2):
    for r, seq in enumerate(seqs):
        at, p = len(prompts[r]) - 1, PENALTIES
        x = loop.target.dense(torch.tensor(seq, device="cuda"))[at:-1].cpu().numpy()
        words = np.packbits(np.pad(mask.numpy(), (0, -len(mask) % 32)), bitorder="little").view(np.int32)[None]
        want, _ = ref.adjusted(
            x, np.array(seq[at:-1]), [0, len(seq) - 1 - at], np.array([seq[:at]], dtype=np.int64).reshape(1, -1), [at],
            [len(prompts[r])], [p["repetition"]], [p["frequency"]], [p["presence"]], np.array([list(p["bias"])]),
            np.array([list(p["bias"].values())]), words, np.zeros(len(x), int))
        want = torch.log_softmax(torch.from_numpy(want), 1)[torch.arange(len(x)), torch.tensor(seq[at + 1:])]
        assert (torch.tensor(lps[r]) - want).abs().max() < tol, (r, (torch.tensor(lps[r]) - want).abs().max())


@pytest.mark.parametrize("block", [512, 100])
def test_rounds_answer_what_the_dense_model_says(b, block):
    """Prompts of one block and of several, the blocks above and below what a warp-per-row call takes."""
    prompts = _prompts([700, 2, 129, 513, 40], seed=11)
    mask = _mask(1024)
    loop = _loop(torch.bfloat16, prompts, num_pages=5 * 50, rotary=True, adjust=dict(PENALTIES, mask=mask), block=block)
    seqs, lps = _answers(loop, prompts, 6)
    for seq, p in zip(seqs, prompts):
        said = torch.tensor(seq[len(p):])
        assert mask[said].all() and 8 not in seq[len(p):]  # what the mask or a bias forbids is never answered
    assert sum(map(len, lps)) > 6 * len(prompts)  # some drafts were accepted
    _check(loop, prompts, seqs, lps, mask)


def test_positions_matter_and_shift(b):
    """Without rotary positions the same prompts give other probabilities, by more than the tolerance; an
    8-bit cache keeps the loop's books."""
    prompts = _prompts([300, 50], seed=5)
    probs = []
    for rotary in (False, True):
        loop = _loop(torch.bfloat16, prompts, num_pages=100, rotary=rotary)
        probs.append(torch.log_softmax(loop.target.dense(torch.tensor(prompts[0], device="cuda")), 1))
    assert (probs[0] - probs[1]).abs().max() > 0.5
    loop = _loop(torch.float8_e4m3fn, prompts, num_pages=100, rotary=True, adjust=dict(repetition=1.25))
    _answers(loop, prompts, 4)


def test_a_chunk_and_its_adjustment_in_a_graph(b):
    """A chunk of prompts through append, attention and adjustment, captured once and replayed: the same
    bits as the eager calls, and the same cache."""
    g = torch.Generator(device="cuda").manual_seed(2)
    R, n, Hq, Hkv, D, V = 3, [200, 0, 150], 8, 2, 64, 1000
    T = sum(n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    q, k, v, logits = rnd(T, Hq, D), rnd(T, Hkv, D), rnd(T, Hkv, D), rnd(T, V)
    q_start = i32([0, 200, 200, 350])
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    history = torch.randint(0, V, (R, 64), generator=g, device="cuda", dtype=torch.int32)
    rates = b.rotary_rates(D)
    args = dict(history=history, history_len=i32([64, 0, 9]), repetition=torch.full((R,), 1.25, device="cuda"),
                frequency=torch.full((R,), 0.5, device="cuda"))

    def caches():
        c = b.PagedCache(R, 64, 16, 20, 1, Hkv, D)
        c.reserve(i32(n))
        return c

    def run(c, out, turned, adjusted):
        c.append(0, q, k, v, q_start, rates, q_out=turned)
        c.attend(0, turned, q_start, max(n), D ** -0.5, out=out)
        b.adjust_logits(logits, tokens, q_start, out=adjusted, **args)

    made = lambda: (dict(out=torch.empty_like(q), lse=torch.empty((T, Hq), device="cuda")), torch.empty_like(q),
                    torch.empty_like(logits))
    eager, c0 = made(), caches()
    run(c0, *eager)
    graphed, c1 = made(), caches()
    warm, c2 = made(), caches()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(c2, *warm)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c1, *graphed)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in ((eager[0]["out"], graphed[0]["out"]), (eager[0]["lse"], graphed[0]["lse"]), (eager[1], graphed[1]),
                 (eager[2], graphed[2]), (c0.k, c1.k), (c0.v, c1.v), (eager[0]["out"], warm[0]["out"])):
        assert torch.equal(x, y)
    assert c0.status() == c1.status() == c2.status() == 0
