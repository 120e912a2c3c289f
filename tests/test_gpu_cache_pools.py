"""The page operations over the pools of many layers (more than one kernel's short list of pools
holds), and compaction between the rounds of a serving loop."""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache import Both, _i32
from tests.test_gpu_serving_loop import _loop, _prompts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


@pytest.mark.parametrize("layers", [12, 13, 40, 256])  # 24, 26, 80 and 512 pools
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_rounds_over_many_pools(b, layers, dtype):
    rng = np.random.default_rng(layers)
    c = Both(b, 20, 150, 4, 6, layers, 0.6, H=1, D=16, layers=layers, dtype=dtype)
    for k in range(3):
        empty = [r for r in range(20) if c.m.lens[r] == 0]
        full = [r for r in range(20) if c.m.lens[r] > 0]
        if empty and full:
            c.fork([int(rng.choice(full)) for _ in empty[:4]], empty[:4])
        before = list(c.m.lens)
        granted = c.reserve([int(x) for x in rng.integers(0, 6, 20)])
        c.check()
        c.truncate([n + int(rng.integers(0, g + 1)) for n, g in zip(before, granted)])
        c.truncate([0 if rng.random() < 0.3 else 1 << 30 for _ in range(20)])
        c.compact()
        c.check()


def test_more_pools_than_a_call_takes_are_refused(b):
    c = Both(b, 2, 8, 4, 2, 0, 0.0, H=1, D=16, layers=257)
    with pytest.raises(b.DSparkError):
        b.cache_reserve(*c.args(), _i32([1, 1]), 4, c.pools, ws=c.ws)
    with pytest.raises(b.DSparkError):
        b.cache_compact(*c.args(), 4, c.pools, ws=c.ws)
    c.check()


def test_compaction_that_moves_pages_changes_nothing(b):
    """The same rounds after one request's context went to other pages, with the holes left as they are
    and with every page moved down."""
    answers, moved = [], []
    for compact in (False, True):
        loop = _loop(torch.bfloat16, _prompts([40, 90, 25]), page_size=8, num_pages=96)
        c = loop.cache
        for _ in range(2):
            loop.step()
        # the second request moves: a slot's pages are copied by hand to the last pages of the pool
        n = -(-int(c.seq_len[1]) // 8)
        old, new = c.page_table[1, :n].long(), torch.arange(96 - n, 96, device="cuda")
        for pool in (c.k, c.v):
            pool[:, new] = pool[:, old]
            pool[:, old] = float("nan")
        c.ref_count[new], c.ref_count[old] = 1, 0
        c.page_table[1, :n] = new.int()
        if compact:
            moved.append(c.compact().item())
            used = int((c.ref_count > 0).sum())
            assert moved[0] >= n - 1 and (c.ref_count[:used] == 1).all() and int(c.page_table.max()) == used - 1
        got = []
        for _ in range(6):
            o = loop.step()
            got.append((o["tokens"].tolist(), o["n_out"].tolist(), o["logprob"].nan_to_num().tolist()))
        assert c.status() == 0
        answers.append(got)
    assert moved[0] > 0 and answers[0] == answers[1]
