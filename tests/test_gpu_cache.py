"""The paged cache's page operations against Python lists: which pages are taken and freed,
reference counts, copies on write, moved data (bit for bit), and reported bad tables."""
import numpy as np
import pytest
import torch

from tests.serving_ref import Tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import binding
    return binding


def _i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


class Both:
    """A cache on the GPU and its Python model."""

    def __init__(self, b, R, P, ps, W, seed, fill, H=2, D=16, layers=2, dtype=torch.bfloat16, pad=0):
        rng = np.random.default_rng(seed)
        self.b, self.ps = b, ps
        lens = [int(rng.integers(0, W * ps + 1)) if rng.random() < fill else 0 for _ in range(R)]
        order, at = rng.permutation(P), 0
        table = np.full((R, W), -1)
        for r in range(R):
            n = -(-lens[r] // ps)
            if at + n > P:
                lens[r] = n = 0
            table[r, :n] = order[at:at + n]
            at += n
        ref = np.zeros(P, int)
        ref[table[table >= 0]] = 1
        self.m = Tables(table, lens, ref, ps)
        wide = torch.full((R, W + pad), -7, dtype=torch.int32, device="cuda")
        self.table = wide[:, :W]
        self.table.copy_(_i32(table))
        self.wide = wide
        self.len, self.ref = _i32(lens), _i32(ref)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = [torch.randint(0, 256, (P, H, ps, D * torch.empty(0, dtype=dtype).element_size()), generator=g,
                                   device="cuda", dtype=torch.uint8).view(dtype) for _ in range(2 * layers)]
        self.want = [self.bytes(p).clone() for p in self.pool]
        self.pools = b.cache_pools(self.pool)
        self.ws = b.workspace(b.cache_workspace_size(R, P), "cuda")

    @staticmethod
    def bytes(p):
        return p.view(torch.uint8)

    def args(self):
        return self.table, self.len, self.ref

    def reserve(self, n_new):
        o = self.b.cache_reserve(*self.args(), _i32(n_new), self.ps, self.pools, ws=self.ws)
        granted, copies = self.m.reserve(n_new)
        for a, c in copies:
            if a >= 0:
                for w in self.want:
                    w[c] = w[a]
        assert o["granted"].tolist() == granted
        assert [tuple(x) for x in o["copies"].tolist()] == [tuple(x) for x in copies]
        return granted

    def fork(self, src, dst):
        self.b.cache_fork(*self.args(), _i32(src), _i32(dst), self.ps, ws=self.ws)
        self.m.fork(src, dst)

    def truncate(self, n):
        self.b.cache_truncate(*self.args(), _i32(n), self.ps, ws=self.ws)
        self.m.truncate(n)

    def compact(self):
        n = self.b.cache_compact(*self.args(), self.ps, self.pools, ws=self.ws)
        moves = self.m.compact()
        for a, c in moves:
            for w in self.want:
                w[c] = w[a]
        assert n.item() == len(moves)

    def check(self, status=0):
        assert self.table.tolist() == self.m.table
        assert self.len.tolist() == self.m.lens
        assert self.ref.tolist() == self.m.ref
        assert (self.wide[:, self.table.shape[1]:] == -7).all()
        for p, w in zip(self.pool, self.want):
            assert torch.equal(self.bytes(p), w)
        assert self.b.device_status(self.ws) == status


@pytest.mark.parametrize("R,P,ps,W,pad", [(1, 1, 1, 1, 0), (3, 17, 4, 5, 3), (40, 500, 16, 6, 0), (300, 4096, 8, 7, 1),
                                          (70, 5001, 5, 40, 2), (1100, 33000, 16, 12, 0)])
def test_rounds(b, R, P, ps, W, pad):
    rng = np.random.default_rng(R + P)
    c = Both(b, R, P, ps, W, R, 0.6, pad=pad)
    c.check()
    for k in range(4):
        empty = [r for r in range(R) if c.m.lens[r] == 0]
        full = [r for r in range(R) if c.m.lens[r] > 0]
        if empty and full:
            dst = [int(r) for r in rng.permutation(empty)[: 1 + len(empty) // 2]]
            c.fork([int(rng.choice(full)) for _ in dst], dst)
            c.check()
        before = list(c.m.lens)
        granted = c.reserve([int(x) for x in rng.integers(0, 2 * ps + 2, R)])
        c.check()
        c.truncate([n + int(rng.integers(0, g + 1)) for n, g in zip(before, granted)])
        c.check()
        if k % 2:
            c.truncate([0 if rng.random() < 0.3 else 1 << 30 for _ in range(R)])
            c.check()
            c.compact()
            c.check()
            used = sum(x > 0 for x in c.m.ref)
            assert all(x > 0 for x in c.m.ref[:used])


def test_pool_runs_out_in_slot_order(b):
    c = Both(b, 6, 10, 4, 8, 0, 0.0)
    assert c.reserve([8, 12, 4, 24, 4, 0]) == [8, 12, 4, 0, 0, 0]  # 2+3+1 pages, then 6 of the 4 left
    c.check()
    assert c.reserve([0, 0, 0, 0, 16, 0]) == [0, 0, 0, 0, 16, 0]
    c.check()
    assert c.reserve([1, 0, 0, 0, 0, 1]) == [0, 0, 0, 0, 0, 0]
    c.truncate([7, 1 << 30, 0, 0, 0, 0])
    c.check()
    assert c.reserve([1, 1, 33, 1, 0, 0]) == [1, 1, 0, 1, 0, 0]  # slot 2's row is too short
    c.check()


def test_huge_demands_are_not_granted(b):
    R = 2100  # 2100 slots that ask for 8 pages each of a pool of 50
    table = torch.full((R, 8), -1, dtype=torch.int32, device="cuda")
    lens, ref = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(50, dtype=torch.int32, device="cuda")
    n = torch.full((R,), 8 << 27, dtype=torch.int32, device="cuda")
    n[0] = 1
    o = b.cache_reserve(table, lens, ref, n, 1 << 27, None)
    assert o["granted"].tolist() == [1] + [8 << 27] * 6 + [0] * (R - 7)
    assert ref.sum().item() == 1 + 48


def test_copy_on_write(b):
    c = Both(b, 5, 20, 4, 4, 1, 0.0, dtype=torch.float8_e4m3fn)
    c.reserve([6, 8, 0, 0, 0])
    c.fork([0, 0, 1], [2, 3, 4])
    c.check()
    assert c.m.ref[:4] == [3, 3, 2, 2]
    c.reserve([0, 0, 1, 0, 1])  # slot 2 copies its half-filled page; slot 4's pages are full
    assert c.m.table[2][:2] == [0, 4] and c.m.table[4][:3] == [2, 3, 5]
    c.check()
    c.reserve([2, 0, 0, 2, 0])  # both remaining holders write: each takes a copy
    c.check()
    assert c.m.ref[1] == 0
    c.reserve([0, 0, 1, 1, 0])
    c.check()


def test_bad_tables_are_reported_and_harmless(b):
    for what in ("len", "n_new", "page", "keep", "fork_full", "fork_range", "fork_chain", "fork_twice"):
        c = Both(b, 4, 12, 4, 4, 2, 0.0)
        c.reserve([6, 5, 0, 0])
        c.check()
        table, lens, ref = (x.clone() for x in c.args())
        if what == "len":
            c.len[1] = 17
            o = b.cache_reserve(*c.args(), _i32([1, 1, 0, 0]), 4, c.pools, ws=c.ws)
            assert o["granted"].tolist() == [1, 0, 0, 0]
        elif what == "n_new":
            o = b.cache_reserve(*c.args(), _i32([1, -1, 0, 0]), 4, c.pools, ws=c.ws)
            assert o["granted"].tolist() == [1, 0, 0, 0]
        elif what == "page":
            c.table[1, 1] = 99
            o = b.cache_reserve(*c.args(), _i32([1, 1, 0, 0]), 4, c.pools, ws=c.ws)
            assert o["granted"].tolist() == [1, 0, 0, 0]
            b.cache_truncate(*c.args(), _i32([0, 0, 0, 0]), 4, ws=c.ws)
            assert c.ref.tolist()[:4] == [0, 0, 0, 1]
        elif what == "keep":
            b.cache_truncate(*c.args(), _i32([-3, 9, 9, 9]), 4, ws=c.ws)
            assert c.len.tolist() == [0, 5, 0, 0]
        else:
            src, dst = {"fork_full": ([0], [1]), "fork_range": ([0, 7], [-1, 2]), "fork_chain": ([0, 2], [2, 3]),
                        "fork_twice": ([0, 1], [3, 3])}[what]
            b.cache_fork(*c.args(), _i32(src), _i32(dst), 4, ws=c.ws)
            if what in ("fork_full", "fork_range"):
                assert torch.equal(c.table, table) and torch.equal(c.ref, ref) and torch.equal(c.len, lens)
            else:
                c.m.fork(src, dst)
                assert c.len.tolist() == c.m.lens and c.ref.tolist() == c.m.ref
        assert b.device_status(c.ws, reset=True) == 1, what


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3_bf16", "e4m3_f16"])
@pytest.mark.parametrize("H,D,ps,nhd", [(1, 16, 1, False), (3, 48, 5, False), (2, 128, 16, True), (8, 256, 64, False)])
def test_write(b, kind, H, D, ps, nhd):
    io = torch.float16 if kind.endswith("f16") and not kind.endswith("bf16") else torch.bfloat16
    cache = torch.float8_e4m3fn if kind.startswith("e4m3") else io
    R, W, P = 5, 6, 40
    rng = np.random.default_rng(D + ps)
    new = [0, 1, 3, 2 * ps, 2]
    lens = [7 % (W * ps), 1, 3 + (W - 3) * ps - (ps > 3) * 2, 2 * ps, min(W * ps, 9)]
    lens = [max(n, m) for n, m in zip(lens, new)]
    table = rng.permutation(P)[: R * W].reshape(R, W)
    T = sum(new)
    q_start = np.concatenate([[0], np.cumsum(new)])
    granted = [1, 1, 0, 1, 1]
    g = torch.Generator().manual_seed(D)
    # rows of a wider projection: strided input
    wide = (torch.randn((T + 2, 2 * H, D + 8), generator=g) * 3).to(io)
    wide[0, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0], dtype=io)
    dev = wide.cuda()
    k, v = dev[:, :H, :D], dev[:, H:, :D]
    shape = (P, ps, H, D) if nhd else (P, H, ps, D)
    pools = [torch.zeros(shape, dtype=torch.uint8, device="cuda").to(cache) if cache != torch.float8_e4m3fn
             else torch.zeros(shape, dtype=torch.uint8, device="cuda").view(cache) for _ in range(2)]
    view = [p.permute(0, 2, 1, 3) if nhd else p for p in pools]
    scales = None
    if cache == torch.float8_e4m3fn:
        scales = [torch.rand(H, generator=g) * 0.05 + 0.01 for _ in range(2)]
    ws = b.workspace(256, "cuda")
    b.cache_write(k, v, view[0], view[1], _i32(table), _i32(lens), _i32(q_start), granted=_i32(granted),
                  k_scale=scales and scales[0].cuda(), v_scale=scales and scales[1].cuda(), ws=ws)
    assert b.device_status(ws) == 0
    for which in range(2):
        want = torch.zeros((P, H, ps, D), dtype=torch.uint8).view(cache) if cache == torch.float8_e4m3fn else \
            torch.zeros((P, H, ps, D), dtype=cache)
        raw = want.view(torch.uint8).view(P, H, ps, -1)
        for r in range(R):
            if not granted[r]:
                continue
            for i in range(new[r]):
                pos = lens[r] - new[r] + i
                x = wide[q_start[r] + i, which * H:(which + 1) * H, :D]
                if scales:
                    x = (x.float() / scales[which][:, None]).clamp(-448, 448)
                raw[table[r, pos // ps], :, pos % ps] = x.to(cache).contiguous().view(torch.uint8).view(H, -1)
        got = view[which].contiguous().cpu()
        same = got.view(torch.uint8).view(P, H, ps, -1) == raw
        if not same.all():  # NaN has several patterns
            a, c = got.float(), want.float()
            assert torch.equal(a.isnan(), c.isnan()) and torch.equal(a.nan_to_num(), c.nan_to_num())


def test_write_of_few_among_many(b):
    """Rows of no slot before the first and past the last, empty slots between, and many slots: a
    warp's tokens lie in different slots."""
    for R, lead, tail in ((1, 2, 1), (37, 1, 3), (1100, 5, 0), (4000, 3, 2)):
        rng = np.random.default_rng(R)
        new = (rng.random(R) < 0.4) * rng.integers(1, 4, R)
        T = int(new.sum())
        q_start = lead + np.concatenate([[0], np.cumsum(new)])
        table = np.arange(R)[:, None]
        k = torch.arange(1, lead + T + tail + 1, device="cuda").float().view(-1, 1, 1).expand(-1, 1, 16)
        k = (k % 251).bfloat16().contiguous()
        pool = [torch.zeros((R, 1, 4, 16), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        ws = b.workspace(256, "cuda")
        b.cache_write(k, -k, pool[0], pool[1], _i32(table), _i32(new), _i32(q_start), ws=ws)
        assert b.device_status(ws) == 0
        want = torch.zeros((R, 1, 4, 16))
        for r in range(R):
            for i in range(new[r]):
                want[r, 0, i] = float((q_start[r] + i + 1) % 251)
        assert torch.equal(pool[0].float().cpu(), want) and torch.equal(pool[1].float().cpu(), -want)


def test_write_reports_bad_places(b):
    pool = torch.zeros((4, 1, 4, 16), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((3, 1, 16), dtype=torch.bfloat16, device="cuda")
    for lens, table, q in (([2], [[0, 1]], [0, 3]), ([9], [[0, 1]], [0, 3]), ([8], [[0, 9]], [0, 3]),
                           ([8], [[0, -1]], [0, 3])):
        ws = b.workspace(256, "cuda")
        pool.zero_()
        b.cache_write(x, x, pool, pool, _i32(table), _i32(lens), _i32(q), ws=ws)
        assert b.device_status(ws) == 1, (lens, table)
        assert pool[1:].sum().item() == 0 or lens == [9]
    b.cache_write(x[:0], x[:0], pool, pool, _i32([[0, 1]]), _i32([3]), _i32([0, 0]))


def test_graph_and_stream(b):
    """A serving round's cache calls, captured: the replay gives what the eager calls give."""
    def make():
        c = b.PagedCache(6, 64, 8, 6, 2, 2, 32)
        c.reserve(_i32([5, 9, 0, 16, 1, 0]))
        return c

    g = torch.Generator().manual_seed(1)
    new = _i32([1, 3, 0, 2, 4, 5])
    q_start = _i32(np.concatenate([[0], np.cumsum([1, 3, 0, 2, 4, 5])]))
    k, v = (torch.randn((15, 2, 32), generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn((15, 4, 32), generator=g).bfloat16().cuda()
    src, dst, keep = _i32([3]), _i32([2]), _i32([6, 10, 16, 17, 2, 3])

    def step(c):
        c.fork(src, dst)
        c.reserve(new)
        for n in range(2):
            c.write(n, k, v, q_start)
        o = c.attend(0, q, q_start, 5, 0.2)
        c.truncate(keep)
        c.compact()
        return o

    eager, graphed = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step(eager)
    side.synchronize()
    graphed.attend(0, q, q_start, 5, 0.2)  # makes the workspace
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(graphed)
    graph.replay()
    torch.cuda.synchronize()
    for a in ("page_table", "seq_len", "ref_count", "k", "v"):
        assert torch.equal(getattr(eager, a), getattr(graphed, a)), a
    assert torch.equal(want["out"], got["out"]) and torch.equal(want["lse"], got["lse"])
    assert eager.status() == 0 and graphed.status() == 0
