"""The binding's own host logic around the serving-side calls, on the CPU: the library's work is
replaced by stand-ins that record what they were given."""
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def b():
    from speculative_decoding_draft_03_gb300 import build
    build.build()
    from speculative_decoding_draft_03_gb300 import binding
    return binding


class Streams:
    """Stands for the CUDA streams: which one is current, and on which each buffer was made."""

    def __init__(self, b, monkeypatch):
        self.current, self.made, self.calls, self.capturing = 7, [], [], False
        zeros, empty = torch.zeros, torch.empty

        @contextlib.contextmanager
        def switched(stream):
            before, self.current = self.current, stream
            yield
            self.current = before

        def noting(make):
            def f(*a, **kw):
                t = make(*a, **{**kw, "device": "cpu"})
                self.made.append((self.current, t.numel()))
                return t
            return f

        def attention(q, k, v, table, lens, q_start, max_q, scale, ws=None, stream=None, **kw):
            self.calls.append((stream if stream is not None else self.current, ws))

        monkeypatch.setattr(torch.cuda, "stream", switched)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        monkeypatch.setattr(torch, "zeros", noting(zeros))
        monkeypatch.setattr(torch, "empty", noting(empty))
        monkeypatch.setattr(b, "_raw_stream", lambda s: self.current if s is None else s)
        monkeypatch.setattr(b, "paged_attention", attention)


def _cache(b, slots=32):
    c = object.__new__(b.PagedCache)
    c.page_table, c.seq_len = torch.zeros((slots, 4), dtype=torch.int32), torch.zeros(slots, dtype=torch.int32)
    c.k = c.v = torch.zeros((2, 8, 8, 16, 128), dtype=torch.bfloat16)
    c.k_scale = c.v_scale = None
    c.not_refused = torch.ones(slots, dtype=torch.int32)
    c._attention_ws = {}
    return c


def test_attend_keeps_one_scratch_for_any_number_of_rows(b, monkeypatch):
    c, s = _cache(b), Streams(b, monkeypatch)
    for T in (1, 17, 32, 100, 256):
        c.attend(0, torch.zeros((T, 32, 128), dtype=torch.bfloat16).as_strided((T, 32, 128), (4096, 128, 1)), None, 8, 0.1)
    assert len({ws.data_ptr() for _, ws in s.calls}) == 1 and len(c._attention_ws) == 1
    # one more for each class of query rows, however many sizes there are
    for max_q in range(1, 129):
        c.attend(0, torch.ones((4, 32, 128), dtype=torch.bfloat16), None, max_q, 0.1)
    assert len(c._attention_ws) <= 6


def test_attend_makes_its_scratch_on_the_stream_it_runs_on(b, monkeypatch):
    c, s = _cache(b), Streams(b, monkeypatch)
    q = torch.ones((4, 32, 128), dtype=torch.bfloat16)
    for stream in (None, 11, 12, 11, None):
        s.made.clear()
        c.attend(0, q, None, 4, 0.1, stream=stream)
        assert all(on == (stream or 7) for on, _ in s.made)
    by_stream = {}
    for stream, ws in s.calls:
        by_stream.setdefault(stream, set()).add(ws.data_ptr())
    assert set(by_stream) == {7, 11, 12}
    assert all(len(v) == 1 for v in by_stream.values()) and len(set.union(*by_stream.values())) == 3
    # a capture does not take the scratch of the stream's eager calls
    s.capturing = True
    c.attend(0, q, None, 4, 0.1)
    assert s.calls[-1][1].data_ptr() not in by_stream[7]


def test_attend_clears_only_the_status_block(b):
    ws = b._attention_workspace(5000, "cpu")
    assert ws.numel() == 5000 and ws.data_ptr() % 256 == 0 and (ws[:256] == 0).all()
    assert b._attention_workspace(0, "cpu").numel() == 256


def test_refusals_of_the_granted_form(b):
    """The entry point with `granted` refuses what the one without refuses, and takes a null."""
    import ctypes

    from tests.test_serving_abi import INVALID, OK, P, UNSUPPORTED
    need = b.paged_attention_workspace_size(3, 4, 8, 2, 64, 1)

    def call(T=3, Hq=8, max_q=1, granted=P[9], null=(), scale=0.1):
        p = [None if i in null else x for i, x in enumerate(P)]
        return b.lib.dspark_paged_attention_granted(T, 4, Hq, 2, 64, 64, 16, 8, max_q, 1, 1, p[0], 512, 64, p[1], p[2], 2048,
                                                    1024, 64, p[3], 8, p[4], p[5], granted, scale, None, None, 0, p[6], p[7],
                                                    p[8], need, None)

    assert call(Hq=7) == INVALID and call(max_q=129) == UNSUPPORTED and call(scale=float("inf")) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 6, 8):
        assert call(null=[i]) == INVALID, i
    assert call(T=0, null=[0, 6]) == OK and call(T=0, null=[0, 6], granted=None) == OK


def test_write_refuses_pools_whose_rows_lie_on_one_another(b):
    """Which of two heads' rows such a pool would hold is chance."""
    from tests.test_serving_abi import INVALID, OK, P

    def call(H=2, pages=64, ps=16, strides=(2048, 1024, 64), T=3):
        return b.lib.dspark_cache_write(T, 4, H, 64, pages, ps, 8, 1, 1, P[0], P[1], 128, 64, P[2], P[3], *strides, P[4], 8,
                                        P[5], P[6], None, None, None, P[7], 256, None)

    for strides in ((0, 1024, 64), (2048, 0, 64), (2048, 1024, 0)):
        assert call(strides=strides) == INVALID, strides
        assert "lie on one another" in b.lib.dspark_last_error_message().decode()
        assert call(strides=strides, T=0) == INVALID
    assert call(H=1, pages=1, ps=1, strides=(0, 0, 0), T=0) == OK


def test_calls_of_a_round_do_not_need_the_marshalling_module(b, tmp_path):
    """Importing the binding, and the calls that go through ctypes, work where it is not built; the
    serving-side calls say so."""
    import subprocess
    import sys

    code = f"""
import torch
from speculative_decoding_draft_03_gb300 import build
build.MARSHAL = {str(tmp_path / "none.so")!r}
from speculative_decoding_draft_03_gb300 import binding as b
assert b.schedule_workspace_size(4, 4) > 0 and b.cache_workspace_size(4, 64) > 0
t = torch.zeros(4, dtype=torch.int32)
for path in (build.MARSHAL, {str(tmp_path / "bad.so")!r}):
    build.MARSHAL = path
    try:
        b.cache_truncate(t.view(1, 4), t, t, t, 16, ws=t)
    except b.DSparkError as e:
        assert "_marshal.so" in str(e), e
    else:
        raise AssertionError("not refused")
"""
    (tmp_path / "bad.so").write_bytes(b"not a library")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=b._build.os.path.dirname(b._build.HERE))
    assert r.returncode == 0, r.stderr


def test_another_pytorch_compiles_its_own_marshalling_module(b, monkeypatch, tmp_path):
    import os
    import subprocess
    import types

    build, ran = b._build, []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", os.path.join(tmp_path, "libdspark.so"))
    monkeypatch.setattr(build, "MARSHAL", os.path.join(tmp_path, "_marshal.so"))
    monkeypatch.setattr(subprocess, "run", run)
    build.build(build_dir=str(tmp_path))
    assert sum("marshal.cpp" in a for cmd in ran for a in cmd) == 1
    ran.clear()
    build.build(build_dir=str(tmp_path))
    assert ran == []
    monkeypatch.setattr(torch, "__version__", "99.0")
    build.build(build_dir=str(tmp_path))
    assert [any("marshal.cpp" in a for a in cmd) for cmd in ran].count(True) == 1  # compiled again
    assert any(cmd[cmd.index("-o") + 1].startswith(build.MARSHAL) for cmd in ran)  # and linked
    assert not any(a.endswith(".cu") for cmd in ran for a in cmd)
