"""What a call given a `stream` allocates comes from that stream's pool (no GPU: streams and launches are fakes that keep
a record).  A block from the current stream's pool would be handed to that stream's next allocation while the kernels on
`stream` still use it."""
import contextlib

import pytest
import torch

CPU = torch.device("cpu")
CURRENT, SIDE = 11, 22


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, CPU


class FakeLib:
    """Every entry succeeds; workspace queries ask for 4096 bytes."""

    def __init__(self, calls):
        self.calls = calls

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            if name == "dsa_tree_attn_workspace_size":
                args[1]._obj.value = 4096
            elif name.endswith("_workspace_size"):
                return 4096
            return 0

        return fn


class Record:
    def __init__(self):
        self.now, self.made, self.back, self.calls = CURRENT, [], [], []

    def streams_of(self, *tensors):
        at = {t.data_ptr(): s for t, s in self.made}
        return [at[t.data_ptr()] for t in tensors]


@pytest.fixture()
def rec(monkeypatch):
    from top_sparse_attention_gb300 import build

    build.build()
    from top_sparse_attention_gb300 import api

    r = Record()

    @contextlib.contextmanager
    def on(stream):
        before, r.now = r.now, stream.cuda_stream
        yield
        r.now = before

    def logged(make):
        def fn(*a, **kw):
            t = make(*a, **kw)
            r.made.append((t, r.now))
            return t

        return fn

    monkeypatch.setattr(torch, "empty", logged(torch.empty))
    monkeypatch.setattr(torch, "zeros", logged(torch.zeros))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream(r.now))
    monkeypatch.setattr(api, "_raw_stream", lambda i: r.now)
    monkeypatch.setattr(api, "_current_device", lambda: None)
    monkeypatch.setattr(api, "_cuda_device", lambda what, t: CPU)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: r.back.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(api.N, "lib", FakeLib(r.calls))
    r.api = api
    return r


def _i32(*shape):
    return torch.ones(*shape, dtype=torch.int32)


def _plan(rec, stream):
    return rec.api.dsa_block_plan(_i32(2), _i32(2), _i32(8), _i32(2, 4), block_size=64, num_blocks=8, rows=5, stream=stream)


def _rope(rec, stream):
    return [rec.api.dsa_rope(torch.ones(3, 64, dtype=torch.bfloat16), _i32(3), torch.ones(32), stream=stream)]


def _tree(rec, stream):
    kv = torch.ones(1, 8, 576, dtype=torch.bfloat16)
    return rec.api.dsa_tree_attn(torch.ones(2, 4, 576, dtype=torch.bfloat16), kv, _i32(1), sm_scale=1.0, q_per_seq=2, stream=stream)


@pytest.mark.parametrize("call", [_plan, _rope, _tree])
def test_serving_step_calls_allocate_on_the_stream_they_run_on(rec, call):
    outs = call(rec, FakeStream(SIDE))
    assert rec.streams_of(*outs) == [SIDE] * len(outs)
    # outputs go back to the caller, whose current stream reads them
    assert {(t.data_ptr(), CURRENT) for t in outs} <= set(rec.back)
    # the workspace: whatever the kernel was given beside the outputs
    assert all(s == SIDE for t, s in rec.made if t.dtype == torch.uint8)
    name, args = rec.calls[-1]
    assert args[-1] == SIDE
    if call is _tree:
        assert any(t.data_ptr() == args[1] and s == SIDE and t.numel() == 4096 for t, s in rec.made)


@pytest.mark.parametrize("call", [_plan, _rope, _tree])
@pytest.mark.parametrize("stream", [None, CURRENT])
def test_serving_step_calls_on_the_current_stream_stay_as_they_are(rec, call, stream):
    outs = call(rec, stream and FakeStream(stream))
    assert rec.streams_of(*outs) == [CURRENT] * len(outs) and not rec.back
    assert rec.calls[-1][1][-1] == CURRENT
