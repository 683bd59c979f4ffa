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


    def wait_event(self, event):
        event.rec.waits.append((self.cuda_stream, event.at))


class FakeEvent:
    def __init__(self, rec):
        self.rec, self.at = rec, None

    def record(self, stream):
        self.at = stream.cuda_stream


class FakeLib:
    """Every entry succeeds; workspace queries ask for 4096 bytes."""

    def __init__(self, calls):
        self.calls = calls

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            if name in ("dsa_tree_attn_workspace_size", "dsa_workspace_size", "dsa_launch_count"):
                args[-1]._obj.value = 4096
            elif name.endswith("_workspace_size"):
                return 4096
            return 0

        return fn


class Record:
    def __init__(self):
        self.now, self.made, self.back, self.calls, self.waits, self.capturing = CURRENT, [], [], [], [], set()

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
    monkeypatch.setattr(torch.cuda, "Event", lambda: FakeEvent(r))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: r.now in r.capturing)
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


# ---- the other entries: each makes its outputs and, where it has one, a zero-filled workspace

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
OLDER = {
    "dsa_index_score": lambda a, s: [a.dsa_index_score(torch.ones(2, 4, 128, dtype=BF), torch.ones(2, 4), torch.ones(1, 8, 128, dtype=BF), stream=s)],
    "dsa_topk": lambda a, s: [a.dsa_topk(torch.ones(2, 8), 4, L=8, stream=s)],
    "dsa_topk_noalloc": lambda a, s: [a.dsa_topk_noalloc(torch.ones(2, 8), 4, L=8, stream=s)],
    "dsa_topk_pairs": lambda a, s: a.dsa_topk_pairs(torch.ones(2, 8), 4, L=8, pos_offset=0, cand_pos=_i32(2, 4), cand_scores=torch.ones(2, 4), stream=s),
    "dsa_topk_merge": lambda a, s: [a.dsa_topk_merge(torch.ones(2, 8), _i32(2, 8), 4, stream=s)],
    "dsa_sparse_attn": lambda a, s: a.dsa_sparse_attn(torch.ones(2, 4, 576, dtype=BF), torch.ones(1, 8, 576, dtype=BF), _i32(2, 4), sm_scale=1.0, stream=s),
    "dsa_sparse_attn_partial": lambda a, s: a.dsa_sparse_attn_partial(torch.ones(2, 4, 576, dtype=BF), torch.ones(1, 8, 576, dtype=BF), _i32(2, 4), sm_scale=1.0, pos_lo=0, stream=s),
    "dsa_attn_combine": lambda a, s: a.dsa_attn_combine(torch.ones(2, 2, 4, 512), torch.ones(2, 2, 4), stream=s),
    "dsa_quantize_mxfp8": lambda a, s: a.dsa_quantize_mxfp8(torch.ones(2, 64, dtype=BF), stream=s),
    "dsa_quantize_fp8_rows": lambda a, s: a.dsa_quantize_fp8_rows(torch.ones(2, 64, dtype=BF), stream=s),
    "dsa_quantize_fp8_tiles": lambda a, s: a.dsa_quantize_fp8_tiles(torch.ones(2, 64, dtype=BF), stream=s),
}


@pytest.mark.parametrize("name", sorted(OLDER))
def test_the_other_entries_allocate_on_the_stream_they_run_on(rec, name):
    outs = list(OLDER[name](rec.api, FakeStream(SIDE)))  # (torch.ones, the inputs, does not go through the record)
    assert all(s == SIDE for _, s in rec.made)
    made = {t.data_ptr() for t, _ in rec.made}
    assert {(t.data_ptr(), CURRENT) for t in outs if t.data_ptr() in made} <= set(rec.back)
    assert rec.calls[-1][0] == name and rec.calls[-1][1][-1].value == SIDE
    if name in ("dsa_topk", "dsa_topk_pairs", "dsa_sparse_attn", "dsa_sparse_attn_partial"):
        assert any(t.dtype == U8 and t.numel() >= 4096 for t, _ in rec.made)
    rec.made.clear()
    rec.back.clear()
    OLDER[name](rec.api, None)
    assert all(s == CURRENT for _, s in rec.made) and not rec.back


def test_buffers_of_an_object_are_ready_on_every_stream_it_is_called_on(rec):
    a, b = torch.ones(4), torch.ones(5)
    own = rec.api.Owned(a, None, b)
    own.follow(None)
    own.follow(FakeStream(CURRENT))
    assert not rec.waits and not rec.back
    own.follow(FakeStream(SIDE))
    own.follow(FakeStream(SIDE))
    assert rec.waits == [(SIDE, CURRENT)] and rec.back == [(a.data_ptr(), SIDE), (b.data_ptr(), SIDE)]
    rec.now = 33  # another current stream
    own.follow(None)
    assert rec.waits[1:] == [(33, CURRENT)]
    # a capturing stream cannot wait for what is outside of the graph; the first call outside of it does
    rec.capturing = {44}
    own.follow(FakeStream(44))
    assert len(rec.waits) == 2
    rec.capturing = set()
    own.follow(FakeStream(44))
    assert rec.waits[2:] == [(44, CURRENT)]


def test_configured_calls_and_split_steps_follow_the_stream(rec):
    kw = dict(q_idx=torch.ones(2, 4, 128, dtype=BF), w=torch.ones(2, 4), k_idx=torch.ones(1, 8, 128, dtype=BF),
              q=torch.ones(2, 4, 576, dtype=BF), kv=torch.ones(1, 8, 576, dtype=BF), K=4, sm_scale=1.0)
    call = rec.api.DsaCall(**kw)
    call()
    assert not rec.waits
    call(FakeStream(SIDE))
    assert rec.waits == [(SIDE, CURRENT)]
    assert {p for p, s in rec.back if s == SIDE} == {t.data_ptr() for t in (call.out, call.lse, call.idx, call.ws)}
    from top_sparse_attention_gb300 import split

    plan = split.SplitPlan(8, (0, 4, 8))
    caches = [{"k_idx": torch.ones(1, 4, 128, dtype=BF), "k_idx_sf": None, "kv": torch.ones(1, 4, 576, dtype=BF), "kv_scale": None,
               "kv_v": None}] * 2
    whole = split.SplitDecode(plan, caches, K=4, sm_scale=1.0, T=2, H=4, D_v=512)
    rec.back.clear()
    whole(kw["q_idx"], None, kw["w"], kw["q"], stream=FakeStream(SIDE))
    held = {p for p, s in rec.back if s == SIDE}
    for st in whole.steps:
        assert {st.scores.data_ptr(), st.topk_ws.data_ptr(), st.attn_ws.data_ptr()} <= held
    assert {whole.out.data_ptr(), whole.lse.data_ptr(), whole.idx.data_ptr(), whole.o_parts.data_ptr(), whole.cand_pos.data_ptr()} <= held
