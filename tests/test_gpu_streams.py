"""Calls on a stream other than the current one: their scratch and outputs belong to that stream's pool, and calls on
two streams at once, with work of the current stream beside them, give what the same calls give one after another."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_sparse_attention_gb300 import build

    build.build()
    import top_sparse_attention_gb300 as m

    torch.cuda.set_device(0)
    yield m
    torch.cuda.synchronize()
    assert m.dsa_get_device_error() == 0


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _pool_of(t):
    """The stream whose pool holds t's block."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in any pool")


def _tree_inputs(seed, n_seq=2, ctx=9000, N=3, H=16):
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn(n_seq, ctx + N, 576, generator=g).bfloat16().cuda()
    q = torch.randn(n_seq * N, H, 576, generator=g).bfloat16().cuda()
    return q, kv, _i32([ctx, ctx - 100 * seed])


def test_outputs_belong_to_the_stream_of_the_call(dsa):
    s = torch.cuda.Stream()
    q, kv, ctx = _tree_inputs(1)
    f = torch.ones(32, device="cuda")
    x = torch.ones(5, 64, dtype=torch.bfloat16, device="cuda")
    one = _i32([1, 1])
    torch.cuda.synchronize()
    outs = list(dsa.dsa_tree_attn(q, kv, ctx, sm_scale=1 / 24, q_per_seq=3, stream=s))
    outs.append(dsa.dsa_rope(x, _i32(np.arange(5)), f, stream=s))
    outs += dsa.dsa_block_plan(one, one, _i32(np.arange(8)), _i32(np.zeros((2, 4))), block_size=64, num_blocks=8, rows=2, stream=s)
    s.synchronize()
    assert {_pool_of(t) for t in outs} == {s.cuda_stream}
    assert _pool_of(dsa.dsa_rope(x, _i32(np.arange(5)), f)) == torch.cuda.current_stream().cuda_stream


def test_tree_attention_on_two_side_streams_without_a_workspace(dsa):
    cases = [_tree_inputs(k) for k in (1, 2)]
    kw = dict(sm_scale=1 / 24, q_per_seq=3)
    want = [dsa.dsa_tree_attn(q, kv, ctx, **kw) for q, kv, ctx in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for (q, kv, ctx), s in zip(cases, streams):
            got.append(dsa.dsa_tree_attn(q, kv, ctx, stream=s, **kw))
            # the current stream's next allocation of the workspace's size, written at once
            torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for k, (out, lse) in enumerate(got):
        assert torch.equal(out, want[k % 2][0]) and torch.equal(lse, want[k % 2][1])


def test_outputs_of_a_side_stream_outlive_their_last_reader(dsa):
    # `got` is dropped while the current stream still reads it; the side stream's next output may not take its block
    s = torch.cuda.Stream()
    f, pos = torch.ones(32, device="cuda"), _i32(np.arange(1 << 14))
    x = torch.randn(1 << 14, 16, 64, device="cuda").bfloat16()
    want = dsa.dsa_rope(x, pos, f)
    torch.cuda.synchronize()
    sums = []
    for _ in range(10):
        got = dsa.dsa_rope(x, pos, f, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(2_000_000)  # (about a millisecond of waiting in front of the read)
        sums.append(got.clone())
        del got
        dsa.dsa_rope(x, pos, f, inverse=True, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in sums)


def test_chain_entries_on_side_streams_without_workspaces(dsa):
    # the separate entries and the fused call, each with what it allocates itself, two streams in turn, the current
    # stream writing blocks of the same sizes beside them
    import synth

    wl = synth.small_workload("decode_b8_l32k_bf16", T=4, L=9000, K=512, name="streams")
    dev = {k: (v.cuda() if v is not None else None) for k, v in synth.make_inputs(wl).items()}
    kw = dict(K=wl.K, sm_scale=wl.sm_scale, q_per_seq=wl.q_per_seq, q_pos0=wl.q_pos0)
    want, want_lse, want_idx = (t.clone() for t in dsa.call_from_tensors(dev, **kw)())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for k in range(12):
        s = streams[k % 2]
        scores = dsa.dsa_index_score(dev["q_idx"], dev["w"], dev["k_idx"], n_valid=dev["n_valid"], stream=s)
        idx = dsa.dsa_topk(scores, wl.K, L=wl.L, n_valid=dev["n_valid"], stream=s)
        got.append(dsa.dsa_sparse_attn(dev["q"], dev["kv"], idx, sm_scale=wl.sm_scale, stream=s) + (idx,))
        got.append(dsa.call_from_tensors(dev, **kw)(s))  # the call object is dropped at once
        torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    fused = got[1::2]
    for out, lse, idx in fused:
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(idx, want_idx)
    for out, lse, idx in got[0::2]:
        assert torch.equal(idx.sort(1).values, want_idx.sort(1).values)
        assert torch.equal(out, got[0][0]) and (out.float() - want.float()).abs().max() <= 2e-2


def test_calls_on_a_forked_stream_of_a_capture(dsa):
    # scratch and outputs of calls on a side stream inside a capture come from the graph's pool; replays repeat them
    q, kv, ctx = _tree_inputs(3)
    f, pos = torch.ones(32, device="cuda"), _i32(np.arange(6))
    kw = dict(sm_scale=1 / 24, q_per_seq=3)

    def step(stream):
        turned = dsa.dsa_rope(q, pos, f, rot_off=512, stream=stream)
        return (turned,) + dsa.dsa_tree_attn(turned, kv, ctx, stream=stream, **kw)

    want = step(None)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        a = step(side)
        b = step(None)
        main.wait_stream(side)
        c = [t.clone() for t in a]
    for _ in range(3):
        for t in (*a, *b, *c):
            t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        for got in (a, b, c):
            assert all(torch.equal(x, y) for x, y in zip(got, want))
