"""The latent-layer operators on streams other than the current one, several calls at once, and graphs that share a workspace one after
another: what the same calls give alone."""
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


def calls(dsa, seed):
    """One call of each operator: name -> function of the stream."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    freq, pos = torch.rand(32, generator=g, device="cuda"), _i32(np.arange(500))
    x, rows = rand(500, 7, 192), rand(500, 576)
    pool = torch.zeros(512, 576, dtype=torch.uint8, device="cuda")
    scale = torch.ones(512, 5, device="cuda")
    kv, w, start = rand(2, 700, 576), rand(3, 256, 512), _i32([0, 700, 1300])
    q, kvx, kr, qs = rand(600, 3, 192), rand(1300, 3, 256), rand(1300, 64), _i32([0, 300, 600])
    qt, ctx, one, shared = rand(6, 16, 576), _i32([650, 640]), _i32([0, 2]), _i32([600])
    kv[1, :600] = kv[0, :600]

    def append(s):
        dsa.dsa_norm_rope_append(rows, pos, freq, pool, scale=scale, norm_dim=512, rot_off=512, stream=s)
        return pool, scale

    return {
        "norm": lambda s: (dsa.dsa_norm_rope(x, pos, freq, rot_off=128, stream=s),),
        "append": append,
        "expand": lambda s: dsa.dsa_latent_expand(kv, w, start, rows=1300, stream=s),
        "attn": lambda s: dsa.dsa_expanded_attn(q, kvx[..., :128], kr, kvx[..., 128:], qs, start, sm_scale=0.07, stream=s),
        "prefix": lambda s: dsa.dsa_prefix_attn(qt, kv, ctx, sm_scale=1 / 24, q_per_seq=3, group_start=one, n_shared=shared, stream=s),
    }


NAMES = ["norm", "append", "expand", "attn", "prefix"]


@pytest.mark.parametrize("name", NAMES)
def test_two_side_streams_at_once(dsa, name):
    fns = [calls(dsa, k)[name] for k in (1, 2)]
    want = [[t.clone() for t in f(None)] for f in fns]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for f, s in zip(fns, streams):
            got.append(f(s))
            torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")  # the current stream's next allocation, written at once
    torch.cuda.synchronize()
    for k, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[k % 2]))


def test_all_operators_side_by_side(dsa):
    fns = calls(dsa, 3)
    want = {n: [t.clone() for t in f(None)] for n, f in fns.items()}
    streams = {n: torch.cuda.Stream() for n in fns}
    torch.cuda.synchronize()
    for _ in range(5):
        got = {n: f(streams[n]) for n, f in fns.items()}
    torch.cuda.synchronize()
    for n in fns:
        assert all(torch.equal(a, b) for a, b in zip(got[n], want[n])), n


@pytest.mark.parametrize("name", NAMES)
def test_captured_on_a_forked_stream(dsa, name):
    f = calls(dsa, 4)[name]
    want = [t.clone() for t in f(None)]
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = f(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graphs_that_share_a_workspace_one_after_another(dsa):
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda").random_(0, 256)
    cases = []
    for seed, new, lens in ((5, [300, 20], [900, 4000]), (6, [1, 2, 700], [3000, 2, 700])):
        g = torch.Generator(device="cuda").manual_seed(seed)
        qs, ks = _i32(np.concatenate([[0], np.cumsum(new)])), _i32(np.concatenate([[0], np.cumsum(lens)]))
        q = torch.randn(sum(new), 2, 192, generator=g, device="cuda").bfloat16()
        kv = torch.randn(sum(lens), 2, 256, generator=g, device="cuda").bfloat16()
        kr = torch.randn(sum(lens), 64, generator=g, device="cuda").bfloat16()
        out, lse = torch.zeros(sum(new), 2, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(sum(new), 2, device="cuda")

        def call(q=q, kv=kv, kr=kr, qs=qs, ks=ks, out=out, lse=lse):
            dsa.dsa_expanded_attn(q, kv[..., :128], kr, kv[..., 128:], qs, ks, sm_scale=0.07, out=out, lse=lse, ws=ws)

        call()
        want = out.clone(), lse.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        cases.append((graph, out, lse, want))
    for _ in range(3):
        for graph, out, lse, want in cases:
            out.zero_(), lse.zero_()
            graph.replay()
    torch.cuda.synchronize()
    for _, out, lse, want in cases:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
