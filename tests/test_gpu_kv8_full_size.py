"""8-bit paged cache on the GPU at a full layer's sizes, by the calls' own split, a
sample of the rows against the fp64 oracle; and calls timed by events."""
import numpy as np
import pytest
import torch

from tests.kv8_util import make_cache, pp
from tests.test_gpu_kv8_attn import DEV, ids, queries
from tests.test_gpu_kv8_tables import compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,g,d,page,N,P,kind", [
    (32, 1, 128, 32, 16384, 256, "decode"), (8, 4, 128, 16, 12289, 61, "decode"),
    (32, 1, 128, 64, 8192, 64, "decode"), (32, 1, 64, 128, 9000, 70, "decode"),
    (32, 1, 128, 32, 12000, 20, "prefill"), (8, 4, 64, 16, 7777, 20, "prefill"),
])
def test_full_size(H, g, d, page, N, P, kind):
    m = pp()
    rng = np.random.default_rng(N)
    lens = [int(x) for x in rng.integers(16, 49, P)]
    layer, doc, segs = make_cache(H, d, page, N, lens, seed=N)
    if kind == "decode":
        sid = [int(x) + 1 for x in rng.permutation(P)]
        pos = [N + lens[x - 1] - 1 for x in sid]
    else:
        sid = sum(([i + 1] * n for i, n in enumerate(lens)), [])
        pos = sum((list(range(N, N + n)) for n in lens), [])
    R = len(sid)
    q = queries(R, H * g, d, 1)
    s, p = ids(sid, pos)
    fn = m.kv8_decode_attn if kind == "decode" else m.kv8_prefill_attn
    lse = torch.zeros((R, H * g), device=DEV)
    o = fn(layer, N, q, s, p, d ** -0.5, lse=lse, opt=m.Options(wait_limit_log2=26))
    torch.cuda.synchronize()
    assert m.kv8_device_status(layer) == 0 and torch.isfinite(o.float()).all()
    compare(layer, doc, segs, N, q, o, lse, sid, pos, d ** -0.5,
            sorted(set([0, R - 1] + [int(x) for x in rng.permutation(R)[:14]])), kind)
    lse2 = torch.zeros_like(lse)
    o2 = fn(layer, N, q, s, p, d ** -0.5, lse=lse2)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)        # the same bits again


@pytest.mark.parametrize("N", [100, 5000])
def test_events_around_the_passes(N):
    """Events between the two kernels, of which the second may start under the first:
    eagerly and as nodes of a graph, with the same results."""
    m = pp()
    P, H, d = 140, 4, 128
    layer, doc, segs = make_cache(H, d, 32, N, [9] * P, seed=2)
    q = queries(P, H, d, 1)
    s, p = ids(list(range(1, P + 1)), [N + 8] * P)
    want = m.kv8_decode_attn(layer, N, q, s, p, 0.09)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for e in ev:
        e.record()
    opt = m.Options()
    opt.set_events(ev)
    o = m.kv8_decode_attn(layer, N, q, s, p, 0.09, opt=opt)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and 0 <= ev[0].elapsed_time(ev[1]) <= ev[0].elapsed_time(ev[2])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = m.workspace(m.kv8_decode_workspace_bytes(P, H, H, d, N), DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        m.kv8_decode_attn(layer, N, q, s, p, 0.09, o=o, ws=ws, opt=opt)
    for _ in range(3):
        o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        assert 0 <= ev[0].elapsed_time(ev[1]) <= ev[0].elapsed_time(ev[2])
