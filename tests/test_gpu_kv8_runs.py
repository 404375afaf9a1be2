"""8-bit paged cache on the GPU: document passes whose CTAs get runs of a single
tile (a stream of the CTA without any), at sizes of a full layer, by the calls' own
split, against the fp64 oracle."""
import pytest
import torch

from tests.kv8_util import make_cache, pp
from tests.test_gpu_kv8_attn import DEV, ids, queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,g,rows,d,page,N", [
    (32, 1, 64, 128, 32, 3000), (32, 1, 64, 128, 64, 4096), (64, 1, 40, 128, 16, 2000),
    (32, 1, 64, 64, 16, 4096), (64, 1, 33, 64, 128, 2000), (24, 2, 60, 128, 16, 4200),
])
def test_runs_of_one_tile(H, g, rows, d, page, N):
    m = pp()
    plan = m.kv8_runs(rows, H * g, H, N)
    lone = [i for i, r in enumerate(plan["runs"][:-1])
            if r[5] == 1 and plan["runs"][i + 1][0] == r[0]]
    assert lone                         # a run of one tile with another behind it
    layer, doc, segs = make_cache(H, d, page, N, [3 + i % 9 for i in range(rows)], seed=H + d)
    sid = list(range(1, rows + 1))
    pos = [N + 2 + i % 9 for i in range(rows)]
    opt = m.Options(wait_limit_log2=24)
    for kind in ("decode", "prefill", "decode"):
        run(layer, doc, segs, N, sid, pos, g, kind, opt=opt, what=kind)
        assert m.kv8_device_status(layer) == 0


@pytest.mark.parametrize("kind,rows,P", [("decode", 150, 150), ("prefill", 3000, 60)])
def test_partials_of_the_call_before_are_not_read(kind, rows, P):
    """Two calls in turn on one workspace, whose kernels start under each other: the
    same bits every time, eagerly and in a graph."""
    m = pp()
    N, H = 5000, 4
    lens = [60] * P
    layer, doc, segs = make_cache(H, 128, 32, N, lens, seed=3)
    sid = [1 + i * P // rows for i in range(rows)]
    pos = [N + i % 60 for i in range(rows)]
    s, p = ids(sid, pos)
    q = [queries(rows, H, 128, i) for i in (1, 2)]
    fn = m.kv8_decode_attn if kind == "decode" else m.kv8_prefill_attn
    size = (m.kv8_decode_workspace_bytes if kind == "decode" else m.kv8_prefill_workspace_bytes)(
        rows, H, H, 128, N)
    assert size > 0
    want = []
    for x in q:
        ws = m.workspace(size, DEV)
        ws.fill_(0xff)
        want.append(fn(layer, N, x, s, p, 0.09, ws=ws))
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    outs = [torch.empty_like(want[0]) for _ in range(20)]

    def go():
        for i, o in enumerate(outs):
            fn(layer, N, q[i & 1], s, p, 0.09, o=o, ws=ws)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        go()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        go()
    for _ in range(3):
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert torch.equal(o, want[i & 1])
            o.zero_()
        g.replay()
