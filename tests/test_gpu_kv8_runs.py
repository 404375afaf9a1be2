"""8-bit paged cache on the GPU: document passes whose CTAs get runs of a single
tile (a stream of the CTA without any), at sizes of a full layer, by the calls' own
split, against the fp64 oracle."""
import pytest

from tests.kv8_util import make_cache, pp
from tests.test_gpu_kv8_attn import run

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
