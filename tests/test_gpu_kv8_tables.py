"""8-bit paged cache on the GPU: page tables with room for far more tokens than the
streams hold, rows of short and long segments side by side in one call, against the
fp64 oracle."""
import numpy as np
import pytest
import torch

from tests.kv8_util import check, make_cache, oracle_attn, pp
from tests.test_gpu_kv8_attn import DEV, ids, queries

pytestmark = pytest.mark.gpu


def compare(layer, doc, segs, N, q, o, lse, sid, pos, scale, rows, what):
    """The rows `rows` of a call against the oracle, over their own streams alone."""
    streams = sorted({sid[i] for i in rows if sid[i] > 0})
    at = {s: i + 1 for i, s in enumerate(streams)}
    ref = oracle_attn(doc, [segs[s - 1] for s in streams], N, q[rows].cpu(),
                      np.array([at.get(sid[i], -1) for i in rows]), np.array([pos[i] for i in rows]),
                      scale)
    check(o[rows], lse[rows], ref, what)


# heads, query heads per head, d, rows: items enough to fill the GPU (base 1 warp an
# item), or half of that (base 2); blocks of four, two or one warps; items of 16 pairs;
# items so many that none is cut
SHAPES = [(16, 1, 128, 256), (8, 10, 64, 350), (5, 1, 128, 400), (8, 4, 64, 230),
          (2, 2, 64, 900), (1, 1, 64, 1800), (7, 3, 64, 150), (3, 12, 128, 600), (6, 12, 64, 300), (4, 9, 128, 460)]


@pytest.mark.parametrize("N,splits", [(0, 0), (150, 0), (300, 37)])
@pytest.mark.parametrize("H,g,d,P", SHAPES)
def test_decode_rows_of_short_and_long_segments(H, g, d, P, N, splits):
    m = pp()
    rng = np.random.default_rng(P + N)
    lens = [int(x) for x in rng.integers(1, 90, P)]
    # around the lengths where a row's items are cut (16 and 32 chunks of 16), to the table's end
    edge = [255, 256, 257, 271, 272, 511, 512, 513, 543, 544, 400, 300]
    for i, n in enumerate(edge):
        lens[i * 9] = n
    layer, doc, segs = make_cache(H, d, 16, N, lens, seed=P, seg_pages=34)
    sid = [int(s) + 1 for s in rng.permutation(P)]
    pos = [N + lens[s - 1] - 1 for s in sid]
    special = [sid.index(i * 9 + 1) for i in range(len(edge))]
    idle = [i for i in range(P) if i not in special][:5]
    sid[idle[0]] = sid[idle[1]] = -1
    pos[idle[0]] = N + 500              # an idle row's position says nothing
    pos[idle[2]] = N - 1                # sees nothing of its segment
    pos[idle[3]] = -2 ** 31
    sid[idle[4]] = -7
    q = queries(P, H * g, d, 3)
    s, p = ids(sid, pos)
    o = torch.full((P + 1, H * g, d), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((P + 1, H * g), 9.0, device=DEV)
    m.kv8_decode_attn(layer, N, q, s, p, d ** -0.5, o=o[:P], lse=lse[:P], opt=m.Options(splits=splits))
    torch.cuda.synchronize()
    assert (o[P:] == 9).all() and (lse[P:] == 9).all() and torch.isfinite(o.float()).all()
    assert m.kv8_device_status(layer) == 0
    some = sorted(set(special + idle + [int(i) for i in rng.permutation(P)[:30]]))
    compare(layer, doc, segs, N, q, o, lse, sid, pos, d ** -0.5, some, "decode")
    # the call again gives the same bits; a stream that is none gives zeros beside it
    sid[special[3]] = 0
    pos[special[4]] = 2 ** 31 - 1       # past its table: all of its slots
    s, p = ids(sid, pos)
    o2 = m.kv8_decode_attn(layer, N, q, s, p, d ** -0.5, opt=m.Options(splits=splits))
    torch.cuda.synchronize()
    assert m.kv8_device_status(layer) == m.PP_DEV_BAD_STREAM
    assert (o2[special[3]] == 0).all()
    same = [i for i in range(P) if i not in (special[3], special[4])]
    assert torch.equal(o2[same], o[same])


@pytest.mark.parametrize("H,g,d", [(8, 1, 128), (4, 3, 64), (2, 8, 128)])
def test_question_rows_with_room_in_their_tables(H, g, d):
    m = pp()
    N, rng = 400, np.random.default_rng(H)
    lens = [int(x) for x in rng.integers(1, 60, 90)] + [500, 3, 333]
    layer, doc, segs = make_cache(H, d, 32, N, lens, seed=H, seg_pages=40)
    sid = sum(([i + 1] * n for i, n in enumerate(lens)), [])
    pos = sum((list(range(N, N + n)) for n in lens), [])
    R = len(sid)
    q = queries(R, H * g, d, 4)
    s, p = ids(sid, pos)
    lse = torch.zeros((R, H * g), device=DEV)
    o = m.kv8_prefill_attn(layer, N, q, s, p, d ** -0.5, lse=lse)
    torch.cuda.synchronize()
    assert m.kv8_device_status(layer) == 0 and torch.isfinite(o.float()).all()
    some = sorted(set([0, R - 1, R - 336] + [int(i) for i in rng.permutation(R)[:60]]))
    compare(layer, doc, segs, N, q, o, lse, sid, pos, d ** -0.5, some, "prefill")


@pytest.mark.parametrize("N", [0, 300, 2000])
@pytest.mark.parametrize("H,g,d,P", [(4, 1, 64, 5), (5, 2, 128, 30), (1, 8, 128, 40), (2, 4, 64, 90),
                                     (3, 3, 128, 1)])
def test_few_decode_rows_with_room_in_their_tables(H, g, d, P, N):
    """Items few enough for sixteen warps each, of rows around the length from which
    they get them (40 chunks of 16), far longer and far shorter."""
    m = pp()
    lens = [[639, 640, 641, 1, 2000, 656, 657, 37, 100, 2047][i % 10] for i in range(P)]
    layer, doc, segs = make_cache(H, d, 16, N, lens, seed=P, seg_pages=128)
    sid = list(range(P, 0, -1))
    pos = [N + lens[x - 1] - 1 for x in sid]
    if P > 3:
        sid[2] = -1
        pos[3] = N - 1
    q = queries(P, H * g, d, 3)
    s, p = ids(sid, pos)
    lse = torch.zeros((P, H * g), device=DEV)
    o = m.kv8_decode_attn(layer, N, q, s, p, d ** -0.5, lse=lse)
    torch.cuda.synchronize()
    assert m.kv8_device_status(layer) == 0
    compare(layer, doc, segs, N, q, o, lse, sid, pos, d ** -0.5, list(range(P)), "decode")
    # a few rows by themselves: the same within the bound, whatever shares a block
    o2 = m.kv8_decode_attn(layer, N, q[:1], s[:1], p[:1], d ** -0.5, lse=lse[:1])
    compare(layer, doc, segs, N, q, o2, lse, sid, pos, d ** -0.5, [0], "one row")
