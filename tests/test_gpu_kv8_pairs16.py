"""8-bit paged cache on the GPU: calls whose segment items hold sixteen (row, query
head) pairs, which take about 1800 items: thousands of question rows, or decode rows
of many query heads a key head.  Against the fp64 oracle, a sample of the rows."""
import numpy as np
import pytest
import torch

from tests.kv8_util import make_cache, pp
from tests.test_gpu_kv8_attn import DEV, ids, queries
from tests.test_gpu_kv8_tables import compare

pytestmark = pytest.mark.gpu


def sixteen(rows, g, H, N, decode, splits=0):
    plan = pp().kv8_runs(rows, H * g, H, N, decode=decode, splits=splits)
    assert plan["pairs"] == 16 and plan["items"] >= 1776
    return plan


def question_rows(rng, streams, most, rows):
    lens = [int(x) for x in rng.integers(1, most, streams)]
    lens[-1] = max(1, rows - sum(lens[:-1]))
    sid = sum(([i + 1] * n for i, n in enumerate(lens)), [])
    return lens, sid[:rows], sum((list(range(n)) for n in lens), [])[:rows]


# splits: the document read by the segment kernel (None: its own choice), or by a pass of
# so many CTAs: one partial a row, several, two M tiles and one in a row group
CASES = [(H, g, d, rows, N, splits)
         for H, g, d, rows in ((8, 1, 128, 4100), (8, 3, 64, 1700), (4, 8, 128, 1100),
                               (9, 16, 64, 260), (6, 5, 128, 1777))
         for N, splits in ((0, 0), (40, 0), (700, 0), (700, 400), (1300, 5))]


@pytest.mark.parametrize("H,g,d,rows,N,splits", CASES)
def test_question_rows(H, g, d, rows, N, splits):
    m = pp()
    sixteen(rows, g, H, N, False, splits)
    rng = np.random.default_rng(rows + N)
    lens, sid, at = question_rows(rng, 90, 2 * rows // 90 - 2, rows)
    layer, doc, segs = make_cache(H, d, 16, N, lens, seed=rows)
    pos = [N + x for x in at]
    q = queries(rows, H * g, d, 5, pad=1)
    opt = m.Options(splits=splits)
    pick = sorted(set([0, 1, rows - 2, rows - 1] + [int(i) for i in rng.permutation(rows)[:40]]))
    for order in ("runs", "mixed"):
        if order == "mixed":            # any order, idle rows, rows that see none of their segment
            p = rng.permutation(rows)
            sid, pos = [sid[i] for i in p], [pos[i] for i in p]
            for i in range(0, rows, 7):
                sid[i] = -1
            for i in range(3, rows, 11):
                pos[i] = N - 1
        s, p = ids(sid, pos)
        o = torch.full((rows + 1, H * g, d), 9.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((rows + 1, H * g), 9.0, device=DEV)
        m.kv8_prefill_attn(layer, N, q, s, p, d ** -0.5, o=o[:rows], lse=lse[:rows], opt=opt)
        torch.cuda.synchronize()
        assert m.kv8_device_status(layer) == 0
        assert (o[rows:] == 9).all() and (lse[rows:] == 9).all() and torch.isfinite(o.float()).all()
        compare(layer, doc, segs, N, q, o, lse, sid, pos, d ** -0.5, pick, order)


@pytest.mark.parametrize("N,splits", [(0, 0), (30, 0), (900, 0), (900, 300)])
def test_nan_reaches_the_rows_that_see_it_and_no_others(N, splits):
    m = pp()
    H, g, d, rows = 8, 2, 64, 2100
    sixteen(rows, g, H, N, False, splits)
    lens, sid, at = question_rows(np.random.default_rng(N), 50, 80, rows)
    layer, doc, segs = make_cache(H, d, 32, N, lens, seed=N + 1)
    pos = [N + x for x in at]
    q = queries(rows, H * g, d, 6).clone()
    far = max(range(len(lens)), key=lambda i: lens[i])              # a key in the middle of a long stream
    t = lens[far] // 2
    layer.k.view(torch.uint8)[int(layer.seg_table[far, t // 32]), 3, t % 32, 0] = 0x7f
    lone = 1234
    q[lone, 5, 9] = float("inf")                                    # a query, key head 2
    s, p = ids(sid, pos)
    lse = torch.zeros((rows, H * g), device=DEV)
    o = m.kv8_prefill_attn(layer, N, q, s, p, d ** -0.5, lse=lse, opt=m.Options(splits=splits))
    torch.cuda.synchronize()
    want = torch.zeros((rows, H * g), dtype=torch.bool)
    for i in range(rows):
        if sid[i] == far + 1 and at[i] >= t:
            want[i, 6:8] = True
    want[lone, 5] = True
    assert want.sum() > 20
    assert torch.equal(o.isnan().all(-1).cpu(), want) and torch.equal(o.isnan().any(-1).cpu(), want)
    assert torch.equal(lse.isnan().cpu(), want)


def test_partials_that_saw_no_key():
    """Document pages that are not there, over whole runs of the pass."""
    m = pp()
    H, g, d, rows, N = 8, 1, 128, 4000, 1500
    plan = sixteen(rows, g, H, N, False, 600)
    assert plan["max_chunks"] >= 4
    lens, sid, at = question_rows(np.random.default_rng(1), 120, 60, rows)
    layer, doc, segs = make_cache(H, d, 32, N, lens, seed=9)
    gone = [*range(0, 18), *range(30, 35)]              # 16 pages are four tiles
    layer.doc_table[gone] = -1
    keep = torch.ones(N, dtype=torch.bool)
    for i in gone:
        keep[i * 32:(i + 1) * 32] = False
    q = queries(rows, H * g, d, 7)
    s, p = ids(sid, [N + x for x in at])
    lse = torch.zeros((rows, H * g), device=DEV)
    o = m.kv8_prefill_attn(layer, N, q, s, p, d ** -0.5, lse=lse, opt=m.Options(splits=600))
    torch.cuda.synchronize()
    assert m.kv8_device_status(layer) == m.PP_DEV_BAD_PAGE
    n2 = int(keep.sum())
    compare(layer, [x[keep] for x in doc], segs, n2, q, o, lse, sid, [n2 + x for x in at], d ** -0.5,
            list(range(0, rows, 71)), "")


@pytest.mark.parametrize("H,g,d,P,N,splits", [(2, 12, 128, 900, 0, 0), (4, 33, 64, 170, 100, 0),
                                              (2, 16, 128, 900, 1100, 0), (6, 9, 64, 300, 800, 77)])
def test_decode_of_many_query_heads(H, g, d, P, N, splits):
    m = pp()
    sixteen(P, g, H, N, True, splits)
    rng = np.random.default_rng(P)
    lens = [int(x) for x in rng.integers(1, 120, P)]
    layer, doc, segs = make_cache(H, d, 64, N, lens, seed=P)
    sid = [int(x) + 1 for x in rng.permutation(P)]
    pos = [N + lens[x - 1] - 1 for x in sid]
    sid[5] = -1
    q = queries(P, H * g, d, 8)
    s, p = ids(sid, pos)
    lse = torch.zeros((P, H * g), device=DEV)
    o = m.kv8_decode_attn(layer, N, q, s, p, d ** -0.5, lse=lse, opt=m.Options(splits=splits))
    torch.cuda.synchronize()
    assert m.kv8_device_status(layer) == 0 and torch.isfinite(o.float()).all()
    compare(layer, doc, segs, N, q, o, lse, sid, pos, d ** -0.5, list(range(0, P, 13)) + [5], "decode")
