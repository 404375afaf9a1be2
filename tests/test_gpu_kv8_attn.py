"""8-bit paged cache on the GPU: decode and question prefill attention against
the fp64 oracle over the dequantised rows."""
import numpy as np
import pytest
import torch

from tests.kv8_util import check, make_cache, oracle_attn, pp

pytestmark = pytest.mark.gpu
DEV = "cuda"


def queries(rows, Hq, d, seed, pad=0):
    """Query rows, `pad` further heads between them (a fused projection's)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, Hq + pad, d), generator=g).to(torch.bfloat16).to(DEV)
    return x[:, :Hq]


def ids(sid, pos):
    return (torch.tensor(sid, dtype=torch.int16, device=DEV),
            torch.tensor(pos, dtype=torch.int32, device=DEV))


def run(layer, doc, segs, N, sid, pos, g, kind, seed=1, doc_len=None, pad=0, what="", opt=None):
    m = pp()
    rows, Hq = len(sid), layer.H * g
    q = queries(rows, Hq, layer.d, seed, pad)
    qs, qp = ids(sid, pos)
    scale = layer.d ** -0.5
    o = torch.full((rows + 2, Hq, layer.d), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((rows + 2, Hq), 9.0, device=DEV)
    fn = m.kv8_decode_attn if kind == "decode" else m.kv8_prefill_attn
    dl = N if doc_len is None else doc_len
    fn(layer, dl, q, qs, qp, scale, o=o[:rows], lse=lse[:rows], opt=opt)
    torch.cuda.synchronize()
    assert (o[rows:] == 9).all() and (lse[rows:] == 9).all()     # rows behind the last one
    ref = oracle_attn(doc, segs, N, q.cpu(), np.array(sid), np.array(pos), scale, dl)
    check(o[:rows], lse[:rows], ref, what)
    return q, o[:rows], lse[:rows]


# heads, query heads per head, d, page, document, streams
SHAPES = [
    (1, 1, 64, 16, 1, 1), (2, 1, 128, 16, 0, 5), (4, 2, 64, 16, 257, 16), (3, 7, 128, 32, 1001, 9),
    (2, 4, 128, 64, 130, 61), (1, 16, 64, 128, 300, 3), (1, 33, 128, 16, 129, 4),
    (8, 1, 128, 32, 640, 130), (2, 3, 64, 64, 2049, 100), (2, 8, 128, 16, 999, 70),
]


# splits: the document pass is taken, however small the work
@pytest.mark.parametrize("splits", [0, 37])
@pytest.mark.parametrize("H,g,d,page,N,P", SHAPES)
def test_decode(H, g, d, page, N, P, splits):
    opt = pp().Options(splits=splits)
    rng = np.random.default_rng(N + P)
    lens = [int(x) for x in rng.integers(1, 90, P)]
    layer, doc, segs = make_cache(H, d, page, N, lens, seed=N)
    sid = [s + 1 for s in rng.permutation(P)]
    pos = [N + lens[s - 1] - 1 for s in sid]
    run(layer, doc, segs, N, sid, pos, g, "decode", opt=opt, pad=1)
    assert pp().kv8_device_status(layer) == 0
    sid[0] = -1                          # inactive rows, rows that see nothing of their segment
    if P > 2:
        sid[2] = -1
        pos[1] = N - 1
    run(layer, doc, segs, N, sid, pos, g, "decode", opt=opt, seed=2)
    run(layer, doc, segs, N, sid, pos, g, "decode", opt=opt, seed=3, doc_len=0)
    if N > 3:                            # a document read in part
        run(layer, doc, segs, N, sid, pos, g, "decode", opt=opt, seed=3, doc_len=N - 3)
    assert pp().kv8_device_status(layer) == 0


@pytest.mark.parametrize("splits", [0, 37])
@pytest.mark.parametrize("H,g,d,page,N,P", SHAPES)
def test_prefill(H, g, d, page, N, P, splits):
    opt = pp().Options(splits=splits)
    rng = np.random.default_rng(N + P)
    lens = [int(x) for x in rng.integers(1, 40, P)]
    layer, doc, segs = make_cache(H, d, page, N, lens, seed=N + 1)
    order = rng.permutation(P)
    sid = sum(([int(s) + 1] * lens[s] for s in order), [])
    pos = sum((list(range(N, N + lens[s])) for s in order), [])
    run(layer, doc, segs, N, sid, pos, g, "prefill", opt=opt, pad=2)
    # any order, idle rows among them, a part of the rows only
    mix = rng.permutation(len(sid))[:max(1, len(sid) * 2 // 3)]
    sid, pos = [sid[i] if i % 7 else -1 for i in mix], [pos[i] for i in mix]
    run(layer, doc, segs, N, sid, pos, g, "prefill", opt=opt, seed=4)
    run(layer, doc, segs, N, sid, pos, g, "prefill", opt=opt, seed=5, doc_len=0)
    assert pp().kv8_device_status(layer) == 0


def test_more_rows_than_one_group():
    """Row groups of 256 (row, head) pairs, the last one partly filled."""
    lens = [20] * 30
    layer, doc, segs = make_cache(2, 128, 32, 700, lens, seed=3)
    sid = sum(([s + 1] * 20 for s in range(30)), [])[:-7]
    pos = (list(range(700, 720)) * 30)[:-7]
    for splits in (0, 5):
        opt = pp().Options(splits=splits)
        run(layer, doc, segs, 700, sid, pos, 1, "prefill", opt=opt)
        run(layer, doc, segs, 700, sid, pos, 3, "prefill", opt=opt)


def test_long_segments():
    lens = [1, 1500, 3, 700, 64]
    layer, doc, segs = make_cache(2, 64, 16, 50, lens, seed=5)
    sid = [1, 2, 3, 4, 5]
    run(layer, doc, segs, 50, sid, [50 + n - 1 for n in lens], 4, "decode")
    run(layer, doc, segs, 50, [2] * 40 + [4] * 3, list(range(1510, 1550)) + [749, 50, 700], 2, "prefill")


def test_all_rows_idle_and_no_rows():
    m = pp()
    layer, doc, segs = make_cache(2, 64, 16, 40, [3, 4], seed=6)
    run(layer, doc, segs, 40, [-1, -1], [0, 0], 2, "decode")
    run(layer, doc, segs, 40, [-1], [0], 2, "prefill")
    q = queries(0, 4, 64, 1)
    s, p = ids([], [])
    assert m.kv8_decode_attn(layer, 40, q, s, p, 0.1).shape == (0, 4, 64)


def test_rows_of_no_stream_are_zero_and_reported():
    m = pp()
    layer, doc, segs = make_cache(2, 64, 16, 300, [3, 4, 5], seed=7)
    for fn in (m.kv8_decode_attn, m.kv8_prefill_attn):
        q = queries(3, 2, 64, 1)
        s, p = ids([0, 4, 2], [300, 300, 302])
        lse = torch.zeros((3, 2), device=DEV)
        o = fn(layer, 300, q, s, p, 0.125, lse=lse)
        torch.cuda.synchronize()
        assert m.kv8_device_status(layer) == m.PP_DEV_BAD_STREAM
        m.kv8_reset(layer)
        assert (o[:2] == 0).all() and (lse[:2] == -torch.inf).all()
        ref = oracle_attn(doc, segs, 300, q.cpu()[2:], np.array([2]), np.array([302]), 0.125)
        check(o[2:], lse[2:], ref)


@pytest.mark.parametrize("N", [40, 700])
def test_pages_that_are_not_there_are_skipped(N):
    m = pp()
    layer, doc, segs = make_cache(2, 128, 16, N, [40, 20], seed=8)
    layer.doc_table[1] = -1
    layer.doc_table[2] = layer.n_pages
    layer.seg_table[0, 1] = -7
    keep = torch.ones(N, dtype=torch.bool)
    keep[16:48] = False
    doc2 = [x[keep] for x in doc]
    ks = torch.ones(40, dtype=torch.bool)
    ks[16:32] = False
    segs2 = [[x[ks] for x in segs[0]], segs[1]]
    q = queries(2, 4, 128, 1)
    s, p = ids([1, 2], [N + 39, N + 19])
    n2 = int(keep.sum())
    for fn, splits in ((f, n) for f in (m.kv8_decode_attn, m.kv8_prefill_attn) for n in (0, 3)):
        lse = torch.zeros((2, 4), device=DEV)
        o = fn(layer, N, q, s, p, 0.09, lse=lse, opt=m.Options(splits=splits))
        torch.cuda.synchronize()
        assert m.kv8_device_status(layer) == m.PP_DEV_BAD_PAGE
        m.kv8_reset(layer)
        ref = oracle_attn(doc2, segs2, n2, q.cpu(), np.array([1, 2]), np.array([n2 + 39, n2 + 19]), 0.09)
        check(o, lse, ref)


@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("N", [40, 900])
@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_nan_reaches_the_rows_that_see_it_and_no_others(N, kind, splits):
    m = pp()
    layer, doc, segs = make_cache(2, 64, 32, N, [30, 30, 30], seed=9)
    fn = m.kv8_decode_attn if kind == "decode" else m.kv8_prefill_attn
    q = queries(3, 4, 64, 1)
    s, p = ids([1, 2, 3], [N + 19, N + 20, N + 29])
    scale = 0.125

    def go():
        lse = torch.zeros((3, 4), device=DEV)
        o = fn(layer, N, q, s, p, scale, lse=lse, opt=m.Options(splits=splits))
        torch.cuda.synchronize()
        return o, lse

    # key 20 of stream 2, head 1: its row sees it, nobody else does
    pg = int(layer.seg_table[1, 0])
    layer.k.view(torch.uint8)[pg, 1, 20, 0] = 0x7f
    pg = int(layer.seg_table[0, 0])
    layer.k.view(torch.uint8)[pg, 0, 20, 0] = 0x7f       # behind row 0's position
    o, lse = go()
    assert o[1, 2:].isnan().all() and lse[1, 2:].isnan().all()
    o[1, 2:], lse[1, 2:] = 0, 0
    assert not o.isnan().any() and not lse.isnan().any()
    ref = oracle_attn(doc, segs, N, q.cpu()[[0, 2]], np.array([1, 3]), np.array([N + 19, N + 29]), scale)
    check(o[[0, 2]], lse[[0, 2]], ref)
    # a document key: everybody in its head
    layer.k.view(torch.uint8)[int(layer.doc_table[N // 32]), 0, N % 32 - 1, 0] = 0x7f
    o, lse = go()
    assert o[:, :2].isnan().all() and lse[:, :2].isnan().all()
    assert not o[0, 2:].isnan().any() and not o[2, 2:].isnan().any()


@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("N", [0, 40, 900])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_queries_give_nan_in_their_row(N, bad, splits):
    m = pp()
    layer, doc, segs = make_cache(2, 64, 32, N, [30, 30, 30], seed=9)
    q = queries(3, 4, 64, 1)
    q[1, 2, 60] = bad
    s, p = ids([1, 2, 3], [N + 19, N + 20, N + 29])
    for fn in (m.kv8_decode_attn, m.kv8_prefill_attn):
        lse = torch.zeros((3, 4), device=DEV)
        o = fn(layer, N, q, s, p, 0.125, lse=lse, opt=m.Options(splits=splits))
        torch.cuda.synchronize()
        assert o[1, 2].isnan().all() and lse[1, 2].isnan()
        o[1, 2], lse[1, 2] = 0, 0
        assert not o.isnan().any() and not lse.isnan().any()


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("d,N", [(64, 100), (128, 1500)])
def test_scales_far_apart_and_large_scores(d, N, splits):
    """Pages 2^-30 to 2^30 apart in value scale; keys large enough that one key
    takes all the weight."""
    m = pp()
    layer, doc, segs = make_cache(1, d, 16, N, [50, 20], seed=10)
    g = torch.Generator().manual_seed(3)
    e = torch.randint(-30, 31, layer.v_scale.shape, generator=g).float()
    old = layer.v_scale.cpu()
    layer.v_scale.copy_(torch.exp2(e - 6))
    ratio = torch.exp2(e - 6) / old
    layer.k_scale *= 16

    def scaled(x, tab, n):
        f = ratio[tab.cpu().long()][:, :, None, None].expand(-1, -1, 16, d)
        return x * f.transpose(1, 2).reshape(-1, 1, d)[:n]

    doc = [doc[0] * 16, scaled(doc[1], layer.doc_table, N)]
    segs = [[sg[0] * 16, scaled(sg[1], layer.seg_table[i], len(sg[0]))] for i, sg in enumerate(segs)]
    q = queries(2, 3, d, 1)
    s, p = ids([1, 2], [N + 49, N + 19])
    lse = torch.zeros((2, 3), device=DEV)
    o = m.kv8_decode_attn(layer, N, q, s, p, d ** -0.5, lse=lse, opt=m.Options(splits=splits))
    torch.cuda.synchronize()
    ro, rl, ra = oracle_attn(doc, segs, N, q.cpu(), np.array([1, 2]), np.array([N + 49, N + 19]), d ** -0.5)
    # scores reach |q||k| scale ~ 600: their fp32 sums err by up to 2^-24 * 128
    # terms * 600 ~ 2^-8 in the worst case, so probabilities by 2^-8 relative in
    # numerator and denominator (and lse by as much), beside check()'s bound
    err = np.abs(o.float().cpu().numpy() - ro)
    assert np.isfinite(o.float().cpu().numpy()).all()
    assert (err <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -7 + 2.0 ** -10 + 2.0 ** -12) * ra + 1e-30).all()
    assert np.abs(lse.cpu().numpy() - rl).max() <= 2.0 ** -8


def test_one_workspace_serves_calls_in_order_and_graphs_replay():
    m = pp()
    N, P = 3100, 140
    lens = [10 + i % 50 for i in range(P)]
    layer, doc, segs = make_cache(2, 128, 32, N, lens, seed=11)
    q = queries(P, 4, 128, 1)
    s, p = ids(list(range(1, P + 1)), [N + n - 1 for n in lens])
    n_ws = max(m.kv8_decode_workspace_bytes(P, 4, 2, 128, N), m.kv8_prefill_workspace_bytes(P, 4, 2, 128, N))
    ws = m.workspace(n_ws, DEV)
    ws.fill_(0xff)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        want = m.kv8_decode_attn(layer, N, q, s, p, 0.09, ws=ws)
        want2 = m.kv8_prefill_attn(layer, N, q, s, p, 0.09, ws=ws)
        again = m.kv8_decode_attn(layer, N, q, s, p, 0.09, ws=ws)
    st.synchronize()
    assert torch.equal(want, again)
    o, o2 = torch.empty_like(want), torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        m.kv8_decode_attn(layer, N, q, s, p, 0.09, o=o, ws=ws)
        m.kv8_prefill_attn(layer, N, q, s, p, 0.09, o=o2, ws=ws)
    for _ in range(2):
        o.zero_()
        o2.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(o2, want2)
    ref = oracle_attn(doc, segs, N, q.cpu(), s.cpu().numpy(), p.cpu().numpy(), 0.09)
    check(want, None, ref)
    check(want2, None, ref)
    # calls at once on two streams, each with its own workspace
    st2, ws2 = torch.cuda.Stream(), m.workspace(n_ws, DEV)
    st2.wait_stream(torch.cuda.current_stream())
    st.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        with torch.cuda.stream(st):
            m.kv8_decode_attn(layer, N, q, s, p, 0.09, o=o, ws=ws)
        with torch.cuda.stream(st2):
            m.kv8_prefill_attn(layer, N, q, s, p, 0.09, o=o2, ws=ws2)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(o2, want2)


def test_serving_run():
    """A document, its questions and some answer tokens through append, prefill
    and decode, as a program would run them; each attention against the oracle
    over the cache's own dequantised rows."""
    from oracle.kv8 import Kv8Replay
    m = pp()
    H, g, d, page, N, P = 2, 4, 64, 16, 345, 6
    gen = torch.Generator().manual_seed(12)
    rope = m.Rope.make(N + 100, d, device=DEV)
    seg_pages, doc_pages = 5, -(-N // page)
    tab = torch.randperm(doc_pages + P * seg_pages, generator=gen).to(torch.int32)
    layer = m.KV8Layer(H, d, page, doc_pages + P * seg_pages, P, seg_pages, doc_pages, N, DEV,
                       doc_table=tab[:doc_pages].to(DEV),
                       seg_table=tab[doc_pages:].view(P, seg_pages).contiguous().to(DEV))
    rep = Kv8Replay(H, d, page, layer.n_pages, N, tab[:doc_pages].numpy(),
                    tab[doc_pages:].view(P, seg_pages).numpy())
    have = [0] * P

    def step(sid, pos, fn):
        x = torch.randn((len(sid), (g + 2) * H, d), generator=gen).to(torch.bfloat16).to(DEV)
        q, k, v = x[:, :g * H], x[:, g * H:(g + 1) * H], x[:, (g + 1) * H:]
        s, p = ids(sid, pos)
        qr = m.kv8_append(layer, k, v, s, p, rope=rope, q=q)
        rep.append(k.float().cpu().numpy(), v.float().cpu().numpy(), sid, pos, rope.cos_sin.cpu().numpy())
        if fn is None:
            return
        for i in sid:
            have[i - 1] += 1
        lse = torch.empty((len(sid), g * H), device=DEV)
        o = fn(layer, N, qr, s, p, 0.125, lse=lse)
        torch.cuda.synchronize()
        doc = [torch.from_numpy(x).float() for x in rep.rows(0, N)]
        segs = [[torch.from_numpy(x).float() for x in rep.rows(i + 1, have[i])] for i in range(P)]
        check(o, lse, oracle_attn(doc, segs, N, qr.cpu(), np.array(sid), np.array(pos), 0.125))

    step([0] * N, list(range(N)), None)
    lens = [5, 17, 1, 32, 16, 9]
    step(sum(([i + 1] * n for i, n in enumerate(lens)), []), sum((list(range(N, N + n)) for n in lens), []),
         m.kv8_prefill_attn)
    for t in range(6):
        act = [i for i in range(P) if (i + t) % 5]
        step([i + 1 for i in act], [N + have[i] for i in act], m.kv8_decode_attn)
    assert m.kv8_device_status(layer) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_injected_timeout_reports_status_and_recovers(d):
    """A copy of the document pass that never lands: its waits run out, the call
    ends, the status says so, and the next call is right."""
    m = pp()
    N, P = 3000, 150
    layer, doc, segs = make_cache(2, d, 16, N, [9] * P, seed=13)
    sid, pos = list(range(1, P + 1)), [N + 8] * P
    q = queries(P, 2, d, 1)
    s, p = ids(sid, pos)
    opt = m.Options(debug_inject_timeout=1, wait_limit_log2=22)
    m.kv8_decode_attn(layer, N, q, s, p, 0.1, opt=opt)
    torch.cuda.synchronize()
    assert m.kv8_device_status(layer) & m.PP_DEV_TIMEOUT
    m.kv8_reset(layer)
    run(layer, doc, segs, N, sid, pos, 1, "decode", opt=m.Options(splits=60))
    assert m.kv8_device_status(layer) == 0


@pytest.mark.parametrize("splits", [1, 2, 5, 40, 1000])
def test_any_split_of_the_document_gives_the_same(splits):
    m = pp()
    N, P = 2100, 90
    layer, doc, segs = make_cache(2, 128, 64, N, [9] * P, seed=14)
    sid, pos = list(range(1, P + 1)), [N + 8] * P
    run(layer, doc, segs, N, sid, pos, 1, "decode", opt=m.Options(splits=splits))
    run(layer, doc, segs, N, sid, pos, 5, "decode", opt=m.Options(splits=splits))


@pytest.mark.parametrize("P,page,splits", [(40, 16, 3), (40, 128, 0), (300, 32, 7), (300, 64, 0)])
def test_long_documents_of_64_dims(P, page, splits):
    """Many tiles a run, keys and values brought in by separate warps; the last
    tile ends inside a page."""
    m = pp()
    N = 6001
    layer, doc, segs = make_cache(2, 64, page, N, [5] * P, seed=P + page)
    sid, pos = list(range(1, P + 1)), [N + 4] * P
    run(layer, doc, segs, N, sid, pos, 1, "decode", opt=m.Options(splits=splits) if splits else None)
    assert m.kv8_device_status(layer) == 0


def test_pool_past_four_gib():
    """Pages that lie more than 4 GiB behind the pool's first, read by both
    kernels."""
    m = pp()
    H, d, page, N, g = 32, 128, 128, 400, 1
    n_pages = (1 << 32) // (H * d * page) + 8
    f8 = torch.float8_e4m3fn
    k = torch.empty((n_pages, H, page, d), dtype=torch.uint8, device=DEV).view(f8)
    v = torch.empty((n_pages, H, page, d), dtype=torch.uint8, device=DEV).view(f8)
    far = [n_pages - 1, 1, n_pages - 3, n_pages // 2 + 1]
    seg = [n_pages - 2, n_pages - 5]
    gen = torch.Generator().manual_seed(5)
    ks = torch.ones((n_pages, H), device=DEV)
    vs = torch.ones((n_pages, H), device=DEV)
    rows = {}
    for pg in far + seg:
        for t, pool, sc in (("k", k, ks), ("v", v, vs)):
            x = torch.randn((H, page, d), generator=gen).mul(64).clamp(-448, 448).to(f8)
            pool[pg].view(torch.uint8).copy_(x.view(torch.uint8))
            sc[pg] = 2.0 ** -6
            rows[t, pg] = x.float().mul(2.0 ** -6).transpose(0, 1)       # [page, H, d]
    layer = m.KV8Layer(H, d, page, n_pages, 2, 1, 4, N, DEV, k=k, v=v, k_scale=ks, v_scale=vs,
                       doc_table=torch.tensor(far, dtype=torch.int32, device=DEV),
                       seg_table=torch.tensor([[p] for p in seg], dtype=torch.int32, device=DEV))
    doc = [torch.cat([rows[t, p] for p in far])[:N] for t in "kv"]
    segs = [[rows[t, p][:n] for t in "kv"] for p, n in zip(seg, (100, 128))]
    for splits in (0, 20):
        run(layer, doc, segs, N, [1, 2], [N + 99, N + 127], g, "decode", opt=m.Options(splits=splits))
        run(layer, doc, segs, N, [2] * 9 + [1], list(range(N + 119, N + 128)) + [N + 40], g, "prefill",
            opt=m.Options(splits=splits))


def test_many_pairs_of_one_row():
    """More query heads per key head than a row group has rows."""
    layer, doc, segs = make_cache(1, 64, 32, 500, [40, 3], seed=21)
    for splits in (0, 4):
        run(layer, doc, segs, 500, [1, 2], [539, 502], 300, "decode", opt=pp().Options(splits=splits))


def test_maximum_that_keeps_rising():
    """Keys that grow tile by tile, and a last tile far above: references are
    raised again and again, also where only some rows of a warp are."""
    m = pp()
    N, d, page = 1280, 128, 16
    layer, doc, segs = make_cache(1, d, page, N, [9] * 40, seed=22, spread=0)
    grow = torch.ones(N // page)
    for i in range(N // page):
        grow[i] = 2.0 ** (i // 16 * 1 - 2) if i < N // page - 1 else 2.0 ** 4
    for i, pg in enumerate(layer.doc_table.tolist()):
        layer.k_scale[pg] *= grow[i].item()
    doc = [doc[0] * grow.repeat_interleave(page)[:, None, None], doc[1]]
    rows = 40
    q = queries(rows, 4, d, 3)
    q[::3] *= 0.125                     # rows whose reference stays
    s, p = ids(list(range(1, rows + 1)), [N + 8] * rows)
    ro, rl, ra = oracle_attn(doc, segs, N, q.cpu(), s.cpu().numpy(), p.cpu().numpy(), d ** -0.5)
    for splits in (0, 1, 3):
        lse = torch.zeros((rows, 4), device=DEV)
        o = m.kv8_decode_attn(layer, N, q, s, p, d ** -0.5, lse=lse, opt=m.Options(splits=splits))
        torch.cuda.synchronize()
        # scores up to ~ 16 * |q||k| scale ~ 700: as in the test of far scales
        err = np.abs(o.float().cpu().numpy() - ro)
        tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -7 + 2.0 ** -10 + 2.0 ** -12) * ra + 1e-30
        assert (err <= tol).all(), (err / tol).max()
        assert np.abs(lse.cpu().numpy() - rl).max() <= 2.0 ** -8


@pytest.mark.parametrize("scale", [0.05, 0.22, 0.5, 0.9])
@pytest.mark.parametrize("d", [64, 128])
def test_one_key_far_above_all_before_it(d, scale):
    """A single key, at another place of its 16 in every head, whose score is up to
    1200 binades above the reference that the tiles before it gave."""
    m = pp()
    N, H, rows, page = 900, 16, 40, 32
    layer, doc, segs = make_cache(H, d, page, N, [9] * rows, seed=31, spread=0)
    q = torch.ones((rows, H, d), dtype=torch.bfloat16, device=DEV)
    s, p = ids(list(range(1, rows + 1)), [N + 8] * rows)
    k = layer.k.view(torch.uint8)
    for h in range(H):
        t = 640 + h
        k[layer.doc_table[t // page].item(), h, t % page] = 0x7e          # 448 * 2^-6
        doc[0][t, h] = 7.0
    for splits in (1, 5):
        lse = torch.zeros((rows, H), device=DEV)
        o = m.kv8_decode_attn(layer, N, q, s, p, scale, lse=lse, opt=m.Options(splits=splits))
        torch.cuda.synchronize()
        # the score is 7 d scale <= 807: 1164 in base 2, whose five roundings of 2^-24
        # are 2^-11.5, of a probability and (times ln 2) of lse
        ref = oracle_attn(doc, segs, N, q.cpu(), s.cpu().numpy(), p.cpu().numpy(), scale)
        err = np.abs(o.float().cpu().numpy() - ref[0])
        tol = 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -10 + 2.0 ** -12 + 2.0 ** -10.5) * ref[2] + 1e-30
        assert (err <= tol).all(), (err / tol).max()
        assert np.abs(lse.cpu().numpy() - ref[1]).max() <= 2.0 ** -11.5 + 2.0 ** -12


@pytest.mark.parametrize("splits", [0, 2])
def test_queries_and_pages_of_zeros_and_tiny_factors(splits):
    """Queries of zeros and of bf16's smallest normals, an all-zero page at the
    least scale, softmax scales down to 1e-30: uniform or nearly uniform weights,
    also in the document's last, hidden-tailed tile."""
    m = pp()
    N, d = 203, 64
    layer, doc, segs = make_cache(2, d, 16, N, [20, 7, 3], seed=23)
    pg = int(layer.doc_table[5])
    layer.k.view(torch.uint8)[pg] = 0
    layer.k_scale[pg] = 2.0 ** -40
    doc[0][80:96] = 0
    q = queries(3, 4, d, 1)
    q[0] = 0
    q[1] = 1.2e-38
    s, p = ids([1, 2, 3], [N + 19, N + 6, N + 2])
    for scale in (0.125, 1e-6, 1e-30):
        for fn in (m.kv8_decode_attn, m.kv8_prefill_attn):
            lse = torch.zeros((3, 4), device=DEV)
            o = fn(layer, N, q, s, p, scale, lse=lse, opt=m.Options(splits=splits))
            torch.cuda.synchronize()
            check(o, lse, oracle_attn(doc, segs, N, q.cpu(), np.array([1, 2, 3]),
                                      np.array([N + 19, N + 6, N + 2]), scale), scale)
    assert m.kv8_device_status(layer) == 0


@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("mag", [2.0 ** 8, 2.0 ** 15])
def test_scores_of_a_million(splits, mag):
    """Scores so large that one key takes all: the output is that key's value."""
    m = pp()
    N, d = 500, 128
    layer, doc, segs = make_cache(1, d, 32, N, [5], seed=24)
    q = (doc[0][[7, 130, 480]].transpose(0, 1) * mag).to(torch.bfloat16).to(DEV)      # [1, 3, d]
    s, p = ids([1], [N + 4])
    lse = torch.zeros((1, 3), device=DEV)
    o = m.kv8_decode_attn(layer, N, q, s, p, 1.0, lse=lse, opt=m.Options(splits=splits))
    torch.cuda.synchronize()
    sc = torch.einsum("hd,nd->hn", q[0].cpu().double(), torch.cat([doc[0][:, 0], segs[0][0][:, 0]]).double())
    two = sc.topk(2).values
    # the runner-up is further off than the scores' fp32 error, 128 * 2^-24 of the sum of magnitudes
    gap = (two[:, 0] - two[:, 1]) / (128 * 2.0 ** -24 * two[:, 0])
    assert (gap > 100).all()
    v = torch.cat([doc[1][:, 0], segs[0][1][:, 0]])[sc.argmax(1)]
    assert torch.equal(o[0].float().cpu(), v.to(torch.bfloat16).float())
    assert ((lse[0].cpu().double() - two[:, 0]).abs() <= 2.0 ** -16 * two[:, 0]).all()
