"""8-bit paged cache on the GPU: the rotating, quantising append against the
plain replay, bit for bit (every step of it is defined to the last rounding)."""
import numpy as np
import pytest
import torch

from oracle.kv8 import Kv8Replay
from tests.kv8_util import pp

pytestmark = pytest.mark.gpu
DEV = "cuda"


def new_cache(H, d, page, P, seg_pages, N, seed=0, extra=3, status=0):
    m = pp()
    g = torch.Generator().manual_seed(seed)
    doc_pages = -(-N // page)
    n_pages = doc_pages + P * seg_pages + extra
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    dt = perm[:doc_pages].contiguous()
    st = perm[doc_pages:doc_pages + P * seg_pages].view(P, seg_pages).contiguous()
    layer = m.KV8Layer(H, d, page, n_pages, P, seg_pages, doc_pages, N, DEV,
                       doc_table=dt.to(DEV), seg_table=st.to(DEV))
    return layer, Kv8Replay(H, d, page, n_pages, N, dt.numpy(), st.numpy())


def rows(n, H, Hq, d, seed, mag=1.0):
    """q, k, v as slices of one fused projection's output."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, Hq + 2 * H, d), generator=g)
    x *= torch.exp2(torch.randint(-3, 4, (n, Hq + 2 * H, 1), generator=g).float())
    x = (x * mag).to(torch.bfloat16).to(DEV)
    return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]


def same_cache(layer, rep):
    for t in "kv":
        got = getattr(layer, t).float().cpu().double().numpy()
        want = getattr(rep, t)
        assert np.array_equal(getattr(layer, t + "_scale").cpu().double().numpy(),
                              getattr(rep, t + "_scale")), t + "_scale"
        assert np.array_equal(got, want, equal_nan=True), t


def call(layer, rep, sid, pos, seed, rope=None, mag=1.0, Hq=None, poke=None):
    m = pp()
    Hq = Hq or layer.H
    n = len(sid)
    q, k, v = rows(n, layer.H, Hq, layer.d, seed, mag)
    if poke:
        poke(q, k, v)
    s = torch.tensor(sid, dtype=torch.int16, device=DEV)
    p = torch.tensor(pos, dtype=torch.int32, device=DEV)
    q_out = torch.full((n, Hq, layer.d), 7.0, dtype=torch.bfloat16, device=DEV)
    r = m.kv8_append(layer, k, v, s, p, rope=rope, q=q, q_out=q_out)
    assert r is q_out
    torch.cuda.synchronize()
    cs = None if rope is None else rope.cos_sin.cpu().numpy()
    inter = rope is not None and rope.interleaved
    dropped = rep.append(k.float().cpu().numpy(), v.float().cpu().numpy(), sid, pos, cs, inter)
    same_cache(layer, rep)
    # queries: turned rows, or the row as it was where it has no angle
    from oracle.kv8 import rotate
    for i in range(n):
        if sid[i] < 0 or sid[i] > layer.P_max or pos[i] < 0 or (cs is not None and pos[i] >= len(cs)):
            want = torch.full((Hq, layer.d), 7.0)
        else:
            x = q[i].float().cpu().numpy()
            want = torch.from_numpy(x if cs is None else rotate(x, pos[i], cs, inter))
        assert torch.equal(torch.nan_to_num(q_out[i].cpu(), nan=123.0),
                           torch.nan_to_num(want.to(torch.bfloat16), nan=123.0)), f"query row {i}"
    return dropped


@pytest.mark.parametrize("H,g,d,page,rot,inter", [
    (1, 1, 64, 16, 0, False), (3, 1, 64, 32, 64, False), (2, 4, 128, 16, 64, True),
    (5, 7, 128, 64, 128, False), (4, 2, 128, 128, 16, False), (2, 1, 64, 16, 32, True),
    (33, 1, 128, 32, 128, True),
])
def test_document_questions_and_steps(H, g, d, page, rot, inter):
    N, lens = 77, [1, 33, 16, 17, 2, 64, 15]
    P = len(lens)
    layer, rep = new_cache(H, d, page, P, -(-(64 + 12) // page), N, seed=H)
    rope = pp().Rope.make(N + 200, rot, interleaved=inter, device=DEV) if rot else None
    assert call(layer, rep, [0] * N, list(range(N)), 1, rope, Hq=H * g) == []
    sid = sum(([s + 1] * n for s, n in enumerate(lens)), [])
    pos = sum((list(range(N, N + n)) for n in lens), [])
    assert call(layer, rep, sid, pos, 2, rope, Hq=H * g) == []
    for t in range(10):                 # decode steps whose values grow: pages are rounded again
        act = [s for s in range(P) if (s + t) % 4]
        assert call(layer, rep, [s + 1 for s in act], [N + lens[s] for s in act], 10 + t, rope,
                    mag=2.0 ** (t - 3), Hq=H * g) == []
        for s in act:
            lens[s] += 1
    assert pp().kv8_device_status(layer) == 0


def test_rows_that_are_dropped_leave_the_cache_and_say_why():
    m = pp()
    layer, rep = new_cache(2, 64, 16, 4, 2, 20, seed=3)
    rope = m.Rope.make(46, 32, device=DEV)
    for sid, pos, bit, drop in [
        ([5, 1], [20, 20], m.PP_DEV_BAD_STREAM, [0]),
        ([1, 2], [19, 20], m.PP_DEV_BAD_POSITION, [0]),
        ([1] * 13 + [3], list(range(36, 49)) + [20], m.PP_DEV_BAD_POSITION, [10, 11, 12]),   # past the angles
        ([0, 2], [32, 21], m.PP_DEV_DOC_OUT_OF_RANGE, [0]),
        ([0, 2], [-1, 21], m.PP_DEV_DOC_OUT_OF_RANGE, [0]),
        ([1, 0, 1], [20, 0, 21], m.PP_DEV_ROW_ORDER, [2]),
        ([1, 1, 1], [20, 21, 23], m.PP_DEV_ROW_ORDER, [2]),
        ([1, 1], [21, 21], m.PP_DEV_ROW_ORDER, [1]),
        ([-1, 3, -5], [0, 22, 9], 0, []),
    ]:
        got = call(layer, rep, sid, pos, 5 + len(sid), rope)
        assert got == drop, (sid, pos, got)
        assert m.kv8_device_status(layer) == bit, (sid, pos)
        m.kv8_reset(layer)
    assert call(layer, rep, [2] * 3, [51, 52, 53], 1) == [1, 2]
    assert m.kv8_device_status(layer) == m.PP_DEV_SEGMENT_OVERFLOW
    m.kv8_reset(layer)
    for bad in (-1, layer.n_pages, -2 ** 31):
        layer.seg_table[1, 1] = bad
        rep.seg_table = layer.seg_table.cpu().numpy()
        assert call(layer, rep, [2, 2, 3], [35, 36, 20], 8) == [1]
        assert m.kv8_device_status(layer) == m.PP_DEV_BAD_PAGE
        m.kv8_reset(layer)


def test_zero_huge_and_non_finite_values():
    m = pp()
    layer, rep = new_cache(2, 64, 16, 3, 2, 0, seed=4)

    def poke(q, k, v):
        k[0] = 0.0
        v[0] = 0.0
        k[1] = 3e38
        v[1] = -3e38
        k[2, 0, 5] = float("nan")
        v[2, 1, 9] = float("nan")
        k[3, 1, 0] = float("inf")
        v[3, 0, 63] = -float("inf")
        k[4] = 1e-38
        v[4] = -1e-38

    call(layer, rep, [1, 1, 2, 2, 3], [0, 1, 0, 1, 0], 1, poke=poke)
    assert m.kv8_device_status(layer) == m.PP_DEV_NONFINITE


def test_repeated_call_on_other_streams_and_in_a_graph():
    m = pp()
    layer, rep = new_cache(4, 128, 32, 6, 3, 40, seed=5)
    rope = m.Rope.make(200, 128, device=DEV)
    sid, pos = [1] * 20 + [4] * 45 + [6], list(range(40, 60)) + list(range(40, 85)) + [40]
    call(layer, rep, sid, pos, 1, rope)
    call(layer, rep, [1, 4], [60, 85], 2, rope, mag=64.0)
    call(layer, rep, [1, 4], [60, 85], 2, rope, mag=64.0)           # the same again
    q, k, v = rows(2, 4, 4, 128, 3, 8.0)
    s = torch.tensor([1, 4], dtype=torch.int16, device=DEV)
    p = torch.tensor([61, 86], dtype=torch.int32, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        q2 = m.kv8_append(layer, k, v, s, p, rope=rope, q=q)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    rep.append(k.float().cpu().numpy(), v.float().cpu().numpy(), [1, 4], [61, 86],
               rope.cos_sin.cpu().numpy())
    same_cache(layer, rep)
    # replayed at the next positions: the kernel reads them at run time
    p += 1
    g.replay()
    torch.cuda.synchronize()
    rep.append(k.float().cpu().numpy(), v.float().cpu().numpy(), [1, 4], [62, 87],
               rope.cos_sin.cpu().numpy())
    same_cache(layer, rep)
    q3 = m.kv8_append(layer, k, v, s, p, rope=rope, q=q, q_out=q)    # in place
    assert q3 is q and torch.equal(q, q2)
    assert m.kv8_append(layer, k[:0], v[:0], s[:0], p[:0]) is None
    m.kv8_append(layer, k, v, s, p, rope=rope)                       # without queries
    torch.cuda.synchronize()
    same_cache(layer, rep)


def test_long_runs_over_many_windows():
    """Rows enough for several rows per CTA, with short and long runs."""
    N, page = 5000, 16
    layer, rep = new_cache(9, 64, page, 300, 3, N, seed=6)
    call(layer, rep, [0] * N, list(range(N)), 1)
    g = np.random.default_rng(7)
    sid, pos = [], []
    for s in g.permutation(300):
        n = int(g.integers(1, 40))
        sid += [int(s) + 1] * n
        pos += list(range(N, N + n))
    call(layer, rep, sid, pos, 2)


@pytest.mark.parametrize("H,d,page,rot,inter", [(3, 128, 64, 128, False), (5, 64, 16, 32, True),
                                                (2, 128, 128, 0, False), (9, 64, 32, 64, False)])
def test_long_runs_among_fewer_rows_than_streams(H, d, page, rot, inter):
    """Calls of fewer rows than the cache has streams, with runs of one, two, three and many
    rows side by side, a NaN far inside a run, pages whose scale grows, runs that end the
    angles or repeat."""
    m = pp()
    N, P = 150, 700
    layer, rep = new_cache(H, d, page, P, -(-260 // page), N, seed=H)
    rope = m.Rope.make(N + 230, rot, interleaved=inter, device=DEV) if rot else None
    assert call(layer, rep, [0] * N, list(range(N)), 1, rope, Hq=2 * H) == []
    lens = [1, 2, 3, 4, 1, 200, 1, 1, 5, 65, 2, 1, 1, 1, 3, 130]
    sid = sum(([600 - 7 * s] * n for s, n in enumerate(lens)), [])
    pos = sum((list(range(N, N + n)) for n in lens), [])

    def poke(q, k, v):
        k[60, H - 1, 7] = float("nan")
        v[100, 0, d - 1] = float("nan")
        v[300, 0, 0] = float("inf")

    assert call(layer, rep, sid, pos, 2, rope, Hq=H, poke=poke) == []
    assert m.kv8_device_status(layer) == m.PP_DEV_NONFINITE
    m.kv8_reset(layer)
    more = [3, 1, 9, 17, 2, 25, 1]
    sid = sum(([600 - 7 * s] * n for s, n in enumerate(more)), []) + [600]
    pos = sum((list(range(N + lens[s], N + lens[s] + n)) for s, n in enumerate(more)), []) + [N + 4]
    got = call(layer, rep, sid, pos, 3, rope, mag=256.0)
    assert got == [len(sid) - 1]
    assert m.kv8_device_status(layer) == m.PP_DEV_ROW_ORDER
    m.kv8_reset(layer)
    if rot:          # past the angles
        assert call(layer, rep, [565] * 20, list(range(N + 225, N + 245)), 4, rope) == list(range(5, 20))
        assert m.kv8_device_status(layer) == m.PP_DEV_BAD_POSITION


def test_pages_past_two_and_four_gib():
    """A pool whose last pages lie more than 4 GiB behind its first."""
    m = pp()
    H, d, page = 32, 128, 128
    n_pages = (1 << 32) // (H * d * page) + 4
    dt = torch.tensor([n_pages - 1], dtype=torch.int32, device=DEV)
    st = torch.tensor([[n_pages - 2, 0], [n_pages // 2 + 1, n_pages - 3]], dtype=torch.int32, device=DEV)
    layer = m.KV8Layer(H, d, page, n_pages, 2, 2, 1, 100, DEV, doc_table=dt, seg_table=st)
    n = 100
    q, k, v = rows(n + 130, H, H, d, 1)
    s = torch.tensor([0] * n + [2] * 130, dtype=torch.int16, device=DEV)
    p = torch.tensor(list(range(n)) + list(range(100, 230)), dtype=torch.int32, device=DEV)
    m.kv8_append(layer, k, v, s, p)
    torch.cuda.synchronize()
    assert m.kv8_device_status(layer) == 0
    rep = Kv8Replay(H, d, page, 4, 100, [0], [[1, 2], [2, 3]])
    rep.append(k.float().cpu().numpy(), v.float().cpu().numpy(), s.tolist(), p.tolist())
    for i, pg in enumerate([n_pages - 1, None, n_pages // 2 + 1, n_pages - 3]):
        if pg is None:
            continue
        for t in "kv":
            assert np.array_equal(getattr(layer, t)[pg].float().cpu().double().numpy(), getattr(rep, t)[i])
            assert np.array_equal(getattr(layer, t + "_scale")[pg].cpu().double().numpy(),
                                  getattr(rep, t + "_scale")[i])


@pytest.mark.parametrize("shift", [0, 1, 3, 5])
def test_ids_at_any_alignment(shift):
    """Stream ids that start on any 2-byte boundary, positions on any 4-byte one,
    with a row that breaks its stream's run far behind it."""
    m = pp()
    layer, rep = new_cache(2, 64, 16, 40, 2, 10, seed=8)
    sid = sum(([s] * 20 for s in range(1, 30)), []) + [7, 31] + [-1] * 5 + [32] * 9
    pos = sum((list(range(10, 30)) for s in range(1, 30)), []) + [30, 10] + [0] * 5 + list(range(10, 19))
    n = len(sid)
    q, k, v = rows(n, 2, 2, 64, 4)
    s = torch.tensor([0] * shift + sid, dtype=torch.int16, device=DEV)[shift:]
    p = torch.tensor([0] * shift + pos, dtype=torch.int32, device=DEV)[shift:]
    m.kv8_append(layer, k, v, s, p)
    torch.cuda.synchronize()
    assert rep.append(k.float().cpu().numpy(), v.float().cpu().numpy(), sid, pos) == [580]
    same_cache(layer, rep)
    assert m.kv8_device_status(layer) == m.PP_DEV_ROW_ORDER


def test_one_layer_for_two_calls_at_once():
    """Appends of different streams on two CUDA streams."""
    m = pp()
    layer, rep = new_cache(8, 128, 32, 64, 3, 20, seed=9)
    calls = []
    for half in (0, 1):
        sid = sum(([s] * 33 for s in range(1 + 32 * half, 33 + 32 * half)), [])
        pos = list(range(20, 53)) * 32
        q, k, v = rows(len(sid), 8, 8, 128, 5 + half)
        calls.append((k, v, torch.tensor(sid, dtype=torch.int16, device=DEV),
                      torch.tensor(pos, dtype=torch.int32, device=DEV), torch.cuda.Stream()))
        rep.append(k.float().cpu().numpy(), v.float().cpu().numpy(), sid, pos)
    torch.cuda.synchronize()
    for k, v, s, p, st in calls:
        with torch.cuda.stream(st):
            m.kv8_append(layer, k, v, s, p)
    torch.cuda.synchronize()
    same_cache(layer, rep)
