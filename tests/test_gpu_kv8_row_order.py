"""8-bit paged cache on the GPU: appends whose rows of a stream break off in the
middle of a page and fit again behind the break, bit for bit against the plain
replay, by both forms of the append, on new pages and on pages that hold rows."""
import numpy as np
import pytest
import torch

from tests.kv8_util import pp
from tests.test_gpu_kv8_append import DEV, new_cache, rows, same_cache
from tests.test_kv8_row_order_cpu import BREAKS, dropped_of

pytestmark = pytest.mark.gpu


def go(layer, rep, k, v, sid, pos, rope=None):
    s = torch.tensor(sid, dtype=torch.int16, device=DEV)
    p = torch.tensor(pos, dtype=torch.int32, device=DEV)
    out = []
    for _ in range(2):                  # twice: the same bytes
        pp().kv8_append(layer, k, v, s, p, rope=rope)
        torch.cuda.synchronize()
        out.append([t.clone() for t in (layer.k.view(torch.uint8), layer.v.view(torch.uint8),
                                        layer.k_scale, layer.v_scale)])
        dropped = rep.append(k.float().cpu().numpy(), v.float().cpu().numpy(), sid, pos,
                             None if rope is None else rope.cos_sin.cpu().numpy(),
                             rope is not None and rope.interleaved)
        same_cache(layer, rep)
    assert all(torch.equal(a, b) for a, b in zip(*out))
    return dropped


# P: fewer rows than streams, or more (the two forms)
@pytest.mark.parametrize("P", [12, 120])
@pytest.mark.parametrize("H,d,page,rot", [(3, 128, 16, 0), (9, 64, 16, 32), (2, 128, 64, 128),
                                          (5, 64, 128, 64), (33, 64, 32, 64)])
@pytest.mark.parametrize("held", [False, True])
def test_breaks_inside_a_page(H, d, page, rot, P, held):
    m = pp()
    N = 8
    layer, rep = new_cache(H, d, page, P, -(-100 // page), N, seed=H)
    rope = m.Rope.make(N + 200, rot, device=DEV) if rot else None
    sid, pos, drop = [], [], []
    for i, (b, _) in enumerate(BREAKS):
        drop += [len(sid) + j for j in dropped_of(b, page)]
        sid += [i + 1] * len(b)
        pos += [N + x if x >= 0 else x for x in b]
    first = [min(x for x in b if x >= 0) for b, _ in BREAKS]
    if held:                            # the rows before the calls', small
        s0 = sum(([i + 1] * n for i, n in enumerate(first)), [])
        p0 = sum((list(range(N, N + n)) for n in first), [])
        q, k, v = rows(len(s0), H, H, d, 1, 2.0 ** -6)
        assert go(layer, rep, k, v, s0, p0, rope) == []
    q, k, v = rows(len(sid), H, H, d, 2)
    k, v = k.clone(), v.clone()
    grow = torch.exp2(torch.arange(len(sid), device=DEV) % 12)[:, None, None]
    k *= grow                           # so that every row asks for another scale
    v *= grow.flip(0)
    assert (len(sid) <= P) == (P == 120)
    assert go(layer, rep, k, v, sid, pos, rope) == drop
    # (the row at -1 is no position besides)
    assert m.kv8_device_status(layer) == m.PP_DEV_ROW_ORDER | m.PP_DEV_BAD_POSITION


@pytest.mark.parametrize("shift", [0, 1, 3, 4, 7])
@pytest.mark.parametrize("P", [40, 320])
def test_a_break_far_before_the_row(P, shift):
    """Long runs with one wrong position, ids and positions at any alignment."""
    m = pp()
    N, page, n = 5, 32, 300
    for at in (0, 1, 6, 7, 8, 9, 100, 253, 298, 299):
        layer, rep = new_cache(2, 64, page, P, -(-n // page), N, seed=4)
        sid = [3] * 9 + [7] * n + [9] * 5 + [-1] * 2 + [11] * 4
        pos = [*range(N, N + 9), *range(N, N + n), *range(N, N + 5), 0, 0, *range(N, N + 4)]
        pos[9 + at] += 1 if at else 40
        q, k, v = rows(len(sid), 2, 2, 64, at)
        s = torch.tensor([0] * shift + sid, dtype=torch.int16, device=DEV)[shift:]
        p = torch.tensor([0] * shift + pos, dtype=torch.int32, device=DEV)[shift:]
        m.kv8_append(layer, k, v, s, p)
        torch.cuda.synchronize()
        dropped = rep.append(k.float().cpu().numpy(), v.float().cpu().numpy(), sid, pos)
        assert dropped == [9 + j for j in dropped_of([x - N for x in pos[9:9 + n]], page)]
        same_cache(layer, rep)
        assert m.kv8_device_status(layer) == m.PP_DEV_ROW_ORDER
