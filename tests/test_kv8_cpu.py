"""8-bit paged cache, host side: descriptors, argument checks (nothing is
launched), and the oracle's append pinned by hand examples."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.kv8 import Kv8Replay, e4m3, rotate, scale_for
from tests.test_abi_cpu import header_struct_fields


@pytest.fixture(scope="module")
def pp():
    from shared_context_decode_b200 import ppattn
    return ppattn


def fake(pp, **kw):
    base = dict(H=4, d=128, page=32, n_pages=64, P_max=8, seg_pages=4, doc_pages=16, pos0=500,
                k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, doc_table=0x50000,
                seg_table=0x60000, status=0x70000)
    base.update(kw)
    return pp.KV8LayerStruct(**base)


def test_structs_match_the_header(pp):
    assert [f for f, _ in pp.KV8LayerStruct._fields_] == header_struct_fields("pp_kv8_layer")
    assert [f for f, _ in pp.RopeStruct._fields_] == header_struct_fields("pp_rope")


LAYER_CASES = [
    (dict(d=96), "UNSUPPORTED"), (dict(page=24), "UNSUPPORTED"), (dict(page=256), "UNSUPPORTED"),
    (dict(P_max=0), "UNSUPPORTED"), (dict(P_max=40000), "UNSUPPORTED"),
    (dict(H=0), "INVALID_ARG"), (dict(n_pages=0), "INVALID_ARG"), (dict(seg_pages=0), "INVALID_ARG"),
    (dict(doc_pages=-1), "INVALID_ARG"), (dict(pos0=-1), "INVALID_ARG"),
    (dict(k=0x10008), "INVALID_ARG"), (dict(v=0), "INVALID_ARG"), (dict(k_scale=0x30002), "INVALID_ARG"),
    (dict(doc_table=0), "INVALID_ARG"), (dict(seg_table=0x60001), "INVALID_ARG"),
    (dict(status=0), "INVALID_ARG"), (dict(seg_pages=1 << 27), "UNSUPPORTED"),
    (dict(pos0=0x7fffffff), "UNSUPPORTED"), (dict(doc_pages=1 << 27), "UNSUPPORTED"),
    (dict(n_pages=1 << 30), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,code", LAYER_CASES)
def test_layer_checks(pp, kw, code):
    want = getattr(pp, "PP_ERR_" + code)
    L = fake(pp, **kw)
    assert pp._kv8_reset(ctypes.byref(L), None) == want
    assert append(pp, L) == want
    assert attend(pp, pp._kv8_decode, L) == want
    assert attend(pp, pp._kv8_prefill, L) == want
    out = ctypes.c_int32(0)
    assert pp._kv8_status(ctypes.byref(L), ctypes.byref(out), None) == want


def append(pp, L=None, k=0x1000, k_ld=512, v=0x2000, v_ld=512, q=0x3000, q_ld=1024, Hq=8, sid=0x4000,
           pos=0x5000, n=3, rope=None, q_out=0x6000, qo_ld=1024):
    L = L if L is not None else fake(pp)
    a = pp._pack_append(k, v, q, q_out, k_ld, v_ld, q_ld, qo_ld, sid, pos,
                        0 if rope is None else ctypes.addressof(rope), Hq, n)
    return pp._kv8_append(ctypes.byref(L), a, None)


def attend(pp, fn, L=None, doc_len=500, q=0x1000, q_ld=1024, Hq=8, sid=0x2000, pos=0x3000, rows=4,
           scale=0.1, o=0x4000, lse=0, ws=0x10000, ws_bytes=1 << 40, opt=None):
    L = L if L is not None else fake(pp)
    a = pp._pack_attn(q, q_ld, sid, pos, o, lse, ws, ws_bytes,
                      0 if opt is None else ctypes.addressof(opt), Hq, rows, doc_len, scale)
    return fn(ctypes.byref(L), a, None)


def test_argument_blocks_match_the_header(pp):
    assert list(pp.KV8_APPEND_FIELDS) == header_struct_fields("pp_kv8_append_args")
    assert list(pp.KV8_ATTN_FIELDS) == header_struct_fields("pp_kv8_attn_args")
    assert len(pp._pack_append(*range(13))) == 96 and len(pp._pack_attn(*range(13))) == 88
    L = fake(pp)
    assert pp._kv8_append(ctypes.byref(L), None, None) == pp.PP_ERR_INVALID_ARG
    assert pp._kv8_decode(ctypes.byref(L), None, None) == pp.PP_ERR_INVALID_ARG


def test_append_checks(pp):
    bad, no = pp.PP_ERR_INVALID_ARG, pp.PP_ERR_UNSUPPORTED
    assert append(pp, n=0) == pp.PP_OK
    assert append(pp, n=-1) == bad
    assert append(pp, k=0x1008) == bad and append(pp, v=0) == bad
    assert append(pp, k_ld=511) == bad and append(pp, k_ld=504) == bad and append(pp, v_ld=516) == bad
    assert append(pp, q=0) == bad and append(pp, q_out=0) == bad      # one without the other
    assert append(pp, q_ld=1016) == bad and append(pp, qo_ld=1000) == bad and append(pp, Hq=0) == bad
    assert append(pp, sid=0x4001) == bad and append(pp, pos=0) == bad
    R = pp.RopeStruct
    assert append(pp, rope=R(64, 0, 0, 0, 0x9000)) == bad                    # no positions
    assert append(pp, rope=R(64, 2, 10, 0, 0x9000)) == bad
    assert append(pp, rope=R(64, 0, 10, 0, 0x9004)) == bad                   # misaligned table
    assert append(pp, rope=R(24, 0, 10, 0, 0x9000)) == no
    assert append(pp, rope=R(144, 0, 10, 0, 0x9000)) == no                   # more than d
    assert append(pp, rope=R(0, 0, 10, 0, 0x9000)) == no


@pytest.mark.parametrize("which", ["_kv8_decode", "_kv8_prefill"])
def test_attention_checks(pp, which):
    fn = getattr(pp, which)
    bad, no = pp.PP_ERR_INVALID_ARG, pp.PP_ERR_UNSUPPORTED
    assert attend(pp, fn, rows=0) == pp.PP_OK
    assert attend(pp, fn, rows=-1) == bad and attend(pp, fn, doc_len=-1) == bad
    assert attend(pp, fn, doc_len=513) == pp.PP_ERR_CAPACITY                 # 16 pages of 32
    assert attend(pp, fn, Hq=6) == bad and attend(pp, fn, Hq=0) == bad       # not a multiple of H
    assert attend(pp, fn, q=0x1004) == bad and attend(pp, fn, q_ld=1020) == bad
    assert attend(pp, fn, q_ld=1016) == bad and attend(pp, fn, o=0) == bad
    assert attend(pp, fn, sid=0) == bad and attend(pp, fn, lse=0x5002) == bad
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(pp, fn, scale=s) == bad
    for o in (pp.Options(ablation_doc_per_stream=1), pp.Options(sibling_scan=1),
              pp.Options(suffix_slices=2)):
        assert attend(pp, fn, opt=o) == no
    assert attend(pp, fn, rows=1 << 30, Hq=8) == no
    if which == "_kv8_decode":
        assert attend(pp, fn, rows=9) == no                                  # P > P_max


def test_binding_checks_shapes_and_strides(pp):
    L = pp.KV8Layer(2, 64, 16, 4, 2, 2, 2, 20, "cpu")
    bf = torch.bfloat16
    sid, pos = torch.zeros(3, dtype=torch.int16), torch.zeros(3, dtype=torch.int32)
    k = torch.zeros((3, 2, 64), dtype=bf)
    with pytest.raises(TypeError):
        pp.kv8_append(L, k.float(), k, sid, pos)
    with pytest.raises(ValueError):
        pp.kv8_append(L, k[:2], k, sid, pos)
    with pytest.raises(ValueError):         # heads not packed
        pp.kv8_append(L, torch.zeros((3, 64, 2), dtype=bf).transpose(1, 2), k, sid, pos)
    with pytest.raises(ValueError):         # rows 132 elements apart
        pp.kv8_append(L, torch.zeros((3, 132), dtype=bf)[:, :128].view(3, 2, 64), k, sid, pos)
    with pytest.raises(ValueError):
        pp.kv8_append(L, k, k, sid, pos, q_out=k)
    with pytest.raises(ValueError):
        pp.kv8_append(L, k, k, sid, pos[:2])
    with pytest.raises(ValueError):
        pp.KV8Layer(2, 64, 16, 4, 2, 2, 2, 20, "cpu", k_scale=torch.zeros((4, 3)))
    with pytest.raises(ValueError):
        pp.Rope(torch.zeros(8))
    assert pp._rows(torch.zeros((3, 6, 64), dtype=bf)[:, 2:4], "k", 3, 2, 64, L) == 384
    assert L.nbytes() == 2 * 4 * 2 * 16 * 64 + 2 * 4 * 2 * 4 + 4 * 2 + 4 * 4 + 4


# ---------------------------------------------------------------- oracle ----
def test_oracle_e4m3_matches_torch():
    x = torch.cat([torch.randn(4000, generator=torch.Generator().manual_seed(1)) * s
                   for s in (1e-3, 0.1, 1.0, 100.0)]).clamp(-448, 448)
    assert np.array_equal(e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    assert e4m3(1000.0) == 448.0 and e4m3(-1e30) == -448.0
    assert e4m3(2.0 ** -10) == 0.0 and e4m3(1.5 * 2.0 ** -9) == 2.0 ** -8    # ties to even


def test_oracle_scale_rule():
    assert scale_for(448.0) == 1.0 and scale_for(448.5) == 2.0 and scale_for(224.0) == 0.5
    assert scale_for(0.0) == 2.0 ** -40 and scale_for(1e30) == 2.0 ** 40
    assert scale_for(4.5) == 2.0 ** -6


def test_oracle_rotation_turns_by_the_angle():
    cs = np.array([[1, 1, 0, 0], [0, np.cos(0.5), 1, np.sin(0.5)]], np.float32)
    x = np.array([[1, 2, 3, 4, 5, 6]], np.float32)
    assert np.array_equal(rotate(x, 0, cs, False), x)
    y = rotate(x, 1, cs, False)
    z = (2 + 4j) * np.exp(0.5j)
    assert np.allclose(y, [[-3, z.real, 1, z.imag, 5, 6]], atol=1e-6)
    y = rotate(x, 1, cs, True)
    z = (3 + 4j) * np.exp(0.5j)
    assert np.allclose(y, [[-2, 1, z.real, z.imag, 5, 6]], atol=1e-6)


def test_oracle_page_grows_and_rounds_again():
    r = Kv8Replay(1, 2, 16, 2, 0, [], [[1]])
    k = np.array([[[1.0, 0.3]]], np.float32)
    assert r.append(k, k, [1], [0]) == []
    assert r.k_scale[1, 0] == 2.0 ** -8                      # 1 <= 448 / 256
    x = r.k[1, 0, 0].copy()
    assert abs(x[1] * 2.0 ** -8 - 0.3) <= 0.3 * 2.0 ** -4
    r.append(k * 1000, k, [1], [1])
    assert r.k_scale[1, 0] == 4.0 and r.v_scale[1, 0] == 2.0 ** -8
    assert np.array_equal(r.k[1, 0, 0], e4m3(x * 2.0 ** -10))
    assert r.append(k, k, [1], [0]) == [] and r.k_scale[1, 0] == 2.0 ** -8   # afresh
    assert r.append(np.repeat(k, 3, 0), np.repeat(k, 3, 0), [1, 0, 1], [1, 0, 2]) == [1, 2]


def test_a_layer_in_host_memory_reaches_no_kernel(pp):
    L = pp.KV8Layer(2, 64, 16, 4, 2, 1, 1, 4, device="cpu")
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    s, p = torch.ones(2, dtype=torch.int16), torch.tensor([4, 5], dtype=torch.int32)
    ws = torch.empty(256, dtype=torch.uint8)
    for call in (lambda: pp.kv8_append(L, k, k, s, p), lambda: pp.kv8_reset(L),
                 lambda: pp.kv8_decode_attn(L, 4, k, s, p, 0.1),
                 lambda: pp.kv8_prefill_attn(L, 4, k, s, p, 0.1, ws=ws),
                 lambda: pp.kv8_device_status(L)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
