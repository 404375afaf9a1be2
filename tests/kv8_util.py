"""Helpers of the 8-bit paged cache's tests: a cache filled with known values,
the fp64 oracle's answer for it, and error bounds."""
import numpy as np
import torch

import oracle
from shared_context_decode_b200.workloads import bf16_bits


def pp():
    from shared_context_decode_b200 import ppattn
    return ppattn


def make_cache(H, d, page, N, lens, seed=0, device="cuda", extra_pages=2, seg_pages=None,
               spread=2, dead=0x7f):
    """A KV8Layer with N document tokens and lens[s-1] tokens of stream s at
    scattered pages, slots past the ends filled with the byte `dead` (NaN), and
    the dequantised rows: doc (k, v) [N, H, d] and per stream (k, v)."""
    m = pp()
    g = torch.Generator().manual_seed(seed)
    P = len(lens)
    doc_pages = -(-N // page)
    seg_pages = seg_pages or max(1, -(-max([1] + list(lens)) // page))
    n_pages = doc_pages + P * seg_pages + extra_pages
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    doc_table = perm[:doc_pages].contiguous()
    seg_table = perm[doc_pages:doc_pages + P * seg_pages].view(P, seg_pages).contiguous()
    pools = {}
    for t in "kv":
        x = torch.randn((n_pages, H, page, d), generator=g)
        e = torch.randint(-spread, spread + 1, (n_pages, H), generator=g)
        sc = torch.exp2(e.float() - 6)
        b = (x / 2.0 ** -6).clamp(-448, 448).to(torch.float8_e4m3fn)
        pools[t], pools[t + "_scale"] = b, sc
    val = {t: pools[t].float() * pools[t + "_scale"][..., None, None] for t in "kv"}

    def rows(table, n):
        out = []
        for t in "kv":
            x = val[t][table.long()]                         # [pages, H, page, d]
            out.append(x.transpose(1, 2).reshape(-1, H, d)[:n])
        return out

    doc = rows(doc_table, N)
    segs = [rows(seg_table[s], lens[s]) for s in range(P)]
    used = torch.zeros((n_pages, page), dtype=torch.bool)

    def mark(table, n):
        for i, pg in enumerate(table.tolist()):
            used[pg, :max(0, min(page, n - i * page))] = True

    mark(doc_table, N)
    for s in range(P):
        mark(seg_table[s], lens[s])
    for t in "kv":
        b = pools[t].view(torch.uint8).clone()
        b[~used[:, None].expand(-1, H, -1)] = dead
        pools[t] = b.view(torch.float8_e4m3fn)
    dev = torch.device(device)
    if dev.type == "cuda":
        layer = m.KV8Layer(H, d, page, n_pages, P, seg_pages, doc_pages, N, dev,
                           k=pools["k"].to(dev), v=pools["v"].to(dev),
                           k_scale=pools["k_scale"].to(dev), v_scale=pools["v_scale"].to(dev),
                           doc_table=doc_table.to(dev), seg_table=seg_table.to(dev))
    else:
        layer = None
    return layer, doc, segs


def oracle_attn(doc, segs, N, q, q_sid, q_pos, scale, doc_len=None):
    """fp64 oracle over the dequantised rows (every one a bf16 number).  Returns
    o, lse and the two sums the error bound needs: sum p |v| and
    max p * sum |v| over the visible keys."""
    doc_len = N if doc_len is None else doc_len
    H = doc[0].shape[1]
    g = q.shape[1] // H
    ks = torch.cat([doc[0][:doc_len]] + [s[0] for s in segs])
    vs = torch.cat([doc[1][:doc_len]] + [s[1] for s in segs])
    sid = np.concatenate([np.zeros(doc_len)] + [np.full(len(s[0]), i + 1) for i, s in enumerate(segs)])
    pos = np.concatenate([np.arange(doc_len)] + [N + np.arange(len(s[0])) for s in segs])

    def bits(x):
        b = x.to(torch.bfloat16)
        assert torch.equal(b.float(), x), "a dequantised value is not a bf16 number"
        return bf16_bits(b.repeat_interleave(g, 1))

    kb, vb, va = bits(ks), bits(vs), bits(vs.abs())
    qb = bf16_bits(q)
    o, lse, _ = oracle.masked_attention(qb, q_sid, q_pos, kb, vb, sid, pos, scale)
    a, _, _ = oracle.masked_attention(qb, q_sid, q_pos, kb, va, sid, pos, scale)
    return o, lse, a


def check(o, lse, ref, what=""):
    """Element-wise: |o - ref| within
         2^-8 |ref|       the output's rounding to bf16,
         2^-11 sum p|v|   each probability rounded to f16,
         2^-11 sum p|v|   the probabilities' own error: scores are fp32 sums of
                          128 exact products (128 * 2^-24 of |q||k| scale ~ 20:
                          2^-13), an exponential in fp32 or by a polynomial of
                          2.7e-6 (2^-18), in numerator and denominator,
         2^-12 sum p|v|   probabilities below 2^-14 of the row's reference lose
                          2^-25 of it at most: 2^-13 over 4096 keys, twice
       and the scores' error on lse."""
    ro, rl, ra = ref
    og = o.float().cpu().numpy().astype(np.float64)
    err = np.abs(og - ro)
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -10 + 2.0 ** -12) * ra + 1e-30
    assert np.isfinite(og).all(), f"{what}: non-finite output"
    worst = (err / tol).max()
    assert worst <= 1.0, f"{what}: error {worst:.3f} of its bound, max {err.max():.3e}"
    if lse is not None:
        lg = lse.cpu().numpy().astype(np.float64)
        fin = np.isfinite(rl)
        assert np.array_equal(np.isfinite(lg), fin), f"{what}: lse finiteness differs"
        assert (lg[~fin] == -np.inf).all()
        if fin.any():
            e2 = np.abs(lg[fin] - rl[fin]).max()
            assert e2 <= 2.0 ** -12, f"{what}: lse error {e2:.3e}"
    return worst
