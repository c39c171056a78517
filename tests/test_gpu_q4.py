"""The 4-bit store: rows written by the append, read back, and attended.

Written rows are compared bit for bit: the quantiser works on the bf16 row that the bf16 append
stores, in correctly rounded fp32 steps.  Read rows too (m + s u, one fma, one rounding).

Decode tolerances, per output element, with p the exact weights:
  2^-8 |o|                 the output's rounding to bf16
  2^-11 sum p s u          each weight times a row's scale is rounded to fp16 once (codes enter the
                           products exactly)
  n 2^-30 max p max s 15   weights below 2^-20 of the greatest are fp16 subnormals: off by half a
                           spacing, 2^-25, where the greatest is 2^5 or more
  2^-15 sum p s 15         fp32 accumulation, up to ~2^9 roundings of 2^-24
  2 E sum p |v|            scores off by at most E change a weight by a factor e^(+-2E)
with E = scale 2^-19 sum_g s_g 15 sum_d |q_d| (the score's fp32 sum of codes: 32 roundings) + the
same of the minima, 2^-21 scale sum_g |m_g sum_d q_d|, and lse within E + 2^-20 max(1, |lse|).
"""
import math

import numpy as np
import pytest
import torch

import synth
from prefix_sliding_window_b200 import binding as B
from prefix_sliding_window_b200.cache import PrefixSlidingCache, QuantizedCache
from tests import norm_q4_ref as R
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu
D, THETA, EPS = 128, 1.0e6, 1e-6


def _part(part):
    """(k, v, record) tensors -> numpy payloads and records (float64)."""
    return None if part is None else (part[0].cpu().numpy(), part[1].cpu().numpy(), f64(part[2]))


def _values(part, which):
    """Dequantised rows [..., 128] of K (0) or V (1)."""
    u = R.unpack(part[which])
    rec = part[2][..., 4 * which:4 * which + 4].reshape(*part[2].shape[:-1], 2, 2)
    return rec[..., 1:] + rec[..., :1] * u, u, rec[..., :1]


def _random_store(Bn, hkv, rows, seed, dev, garbage=False):
    """A store part of random rows; garbage: payload bytes of noise and NaN records."""
    if rows == 0:
        return None
    g = torch.Generator(device=dev).manual_seed(seed)
    pay = [torch.randint(0, 256, (Bn, hkv, rows, 64), generator=g, device=dev,
                         dtype=torch.int32).to(torch.uint8) for _ in range(2)]
    s = 0.1 + 0.3 * torch.rand(Bn, hkv, rows, 4, generator=g, device=dev)
    m = -7.5 * s + 0.3 * torch.randn(Bn, hkv, rows, 4, generator=g, device=dev)
    rec = torch.stack((s, m), -1).flatten(-2).bfloat16()
    if garbage:
        rec.fill_(float("nan"))
    return pay[0], pay[1], rec.contiguous()


def _visible(p, lp, w, linear):
    if linear:
        return [(0, r) for r in range(p + 1)]
    pre = [(0, r) for r in range(min(lp, p + 1))]
    return pre + [(1, (x - lp) % w) for x in range(max(lp, p - w + 1), p + 1)]


def _check_decode(params, q, out, lse, rows_of, what):
    """rows_of(b) -> (k, v, u, s) of the visible rows: [n, hkv, 128], codes and scales [n,hkv,2,.]"""
    scale = params.softmax_scale or 1 / math.sqrt(D)
    got, got_l, qv = f64(out), f64(lse), f64(q)
    assert np.isfinite(got).all(), what
    grp = params.n_q_heads // params.n_kv_heads
    for b in range(q.shape[0]):
        rows = rows_of(b)
        if rows is None:
            assert (got[b] == 0).all() and (got_l[b] == -np.inf).all()
            continue
        k, v, sk, u, sv = rows
        for head in range(params.n_q_heads):
            h = head // grp
            sc = k[:, h] @ qv[b, head] * scale
            top = sc.max()
            e = np.exp(sc - top)
            z = e.sum()
            p = e / z
            want, want_l = p @ v[:, h], top + math.log(z)
            aq = np.abs(qv[b, head]).reshape(2, 64).sum(-1)
            Qg = np.abs(qv[b, head].reshape(2, 64).sum(-1))
            least = k[:, h].reshape(-1, 2, 64).min(-1)   # m + s u >= m, so |m| <= |least| + 15 s
            E = scale * (2.0 ** -19 * 15 * (sk[:, h, :, 0] @ aq)
                         + 2.0 ** -21 * ((np.abs(least) + 15 * sk[:, h, :, 0]) @ Qg)).max()
            su = (sv[:, h] * u[:, h]).reshape(-1, 128)
            s1 = sv[:, h, :, 0]
            tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * (p @ su) \
                + len(p) * 2.0 ** -30 * p.max() * s1.max() * 15 \
                + 2.0 ** -15 * 15 * np.repeat(p @ s1, 64) + 2 * E * (p @ np.abs(v[:, h]))
            bad = ~(np.abs(got[b, head] - want) <= tol)
            assert not bad.any(), (what, b, head, int(bad.sum()),
                                   np.abs(got[b, head] - want).max())
            assert abs(got_l[b, head] - want_l) <= E + 2.0 ** -20 * max(1, abs(want_l)), \
                (what, b, head, got_l[b, head], want_l)


def _decode(params, cache, q, pos, dev, lse=True):
    Bn, hq = q.shape[0], params.n_q_heads
    out = torch.full((Bn, hq, D), float("nan"), dtype=torch.bfloat16, device=dev)
    l = torch.full((Bn, hq), float("nan"), device=dev)
    n = B.ps_decode_q4_workspace_bytes(params, Bn)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=dev) if n else None
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    B.ps_decode_attn_q4(params, cache, q, pos, out, l if lse else None, ws, st)
    return out, l, st


def _run_contiguous(dev, hq, hkv, lp, w, positions, scale=0.0, seed=1):
    linear = w == 0
    Bn = len(positions)
    params = B.make_params(hq, hkv, D, lp, max(w, 1), THETA, scale)
    pre, ring = _random_store(Bn, hkv, lp, seed, dev), _random_store(Bn, hkv, w, seed + 1, dev)
    q = synth.normal_bf16((Bn, hq, D), seed + 2, dev)
    host = [_part(pre), _part(ring)]
    # rows nothing visible maps to: noise and NaN
    for i, part in enumerate((pre, ring)):
        for b, p in enumerate(positions):
            if part is None or p < 0:
                continue
            see = {r for j, r in _visible(p, lp, w, linear) if j == i}
            hide = [r for r in range(part[2].shape[2]) if r not in see]
            if hide:
                part[2][b, :, hide] = float("nan")
    pos = torch.tensor(positions, device=dev)
    out, lse, st = _decode(params, B.make_cache_q4(pre, ring, Bn), q, pos, dev)
    assert st.item() == (B.PS_DEV_BAD_POS if min(positions) < 0 else 0)

    def rows_of(b):
        if positions[b] < 0:
            return None
        got = []
        for which in (0, 1):
            xs, us, ss = [], [], []
            for i in (0, 1):
                r = [row for j, row in _visible(positions[b], lp, w, linear) if j == i]
                if r:
                    x, u, s = _values(tuple(a[b][:, r] for a in host[i]), which)
                    xs.append(x), us.append(u), ss.append(s)
            got.append([np.concatenate(a, 1).swapaxes(0, 1) for a in (xs, us, ss)])
        (k, _, sk), (v, u, sv) = got
        return k.reshape(-1, hkv, 128), v.reshape(-1, hkv, 128), sk, u, sv
    _check_decode(params, q, out, lse, rows_of, (hq, hkv, lp, w, positions))


@pytest.mark.parametrize("hq,hkv,lp,w,positions", [
    (1, 1, 0, 1, [0]), (1, 1, 0, 1, [5]), (2, 2, 1, 1, [0, 1]), (16, 2, 100, 512, [0]),
    (16, 2, 100, 512, [611]), (16, 2, 100, 512, [612, 99, 100, 2000, 33]),
    (28, 4, 7, 33, [0, 6, 7, 38, 39, 40, 71, 72, -1, 1000]),
    (8, 1, 0, 300, [298, 299, 300, 10000]), (3, 3, 13, 64, [76, 77, 100, 141]),
    (5, 1, 257, 255, [255, 256, 257, 511, 512, 700]), (16, 2, 2000, 0, [0, 1, 127, 1500, 1999]),
    (4, 4, 64, 4096, [9000, 4159, 4160]), (16, 2, 100, 4096, [131072])])
def test_decode_matches_reference(cuda_device, hq, hkv, lp, w, positions):
    _run_contiguous(cuda_device, hq, hkv, lp, w, positions)


def test_decode_custom_scale_and_far_positions(cuda_device):
    _run_contiguous(cuda_device, 14, 2, 20, 100, [(1 << 31) - 1, 50, 119], scale=0.31, seed=40)


@pytest.mark.parametrize("Bn,hkv", [(160, 2), (40, 8), (600, 1), (1100, 1), (296, 1), (100, 2)])
def test_decode_many_units(cuda_device, Bn, hkv):
    """Around and above the number of blocks the GPU holds, mixed lengths."""
    rng = np.random.default_rng(Bn)
    pos = [int(x) for x in rng.integers(0, 400, Bn)]
    _run_contiguous(cuda_device, 2 * hkv, hkv, 9, 140, pos, seed=Bn)


def test_decode_one_long_among_short(cuda_device):
    _run_contiguous(cuda_device, 8, 2, 3000, 0, [2999, 0, 1, 2, 3, 4, 5])


@pytest.mark.parametrize("hq,hkv,lp,positions", [
    (2, 1, 70000, [69999]),                           # more pieces than a round of the merge
    (4, 2, 5000, [4999, 0, 300, 4000, 31, 2047] * 4),  # a few pieces a unit, short ones among them
    (8, 8, 9000, [8999, 1, 5000] * 8)])
def test_decode_in_pieces(cuda_device, hq, hkv, lp, positions):
    _run_contiguous(cuda_device, hq, hkv, lp, 0, positions, seed=lp)


@pytest.mark.parametrize("back", [False, True])
def test_decode_scales_of_all_sizes(cuda_device, back):
    """V scales that jump by many powers of two from tile to tile, either way: constant groups,
    2^-40, 2^-10, 1, 2^30; a query sees one more of these segments each."""
    dev, hkv, hq, seg = cuda_device, 2, 6, 300
    scales = [0.0, 2.0 ** -40, 2.0 ** -10, 1.0, 2.0 ** 30]
    if back:
        scales.reverse()
    n = seg * len(scales)
    one = _random_store(1, hkv, n, 77, dev)
    g = torch.Generator(device=dev).manual_seed(78)
    rec = one[2].view(1, hkv, n, 4, 2)
    for i, s in enumerate(scales):
        x = rec[:, :, i * seg:(i + 1) * seg, 2:]
        x[..., 0] = s
        m = 1 + torch.rand(x.shape[:-1], generator=g, device=dev)
        x[..., 1] = (m if s < 0.5 else -7.5 * s * m).bfloat16()
    Bn = len(scales)
    part = tuple(x.expand(Bn, *x.shape[1:]).contiguous() for x in one)
    params = B.make_params(hq, hkv, D, n, 1, THETA)
    q = synth.normal_bf16((1, hq, D), 79, dev).expand(Bn, hq, D).contiguous()
    pos = torch.tensor([seg * (i + 1) - 1 for i in range(Bn)], device=dev)
    out, lse, st = _decode(params, B.make_cache_q4(part, None, Bn), q, pos, dev)
    assert st.item() == 0
    host = _part(part)

    def rows_of(b):
        r = seg * (b + 1)
        (k, _, sk), (v, u, sv) = (_values(tuple(a[b, :, :r] for a in host), i) for i in (0, 1))
        return tuple(x.swapaxes(0, 1).reshape(r, hkv, *t) for x, t in (
            (k, (128,)), (v, (128,)), (sk, (2, 1)), (u, (2, 64)), (sv, (2, 1))))
    _check_decode(params, q, out, lse, rows_of, ("scales", back))


@pytest.mark.parametrize("value", [0.0, -1.0, 2.0 ** 29, 2.0 ** -40])
def test_decode_constant_values(cuda_device, value):
    """Every V row is one constant: so is the output (to its rounding and 2^-15 of the sums')."""
    dev, hkv, hq, n = cuda_device, 1, 8, 5000
    part = _random_store(1, hkv, n, 80, dev)
    rec = part[2].view(1, hkv, n, 4, 2)
    rec[..., 2:, 0], rec[..., 2:, 1] = 0.0, value
    params = B.make_params(hq, hkv, D, n, 1, THETA)
    q = synth.normal_bf16((1, hq, D), 81, dev)
    out, _, _ = _decode(params, B.make_cache_q4(part, None, 1), q,
                        torch.tensor([n - 1], device=dev), dev)
    assert (np.abs(f64(out) - value) <= (2.0 ** -8 + 2.0 ** -15) * abs(value)).all()


def _paged(dev, lp, w, positions, bad=None, hq=14, hkv=2):
    Bn = len(positions)
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    nb, per = -(-lp // 64), -(-lp // 64) + w // 64
    blocks = Bn * per + 5
    pool = _random_store(blocks, hkv, 64, 3, dev)
    table = torch.randperm(blocks, generator=torch.Generator().manual_seed(2))[:Bn * per]
    table = table.view(Bn, per).int()
    if Bn > 1 and nb:
        table[1, :nb] = table[0, :nb]                 # a shared prompt
    host, ht = _part(pool), table.numpy().copy()
    if bad is not None:
        table[bad[0], bad[1]] = bad[2]
    seen = np.zeros((blocks, 64), bool)
    where = []
    for b, p in enumerate(positions):
        rows = [(ht[b, (nb if i else 0) + r // 64], r % 64)
                for i, r in _visible(p, lp, w, False)
                if bad is None or (b, (nb if i else 0) + r // 64) != (bad[0], bad[1])]
        for r in rows:
            seen[r] = True
        where.append(rows)
    hide = torch.from_numpy(~seen).to(dev)
    pool[2].masked_fill_(hide[:, None, :, None], float("nan"))
    q = synth.normal_bf16((Bn, hq, D), 4, dev)
    cache = B.make_cache_q4(pool, None, Bn, table.to(dev))
    out, lse, st = _decode(params, cache, q, torch.tensor(positions, device=dev), dev)
    assert st.item() == (0 if bad is None else B.PS_DEV_POS_RANGE)

    def rows_of(b):
        idx = tuple(np.array(where[b]).T)
        (k, _, sk), (v, u, sv) = (_values(tuple(a[idx[0], :, idx[1]] for a in host), i)
                                  for i in (0, 1))
        return k.reshape(-1, hkv, 128), v.reshape(-1, hkv, 128), sk, u, sv
    _check_decode(params, q, out, lse, rows_of, ("paged", lp, w, positions))


@pytest.mark.parametrize("lp,w,positions", [
    (100, 128, [0, 99, 100, 227, 228, 300, 5000]), (0, 64, [0, 63, 64, 100]),
    (64, 192, [63, 64, 255, 256, 400])])
def test_decode_paged(cuda_device, lp, w, positions):
    _paged(cuda_device, lp, w, positions)


@pytest.mark.parametrize("entry", [-1, 1 << 20])
def test_decode_paged_bad_entry(cuda_device, entry):
    _paged(cuda_device, 100, 128, [300, 700], bad=(1, 3, entry))


# ---------------------------------------------------------------- appends and reads
def _rows(Bn, T, hq, hkv, seed, dev):
    rows = synth.normal_bf16((Bn, T, hq + 2 * hkv, D), seed, dev)
    return rows[:, :, :hq], rows[:, :, hq:hq + hkv], rows[:, :, hq + hkv:]


def _same_as_bf16(part, k, v, where):
    """The 4-bit rows `where` (index arrays into [B, hkv, rows]) equal the quantised bf16 rows."""
    pay_k, pay_v, rec = part[0].cpu().numpy(), part[1].cpu().numpy(), f64(part[2])
    for i, (pay, x) in enumerate(((pay_k, f64(k)), (pay_v, f64(v)))):
        u, s, m = R.quantise(x[where])
        assert np.array_equal(pay[where], R.pack(u))
        assert np.array_equal(rec[where][..., 4 * i:4 * i + 4],
                              np.concatenate((s, m), -1).reshape(*s.shape[:-2], 4))


@pytest.mark.parametrize("layout,rd,norm", [("half", 128, True), ("interleaved", 64, True),
                                            ("half", 32, False), ("half", 112, True)])
@pytest.mark.parametrize("T,starts", [(1, [0, 69, 70, 5000]), (257, [0, 10, 69, 333])])
def test_append_and_read(cuda_device, layout, rd, norm, T, starts):
    dev = cuda_device
    Bn, hq, hkv, lp, w = len(starts), 6, 3, 70, 128
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    rope = B.make_rope(params, layout, rd)
    wq, wk = ((1 + 0.3 * torch.randn(2, D, generator=torch.Generator().manual_seed(8))).to(dev))
    nrm = B.make_norm(wq, wk, EPS) if norm else None
    q, k, v = _rows(Bn, T, hq, hkv, 5, dev)
    k[:, :, 0] *= 100.0          # spreads of other sizes, and constant and zero groups
    k[0, 0, 1] = 0.0
    v[0, 0, 0] = 0.25
    v[1, 0, 1, 64:] = 0.0
    pos0 = torch.tensor(starts, device=dev)
    bf = PrefixSlidingCache(Bn, hkv, lp, w, D, dev, fill=9.0)
    q4 = QuantizedCache(Bn, hkv, lp, w, dev)
    for part in (q4.prefix, q4.ring):
        part[0].fill_(0xa5), part[1].fill_(0x5a), part[2].fill_(9.0)
    qa, qb = (torch.empty(Bn, T, hq, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    B.ps_kv_append_norm_rope(params, rope, nrm, bf.struct, k, v, q, qa, pos0, T)
    B.ps_kv_append_norm_rope_q4(params, rope, nrm, q4.struct, k, v, q, qb, pos0, T, st)
    kr, vr = (torch.full((Bn, T, hkv, D), float("nan"), dtype=torch.bfloat16, device=dev)
              for _ in range(2))
    B.ps_kv_read_q4(params, q4.struct, pos0, T, kr, vr, st)
    assert st.item() == 0 and torch.equal(qa, qb)
    wrote = [np.zeros((Bn, n), bool) for n in (lp, w)]
    held = np.zeros((Bn, T), bool)
    rows = {}
    for b, s in enumerate(starts):
        for t in range(T):
            p = s + t
            if p < lp or p > s + T - 1 - w:
                i, r = (0, p) if p < lp else (1, (p - lp) % w)
                wrote[i][b, r] = held[b, t] = True
                rows[b, t] = (i, r)
    for i, (part, kb, vb) in enumerate(((q4.prefix, bf.k_prefix, bf.v_prefix),
                                        (q4.ring, bf.k_ring, bf.v_ring))):
        b, r = np.nonzero(wrote[i])
        if len(b):
            _same_as_bf16([x.transpose(1, 2) for x in part], kb.transpose(1, 2),
                          vb.transpose(1, 2), (b, r))
        hide = torch.from_numpy(~wrote[i]).to(dev)
        assert (part[0].transpose(1, 2)[hide] == 0xa5).all()
        assert (part[2].transpose(1, 2)[hide] == 9.0).all()
    host = [_part(q4.prefix), _part(q4.ring)]
    for which, got in ((0, f64(kr)), (1, f64(vr))):
        assert (got[~held] == 0).all()
        for i in (0, 1):
            at = [(b, t, r) for (b, t), (j, r) in rows.items() if j == i]
            if at:
                b, t, r = np.array(at).T
                x, _, _ = _values(tuple(a[b, :, r] for a in host[i]), which)
                assert np.array_equal(got[b, t], R.bf16(x.reshape(-1, hkv, 128)))


def test_append_values_that_are_not_finite(cuda_device):
    """An infinity or a NaN makes its group NaN, and only its group; huge spreads too."""
    dev = cuda_device
    params = B.make_params(1, 1, D, 8, 8, THETA)
    rope = B.make_rope(params, rotary_dim=0)
    q4 = QuantizedCache(1, 1, 8, 8, dev)
    k = synth.normal_bf16((1, 4, 1, D), 1, dev)
    v = synth.normal_bf16((1, 4, 1, D), 2, dev)
    k[0, 0, 0, 3] = float("inf")
    k[0, 1, 0, 70] = float("nan")
    v[0, 2, 0, 127] = float("-inf")
    v[0, 3, 0, 0], v[0, 3, 0, 1] = 3e38, -3e38
    pos0 = torch.zeros(1, dtype=torch.int64, device=dev)
    B.ps_kv_append_norm_rope_q4(params, rope, None, q4.struct, k, v, None, None, pos0, 4)
    kr, vr = (torch.empty(1, 4, 1, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    B.ps_kv_read_q4(params, q4.struct, pos0, 4, kr, vr)
    nan_k, nan_v = torch.isnan(kr[0, :, 0]).cpu(), torch.isnan(vr[0, :, 0]).cpu()
    want_k, want_v = torch.zeros(4, D, dtype=torch.bool), torch.zeros(4, D, dtype=torch.bool)
    want_k[0, :64] = want_k[1, 64:] = want_v[2, 64:] = want_v[3, :64] = True
    assert torch.equal(nan_k, want_k) and torch.equal(nan_v, want_v)
    only_v = torch.empty_like(vr)
    B.ps_kv_read_q4(params, q4.struct, pos0, 4, None, only_v)
    assert torch.equal(only_v.view(torch.int16), vr.view(torch.int16))


def test_linear_ring_only_and_paged_appends(cuda_device):
    """The same tokens through a linear, a ring-only and a paged 4-bit store hold the same rows."""
    dev = cuda_device
    Bn, T, hq, hkv, lp, w = 2, 90, 4, 2, 70, 64
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    rope = B.make_rope(params)
    q, k, v = _rows(Bn, T, hq, hkv, 6, dev)
    pos0 = torch.tensor([0, 30], device=dev)
    full = QuantizedCache(Bn, hkv, lp, w, dev)
    B.ps_kv_append_norm_rope_q4(params, rope, None, full.struct, k, v, None, None, pos0, T)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    lin = QuantizedCache(Bn, hkv, 118, 0, dev)
    B.ps_kv_append_norm_rope_q4(lin.params(hq), rope, None, lin.struct, k, v, None, None, pos0, T,
                                st)
    assert st.item() == B.PS_DEV_POS_RANGE      # positions 118 and 119 have no row
    for a, b in zip(full.prefix, lin.prefix):
        assert torch.equal(a, b[:, :, :lp])
    for x in range(70, 118):
        for a, b in zip(full.ring, lin.prefix):
            assert torch.equal(a[1, :, x - 70], b[1, :, x])
    read = torch.empty(Bn, T, hkv, D, dtype=torch.bfloat16, device=dev)
    B.ps_kv_read_q4(lin.params(hq), lin.struct, pos0, T, read, None)
    assert (read[1, 88:] == 0).all() and (read[1, 87] != 0).any()
    st.zero_()
    ring = QuantizedCache(Bn, hkv, 0, w, dev)
    B.ps_kv_append_norm_rope_q4(params, rope, None, B.make_cache_q4(None, ring.ring, Bn), k, v,
                                None, None, pos0, T, st)
    assert st.item() == B.PS_DEV_POS_RANGE      # the prompt's rows live elsewhere
    for a, b in zip(full.ring, ring.ring):
        assert torch.equal(a, b)
    pool = QuantizedCache(8, hkv, 64, 0, dev).prefix
    table = torch.tensor([[5, 2, 7], [0, 3, 6]], dtype=torch.int32, device=dev)
    cache = B.make_cache_q4(pool, None, Bn, table)
    B.ps_kv_append_norm_rope_q4(params, rope, None, cache, k, v, None, None, pos0, T)
    for a, pre, rng in zip(pool, full.prefix, full.ring):
        for b in range(Bn):
            t = table[b].tolist()
            assert torch.equal(a[t[0]], pre[b, :, :64])
            assert torch.equal(a[t[1], :, :6], pre[b, :, 64:])
            assert torch.equal(a[t[2]], rng[b])
    reads = [torch.empty(Bn, T, hkv, D, dtype=torch.bfloat16, device=dev) for _ in range(4)]
    B.ps_kv_read_q4(params, cache, pos0, T, reads[0], reads[1])
    B.ps_kv_read_q4(params, full.struct, pos0, T, reads[2], reads[3])
    assert torch.equal(reads[0], reads[2]) and torch.equal(reads[1], reads[3])


def test_offsets_past_32_bits(cuda_device):
    """Rows whose byte offset passes 2^32: the last sequence of a long linear store."""
    dev = cuda_device
    Bn, hkv, lmax, hq = 9, 4, 2_000_000, 8      # payload 4.6e9 bytes each
    params = B.make_params(hq, hkv, D, lmax, 1, THETA)
    part = tuple(torch.empty(Bn, hkv, lmax, n, dtype=t, device=dev)
                 for n, t in ((64, torch.uint8), (64, torch.uint8), (8, torch.bfloat16)))
    cache = B.make_cache_q4(part, None, Bn)
    rope = B.make_rope(params)
    T = 200
    q, k, v = _rows(Bn, T, hq, hkv, 6, dev)
    pos0 = torch.zeros(Bn, dtype=torch.int64, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    qo = torch.empty(Bn, T, hq, D, dtype=torch.bfloat16, device=dev)
    B.ps_kv_append_norm_rope_q4(params, rope, None, cache, k, v, q, qo, pos0, T, st)
    pos = torch.full((Bn,), T - 1, dtype=torch.int64, device=dev)
    qd = qo[:, -1].contiguous()
    out, lse, st2 = _decode(params, cache, qd, pos, dev)
    assert st.item() == 0 and st2.item() == 0
    small = QuantizedCache(Bn, hkv, T, 0, dev)
    ps = small.params(hq)
    B.ps_kv_append_norm_rope_q4(ps, rope, None, small.struct, k, v, None, None, pos0, T)
    host = _part(small.prefix)

    def rows_of(b):
        (kk, _, sk), (vv, u, sv) = (_values(tuple(a[b] for a in host), i) for i in (0, 1))
        return tuple(x.swapaxes(0, 1).reshape(T, hkv, *s) for x, s in (
            (kk, (128,)), (vv, (128,)), (sk, (2, 1)), (u, (2, 64)), (sv, (2, 1))))
    _check_decode(params, qd, out, lse, rows_of, "offsets")


def test_serving_loop_together(cuda_device):
    """A prompt, then decode steps past the window's wrap: append and attend, each step's output
    against 64-bit attention over the rows the store should hold."""
    dev = cuda_device
    Bn, hq, hkv, lp, w, steps = 3, 14, 2, 21, 40, 60
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    rope = B.make_rope(params)
    wq, wk = ((1 + 0.3 * torch.randn(2, D, generator=torch.Generator().manual_seed(8))).to(dev))
    norm = B.make_norm(wq, wk, EPS)
    cache = QuantizedCache(Bn, hkv, lp, w, dev)
    prompts = [21, 5, 30]
    total = max(prompts) + steps
    q, k, v = _rows(Bn, total, hq, hkv, 12, dev)
    # the values each position's row stands for, through a linear store
    lin = QuantizedCache(Bn, hkv, total, 0, dev)
    zero = torch.zeros(Bn, dtype=torch.int64, device=dev)
    B.ps_kv_append_norm_rope_q4(lin.params(hq), rope, norm, lin.struct, k, v, None, None, zero,
                                total)
    host = _part(lin.prefix)
    for b, n in enumerate(prompts):              # prompts of different lengths
        one = B.make_cache_q4(tuple(x[b:b + 1] for x in cache.prefix),
                              tuple(x[b:b + 1] for x in cache.ring), 1)
        B.ps_kv_append_norm_rope_q4(params, rope, norm, one, k[b:b + 1, :n], v[b:b + 1, :n], None,
                                    None, zero[:1], n)
    pos = torch.tensor(prompts, device=dev)
    ar = torch.arange(Bn, device=dev)
    for step in range(steps):
        kt, vt, qt = (x[ar, pos][:, None] for x in (k, v, q))
        qo = torch.empty(Bn, 1, hq, D, dtype=torch.bfloat16, device=dev)
        B.ps_kv_append_norm_rope_q4(params, rope, norm, cache.struct, kt, vt, qt, qo, pos, 1)
        out, lse, st = _decode(params, cache.struct, qo[:, 0], pos, dev)
        assert st.item() == 0
        if step % 7 == 0 or step == steps - 1:
            def rows_of(b):
                p = prompts[b] + step
                r = [x for x in range(p + 1) if x < lp or x > p - w]
                (kk, _, sk), (vv, u, sv) = (_values(tuple(a[b][:, r] for a in host), i)
                                            for i in (0, 1))
                return tuple(x.swapaxes(0, 1).reshape(len(r), hkv, *s) for x, s in (
                    (kk, (128,)), (vv, (128,)), (sk, (2, 1)), (u, (2, 64)), (sv, (2, 1))))
            _check_decode(params, qo[:, 0], out, lse, rows_of, step)
        pos = pos + 1


def test_captured_steps_and_streams(cuda_device):
    """Append + decode captured into two graphs that replay on two streams with workspaces of
    their own give the eager results."""
    dev = cuda_device
    hq, hkv, lp, w, Bn = 16, 2, 100, 600, 4
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    rope = B.make_rope(params)
    runs = []
    for i in range(2):
        cache = QuantizedCache(Bn, hkv, lp, w, dev)
        q, k, v = _rows(Bn, 900, hq, hkv, 60 + i, dev)
        zero = torch.zeros(Bn, dtype=torch.int64, device=dev)
        B.ps_kv_append_norm_rope_q4(params, rope, None, cache.struct, k, v, None, None, zero, 900)
        st = dict(cache=cache, q=q[:, :1].clone(), k=k[:, :1].clone(), v=v[:, :1].clone(),
                  qo=torch.empty(Bn, 1, hq, D, dtype=torch.bfloat16, device=dev),
                  out=torch.empty(Bn, hq, D, dtype=torch.bfloat16, device=dev),
                  lse=torch.empty(Bn, hq, device=dev),
                  pos=torch.tensor([900, 901, 950, 1500], device=dev),
                  ws=torch.empty(max(1, B.ps_decode_q4_workspace_bytes(params, Bn)),
                                 dtype=torch.uint8, device=dev))

        def step(s=st):
            B.ps_kv_append_norm_rope_q4(params, rope, None, s["cache"].struct, s["k"], s["v"],
                                        s["q"], s["qo"], s["pos"], 1)
            B.ps_decode_attn_q4(params, s["cache"].struct, s["qo"], s["pos"], s["out"], s["lse"],
                                s["ws"])
        st["step"] = step
        step()
        torch.cuda.synchronize()
        st["want"] = (st["out"].clone(), st["lse"].clone(), st["qo"].clone())
        st["stream"] = torch.cuda.Stream()
        st["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(st["graph"], stream=st["stream"]):
            step()
        runs.append(st)
    for s in runs:
        s["out"].fill_(float("nan")), s["lse"].fill_(float("nan")), s["qo"].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        for s in runs:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
    torch.cuda.synchronize()
    for s in runs:
        for a, b in zip(s["want"], (s["out"], s["lse"], s["qo"])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("Bn", [256, 257, 700])
def test_append_many_sequences(cuda_device, Bn):
    """More tokens than blocks, from many sequences (some at positions that no store has): the rows
    and queries of slices of the batch appended one by one."""
    dev, T, hq, hkv, lp, w = cuda_device, 3, 4, 2, 5, 4
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    rope = B.make_rope(params)
    weights = [(1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(i))).to(dev)
               for i in (1, 2)]
    norm = B.make_norm(*weights, EPS)
    q, k, v = _rows(Bn, T, hq, hkv, 31, dev)
    pos0 = torch.randint(0, 40, (Bn,), generator=torch.Generator().manual_seed(Bn)).to(dev)
    pos0[3], pos0[Bn - 2], pos0[Bn - 1] = -2, (1 << 31) - 1, 1 << 40
    runs = []
    for step in (Bn, 50):
        bf = PrefixSlidingCache(Bn, hkv, lp, w, D, dev, fill=9.0)
        q4 = QuantizedCache(Bn, hkv, lp, w, dev)
        outs = [torch.full((Bn, T, hq, D), 7.0, dtype=torch.bfloat16, device=dev)
                for _ in range(2)]
        st = torch.zeros(2, dtype=torch.int32, device=dev)
        for b in range(0, Bn, step):
            e = min(b + step, Bn)
            c = B.make_cache(*(x[b:e] for x in (bf.k_prefix, bf.v_prefix, bf.k_ring, bf.v_ring)),
                             e - b)
            c4 = B.make_cache_q4(*(tuple(x[b:e] for x in p) for p in (q4.prefix, q4.ring)), e - b)
            B.ps_kv_append_norm_rope(params, rope, norm, c, k[b:e], v[b:e], q[b:e],
                                     outs[0][b:e], pos0[b:e], T, st[:1])
            B.ps_kv_append_norm_rope_q4(params, rope, norm, c4, k[b:e], v[b:e], q[b:e],
                                        outs[1][b:e], pos0[b:e], T, st[1:])
        runs.append([bf.k_prefix, bf.v_prefix, bf.k_ring, bf.v_ring, *q4.prefix, *q4.ring, *outs,
                     st])
    for x, y in zip(*runs):
        assert torch.equal(x, y)
    assert (runs[0][-1] == (B.PS_DEV_BAD_POS | B.PS_DEV_POS_RANGE)).all()
    assert (runs[0][-2][Bn - 1] == 0).all() and (runs[0][-2][3, :2] == 0).all()
    assert (runs[0][-2][3, 2] != 0).any()     # position 0
