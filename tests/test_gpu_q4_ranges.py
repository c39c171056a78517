"""Decode over 4-bit stores whose V scales differ by many powers of two: between the two groups of
a row, between rows, and against the weights.

A weight times its row's V scale is rounded to fp16 on a scale of its own for every query head and
group, which follows the greatest such product.  Tolerance of an output of group g, with p the
exact weights and M_g = max_k p_k s_kg:
  2^-8 |o|                      the output's rounding to bf16
  2^-11 sum p s u               the products' rounding to fp16
  15 sum min(p s, 2^-21 M_g)    products that are fp16 subnormals: off by half a spacing, 2^-25,
                                where the greatest is 2^-4 or more, and never by more than themselves
  2^-15 sum p (15 s + |m|)      fp32 accumulation, up to ~2^9 roundings of 2^-24
  2 E sum p |v|                 scores off by at most E change a weight by a factor e^(+-2E)
with E = scale (2^-19 sum_g 15 s_g sum_{d in g} |q_d| + 2^-21 sum_g |m_g sum_{d in g} q_d|), s and m
here K's, as in the tests of ordinary stores.
"""
import math

import numpy as np
import pytest
import torch

import synth
from prefix_sliding_window_b200 import binding as B
from prefix_sliding_window_b200.cache import QuantizedCache
from tests import norm_q4_ref as R
from tests.gpu_util import f64
from tests.test_gpu_q4 import _decode, _part, _random_store, _values

pytestmark = pytest.mark.gpu
D, THETA = 128, 1.0e6


def _check(params, q, out, lse, part, lengths, what):
    """Linear store `part` [B, hkv, rows]; sequence b sees its first lengths[b] rows."""
    scale = 1 / math.sqrt(D)
    got, got_l, qv = f64(out), f64(lse), f64(q)
    grp = params.n_q_heads // params.n_kv_heads
    for b, n in enumerate(lengths):
        rows = tuple(a[b, :, :n].swapaxes(0, 1) for a in part)
        (k, _, sk), (v, u, sv) = (_values(rows, i) for i in (0, 1))
        k, v = k.reshape(n, -1, D), v.reshape(n, -1, D)
        mk, mv = rows[2][..., [1, 3]], rows[2][..., [5, 7]]
        want, want_l = R.attend(qv[b], k, v, scale)
        for head in range(params.n_q_heads):
            h = head // grp
            sc = k[:, h] @ qv[b, head] * scale
            p = np.exp(sc - want_l[head])
            aq = np.abs(qv[b, head]).reshape(2, 64).sum(-1)
            Q = qv[b, head].reshape(2, 64).sum(-1)
            E = scale * (2.0 ** -19 * 15 * (sk[:, h, :, 0] @ aq)
                         + 2.0 ** -21 * np.abs(mk[:, h] * Q).sum(-1)).max()
            ps = p[:, None] * sv[:, h, :, 0]                              # [n, 2]
            small = 15 * np.minimum(ps, 2.0 ** -21 * ps.max(0)).sum(0)
            acc = 2.0 ** -15 * (15 * ps.sum(0) + p @ np.abs(mv[:, h]))
            tol = 2.0 ** -8 * np.abs(want[head]) \
                + 2.0 ** -11 * (ps[:, :, None] * u[:, h]).sum(0).reshape(D) \
                + np.repeat(small + acc, 64) + 2 * E * (p @ np.abs(v[:, h]))
            bad = ~(np.abs(got[b, head] - want[head]) <= tol)
            assert not bad.any(), (what, b, head, int(bad.sum()), np.argwhere(bad)[0],
                                   np.abs(got[b, head] - want[head]).max())
            assert abs(got_l[b, head] - want_l[head]) <= E + 2.0 ** -20 * max(1, abs(want_l[head]))


def _scaled(dev, hkv, n, seed, scale_of):
    """A random store whose V groups have the scales scale_of(row) [n, 2] and centred minima."""
    part = _random_store(1, hkv, n, seed, dev)
    rec = part[2].view(1, hkv, n, 4, 2)
    s = torch.as_tensor(scale_of(np.arange(n)), dtype=torch.float64, device=dev)
    rec[..., 2:, 0] = s.bfloat16()
    rec[..., 2:, 1] = (-7.5 * s).bfloat16()
    return part


def _run(dev, hq, hkv, part, q, lengths, what):
    n = part[2].shape[2]
    Bn = len(lengths)
    params = B.make_params(hq, hkv, D, n, 1, THETA)
    part = tuple(x.expand(Bn, *x.shape[1:]).contiguous() for x in part)
    q = q.expand(Bn, hq, D).contiguous()
    pos = torch.tensor([x - 1 for x in lengths], device=dev)
    out, lse, st = _decode(params, B.make_cache_q4(part, None, Bn), q, pos, dev)
    assert st.item() == 0
    _check(params, q, out, lse, _part(part), lengths, what)


@pytest.mark.parametrize("lo,hi", [(0, 34), (34, 0), (-30, 60), (60, -30), (-60, -20), (-100, 100),
                                   (100, -100)])
def test_groups_of_different_scales(cuda_device, lo, hi):
    """The two groups of every row apart by up to 2^200: each keeps its own bits."""
    part = _scaled(cuda_device, 2, 700, 5,
                   lambda r: np.stack((2.0 ** lo + 0 * r, 2.0 ** hi + 0 * r), -1))
    q = synth.normal_bf16((1, 6, D), 6, cuda_device)
    _run(cuda_device, 6, 2, part, q, [1, 33, 700], (lo, hi))


@pytest.mark.parametrize("ratio", [12, 24, 30, 40, 90])
@pytest.mark.parametrize("where", ["first", "last", "each tile"])
def test_large_scales_without_weight(cuda_device, ratio, where):
    """Rows whose V scale is 2^ratio of the others', and whose weight is 2^-(ratio + 40) of theirs
    or less: the others keep their bits, wherever those rows are."""
    dev, n, hq, hkv = cuda_device, 1500, 4, 1
    big = {"first": np.arange(32), "last": np.arange(n - 32, n), "each tile": np.arange(0, n, 32)}
    big = big[where]
    part = _scaled(dev, hkv, n, 7, lambda r: np.where(
        np.isin(r, big), 2.0 ** ratio, 1.0)[:, None] * np.array([1.0, 0.25]))
    # dim 0 of every query is 8 and of those rows' keys far below zero: a whole group of K of
    # codes 0 standing for m
    q = synth.normal_bf16((1, hq, D), 8, dev)
    q[..., :64] = 0.125
    rec = part[2].view(1, hkv, n, 4, 2)
    idx = torch.as_tensor(big, device=dev)
    part[0][:, :, idx] = 0
    rec[:, :, idx, 0, 1] = -2.0 * (ratio + 64)   # score: 64 dims x 0.125 x m / sqrt(128) < -m
    _run(dev, hq, hkv, part, q, [n], (ratio, where))


def test_scales_that_fall_as_weights_rise(cuda_device):
    """Scores rise and V scales fall from tile to tile, so that the greatest product moves on while
    its row's scale is far below the greatest scale."""
    dev, n, hq, hkv = cuda_device, 2048, 8, 1
    part = _scaled(dev, hkv, n, 9, lambda r: 2.0 ** (30 - 0.03 * r)[:, None] * np.ones(2))
    q = torch.full((1, hq, D), 0.125, dtype=torch.bfloat16, device=dev)
    q *= torch.arange(1, hq + 1, device=dev)[None, :, None]
    rec = part[2].view(1, hkv, n, 4, 2)
    part[0].zero_()
    m = (torch.arange(n, device=dev) * 0.05).bfloat16()   # score of row r: head's factor x m
    rec[0, 0, :, :2, 1] = m[:, None]
    _run(dev, hq, hkv, part, q, [n, 1000], "falling")


@pytest.mark.parametrize("value", [2.0 ** 60, -(2.0 ** 90), 2.0 ** -100])
def test_constant_groups_of_any_size(cuda_device, value):
    """V rows of one constant beside a group of ordinary ones."""
    dev, n = cuda_device, 3000
    part = _random_store(1, 1, n, 10, dev)
    rec = part[2].view(1, 1, n, 4, 2)
    rec[..., 2, 0], rec[..., 2, 1] = 0.0, value
    q = synth.normal_bf16((1, 8, D), 11, dev)
    _run(dev, 8, 1, part, q, [n, 40], value)


@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 66, 2.0 ** -40])
def test_queries_of_any_size(cuda_device, size):
    """Large queries (keys scaled down against them) and tiny ones."""
    dev, n = cuda_device, 600
    part = _random_store(1, 2, n, 12, dev)
    rec = part[2].view(1, 2, n, 4, 2)
    rec[..., :2, :] = (rec[..., :2, :].double() / size).bfloat16()
    q = (synth.normal_bf16((1, 4, D), 13, dev).double() * size).bfloat16()
    _run(dev, 4, 2, part, q, [n], size)


def test_rows_that_are_not_numbers(cuda_device):
    """A visible row with a NaN group in V makes that group's outputs NaN and no other; one in K all
    of its head's; the same row out of sight changes nothing."""
    dev, n, hq, hkv = cuda_device, 300, 4, 2
    part = _random_store(1, hkv, n, 14, dev)
    q = synth.normal_bf16((1, hq, D), 15, dev)
    params = B.make_params(hq, hkv, D, n, 1, THETA)
    row = 123
    for which in ("k", "v"):
        bad = tuple(x.clone() for x in part)
        rec = bad[2].view(1, hkv, n, 4, 2)
        rec[0, 1, row, 0 if which == "k" else 3] = float("nan")   # of KV head 1, group 0 / 1
        for last, seen in ((row, True), (n - 1, True), (row - 1, False)):
            pos = torch.tensor([last], device=dev)
            good, gl, _ = _decode(params, B.make_cache_q4(part, None, 1), q, pos, dev)
            out, lse, st = _decode(params, B.make_cache_q4(bad, None, 1), q, pos, dev)
            assert st.item() == 0
            nan = torch.zeros(1, hq, D, dtype=torch.bool, device=dev)
            if seen and which == "k":
                nan[:, 2:] = True
            if seen and which == "v":
                nan[:, 2:, 64:] = True
            assert torch.equal(torch.isnan(out), nan), (which, last)
            assert torch.equal(torch.isnan(lse), nan.all(-1))
            # the other KV head's outputs are untouched; in the row's own one, weights may be held
            # on another scale: products off by 2^-11 of at most 15 x 0.4 each, twice, and the
            # outputs' roundings
            same = ~nan
            if seen:
                near = (out - good).abs() <= 2.0 ** -7 * good.abs() + 2.0 ** -10 * 6
                assert near[~nan].all()
                same[:, 2:] = False
            assert torch.equal(out[same], good[same])


def test_same_bits_again(cuda_device):
    """The same call gives the same bits: pieces, warps and merges add in a fixed order."""
    dev, hq, hkv, lp, w, Bn = cuda_device, 14, 2, 100, 2000, 40
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    pre, ring = (_random_store(Bn, hkv, r, r, dev) for r in (lp, w))
    q = synth.normal_bf16((Bn, hq, D), 16, dev)
    pos = synth.uniform_positions(Bn, 0, 5000, 17, dev)
    cache = B.make_cache_q4(pre, ring, Bn)
    first = _decode(params, cache, q, pos, dev)
    for _ in range(20):
        again = _decode(params, cache, q, pos, dev)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_store_made_by_the_append_with_contrasts(cuda_device):
    """The same through the store's own quantiser: values whose groups differ by 2^34."""
    dev, T, hq, hkv = cuda_device, 200, 4, 2
    cache = QuantizedCache(1, hkv, T, 0, dev)
    params = cache.params(hq)
    rope = B.make_rope(params)
    q, k, v = (synth.normal_bf16((1, T, h, D), 20 + h, dev) for h in (hq, hkv, hkv))
    v[..., :64] *= 2.0 ** 34
    qo = torch.empty_like(q)
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    B.ps_kv_append_norm_rope_q4(params, rope, None, cache.struct, k, v, q, qo, zero, T)
    out, lse, st = _decode(params, cache.struct, qo[:, -1].contiguous(),
                           torch.tensor([T - 1], device=dev), dev)
    assert st.item() == 0
    _check(params, qo[:, -1], out, lse, _part(cache.prefix), [T], "append")


def test_heads_that_attend_rows_of_other_scales(cuda_device):
    """Of two kinds of rows, in every tile, even heads attend one and odd heads the other; the kinds'
    V scales are apart by 2^30, the other way round in the other group."""
    dev, n, hq, hkv = cuda_device, 900, 8, 1
    part = _scaled(dev, hkv, n, 16, lambda r: np.where(
        (r % 3 == 0)[:, None], np.array([1.0, 2.0 ** 30]), np.array([2.0 ** 30, 1.0])))
    rec = part[2].view(1, hkv, n, 4, 2)
    part[0].zero_()
    sign = 1.0 - 2.0 * (torch.arange(n, device=dev) % 3 != 0)
    # scores: 128 dims x 0.125 x (+-40 or a little more) / sqrt(128), 2^-160 between the kinds
    rec[0, 0, :, :2, 1] = (sign * (40 + torch.arange(n, device=dev) % 7 / 8)).bfloat16()[:, None]
    q = torch.full((1, hq, D), 0.125, dtype=torch.bfloat16, device=dev)
    q[:, 1::2] *= -1
    _run(dev, hq, hkv, part, q, [n, 2], "heads")


def test_scores_of_millions(cuda_device):
    """Scores far past where fp32 tells their fractions: nothing overflows on the way."""
    dev, n = cuda_device, 500
    part = _random_store(1, 2, n, 18, dev)
    q = (synth.normal_bf16((1, 8, D), 19, dev).double() * 2.0 ** 22).bfloat16()
    _run(dev, 8, 2, part, q, [n, 64], "millions")
