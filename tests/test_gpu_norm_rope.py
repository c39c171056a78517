"""Norm + rotary pass and the appends that apply it, against 64-bit formulas.

Tolerances (before the first run): an output is rounded to bf16 once, at most 2^-8 of its value.
Everything before is fp32: a sum of 128 squares in 16 + 3 steps, a reciprocal root, two products,
cos and sin within a few 2^-24, and two products and a sum of the pair.  Each of those is at most
a few 2^-24 of the pair's magnitude P = |x_1| + |x_2| (normalised, times the factor on cos and
sin), about 40 roundings in all, so 2^-17 P covers them.  The backward has the same count on
r (|w| G + |n| mean(|w| G |n|)), G the pair's gradient magnitude; a weight gradient adds at most
100 terms in a row per thread and then 12, hence 2^-17 of the sum of magnitudes.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
import synth
from prefix_sliding_window_b200 import binding as B
from prefix_sliding_window_b200.cache import LinearCache, PrefixSlidingCache
from tests import norm_q4_ref as R
from tests.gpu_util import assert_close, assert_close_grad, f64

pytestmark = pytest.mark.gpu
D, THETA, EPS = 128, 1.0e6, 1e-6
SCALE = {"none": {}, "linear": dict(factor=4.0),
         "by_parts": dict(factor=8.0, low=1.0, high=4.0, original_len=8192),
         "yarn": dict(factor=4.0, low=1.0, high=32.0, original_len=32768)}


def _weights(kind, seed, dev):
    if kind is None:
        return None, None
    g = torch.Generator().manual_seed(seed)
    w = 1 + 0.3 * torch.randn(2, D, generator=g)
    w = w.to(dev, torch.bfloat16 if kind == "bf16" else torch.float32)
    return w[0].clone(), w[1].clone()


def _pair_sum(a, layout, rd, attn):
    """|a_1| + |a_2| of every dim's pair times attn (unrotated dims: |a|)."""
    a = np.abs(a)
    i, j = R.pair_index(layout, rd)
    out = a.copy()
    out[..., i] = out[..., j] = (a[..., i] + a[..., j]) * attn
    return out


def _check(got, want, slack, what):
    got = f64(got)
    bad = ~(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * slack)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}"


def _normed(x, w):
    if w is None:
        return x
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + EPS) * w


def _packed(n, hq, hkv, seed, dev, extra=0):
    """q, k, v views of packed projection rows (with `extra` more heads of padding)."""
    rows = synth.normal_bf16((n, hq + 2 * hkv + extra, D), seed, dev)
    return rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:hq + 2 * hkv]


CASES = [
    # n, hq, hkv, layout, rotary_dim, scaling, weights, largest position
    (1, 16, 2, "half", 128, "none", "bf16", 0),
    (1, 1, 1, "interleaved", 128, "none", None, 1 << 20),
    (3, 28, 4, "half", 64, "yarn", "fp32", 131072),
    (77, 5, 5, "interleaved", 32, "by_parts", "bf16", (1 << 31) - 1),
    (1187, 6, 3, "half", 96, "linear", "fp32", 8191),     # one token past the wide blocks' start
    (1186, 3, 1, "interleaved", 112, "yarn", "bf16", 40000),
    (64, 9, 3, "half", 16, "none", "fp32", 1000),
    (33, 16, 2, "half", 0, "none", "bf16", 1000),         # norm alone
]


@pytest.mark.parametrize("n,hq,hkv,layout,rd,scaling,weights,top", CASES)
def test_forward_and_backward(cuda_device, n, hq, hkv, layout, rd, scaling, weights, top):
    dev = cuda_device
    params = B.make_params(hq, hkv, D, 0, 1, THETA)
    attn = 1.25 if scaling == "yarn" else 1.0
    rope = B.make_rope(params, layout, rd, scaling, attn_factor=attn, **SCALE[scaling])
    freq = R.frequencies(THETA, rd, scaling, **SCALE[scaling])
    q, k, _ = _packed(n, hq, hkv, 11 + n, dev, extra=1)
    wq, wk = _weights(weights, n, dev)
    norm = B.make_norm(wq, wk, EPS) if weights else None
    pos = synth.uniform_positions(n, 0, top, n, dev)
    pos[0] = top
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    out = [torch.full((n, h, D), float("nan"), dtype=torch.bfloat16, device=dev)
           for h in (hq, hkv)]
    B.ps_qk_norm_rope(params, rope, norm, q, k, pos, *out, st)
    # gradients go into slices of packed rows whose other heads keep what they held
    grads = torch.full((n, hq + hkv + 1, D), 7.0, dtype=torch.bfloat16, device=dev)
    dq, dk = grads[:, :hq], grads[:, hq:hq + hkv]
    dyq, dyk = (synth.normal_bf16((n, h, D), 50 + h, dev) for h in (hq, hkv))
    dw = [torch.full((D,), float("nan"), device=dev) for _ in range(2)] if weights else [None] * 2
    ws = torch.empty(B.ps_qk_norm_rope_bwd_workspace_bytes(params, n), dtype=torch.uint8,
                     device=dev)
    B.ps_qk_norm_rope_bwd(params, rope, norm, q, k, pos, dyq, dyk, dq, dk, *dw, ws, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert (grads[:, -1] == 7.0).all()
    p = f64(pos)
    for x, w, y, dy, dx, g in ((q, wq, out[0], dyq, dq, dw[0]), (k, wk, out[1], dyk, dk, dw[1])):
        x, dy, w = f64(x), f64(dy), None if w is None else f64(w)
        want = R.norm_rope(x, w, EPS, p, freq, layout, attn)
        _check(y, want, _pair_sum(_normed(x, w), layout, rd, attn), "forward")
        want, want_w = R.norm_rope_bwd(x, w, EPS, p, freq, layout, dy, attn)
        G = _pair_sum(dy, layout, rd, attn)
        if w is None:
            _check(dx, want, G, "backward")
            continue
        r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + EPS)
        nn = np.abs(x * r)
        wg = np.abs(w) * G
        _check(dx, want, r * (wg + nn * (wg * nn).mean(-1, keepdims=True)), "backward")
        err = np.abs(f64(g) - want_w)
        assert (err <= 2.0 ** -17 * (G * nn).sum((0, 1))).all()


def test_gradient_against_differences(cuda_device):
    """dx and dw against central differences of a 64-bit forward along random directions."""
    dev = cuda_device
    n, hq, hkv = 5, 4, 2
    params = B.make_params(hq, hkv, D, 0, 1, THETA)
    rope = B.make_rope(params, "interleaved", 64, "yarn", attn_factor=1.1, **SCALE["yarn"])
    freq = R.frequencies(THETA, 64, "yarn", **SCALE["yarn"])
    q, k, _ = _packed(n, hq, hkv, 3, dev)
    wq, wk = _weights("fp32", 4, dev)
    pos = synth.uniform_positions(n, 0, 5000, 5, dev)
    dy = synth.normal_bf16((n, hq, D), 6, dev)
    dq = torch.empty(n, hq, D, dtype=torch.bfloat16, device=dev)
    dw = torch.empty(D, device=dev)
    ws = torch.empty(B.ps_qk_norm_rope_bwd_workspace_bytes(params, n), dtype=torch.uint8,
                     device=dev)
    # the query side alone
    B.ps_qk_norm_rope_bwd(params, rope, B.make_norm(wq, wk, EPS), q, None, pos, dy, None, dq, None,
                          dw, None, ws)
    x, w, p, dyv = f64(q), f64(wq), f64(pos), f64(dy)
    rng = np.random.default_rng(0)

    def loss(x, w):
        return (R.norm_rope(x, w, EPS, p, freq, "interleaved", 1.1) * dyv).sum()
    h = 1e-5
    for _ in range(4):
        vx, vw = rng.normal(size=x.shape), rng.normal(size=w.shape)
        num = (loss(x + h * vx, w) - loss(x - h * vx, w)) / (2 * h)
        # dq is rounded to bf16: each term is off by up to 2^-8 of itself
        assert abs((f64(dq) * vx).sum() - num) <= \
            2.0 ** -8 * (np.abs(f64(dq) * vx)).sum() + 1e-6 * abs(num) + 1e-6
        num = (loss(x, w + h * vw) - loss(x, w - h * vw)) / (2 * h)
        assert abs((f64(dw) * vw).sum() - num) <= 1e-4 * (np.abs(f64(dw) * vw)).sum() + 1e-6


def test_padding_one_side_in_place_and_repeat(cuda_device):
    """Positions outside [0, 2^31) give zero rows, flags and no weight gradient; q or k alone;
    in place; the same call twice gives the same bits."""
    dev = cuda_device
    n, hq, hkv = 40, 8, 2
    params = B.make_params(hq, hkv, D, 0, 1, THETA)
    rope = B.make_rope(params)
    q, k, _ = (t.contiguous() for t in _packed(n, hq, hkv, 9, dev))
    wq, wk = _weights("bf16", 4, dev)
    norm = B.make_norm(wq, wk, EPS)
    pos = torch.arange(n, device=dev)
    pads = [0, 7, 39]
    pos[pads] = torch.tensor([-1, -5, 1 << 31], device=dev)
    q[7] = float("nan")  # padding may hold anything
    k[39] = float("inf")
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    B.ps_qk_norm_rope(params, rope, norm, q, k, pos, qo, ko, st)
    assert st.item() == B.PS_DEV_BAD_POS | B.PS_DEV_POS_RANGE
    assert (qo[pads] == 0).all() and (ko[pads] == 0).all()
    assert torch.isfinite(qo).all() and torch.isfinite(ko).all()
    alone = torch.empty_like(k)
    B.ps_qk_norm_rope(params, rope, norm, None, k, pos, None, alone)
    assert torch.equal(alone, ko)
    qi = q.clone()
    B.ps_qk_norm_rope(params, rope, norm, qi, None, pos, qi, None)
    assert torch.equal(qi, qo)
    dyq, dyk = synth.normal_bf16((n, hq, D), 1, dev), synth.normal_bf16((n, hkv, D), 2, dev)
    dyq[0] = float("nan")
    ws = torch.empty(B.ps_qk_norm_rope_bwd_workspace_bytes(params, n), dtype=torch.uint8,
                     device=dev)
    res = []
    for _ in range(2):
        ws.fill_(0xff)
        got = [torch.empty_like(q), torch.empty_like(k), torch.empty(D, device=dev),
               torch.empty(D, device=dev)]
        B.ps_qk_norm_rope_bwd(params, rope, norm, q, k, pos, dyq, dyk, *got, ws)
        res.append(got)
    for a, b in zip(*res):
        assert torch.equal(a, b)
    dq, dk, dwq, dwk = res[0]
    assert (dq[pads] == 0).all() and (dk[pads] == 0).all()
    keep = [i for i in range(n) if i not in pads]
    short = [torch.empty_like(q[keep]), torch.empty_like(k[keep]), torch.empty(D, device=dev),
             torch.empty(D, device=dev)]
    B.ps_qk_norm_rope_bwd(params, rope, norm, q[keep], k[keep], pos[keep], dyq[keep], dyk[keep],
                          *short, ws)
    assert torch.equal(short[0], dq[keep]) and torch.equal(short[1], dk[keep])
    for a, b in ((short[2], dwq), (short[3], dwk)):  # the same terms in another order
        assert torch.allclose(a, b, rtol=0, atol=2.0 ** -17 * n * hq * 4)
    # gradients in place of the outputs' gradients, no weight gradients, no workspace
    gi = dyq.clone()
    B.ps_qk_norm_rope_bwd(params, rope, norm, q, None, pos, gi, None, gi, None)
    assert torch.equal(gi, dq)
    # no tokens: weight gradients are zero
    dw = torch.full((D,), 3.0, device=dev)
    B.ps_qk_norm_rope_bwd(params, rope, norm, q[:0], k[:0], pos[:0], dyq[:0], dyk[:0],
                          dq[:0], dk[:0], dw, None, ws)
    assert (dw == 0).all()


def test_binding_refusals(cuda_device):
    dev = cuda_device
    params = B.make_params(4, 2, D, 0, 1, THETA)
    rope = B.make_rope(params)
    q, k, _ = (t.contiguous() for t in _packed(6, 4, 2, 9, dev))
    pos = torch.arange(6, device=dev)
    ok = dict(q=q, k=k, pos=pos, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
    bad = [dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:5]), dict(q=q.transpose(0, 1)),
           dict(q=q[..., ::2]), dict(pos=pos.int()), dict(pos=pos.cpu()), dict(q_out=q[:5]),
           dict(q_out=q.float()), dict(k=k[:, :1]), dict(pos=torch.arange(12, device=dev)[::2])]
    for over in bad:
        with pytest.raises(ValueError):
            B.ps_qk_norm_rope(params, rope, None, *{**ok, **over}.values())
    with pytest.raises(ValueError):
        B.make_norm(torch.ones(128))
    with pytest.raises(ValueError):
        B.make_norm(torch.ones(64, device=dev))
    with pytest.raises(ValueError):
        B.make_norm(torch.ones(128, device=dev), torch.ones(128, device=dev).bfloat16())


def test_training_step_together(cuda_device):
    """norm + rotation -> masked prefill -> its backward -> backward of norm + rotation, gradients
    of the raw projections against the 64-bit chain."""
    dev = cuda_device
    S, hq, hkv, lp, w = 200, 4, 2, 16, 64
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    rope = B.make_rope(params)
    freq = R.frequencies(THETA, 128)
    qr, kr, vr = _packed(S, hq, hkv, 21, dev)
    wq, wk = _weights("bf16", 22, dev)
    norm = B.make_norm(wq, wk, EPS)
    pos = torch.arange(S, device=dev)
    bf = dict(dtype=torch.bfloat16, device=dev)
    q, k = torch.empty(S, hq, D, **bf), torch.empty(S, hkv, D, **bf)
    B.ps_qk_norm_rope(params, rope, norm, qr, kr, pos, q, k)
    v = vr.contiguous()
    out, lse = torch.empty_like(q), torch.empty(1, hq, S, device=dev)
    ws = torch.empty(B.ps_prefill_workspace_bytes(params, 1, S), dtype=torch.uint8, device=dev)
    B.ps_masked_prefill_attn(params, q, k, v, 1, S, out, lse, None, ws)
    do = synth.normal_bf16((S, hq, D), 23, dev)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(B.ps_prefill_bwd_workspace_bytes(params, 1, S), dtype=torch.uint8, device=dev)
    B.ps_masked_prefill_attn_bwd(params, q, k, v, out, do, lse, 1, S, dq, dk, dv, ws)
    dqkv = torch.empty(S, hq + 2 * hkv, D, **bf)
    dw = torch.empty(2, D, device=dev)
    ws = torch.empty(B.ps_qk_norm_rope_bwd_workspace_bytes(params, S), dtype=torch.uint8,
                     device=dev)
    B.ps_qk_norm_rope_bwd(params, rope, norm, qr, kr, pos, dq, dk, dqkv[:, :hq],
                          dqkv[:, hq:hq + hkv], dw[0], dw[1], ws)
    # stage by stage: the attention against the oracle on the kernels' own q and k ...
    want, _ = O.prefill_reference(f64(q), f64(k), f64(v), lp, w, 1 / np.sqrt(D))
    assert_close(f64(out), want, "prefill")
    gq, gk, gv = O.prefill_backward_reference(f64(q), f64(k), f64(v), f64(do), lp, w,
                                              1 / np.sqrt(D), rows=list(range(S)),
                                              keys=list(range(S)))
    for name, a, b in (("dq", dq, gq), ("dk", dk, gk), ("dv", dv, gv)):
        assert_close_grad(f64(a), b, name)
    # ... and the projections' gradients against the 64-bit chain from that dq, dk: the inner
    # gradients' 5e-3 carry over (the map is linear in them), and one more rounding of 2^-8
    p = f64(pos)
    for name, x, w_, g, got, got_w in (("q", qr, wq, gq, dqkv[:, :hq], dw[0]),
                                       ("k", kr, wk, gk, dqkv[:, hq:hq + hkv], dw[1])):
        dx, dwant = R.norm_rope_bwd(f64(x), f64(w_), EPS, p, freq, "half", g)
        for a, b, tol in ((f64(got), dx, 5e-3 + 2.0 ** -8), (f64(got_w), dwant, 2e-2)):
            assert np.linalg.norm(a - b) <= tol * np.linalg.norm(b), name


# ---------------------------------------------------------------- appends
def _append_args(Bn, T, hq, hkv, seed, dev):
    q, k, v = (t.view(Bn, T, t.shape[1], D) for t in _packed(Bn * T, hq, hkv, seed, dev))
    return q, k, v


@pytest.mark.parametrize("Bn,T,lp,w,starts", [
    (3, 1, 5, 64, [0, 4, 1000]), (2, 150, 33, 64, [0, 90]), (1, 700, 256, 128, [100]),
    (2, 1, 0, 1, [0, 77]), (4, 400, 100, 512, [0, 50, 101, 100000])])
def test_append_matches_plain_append(cuda_device, Bn, T, lp, w, starts):
    """Without a norm, with the plain rotary plan: the slots and values of ps_kv_append_rope bit
    for bit, keys and queries within what two fp32 rotations rounded to bf16 can differ (each
    within 2^-8 |y| + 2^-17 P of the exact one, P the pair's magnitude)."""
    dev = cuda_device
    hq, hkv = 8, 2
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    q, k, v = _append_args(Bn, T, hq, hkv, 31, dev)
    pos0 = torch.tensor(starts, device=dev)
    a, b = (PrefixSlidingCache(Bn, hkv, lp, w, D, dev, fill=300.0) for _ in range(2))
    qa = q.contiguous()
    B.ps_kv_append_rope(params, a.struct, k.contiguous(), v.contiguous(), qa, pos0, T)
    qb = torch.empty_like(qa)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    B.ps_kv_append_norm_rope(params, B.make_rope(params), None, b.struct, k, v, q, qb, pos0, T, st)
    assert st.item() == 0

    def same_rotation(x, y):
        x, y = f64(x), f64(y)
        pair = np.hypot(y[..., :64], y[..., 64:])  # the rotation keeps it; P <= sqrt(2) of it
        slack = np.concatenate((pair, pair), -1) * math.sqrt(2) * 2.0 ** -16
        assert (np.abs(x - y) <= 2.0 ** -7 * np.maximum(np.abs(x), np.abs(y)) + slack).all()
    same_rotation(qa, qb)
    for name in ("v_prefix", "v_ring", "k_prefix", "k_ring"):
        x, y = getattr(a, name), getattr(b, name)
        if x is None:
            assert y is None
        elif name[0] == "v":
            assert torch.equal(x, y), name
        else:
            empty = (x == 300.0).all(-1)
            assert torch.equal(empty, (y == 300.0).all(-1)), name
            same_rotation(x[~empty], y[~empty])


@pytest.mark.parametrize("layout,rd,scaling,weights", [
    ("half", 128, "yarn", "bf16"), ("interleaved", 64, "by_parts", "fp32"),
    ("half", 96, "linear", None)])
@pytest.mark.parametrize("T", [1, 333])
def test_append_rows_match_the_norm_rope_pass(cuda_device, layout, rd, scaling, weights, T):
    """Keys in the store (contiguous, paged and linear) and queries equal ps_qk_norm_rope's rows
    bit for bit, values the inputs; everything else in the store stays."""
    dev = cuda_device
    Bn, hq, hkv, lp, w = 3, 10, 2, 70, 128
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    attn = 1.2 if scaling == "yarn" else 1.0
    rope = B.make_rope(params, layout, rd, scaling, attn_factor=attn, **SCALE[scaling])
    wq, wk = _weights(weights, 3, dev)
    norm = B.make_norm(wq, wk, EPS) if weights else None
    q, k, v = _append_args(Bn, T, hq, hkv, 77, dev)
    starts = [0, 60, 900]
    pos0 = torch.tensor(starts, device=dev)
    pos = (pos0[:, None] + torch.arange(T, device=dev)).flatten()
    qr = torch.empty(Bn * T, hq, D, dtype=torch.bfloat16, device=dev)
    kr = torch.empty(Bn * T, hkv, D, dtype=torch.bfloat16, device=dev)
    B.ps_qk_norm_rope(params, rope, norm, q, k, pos, qr, kr)
    kr = kr.view(Bn, T, hkv, D)

    def expect(rows, fill):
        pre = torch.full((Bn, hkv, lp, D), fill, dtype=torch.bfloat16, device=dev)
        ring = torch.full((Bn, hkv, w, D), fill, dtype=torch.bfloat16, device=dev)
        for b, s in enumerate(starts):
            for t in range(T):
                p = s + t
                if p < lp:
                    pre[b, :, p] = rows[b, t]
                elif p > s + T - 1 - w:
                    ring[b, :, (p - lp) % w] = rows[b, t]
        return pre, ring
    want = [x for rows in (kr, v) for x in expect(rows, 3.0)]
    c = PrefixSlidingCache(Bn, hkv, lp, w, D, dev, fill=3.0)
    qo = torch.empty(Bn, T, hq, D, dtype=torch.bfloat16, device=dev)
    B.ps_kv_append_norm_rope(params, rope, norm, c.struct, k, v, q, qo, pos0, T)
    assert torch.equal(qo.view(-1, hq, D), qr)
    for x, y in zip(want, (c.k_prefix, c.k_ring, c.v_prefix, c.v_ring)):
        assert torch.equal(x, y)
    # paged, blocks in random order, without queries
    per = -(-lp // 64) + w // 64
    table = torch.randperm(Bn * per + 3, generator=torch.Generator().manual_seed(1))
    table = table[:Bn * per].view(Bn, per).int().to(dev)
    kp, vp = (torch.full((Bn * per + 3, hkv, 64, D), 3.0, dtype=torch.bfloat16, device=dev)
              for _ in range(2))
    B.ps_kv_append_norm_rope_paged(params, rope, norm, kp, vp, table, Bn, k, v, None, None, pos0, T)
    nb = -(-lp // 64)
    for pool, pre, ring in ((kp, want[0], want[1]), (vp, want[2], want[3])):
        full = torch.full_like(pool, 3.0)
        blocks = torch.full((Bn, hkv, per * 64, D), 3.0, dtype=torch.bfloat16, device=dev)
        blocks[:, :, :lp], blocks[:, :, nb * 64:] = pre, ring
        full[table.flatten().long()] = blocks.view(Bn, hkv, per, 64, D).transpose(1, 2).reshape(
            -1, hkv, 64, D)
        assert torch.equal(pool, full)
    # linear: positions past the end are skipped, flagged, and their queries are zeros
    lin = LinearCache(Bn, hkv, 901, D, dev, fill=3.0)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    B.ps_kv_append_norm_rope(lin.params(hq), rope, norm, lin.struct, k, v, q, qo, pos0, T, st)
    torch.cuda.synchronize()
    assert st.item() == (B.PS_DEV_POS_RANGE if T > 1 else 0)
    for b, s in enumerate(starts):
        n = min(T, 901 - s)
        assert torch.equal(lin.k[b, :, s:s + n].transpose(0, 1), kr[b, :n])
        assert torch.equal(lin.v[b, :, s:s + n].transpose(0, 1), v[b, :n])
        assert (lin.k[b, :, s + n:] == 3.0).all() and (lin.k[b, :, :s] == 3.0).all()
        assert torch.equal(qo[b, :n], qr.view(Bn, T, hq, D)[b, :n]) and (qo[b, n:] == 0).all()


def test_append_skips(cuda_device):
    """A negative position, a ring-only store below its prefix, a bad table entry."""
    dev = cuda_device
    Bn, T, hq, hkv, lp, w = 2, 5, 4, 2, 64, 64
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    rope = B.make_rope(params)
    q, k, v = _append_args(Bn, T, hq, hkv, 5, dev)
    qo = torch.empty(Bn, T, hq, D, dtype=torch.bfloat16, device=dev)
    c = PrefixSlidingCache(Bn, hkv, lp, w, D, dev, fill=3.0)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    pos0 = torch.tensor([-2, 200], device=dev)
    B.ps_kv_append_norm_rope(params, rope, None, c.struct, k, v, q, qo, pos0, T, st)
    assert st.item() == B.PS_DEV_BAD_POS
    assert (qo[0, :2] == 0).all() and (qo[0, 2:] != 0).any() and torch.isfinite(qo).all()
    assert (c.k_prefix[0, :, 3:] == 3.0).all() and (c.k_prefix[0, :, :3] != 3.0).any()
    st.zero_()
    ring = B.make_cache(None, None, c.k_ring, c.v_ring, Bn)
    before = c.k_ring.clone()
    B.ps_kv_append_norm_rope(params, rope, None, ring, k, v, q, qo,
                             torch.tensor([10, 62], device=dev), T, st)
    assert st.item() == B.PS_DEV_POS_RANGE
    assert (qo[0] == 0).all() and (qo[1, :2] == 0).all() and (qo[1, 2:] != 0).any()
    assert torch.equal(c.k_ring[0], before[0]) and torch.equal(c.k_ring[1, :, 3:], before[1, :, 3:])
    st.zero_()
    table = torch.tensor([[0, 1], [9, -1]], dtype=torch.int32, device=dev)
    kp, vp = (torch.full((2, hkv, 64, D), 3.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    B.ps_kv_append_norm_rope_paged(params, rope, None, kp, vp, table, Bn, k, v, q, qo,
                                   torch.tensor([0, 62], device=dev), T, st)
    assert st.item() == B.PS_DEV_POS_RANGE
    assert (qo != 0).any(-1).all()       # a bad entry loses the row, not the query
    assert (kp[0, :, 5:] == 3.0).all() and (kp[1] == 3.0).all() and (kp[0, :, :5] != 3.0).any()
