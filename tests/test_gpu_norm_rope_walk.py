"""The norm + rotary pass, its backward and the appends where a warp goes from token to token, and
at the token count from which tokens are no longer shared by eight warps.

Sizes follow from the GPU: two blocks of eight warps an SM; up to one token a block (2 x SMs) eight
warps share a token, past that every warp has tokens of its own, several of them past 16 x SMs.
Tolerances are those of the tests of single tokens.
"""
import numpy as np
import pytest
import torch

import synth
from prefix_sliding_window_b200 import binding as B
from prefix_sliding_window_b200.cache import LinearCache, PrefixSlidingCache, QuantizedCache
from tests import norm_q4_ref as R
from tests.gpu_util import f64
from tests.test_gpu_norm_rope import _check, _normed, _packed, _pair_sum, _weights
from tests.test_gpu_q4 import _decode, _same_as_bf16

pytestmark = pytest.mark.gpu
D, THETA, EPS = 128, 1.0e6, 1e-6


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


SIZES = {"one a block": lambda s: 2 * s, "one more": lambda s: 2 * s + 1,
         "one a warp": lambda s: 16 * s, "two for one warp": lambda s: 16 * s + 1,
         "several a warp": lambda s: 3 * 16 * s + 396}


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("hq,hkv,layout,rd,sides,pads", [
    (2, 1, "half", 128, "qk", True), (6, 2, "interleaved", 64, "qk", False),
    (5, 5, "half", 96, "k", True), (9, 1, "half", 128, "q", False)])
def test_forward_and_backward_over_tokens(cuda_device, size, hq, hkv, layout, rd, sides, pads):
    """sides: which of q and k are normalised.  pads: positions that a token cannot have, between
    ordinary ones."""
    dev, n = cuda_device, SIZES[size](_sms())
    params = B.make_params(hq, hkv, D, 0, 1, THETA)
    rope = B.make_rope(params, layout, rd)
    freq = R.frequencies(THETA, rd)
    q, k, _ = _packed(n, hq, hkv, 3 + hq, dev, extra=1)
    wq, wk = _weights("fp32", 5, dev)
    wq, wk = (wq if "q" in sides else None), (wk if "k" in sides else None)
    norm = B.make_norm(wq, wk, EPS)
    pos = synth.uniform_positions(n, 0, 100000, 7, dev)
    if pads:
        pos[::7] = -1
        pos[3::11] = 1 << 31
    ok = (f64(pos) >= 0) & (f64(pos) < 2.0 ** 31)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    out = [torch.full((n, h, D), float("nan"), dtype=torch.bfloat16, device=dev)
           for h in (hq, hkv)]
    B.ps_qk_norm_rope(params, rope, norm, q, k, pos, *out, st)
    grads = torch.full((n, hq + hkv + 1, D), 7.0, dtype=torch.bfloat16, device=dev)
    dq, dk = grads[:, :hq], grads[:, hq:hq + hkv]
    dyq, dyk = (synth.normal_bf16((n, h, D), 50 + h, dev) for h in (hq, hkv))
    dw = [torch.full((D,), float("nan"), device=dev) if w is not None else None for w in (wq, wk)]
    ws = torch.empty(B.ps_qk_norm_rope_bwd_workspace_bytes(params, n), dtype=torch.uint8,
                     device=dev)
    B.ps_qk_norm_rope_bwd(params, rope, norm, q, k, pos, dyq, dyk, dq, dk, *dw, ws, st)
    torch.cuda.synchronize()
    assert st.item() == ((B.PS_DEV_BAD_POS | B.PS_DEV_POS_RANGE) if pads else 0)
    assert (grads[:, -1] == 7.0).all()
    p = np.where(ok, f64(pos), 0)
    for x, w, y, dy, dx, g in ((q, wq, out[0], dyq, dq, dw[0]), (k, wk, out[1], dyk, dk, dw[1])):
        for t in (y, dx):
            assert (t[torch.from_numpy(~ok).to(dev)] == 0).all()
        x, dy, w = f64(x)[ok], f64(dy)[ok], None if w is None else f64(w)
        keep = torch.from_numpy(ok).to(dev)
        want = R.norm_rope(x, w, EPS, p[ok], freq, layout)
        _check(y[keep], want, _pair_sum(_normed(x, w), layout, rd, 1.0), "forward")
        want, want_w = R.norm_rope_bwd(x, w, EPS, p[ok], freq, layout, dy)
        G = _pair_sum(dy, layout, rd, 1.0)
        if w is None:
            _check(dx[keep], want, G, "backward")
            continue
        r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + EPS)
        nn = np.abs(x * r)
        wg = np.abs(w) * G
        _check(dx[keep], want, r * (wg + nn * (wg * nn).mean(-1, keepdims=True)), "backward")
        assert (np.abs(f64(g) - want_w) <= 2.0 ** -17 * (G * nn).sum((0, 1))).all()


def _append_inputs(Bn, T, hq, hkv, dev):
    rows = synth.normal_bf16((Bn, T, hq + 2 * hkv, D), 31, dev)
    return rows[:, :, :hq], rows[:, :, hq:hq + hkv], rows[:, :, hq + hkv:]


@pytest.mark.parametrize("Bn,T,starts", [
    (3, 3001, [0, 60, 5000]),            # most of a call's ring rows are evicted by newer ones
    (1, None, [0]), (1, None, [69]),     # one token a block, and one more
    (3, 1700, [-5, (1 << 31) - 800, 7])])
@pytest.mark.parametrize("hq,hkv,layout,rd,norm", [(2, 1, "half", 128, True),
                                                   (6, 3, "interleaved", 64, True),
                                                   (10, 5, "half", 32, False)])
def test_appends_over_tokens(cuda_device, Bn, T, starts, hq, hkv, layout, rd, norm):
    """Contiguous, paged, linear and 4-bit stores and the queries, against the 64-bit formulas."""
    dev, lp, w = cuda_device, 70, 128
    T = T or 2 * _sms() + (1 if starts[0] else 0)
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    rope = B.make_rope(params, layout, rd)
    freq = R.frequencies(THETA, rd)
    wq, wk = _weights("bf16", 6, dev)
    nrm = B.make_norm(wq, wk, EPS) if norm else None
    q, k, v = _append_inputs(Bn, T, hq, hkv, dev)
    pos0 = torch.tensor(starts, device=dev)
    pos = np.array(starts)[:, None] + np.arange(T)
    ok = (pos >= 0) & (pos < 1 << 31)
    flags = (B.PS_DEV_BAD_POS if (pos < 0).any() else 0) \
        | (B.PS_DEV_POS_RANGE if (pos >= 1 << 31).any() else 0)
    c = PrefixSlidingCache(Bn, hkv, lp, w, D, dev, fill=9.0)
    q4 = QuantizedCache(Bn, hkv, lp, w, dev)
    for part in (q4.prefix, q4.ring):
        part[2].fill_(9.0)
    outs = [torch.full((Bn, T, hq, D), float("nan"), dtype=torch.bfloat16, device=dev)
            for _ in range(2)]
    st = torch.zeros(2, dtype=torch.int32, device=dev)
    B.ps_kv_append_norm_rope(params, rope, nrm, c.struct, k, v, q, outs[0], pos0, T, st[:1])
    B.ps_kv_append_norm_rope_q4(params, rope, nrm, q4.struct, k, v, q, outs[1], pos0, T, st[1:])
    assert st.tolist() == [flags, flags]
    assert torch.equal(*outs)
    # queries
    flat, good = np.where(ok, pos, 0).reshape(-1), torch.from_numpy(ok).to(dev)
    assert (outs[0][~good] == 0).all()
    fw = None if not norm else f64(wq)
    xq = f64(q).reshape(-1, hq, D)
    want = R.norm_rope(xq, fw, EPS, flat, freq, layout).reshape(Bn, T, hq, D)
    slack = _pair_sum(_normed(xq, fw), layout, rd, 1.0).reshape(Bn, T, hq, D)
    _check(outs[0][good], want[ok], slack[ok], "queries")
    # rows: which token each slot holds in the end
    fw = None if not norm else f64(wk)
    xk = f64(k).reshape(-1, hkv, D)
    want = R.norm_rope(xk, fw, EPS, flat, freq, layout).reshape(Bn, T, hkv, D)
    slack = _pair_sum(_normed(xk, fw), layout, rd, 1.0).reshape(Bn, T, hkv, D)
    held = [np.full((Bn, n), -1) for n in (lp, w)]
    for b in range(Bn):
        for t in range(T):
            if ok[b, t]:
                i = int(pos[b, t] >= lp)
                # (the newest of the call, whether or not it has a place itself)
                if not i or t >= T - w:
                    held[i][b, (pos[b, t] - lp) % w if i else pos[b, t]] = t
    for i, (kb, vb, part) in enumerate(((c.k_prefix, c.v_prefix, q4.prefix),
                                        (c.k_ring, c.v_ring, q4.ring))):
        b, r = np.nonzero(held[i] >= 0)
        t = held[i][b, r]
        none = torch.from_numpy(held[i] < 0).to(dev)
        kb, vb, part = kb.transpose(1, 2), vb.transpose(1, 2), [x.transpose(1, 2) for x in part]
        assert (kb[none] == 9.0).all() and (vb[none] == 9.0).all() and (part[2][none] == 9.0).all()
        if len(b):
            _check(kb[b, r], want[b, t], slack[b, t], "keys")
            assert torch.equal(vb[b, r], v[b, t])
            _same_as_bf16(part, kb, vb, (b, r))
    # the same tokens into pages, and into a linear store as far as it goes
    nb, per = -(-lp // 64), -(-lp // 64) + w // 64
    table = torch.randperm(Bn * per + 2, generator=torch.Generator().manual_seed(3))[:Bn * per]
    table = table.view(Bn, per).int().to(dev)
    kp, vp = (torch.full((Bn * per + 2, hkv, 64, D), 9.0, dtype=torch.bfloat16, device=dev)
              for _ in range(2))
    B.ps_kv_append_norm_rope_paged(params, rope, nrm, kp, vp, table, Bn, k, v, None, None, pos0, T)
    for pool, pre, ring in ((kp, c.k_prefix, c.k_ring), (vp, c.v_prefix, c.v_ring)):
        got = pool[table.long()].transpose(1, 2).reshape(Bn, hkv, per * 64, D)
        assert torch.equal(got[:, :, :lp], pre) and torch.equal(got[:, :, nb * 64:], ring)
    lin = LinearCache(Bn, hkv, 2000, D, dev, fill=9.0)
    B.ps_kv_append_norm_rope(lin.params(hq), rope, nrm, lin.struct, k, v, q, outs[1], pos0, T)
    for b in range(Bn):
        t = np.nonzero(ok[b] & (pos[b] < 2000))[0]
        if len(t):
            _check(lin.k[b][:, pos[b, t]].transpose(0, 1), want[b, t], slack[b, t], "linear keys")
            assert torch.equal(lin.v[b][:, pos[b, t]].transpose(0, 1), v[b, t])
        rest = np.setdiff1d(np.arange(2000), pos[b, t])
        assert (lin.k[b][:, rest] == 9.0).all()
        assert (outs[1][b, np.setdiff1d(np.arange(T), t)] == 0).all()


@pytest.mark.parametrize("layout,rd,norm", [("half", 128, True), ("interleaved", 48, True),
                                            ("half", 80, True)])
@pytest.mark.parametrize("T,starts", [(1, [0, 63, 64, 900]), (700, [0, 5, 64, 2000])])
def test_paged_4_bit_append_and_decode(cuda_device, layout, rd, norm, T, starts):
    """A paged 4-bit store against the contiguous one: the same rows read back, and the same bits
    out of the decode."""
    dev, Bn, hq, hkv, lp, w = cuda_device, len(starts), 14, 2, 100, 192
    params = B.make_params(hq, hkv, D, lp, w, THETA)
    rope = B.make_rope(params, layout, rd)
    nrm = B.make_norm(*_weights("bf16", 6, dev), EPS)
    flat = QuantizedCache(Bn, hkv, lp, w, dev)
    per = -(-lp // 64) + w // 64
    pool = QuantizedCache(Bn * per + 3, hkv, 64, 0, dev).prefix
    table = torch.randperm(Bn * per + 3, generator=torch.Generator().manual_seed(4))[:Bn * per]
    paged = B.make_cache_q4(pool, None, Bn, table.view(Bn, per).int().to(dev))
    q, k, v = _append_inputs(Bn, T, hq, hkv, dev)
    warm = _append_inputs(Bn, 300, hq, hkv, dev)
    pos0 = torch.tensor(starts, device=dev)
    res = []
    for cache in (flat.struct, paged):
        before = (pos0 - 300).clamp(min=0)
        B.ps_kv_append_norm_rope_q4(params, rope, nrm, cache, warm[1], warm[2], None, None, before,
                                    300)
        qo = torch.empty(Bn, T, hq, D, dtype=torch.bfloat16, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        B.ps_kv_append_norm_rope_q4(params, rope, nrm, cache, k, v, q, qo, pos0, T, st)
        kr, vr = (torch.empty(Bn, T, hkv, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
        B.ps_kv_read_q4(params, cache, pos0, T, kr, vr, st)
        out, lse, st2 = _decode(params, cache, qo[:, -1].contiguous(), pos0 + T - 1, dev)
        assert st.item() == 0 and st2.item() == 0 and torch.isfinite(out).all()
        res.append((qo, kr, vr, out, lse))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    assert (res[0][1][:, -1] != 0).any(-1).all()
