"""Host-side checks of the norm + rotary and 4-bit entry points that need no GPU: rotary plans
against the formulas, and every refusal before a launch."""
import ctypes
import math
import os

import numpy as np
import pytest

from prefix_sliding_window_b200 import binding as B
from prefix_sliding_window_b200 import build as BLD
from tests import norm_q4_ref as R


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        BLD.build(quiet=True)
    return B.load()


def _params(**kw):
    base = dict(n_q_heads=16, n_kv_heads=2, head_dim=128, l_prefix=100, window=512)
    base.update(kw)
    return B.make_params(**base)


def test_struct_sizes():
    assert ctypes.sizeof(B.PsRope) == 528 and B.PsRope.inv_freq.offset == 16
    assert ctypes.sizeof(B.PsRopeScaling) == 40
    assert ctypes.sizeof(B.PsQkNorm) == 24
    assert ctypes.sizeof(B.PsKVCacheQ4) == 80


@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=4.0)),
    ("by_parts", dict(factor=8.0, low=1.0, high=4.0, original_len=8192)),
    ("yarn", dict(factor=4.0, low=1.0, high=32.0, original_len=32768)),
    ("yarn", dict(factor=2.5, low=1.0, high=1.01, original_len=10.0)),  # the ramp is a step
])
@pytest.mark.parametrize("rotary_dim", [128, 64, 16, 112])
def test_rope_init_matches_formulas(lib, scaling, kw, rotary_dim):
    for theta in (1.0e6, 1.0e4):
        r = B.make_rope(_params(rope_theta=theta), "interleaved", rotary_dim, scaling,
                        attn_factor=1.25, **kw)
        want = R.frequencies(theta, rotary_dim, scaling, **kw)
        # both sides are a handful of 64-bit operations; near a ramp's border the blend moves by
        # the same rounding
        np.testing.assert_allclose(list(r.inv_freq)[:rotary_dim // 2], want, rtol=1e-12)
        assert list(r.inv_freq)[rotary_dim // 2:] == [0.0] * (64 - rotary_dim // 2)
        assert (r.layout, r.rotary_dim) == (B.PS_ROPE_INTERLEAVED, rotary_dim)
        assert r.attn_factor == 1.25


def test_rope_init_no_rotation(lib):
    r = B.make_rope(_params(), "half", 0)
    assert r.rotary_dim == 0 and set(r.inv_freq) == {0.0}


@pytest.mark.parametrize("kw,code", [
    (dict(rotary_dim=24), B.PS_ERR_UNSUPPORTED),
    (dict(rotary_dim=144), B.PS_ERR_UNSUPPORTED),
    (dict(rotary_dim=-16), B.PS_ERR_UNSUPPORTED),
    (dict(attn_factor=0.0), B.PS_ERR_INVALID_ARG),
    (dict(attn_factor=math.nan), B.PS_ERR_INVALID_ARG),
    (dict(scaling="linear", factor=0.5), B.PS_ERR_INVALID_ARG),
    (dict(scaling="yarn", factor=math.inf), B.PS_ERR_INVALID_ARG),
    (dict(scaling="by_parts", factor=2.0, low=4.0, high=4.0), B.PS_ERR_INVALID_ARG),
    (dict(scaling="by_parts", factor=2.0, low=0.0), B.PS_ERR_INVALID_ARG),
    (dict(scaling="yarn", factor=2.0, original_len=0.0), B.PS_ERR_INVALID_ARG),
])
def test_rope_init_refusals(lib, kw, code):
    with pytest.raises(B.PsError) as e:
        B.make_rope(_params(), **kw)
    assert e.value.code == code


def test_rope_theta_below_one_refused(lib):
    for theta, scaling in ((0.5, "none"), (1.0, "yarn")):
        with pytest.raises(B.PsError) as e:
            B.make_rope(_params(rope_theta=theta), scaling=scaling)
        assert e.value.code == B.PS_ERR_UNSUPPORTED


def _call(fn, args, over):
    """fn with named arguments, some replaced."""
    assert set(over) <= set(args), set(over) - set(args)
    return fn(*{**args, **over}.values())


FWD = dict(params=None, rope=None, norm=None, q=256, qs=2048, k=256, ks=256, pos=256, n=4,
           q_out=512, k_out=512, status=None, stream=None)


def _fwd_args():
    p = _params()
    return {**FWD, "params": p, "rope": B.make_rope(p)}


def _bad_rope(**kw):
    r = B.make_rope(_params())
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _steep():
    r = B.make_rope(_params())
    r.inv_freq[3] = 1.5
    return r


@pytest.mark.parametrize("over,code", [
    (dict(rope=None), B.PS_ERR_INVALID_ARG),
    (dict(rope="layout"), B.PS_ERR_INVALID_ARG),
    (dict(rope="dim"), B.PS_ERR_UNSUPPORTED),
    (dict(rope="steep"), B.PS_ERR_INVALID_ARG),
    (dict(rope="reserved"), B.PS_ERR_INVALID_ARG),
    (dict(norm=B.PsQkNorm(256, 256, 7, 1e-6)), B.PS_ERR_INVALID_ARG),
    (dict(norm=B.PsQkNorm(256, 256, 0, -1.0)), B.PS_ERR_INVALID_ARG),
    (dict(norm=B.PsQkNorm(256, 264, 0, 1e-6)), B.PS_ERR_INVALID_ARG),
    (dict(n=-1), B.PS_ERR_INVALID_ARG),
    (dict(q=264), B.PS_ERR_INVALID_ARG),
    (dict(q_out=None), B.PS_ERR_INVALID_ARG),
    (dict(k=None), B.PS_ERR_INVALID_ARG),
    (dict(q=None, q_out=None, k=None, k_out=None), B.PS_ERR_INVALID_ARG),
    (dict(qs=2047), B.PS_ERR_INVALID_ARG),
    (dict(qs=2052), B.PS_ERR_INVALID_ARG),
    (dict(ks=255), B.PS_ERR_INVALID_ARG),
    (dict(q_out=256, qs=4096), B.PS_ERR_INVALID_ARG),   # in place on strided rows
    (dict(pos=None), B.PS_ERR_INVALID_ARG),
    (dict(pos=260), B.PS_ERR_INVALID_ARG),
    (dict(status=258), B.PS_ERR_INVALID_ARG),
])
def test_norm_rope_refusals(lib, over, code):
    named = {"layout": _bad_rope(layout=2), "dim": _bad_rope(rotary_dim=20), "steep": _steep(),
             "reserved": _bad_rope(reserved=1)}
    over = {k: named.get(v, v) if k == "rope" else v for k, v in over.items()}
    assert _call(lib.ps_qk_norm_rope, _fwd_args(), over) == code
    assert B.last_error() != ""


def test_norm_rope_no_tokens(lib):
    assert _call(lib.ps_qk_norm_rope, _fwd_args(), dict(n=0)) == B.PS_OK


def _bwd_args():
    p = _params()
    need = lib_bytes(p, 4)
    return dict(params=p, rope=B.make_rope(p), norm=B.PsQkNorm(256, 256, 0, 1e-6), q=256, qs=2048,
                k=256, ks=256, pos=256, n=4, gq=256, gk=256, dq=512, dqs=2048, dk=512, dks=256,
                dwq=256, dwk=256, ws=256, wsb=need, status=None, stream=None)


def lib_bytes(p, n):
    return B.ps_qk_norm_rope_bwd_workspace_bytes(p, n)


@pytest.mark.parametrize("over,code", [
    (dict(gq=None), B.PS_ERR_INVALID_ARG),
    (dict(dk=None), B.PS_ERR_INVALID_ARG),
    (dict(gq=None, dq=None, gk=None, dk=None, dwq=None, dwk=None), B.PS_ERR_INVALID_ARG),
    (dict(gq=None, dq=None), B.PS_ERR_INVALID_ARG),        # dq_weight without dq_out
    (dict(norm=None), B.PS_ERR_INVALID_ARG),               # dq_weight without a weight
    (dict(norm=B.PsQkNorm(256, None, 0, 1e-6)), B.PS_ERR_INVALID_ARG),
    (dict(q=None), B.PS_ERR_INVALID_ARG),                  # a normalised input is needed
    (dict(k=260), B.PS_ERR_INVALID_ARG),
    (dict(qs=0), B.PS_ERR_INVALID_ARG),
    (dict(dqs=2040), B.PS_ERR_INVALID_ARG),
    (dict(dks=260), B.PS_ERR_INVALID_ARG),
    (dict(dq=256, dqs=4096), B.PS_ERR_INVALID_ARG),
    (dict(dwq=260), B.PS_ERR_INVALID_ARG),
    (dict(ws=None), B.PS_ERR_WORKSPACE),
    (dict(ws=264), B.PS_ERR_INVALID_ARG),
    (dict(wsb=8), B.PS_ERR_WORKSPACE),
    (dict(pos=None), B.PS_ERR_INVALID_ARG),
    (dict(n=-1), B.PS_ERR_INVALID_ARG),
])
def test_norm_rope_bwd_refusals(lib, over, code):
    assert _call(lib.ps_qk_norm_rope_bwd, _bwd_args(), over) == code


def test_norm_rope_bwd_nothing_to_do(lib):
    assert _call(lib.ps_qk_norm_rope_bwd, _bwd_args(), dict(n=0, dwq=None, dwk=None)) == B.PS_OK
    p = _params()
    assert lib_bytes(p, 1) >= 1024 and lib_bytes(p, 1 << 20) >= lib_bytes(p, 1)
    assert lib_bytes(p, 1 << 40) == lib_bytes(p, 1 << 20)  # partials per block, not per token
    assert lib_bytes(_params(head_dim=64), 4) == 0


APPEND = dict(k=256, ks=256, v=256, vs=256, q=256, qs=2048, q_out=512, pos0=256, T=1, status=None,
              stream=None)


def _append_calls(lib, params):
    rope = B.make_rope(_params())
    q4 = B.PsKVCacheQ4(256, 256, 256, 256, 256, 256, 4, None, 0, 0, 0)
    yield lib.ps_kv_append_norm_rope, dict(params=params, rope=rope, norm=None,
                                           cache=B.PsKVCache(256, 256, 256, 256, 4), **APPEND)
    yield lib.ps_kv_append_norm_rope_q4, dict(params=params, rope=rope, norm=None, cache=q4,
                                              **APPEND)
    yield lib.ps_kv_append_norm_rope_paged, dict(params=params, rope=rope, norm=None, kp=256,
                                                 vp=256, nb=64, table=256, stride=10, batch=4,
                                                 **APPEND)


@pytest.mark.parametrize("over", [
    dict(rope=None), dict(k=None), dict(v=264), dict(ks=128), dict(vs=258), dict(q=None),
    dict(q_out=None), dict(qs=1024), dict(q_out=256, qs=4096), dict(pos0=None), dict(pos0=260),
    dict(T=0), dict(status=257), dict(norm=B.PsQkNorm(256, 256, 2, 1e-6)),
])
def test_append_refusals(lib, over):
    for fn, args in _append_calls(lib, _params()):
        assert _call(fn, args, over) == B.PS_ERR_INVALID_ARG, fn.__name__


def test_append_store_refusals(lib):
    (f, fa), (g, ga), (h, ha) = _append_calls(lib, _params())
    for c in (B.PsKVCache(256, 256, None, 256, 4), B.PsKVCache(256, None, 256, 256, 4),
              B.PsKVCache(256, 264, 256, 256, 4), B.PsKVCache(None, None, None, None, 4),
              B.PsKVCache(256, 256, 256, 256, -1), None):
        assert _call(f, fa, dict(cache=c)) == B.PS_ERR_INVALID_ARG
    linear0 = dict(params=_params(l_prefix=0), cache=B.PsKVCache(256, 256, None, None, 4))
    assert _call(f, fa, linear0) == B.PS_ERR_INVALID_ARG
    six = [256] * 6
    for i in range(6):
        ptrs = list(six)
        ptrs[i] = None
        assert _call(g, ga, dict(cache=B.PsKVCacheQ4(*ptrs, 4, None, 0, 0, 0))) == \
            B.PS_ERR_INVALID_ARG
    for tail in ((4, None, 1, 0, 0), (4, None, 0, 1, 0), (4, None, 0, 0, 1), (-1, None, 0, 0, 0),
                 (4, 256, 64, 10, 0)):                      # the last: ring pointers and a table
        assert _call(g, ga, dict(cache=B.PsKVCacheQ4(*six, *tail))) == B.PS_ERR_INVALID_ARG
    pool = [256, 256, 256, None, None, None]
    for tail, code in (((4, 256, 64, 9, 0), B.PS_ERR_INVALID_ARG),
                       ((4, 256, 0, 10, 0), B.PS_ERR_INVALID_ARG),
                       ((4, 258, 64, 10, 0), B.PS_ERR_INVALID_ARG)):
        assert _call(g, ga, dict(cache=B.PsKVCacheQ4(*pool, *tail))) == code
    paged = B.PsKVCacheQ4(*pool, 4, 256, 64, 10, 0)
    assert _call(g, ga, dict(cache=paged, params=_params(window=500))) == B.PS_ERR_UNSUPPORTED
    for over, code in ((dict(stride=9), B.PS_ERR_INVALID_ARG), (dict(nb=0), B.PS_ERR_INVALID_ARG),
                       (dict(table=None), B.PS_ERR_INVALID_ARG),
                       (dict(table=258), B.PS_ERR_INVALID_ARG),
                       (dict(kp=None), B.PS_ERR_INVALID_ARG), (dict(batch=-1), B.PS_ERR_INVALID_ARG),
                       (dict(params=_params(window=500)), B.PS_ERR_UNSUPPORTED)):
        assert _call(h, ha, over) == code


def test_empty_batches_do_nothing(lib):
    (f, fa), (g, ga), (h, ha) = _append_calls(lib, _params())
    assert _call(f, fa, dict(cache=B.PsKVCache(None, None, None, None, 0))) == B.PS_OK
    none = B.PsKVCacheQ4(*[None] * 6, 0, None, 0, 0, 0)
    assert _call(g, ga, dict(cache=none)) == B.PS_OK
    assert _call(h, ha, dict(batch=0)) == B.PS_OK
    p = _params()
    assert lib.ps_kv_read_q4(p, none, 256, 1, 256, 256, None, None) == B.PS_OK
    assert lib.ps_decode_attn_q4(p, none, 256, 256, 256, None, None, 0, None, None) == B.PS_OK


def test_read_and_decode_refusals(lib):
    p = _params()
    cache = B.PsKVCacheQ4(*[256] * 6, 4, None, 0, 0, 0)
    read = dict(params=p, cache=cache, pos0=256, T=1, k=256, v=256, status=None, stream=None)
    for over in (dict(cache=None), dict(pos0=None), dict(pos0=260), dict(T=0),
                 dict(k=None, v=None), dict(k=264), dict(status=258)):
        assert _call(lib.ps_kv_read_q4, read, over) == B.PS_ERR_INVALID_ARG, over
    need = B.ps_decode_q4_workspace_bytes(p, 4)
    dec = dict(params=p, cache=cache, q=256, pos=256, out=256, lse=None, ws=256, wsb=need,
               status=None, stream=None)
    half = B.PsKVCacheQ4(None, None, None, 256, 256, 256, 4, None, 0, 0, 0)
    for over, code in ((dict(cache=None), B.PS_ERR_INVALID_ARG),
                       (dict(cache=half), B.PS_ERR_INVALID_ARG),  # a decode reads the prefix
                       (dict(q=264), B.PS_ERR_INVALID_ARG), (dict(pos=None), B.PS_ERR_INVALID_ARG),
                       (dict(pos=260), B.PS_ERR_INVALID_ARG), (dict(out=None), B.PS_ERR_INVALID_ARG),
                       (dict(lse=258), B.PS_ERR_INVALID_ARG),
                       (dict(status=258), B.PS_ERR_INVALID_ARG),
                       (dict(params=_params(n_q_heads=32)), B.PS_ERR_UNSUPPORTED)):
        assert _call(lib.ps_decode_attn_q4, dec, over) == code, over
    if need:
        assert _call(lib.ps_decode_attn_q4, dec, dict(wsb=need - 1)) == B.PS_ERR_WORKSPACE
        assert _call(lib.ps_decode_attn_q4, dec, dict(ws=None)) == B.PS_ERR_WORKSPACE
        assert _call(lib.ps_decode_attn_q4, dec, dict(ws=264)) == B.PS_ERR_INVALID_ARG
    assert B.ps_decode_q4_workspace_bytes(_params(head_dim=64), 4) == 0


def test_reference_pack_and_quantiser():
    """The tests' own packing is the documented one, and a row's values are within half a step."""
    rng = np.random.default_rng(5)
    x = R.bf16(rng.normal(size=(7, 128)) * 3)
    u, s, m = R.quantise(x)
    assert np.array_equal(R.unpack(R.pack(u)), u)
    # s is rounded to bf16 (2^-8 either way): the greatest value is off by up to 15 s 2^-8 more
    err = np.abs(R.values(u, s, m).reshape(7, 2, 64) - x.reshape(7, 2, 64))
    assert (err <= s * (0.5 + 15 * 2.0 ** -8)).all()
    row = np.zeros(64, np.uint8)
    row[4 * 2 * 3 + 1] = 0x50   # word 6 (block 3 of group 0), bits 8-15: code at bit 12 is 5
    u = R.unpack(row)
    assert u[0, 24 + 6] == 5 and u.sum() == 5
