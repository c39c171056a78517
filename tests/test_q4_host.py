"""Refusals of the 4-bit store's calls that need no GPU."""
import os

import pytest
import torch

from prefix_sliding_window_b200 import binding as B
from prefix_sliding_window_b200 import build as BLD


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        BLD.build(quiet=True)
    return B.load()


@pytest.mark.parametrize("scale,code", [(2.0 ** 33, B.PS_ERR_UNSUPPORTED),
                                        (float("inf"), B.PS_ERR_INVALID_ARG),
                                        (-1.0, B.PS_ERR_INVALID_ARG)])
def test_decode_scale_refused(lib, scale, code):
    p = B.make_params(16, 2, 128, 100, 512, softmax_scale=scale)
    cache = B.PsKVCacheQ4(*[256] * 6, 4, None, 0, 0, 0)
    rc = lib.ps_decode_attn_q4(p, cache, 256, 256, 256, None, 256, 1 << 30, None, None)
    assert rc == code and B.last_error() != ""


class _Fake:
    """What make_cache_q4 asks of a tensor, without a GPU."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.uint8, device=0):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, device

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 256


def _part(*rows, device=0):
    return (_Fake(*rows, 64, device=device), _Fake(*rows, 64, device=device),
            _Fake(*rows, 8, dtype=torch.bfloat16, device=device))


def _table(*shape, device=0):
    return _Fake(*shape, dtype=torch.int32, device=device)


PREFIX, RING = (4, 2, 100), (4, 2, 512)


@pytest.mark.parametrize("prefix,ring,batch,geometry", [
    (PREFIX, RING, 4, (2, 100, 512)),
    (PREFIX, RING, 3, (2, 100, 512)),          # a batch below the tensors'
    (None, RING, 4, (2, 100, 512)),            # ring only
    (PREFIX, RING, 4, (2, 0, 512)),            # no prefix row is asked for
    (PREFIX, None, 4, (2, 100, 1)),            # linear
    ((4, 2, 0), RING, 4, (2, 0, 512)),
    ((8, 100), RING, 4, (2, 100, 512)),        # the same rows without the batch's dim
])
def test_stores_that_hold_the_geometry(prefix, ring, batch, geometry):
    cache = B.make_cache_q4(prefix and _part(*prefix), ring and _part(*ring), batch)
    p = B.make_params(16, geometry[0], 128, *geometry[1:])
    for _ in range(2):
        B._store_q4_fits(p, cache)
    B._store_q4_fits(p, B.PsKVCacheQ4(*[256] * 6, 4, None, 0, 0, 0))  # addresses alone


@pytest.mark.parametrize("prefix,ring,batch,geometry", [
    (PREFIX, RING, 5, (2, 100, 512)),          # more sequences than the tensors have
    (PREFIX, RING, 4, (4, 100, 512)),          # more KV heads
    (PREFIX, RING, 4, (1, 100, 512)),
    (PREFIX, RING, 4, (2, 101, 512)),          # a longer prefix
    (PREFIX, RING, 4, (2, 100, 513)),          # a larger window
    (PREFIX, RING, 4, (2, 100, 256)),
    (PREFIX, (2, 2, 512), 4, (2, 100, 512)),   # the ring of another batch
    (PREFIX, None, 4, (2, 128, 1)),
    ((8, 99), RING, 4, (2, 100, 512)),
])
def test_stores_that_do_not(prefix, ring, batch, geometry):
    cache = B.make_cache_q4(prefix and _part(*prefix), ring and _part(*ring), batch)
    p = B.make_params(16, geometry[0], 128, *geometry[1:])
    for _ in range(2):
        with pytest.raises(ValueError):
            B._store_q4_fits(p, cache)


def test_a_store_is_looked_at_again_for_another_geometry():
    cache = B.make_cache_q4(_part(*PREFIX), _part(*RING), 4)
    B._store_q4_fits(B.make_params(16, 2, 128, 100, 512), cache)
    with pytest.raises(ValueError):
        B._store_q4_fits(B.make_params(16, 2, 128, 100, 600), cache)
    cache.batch = 9
    with pytest.raises(ValueError):
        B._store_q4_fits(B.make_params(16, 2, 128, 100, 512), cache)


def test_paged_stores():
    p = B.make_params(16, 2, 128, 100, 512)
    pool, table = _part(30, 2, 64), _table(4, 10)
    B._store_q4_fits(p, B.make_cache_q4(pool, None, 4, table))
    for bad in (_part(30, 4, 64), _part(30, 2, 32), _part(60, 64)):
        with pytest.raises(ValueError):
            B._store_q4_fits(p, B.make_cache_q4(bad, None, 4, table))
    with pytest.raises(ValueError):
        B.make_cache_q4(pool, None, 5, table)  # more sequences than the table has
    cache = B.make_cache_q4(pool, None, 4, table)
    cache.batch = 5
    with pytest.raises(ValueError):
        B._store_q4_fits(p, cache)


def test_parts_on_several_devices_refused():
    with pytest.raises(ValueError):
        B.make_cache_q4(_part(*PREFIX), _part(*RING, device=1), 4)
    with pytest.raises(ValueError):
        B.make_cache_q4(_part(30, 2, 64), None, 4, _table(4, 10, device=1))


def test_bf16_stores():
    def part(*shape, dtype=torch.bfloat16, device=0):
        t = _Fake(*shape, dtype=dtype, device=device)
        t.device = f"cuda:{device}"
        return t
    p = B.make_params(16, 2, 128, 100, 512)
    pre, ring = (4, 2, 100, 128), (4, 2, 512, 128)
    good = B.make_cache(part(*pre), part(*pre), part(*ring), part(*ring), 4)
    for _ in range(2):
        B._store_fits(p, good, 0)
    B._store_fits(p, B.PsKVCache(256, 256, 256, 256, 4), 0)  # addresses alone
    B._store_fits(p, B.make_cache(None, None, part(*ring), part(*ring), 4), 0)
    with pytest.raises(ValueError):
        B._store_fits(p, good, 1)
    for args in ((part(*pre), part(*pre), part(*ring), part(*ring), 5),
                 (part(*pre), part(3, 2, 100, 128), part(*ring), part(*ring), 4),
                 (part(*pre), part(*pre), part(*ring), part(4, 2, 500, 128), 4),
                 (part(*pre, dtype=torch.float32), part(*pre), part(*ring), part(*ring), 4),
                 (part(*pre), part(*pre, device=1), part(*ring), part(*ring), 4)):
        with pytest.raises(ValueError):
            B._store_fits(p, B.make_cache(*args), 0)


def test_one_of_a_pair_refused():
    """An input without its output, or the other way round: left out without a word it would leave
    an output unwritten."""
    p = B.make_params(4, 2, 128, 100, 512)
    rope = B.make_rope(p)
    q, k = (torch.zeros(3, h, 128, dtype=torch.bfloat16) for h in (4, 2))
    pos = torch.zeros(3, dtype=torch.int64)
    for args in ((None, k, pos, q, k), (q, k, pos, None, k), (q, None, pos, q, k),
                 (q, k, pos, q, None)):
        with pytest.raises(ValueError, match="go together"):
            B.ps_qk_norm_rope(p, rope, None, *args)
    for args in ((None, k, q, k), (q, k, None, k), (q, None, q, k), (q, k, q, None)):
        with pytest.raises(ValueError, match="go together"):
            B.ps_qk_norm_rope_bwd(p, rope, None, q, k, pos, *args)
    for args in ((None, q), (q, None)):
        with pytest.raises(ValueError, match="go together"):
            B._append_rows(p, 3, k, k, *args, pos, 1, 0)
