"""Calls whose store is too small for their geometry are refused before anything is launched."""
import pytest
import torch

from prefix_sliding_window_b200 import binding as B
from prefix_sliding_window_b200.cache import PrefixSlidingCache, QuantizedCache

pytestmark = pytest.mark.gpu
D = 128


def test_short_stores_refused(cuda_device):
    dev, Bn, hq, hkv, lp, w = cuda_device, 3, 8, 2, 40, 64
    params = B.make_params(hq, hkv, D, lp, w)
    rope = B.make_rope(params)
    bf = dict(dtype=torch.bfloat16, device=dev)
    pos = torch.zeros(Bn, dtype=torch.int64, device=dev)
    q, qo = (torch.zeros(Bn, hq, D, **bf) for _ in range(2))
    k, v = (torch.zeros(Bn, hkv, D, **bf) for _ in range(2))
    ws = torch.empty(max(1, B.ps_decode_q4_workspace_bytes(params, Bn)), dtype=torch.uint8,
                     device=dev)

    def calls(c):
        yield lambda: B.ps_kv_append_norm_rope_q4(params, rope, None, c, k, v, q, qo, pos, 1)
        yield lambda: B.ps_kv_read_q4(params, c, pos, 1, k, v)
        yield lambda: B.ps_decode_attn_q4(params, c, q, pos, qo, None, ws)
    for call in calls(QuantizedCache(Bn, hkv, lp, w, dev).struct):
        call()
    for shape in ((Bn - 1, hkv, lp, w), (Bn, 1, lp, w), (Bn, hkv, lp - 1, w), (Bn, hkv, lp, w // 2)):
        small = QuantizedCache(*shape, dev)
        c = B.make_cache_q4(small.prefix, small.ring, Bn)
        for call in calls(c):
            with pytest.raises(ValueError):
                call()
        if shape[1] == hkv:
            small = PrefixSlidingCache(*shape, D, dev)
            c = B.make_cache(small.k_prefix, small.v_prefix, small.k_ring, small.v_ring, Bn)
            with pytest.raises(ValueError):
                B.ps_kv_append_norm_rope(params, rope, None, c, k, v, q, qo, pos, 1)
    pool = QuantizedCache(9, hkv, 32, 0, dev).prefix
    table = torch.zeros(Bn, 2, dtype=torch.int32, device=dev)
    for call in calls(B.make_cache_q4(pool, None, Bn, table)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
