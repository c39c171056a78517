"""Cases for the query/key norm with rotary positions (forward and backward), the appends that
apply it on the way into the bf16 and the 4-bit store, and decode attention over the 4-bit store.

Each case names an operator ("op") and its sizes.  `run` computes it from elementary torch
operations where `own` is false, and through the library's entry points where it is true.

Sizes are the repository's: 16 query / 2 KV heads and 28 / 4 heads of 128, prefixes of 100 to
2000 rows, windows of 512 to 8192, positions up to 131072, training slices of 8192 tokens.

4-bit rows: a row of 128 dims is two groups of 64; a group keeps bf16 (scale s, minimum m) and
4-bit codes u, and stands for m + s u.  Its 64 bytes are sixteen 32-bit words; word 2 b + g
holds dims 64 g + 8 b + e (e = 0..7), code e at bit 4 (e >> 1) + 16 (e & 1).  One record of
eight bf16 per row: K s, m of group 0, s, m of group 1, then V's four.
"""
import math

import torch

own = False

D = 128
EPS = 1e-6
THETA = 1.0e6


# ------------------------------------------------------------------ cases
def listed():
    half = {"layout": "half", "rotary_dim": 128, "scaling": "none"}
    return [
        # one short prompt chunk of the small model: latency is what counts
        {"name": "norm_rope 64 tokens", "op": "fwd", "tokens": 64, "hq": 16, "hkv": 2,
         "pos_hi": 131072, "norm": True, "weights": "bf16", **half},
        # the truncated-backprop slice: 4 sequences of 8192 tokens, q/k inside packed qkv rows
        {"name": "norm_rope 4x8192 tokens", "op": "fwd", "tokens": 32768, "hq": 28, "hkv": 4,
         "pos_hi": 8191, "norm": True, "weights": "bf16", **half},
        # an odd packed batch with half the head rotated in pairs and stretched frequencies
        {"name": "norm_rope_bwd 1021 tokens", "op": "bwd", "tokens": 1021, "hq": 16, "hkv": 2,
         "pos_hi": 40000, "norm": True, "weights": "fp32", "layout": "interleaved",
         "rotary_dim": 64, "scaling": "by_parts"},
        # the backward of the training slice
        {"name": "norm_rope_bwd 4x8192 tokens", "op": "bwd", "tokens": 32768, "hq": 28, "hkv": 4,
         "pos_hi": 8191, "norm": True, "weights": "bf16", **half},
        # one decode step's append, 64 sequences past their window
        {"name": "append b64 T1", "op": "append", "batch": 64, "T": 1, "hq": 16, "hkv": 2,
         "lp": 100, "w": 4096, "pos_lo": 8192, "pos_hi": 131072, "norm": True, "weights": "bf16",
         **half},
        # prompts of 2125 tokens into the paged store: part prefix, part ring, longer than the ring
        {"name": "append paged b4 T2125", "op": "append_paged", "batch": 4, "T": 2125, "hq": 28,
         "hkv": 4, "lp": 250, "w": 1024, "pos_lo": 0, "pos_hi": 0, "norm": True,
         "weights": "bf16", "layout": "half", "rotary_dim": 128, "scaling": "yarn"},
        # one decode step's append into the 4-bit store (and the rows read back)
        {"name": "append_q4 b64 T1", "op": "append_q4", "batch": 64, "T": 1, "hq": 16, "hkv": 2,
         "lp": 100, "w": 4096, "pos_lo": 8192, "pos_hi": 131072, "norm": True, "weights": "bf16",
         **half},
        # long prompts into the 4-bit store: only the prefix and the last W tokens survive
        {"name": "append_q4 b4 T8192", "op": "append_q4", "batch": 4, "T": 8192, "hq": 28,
         "hkv": 4, "lp": 256, "w": 4096, "pos_lo": 0, "pos_hi": 0, "norm": True,
         "weights": "bf16", **half},
        # one sequence, W = 512: latency
        {"name": "decode_q4 b1 w512", "op": "decode_q4", "batch": 1, "hq": 16, "hkv": 2,
         "lp": 100, "w": 512, "pos_lo": 100, "pos_hi": 2147},
        # the headline decode shape, every window full
        {"name": "decode_q4 b64 w4096", "op": "decode_q4", "batch": 64, "hq": 16, "hkv": 2,
         "lp": 100, "w": 4096, "pos_lo": 8192, "pos_hi": 131072},
        # a large batch of the larger model (7 heads a KV head), some windows not yet full
        {"name": "decode_q4 b256 ragged", "op": "decode_q4", "batch": 256, "hq": 28, "hkv": 4,
         "lp": 100, "w": 4096, "pos_lo": 2000, "pos_hi": 131072},
        # full attention: four long linear caches of different lengths
        {"name": "decode_q4 linear b4 131072", "op": "decode_q4", "batch": 4, "hq": 16, "hkv": 2,
         "lp": 131072, "w": 0, "pos_lo": 60000, "pos_hi": 131071},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "append", "append_paged", "append_q4", "decode_q4"])
    hq, hkv = rng.choice([(16, 2), (28, 4), (8, 1), (4, 4), (32, 8)])
    c = {"op": op, "hq": hq, "hkv": hkv}
    if op != "decode_q4":
        c["layout"] = rng.choice(["half", "interleaved"])
        c["rotary_dim"] = rng.choice([128, 128, 64, 32, 96])
        c["scaling"] = rng.choice(["none", "linear", "by_parts", "yarn"])
        c["norm"] = rng.random() < 0.75
        c["weights"] = rng.choice(["bf16", "fp32"])
    if op in ("fwd", "bwd"):
        c["tokens"] = _log(rng, 1, 24000)
        c["pos_hi"] = rng.choice([8191, 131072, 1 << 20])
        return c
    if op == "decode_q4":
        if rng.random() < 0.25:
            c["lp"], c["w"] = _log(rng, 1000, 131072), 0
            c["batch"] = max(1, min(_log(rng, 1, 64), int(1.0e6 / (c["lp"] * hkv))))
            c["pos_lo"], c["pos_hi"] = rng.randint(0, c["lp"] // 2), c["lp"] - 1
            return c
        c["lp"] = rng.choice([0, 33, 100, 256, 2000])
        c["w"] = _log(rng, 64, 8192)
        c["batch"] = max(1, min(_log(rng, 1, 512), int(4.0e6 / ((c["lp"] + c["w"]) * hkv))))
        c["pos_lo"] = rng.choice([0, c["lp"] + c["w"]])
        c["pos_hi"] = c["pos_lo"] + _log(rng, 64, 131072)
        return c
    c["lp"] = rng.choice([0, 33, 100, 256, 2000])
    c["w"] = 64 * _log(rng, 1, 64) if op == "append_paged" else _log(rng, 64, 4096)
    c["T"] = _log(rng, 1, 8192)
    c["batch"] = max(1, min(_log(rng, 1, 256), int(40000 / c["T"]), int(1.5e6 / (c["w"] * hkv))))
    c["pos_lo"] = rng.choice([0, c["lp"] + c["w"]])
    c["pos_hi"] = c["pos_lo"] + (0 if c["pos_lo"] == 0 else 100000)
    return c


# ------------------------------------------------------------------ frequencies
SCALE = {"none": None,
         "linear": {"factor": 4.0},
         "by_parts": {"factor": 8.0, "low": 1.0, "high": 4.0, "original_len": 8192},
         "yarn": {"factor": 4.0, "low": 1.0, "high": 32.0, "original_len": 32768}}


def _attn_factor(case):
    return 0.1 * math.log(SCALE["yarn"]["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0


def _frequencies(case):
    """Angle per position of each rotated pair (floats, 64 bits)."""
    R, s = case["rotary_dim"], SCALE[case["scaling"]]
    f = [THETA ** (-2.0 * i / R) for i in range(R // 2)]
    if s is None:
        return f
    if case["scaling"] == "linear":
        return [x / s["factor"] for x in f]
    if case["scaling"] == "by_parts":
        turns = [s["original_len"] * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (r - s["low"]) / (s["high"] - s["low"]))) for r in turns]
    else:
        def index_of(turn):
            return R * math.log(s["original_len"] / (2 * math.pi * turn)) / (2 * math.log(THETA))
        lo = max(math.floor(index_of(s["high"])), 0)
        hi = min(math.ceil(index_of(s["low"])), R - 1)
        hi = hi if hi > lo else lo + 0.001
        keep = [1.0 - min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(R // 2)]
    return [(1 - k) * x / s["factor"] + k * x for k, x in zip(keep, f)]


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).bfloat16()


def _positions(g, lo, hi, n):
    return torch.randint(int(lo), int(hi) + 1, (n,), generator=g, device="cuda",
                         dtype=torch.int64)


def _weight(g, case):
    w = (1.0 + 0.3 * torch.randn(D, generator=g, device="cuda")).clamp_(0.1, 3.0)
    return w.bfloat16() if case["weights"] == "bf16" else w


def _quantise(x):
    """x: values on the bf16 grid [..., 128] (fp32) -> (codes, s, m), groups [..., 2, 64]."""
    x = x.unflatten(-1, (2, 64))
    m = x.amin(-1, keepdim=True)
    s = ((x.amax(-1, keepdim=True) - m) / 15).bfloat16().float()
    u = torch.round((x - m) / torch.where(s > 0, s, 1.0)).clamp_(0, 15)
    return u, s, m


def _pack(u):
    """codes [..., 2, 64] -> bytes [..., 64]."""
    u = u.to(torch.uint8).unflatten(-1, (8, 8)).transpose(-2, -3)  # [..., 8 blocks, 2 groups, 8]
    lo, hi = u[..., [0, 4, 1, 5]], u[..., [2, 6, 3, 7]]
    return (lo | (hi << 4)).flatten(-3).contiguous()


def _unpack(p):
    """bytes [..., 64] -> codes [..., 2, 64], fp32."""
    p = p.unflatten(-1, (8, 2, 4))
    u = torch.stack((p & 15, p >> 4), -1).flatten(-2)[..., [0, 4, 1, 5, 2, 6, 3, 7]]
    return u.transpose(-2, -3).flatten(-2).float()


def _store4(g, *rows):
    """A 4-bit store of random keys and values: payloads [*rows, 64] and records [*rows, 8]."""
    rec = []
    pay = []
    chan = 0.5 + torch.rand(D, generator=g, device="cuda")  # keys differ by channel
    for scale in (chan, 1.0):
        x = (torch.randn(*rows, D, generator=g, device="cuda") * scale).bfloat16().float()
        u, s, m = _quantise(x)
        pay.append(_pack(u))
        rec.append(torch.cat((s, m), -1).flatten(-2))
        del x, u
    return pay[0], pay[1], torch.cat(rec, -1).bfloat16().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hkv, op = case["hq"], case["hkv"], case["op"]
    s = {"case": case}
    if op == "decode_q4":
        B, lp, w = case["batch"], case["lp"], case["w"]
        s["pre"] = _store4(g, B, hkv, lp) if lp else None
        s["ring"] = _store4(g, B, hkv, w) if w else None
        s["q"] = 1.5 * _normal(g, B, hq, D)
        s["pos"] = _positions(g, case["pos_lo"], case["pos_hi"], B)
        s["out"] = torch.empty(B, hq, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(B, hq, dtype=torch.float32, device="cuda")
        return s
    s["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    s["wq"], s["wk"] = (_weight(g, case), _weight(g, case)) if case["norm"] else (None, None)
    n = case["tokens"] if op in ("fwd", "bwd") else case["batch"] * case["T"]
    heads = hq + 2 * hkv
    # packed rows of one projection: q heads, k heads, v heads
    qkv = _normal(g, n, heads, D) * (0.5 + torch.rand(heads, D, generator=g, device="cuda"))
    s["qkv"] = qkv.bfloat16()
    s["q"], s["k"], s["v"] = s["qkv"].split((hq, hkv, hkv), 1)
    bf = {"dtype": torch.bfloat16, "device": "cuda"}
    s["q_out"] = torch.empty(n, hq, D, **bf)
    if op in ("fwd", "bwd"):
        s["pos"] = _positions(g, 0, case["pos_hi"], n)
        s["k_out"] = torch.empty(n, hkv, D, **bf)
        if op == "bwd":
            s["dyq"], s["dyk"] = _normal(g, n, hq, D), _normal(g, n, hkv, D)
            s["dqkv"] = torch.zeros(n, heads, D, **bf)
            s["dq"], s["dk"], _ = s["dqkv"].split((hq, hkv, hkv), 1)
            s["dwq"] = torch.empty(D, device="cuda") if case["norm"] else None
            s["dwk"] = torch.empty(D, device="cuda") if case["norm"] else None
        return s
    B, T, lp, w = case["batch"], case["T"], case["lp"], case["w"]
    s["pos0"] = _positions(g, case["pos_lo"], case["pos_hi"], B)
    if op == "append_q4":
        s["pre"] = _empty4(B, hkv, lp) if lp else None
        s["ring"] = _empty4(B, hkv, w)
        s["k_read"], s["v_read"] = (torch.empty(B, T, hkv, D, **bf) for _ in range(2))
        return s
    if op == "append_paged":
        per = -(-lp // 64) + w // 64
        s["table"] = torch.randperm(B * per, generator=g, device="cuda").int().view(B, per)
        rows = B * per * hkv * 64
    else:
        rows = B * hkv * (lp + w)
    # one allocation a tensor, with a row at its end that belongs to no store
    s["k_flat"], s["v_flat"] = (torch.zeros(rows + 1, D, **bf) for _ in range(2))
    if op == "append_paged":
        s["k_pool"], s["v_pool"] = (f[:rows].view(B * per, hkv, 64, D)
                                    for f in (s["k_flat"], s["v_flat"]))
    else:
        cut = B * hkv * lp
        for x in "kv":
            f = s[x + "_flat"]
            s[x + "_pre"] = f[:cut].view(B, hkv, lp, D)
            s[x + "_ring"] = f[cut:rows].view(B, hkv, w, D)
    return s


def _empty4(*rows):
    z = {"dtype": torch.uint8, "device": "cuda"}
    return (torch.zeros(*rows, 64, **z), torch.zeros(*rows, 64, **z),
            torch.zeros(*rows, 8, dtype=torch.bfloat16, device="cuda"))


# ------------------------------------------------------------------ plain forms
def _cos_sin(s, pos):
    a = pos.double()[:, None, None] * s["freq"]
    f = _attn_factor(s["case"])
    return (torch.cos(a) * f).float(), (torch.sin(a) * f).float()


def _turn(x, cos, sin, case):
    """Rotates the first rotary_dim dims of x [n, H, D] (fp32)."""
    R = case["rotary_dim"]
    if case["layout"] == "half":
        a, b, rest = x[..., :R // 2], x[..., R // 2:R], x[..., R:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
    a, b, rest = x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest),
                     -1)


def _normed(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _plain_forward(s, x, w, cos, sin):
    return _turn(_normed(x.float(), w), cos, sin, s["case"]).bfloat16()


def _plain_backward(s, x, w, dy, cos, sin):
    g = _turn(dy.float(), cos, -sin, s["case"])
    if w is None:
        return g.bfloat16(), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n, gw = x * r, g * w.float()
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    return dx.bfloat16(), (g * n).double().sum((0, 1)).float()


def _token_positions(s):
    c = s["case"]
    return (s["pos0"][:, None] + torch.arange(c["T"], device="cuda")).flatten()


def _held(s, pos):
    """Per token: it goes to the prefix, it goes to the ring (the newest of its slot)."""
    c = s["case"]
    last = (s["pos0"] + c["T"] - 1).repeat_interleave(c["T"])
    return pos < c["lp"], (pos >= c["lp"]) & (pos > last - c["w"])


def _plain_rows(s):
    pos = _token_positions(s)
    cos, sin = _cos_sin(s, pos)
    q = _plain_forward(s, s["q"], s["wq"], cos, sin)
    k = _plain_forward(s, s["k"], s["wk"], cos, sin)
    return pos, q, k


def _plain_append(s):
    c = s["case"]
    B, T, lp, w, hkv = c["batch"], c["T"], c["lp"], c["w"], c["hkv"]
    pos, q, k = _plain_rows(s)
    pre, ring = _held(s, pos)
    seq = torch.arange(B, device="cuda").repeat_interleave(T)
    h = torch.arange(hkv, device="cuda")
    slot = torch.remainder(pos - lp, w)
    if c["op"] == "append_paged":
        block = torch.where(pre, pos // 64, -(-lp // 64) + slot // 64)
        row = torch.where(pre, pos, slot) % 64
        at = (s["table"][seq, block.clamp(0, s["table"].shape[1] - 1)].long()[:, None] * hkv
              + h) * 64 + row[:, None]
    else:
        at = torch.where(pre[:, None], (seq[:, None] * hkv + h) * lp + pos[:, None],
                         B * hkv * lp + (seq[:, None] * hkv + h) * w + slot[:, None])
    at = torch.where((pre | ring)[:, None], at, s["k_flat"].shape[0] - 1).flatten()
    s["k_flat"][at] = k.view(-1, D)
    s["v_flat"][at] = s["v"].reshape(-1, D)
    return q


def _four_bit(x):
    u, sc, m = _quantise(x.float())
    return (m + sc * u).flatten(-2)


def _plain_append_q4(s):
    c = s["case"]
    pos, q, k = _plain_rows(s)
    pre, ring = _held(s, pos)
    here = (pre | ring)[:, None, None]
    shape = (c["batch"], c["T"], c["hkv"], D)
    k = torch.where(here, _four_bit(k), 0.0).bfloat16().view(shape)
    v = torch.where(here, _four_bit(s["v"]), 0.0).bfloat16().view(shape)
    return {"q": q, "k": k, "v": v}


def _row_positions(case, pos):
    """Which position each row of [prefix, ring] holds for a query at pos, and if it sees it."""
    lp, w = case["lp"], case["w"]
    r = torch.arange(lp, device="cuda").expand(len(pos), lp)
    if w:
        slot = torch.arange(w, device="cuda")
        newest = pos[:, None] - torch.remainder(pos[:, None] - lp - slot, w)
        r = torch.cat((r, newest), 1)
    edge = torch.arange(lp + w, device="cuda") < lp
    return (r <= pos[:, None]) & (edge | (r >= lp))


def _plain_decode(s):
    c = s["case"]
    B, hq, hkv = c["batch"], c["hq"], c["hkv"]
    parts = [p for p in (s["pre"], s["ring"]) if p is not None]
    rec = torch.cat([p[2] for p in parts], 2).float()
    see = _row_positions(c, s["pos"])[:, None, None, :]

    def values(i):
        u = _unpack(torch.cat([p[i] for p in parts], 2))
        a = rec[..., 4 * i:4 * i + 4].unflatten(-1, (2, 2))
        return (a[..., 1:] + a[..., :1] * u).flatten(-2)

    q = s["q"].float().view(B, hkv, hq // hkv, D)
    sc = (q @ values(0).transpose(-1, -2)) * (1.0 / math.sqrt(D))
    sc = sc.masked_fill(~see, -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - top)
    z = p.sum(-1, keepdim=True)
    out = ((p @ values(1)) / z).view(B, hq, D).bfloat16()
    return {"out": out, "lse": (top + torch.log(z)).view(B, hq)}


# ------------------------------------------------------------------ one pass
def _handles(s):
    """What a program keeps: the rotary plan, the norm, the cache views and a workspace."""
    from prefix_sliding_window_b200 import binding as B
    c = s["case"]
    lp, w = c.get("lp", 0), c.get("w", 1)
    h = {"params": B.make_params(c["hq"], c["hkv"], D, lp, max(w, 1), THETA)}
    if c["op"] != "decode_q4":
        h["rope"] = B.make_rope(h["params"], c["layout"], c["rotary_dim"], c["scaling"],
                                attn_factor=_attn_factor(c), **(SCALE[c["scaling"]] or {}))
        h["norm"] = B.make_norm(s["wq"], s["wk"], EPS) if c["norm"] else None
    ws = 0
    if c["op"] == "bwd":
        ws = B.ps_qk_norm_rope_bwd_workspace_bytes(h["params"], c["tokens"])
    if c["op"] == "decode_q4":
        ws = B.ps_decode_q4_workspace_bytes(h["params"], c["batch"])
    h["ws"] = torch.empty(ws, dtype=torch.uint8, device="cuda") if ws else None
    if c["op"] in ("append_q4", "decode_q4"):
        h["cache"] = B.make_cache_q4(s["pre"], s["ring"], c["batch"])
    if c["op"] == "append":
        h["cache"] = B.make_cache(s["k_pre"] if lp else None, s["v_pre"] if lp else None,
                                  s["k_ring"], s["v_ring"], c["batch"])
    return h


def _run_own(s):
    from prefix_sliding_window_b200 import binding as B
    if "handles" not in s:
        s["handles"] = _handles(s)
    h, c = s["handles"], s["case"]
    op, par = c["op"], h["params"]
    if op == "fwd":
        B.ps_qk_norm_rope(par, h["rope"], h["norm"], s["q"], s["k"], s["pos"], s["q_out"],
                          s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "bwd":
        B.ps_qk_norm_rope_bwd(par, h["rope"], h["norm"], s["q"], s["k"], s["pos"], s["dyq"],
                              s["dyk"], s["dq"], s["dk"], s["dwq"], s["dwk"], h["ws"])
        return {"dq": s["dq"], "dk": s["dk"], "dwq": s["dwq"], "dwk": s["dwk"]}
    if op == "append":
        B.ps_kv_append_norm_rope(par, h["rope"], h["norm"], h["cache"], s["k"], s["v"], s["q"],
                                 s["q_out"], s["pos0"], c["T"])
        return {"q": s["q_out"], **{x: s[x] for x in ("k_pre", "v_pre", "k_ring", "v_ring")}}
    if op == "append_paged":
        B.ps_kv_append_norm_rope_paged(par, h["rope"], h["norm"], s["k_pool"], s["v_pool"],
                                       s["table"], c["batch"], s["k"], s["v"], s["q"], s["q_out"],
                                       s["pos0"], c["T"])
        return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op == "append_q4":
        B.ps_kv_append_norm_rope_q4(par, h["rope"], h["norm"], h["cache"], s["k"], s["v"], s["q"],
                                    s["q_out"], s["pos0"], c["T"])
        B.ps_kv_read_q4(par, h["cache"], s["pos0"], c["T"], s["k_read"], s["v_read"])
        return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}
    B.ps_decode_attn_q4(par, h["cache"], s["q"], s["pos"], s["out"], s["lse"], h["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op in ("fwd", "bwd"):
        cos, sin = _cos_sin(s, s["pos"])
        if op == "fwd":
            return {"q": _plain_forward(s, s["q"], s["wq"], cos, sin),
                    "k": _plain_forward(s, s["k"], s["wk"], cos, sin)}
        dq, dwq = _plain_backward(s, s["q"], s["wq"], s["dyq"], cos, sin)
        dk, dwk = _plain_backward(s, s["k"], s["wk"], s["dyk"], cos, sin)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if op == "append":
        q = _plain_append(s)
        return {"q": q, **{x: s[x] for x in ("k_pre", "v_pre", "k_ring", "v_ring")}}
    if op == "append_paged":
        q = _plain_append(s)
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op == "append_q4":
        return _plain_append_q4(s)
    return _plain_decode(s)


# ------------------------------------------------------------------ what a pass cannot do without
def _stored_tokens(c):
    """Tokens of one sequence that an append leaves in its store."""
    pre = max(0, min(c["T"], c["lp"] - c["pos_lo"]))
    return pre + min(c["T"] - pre, c["w"])


def work(case):
    hq, hkv, op = case["hq"], case["hkv"], case["op"]
    row = 2 * D
    if op in ("fwd", "bwd"):
        n, el = case["tokens"], case["tokens"] * (hq + hkv) * D
        return {"bytes": (2 if op == "fwd" else 3) * n * (hq + hkv) * row + 8 * n,
                "flops": (7 if op == "fwd" else 14) * el}
    if op == "decode_q4":
        cap = case["lp"] + case["w"]
        lo, hi = case["pos_lo"] + 1, case["pos_hi"] + 1
        short = max(0, min(hi, cap) - lo + 1)  # lengths lo .. min(hi, cap), one each
        total = short * (lo + min(hi, cap)) / 2 + (hi - lo + 1 - short) * cap
        keys = case["batch"] * total / (hi - lo + 1)
        return {"bytes": keys * hkv * 144 + case["batch"] * hq * (2 * row + 4),
                "flops": keys * hq * 4 * D}
    B, T = case["batch"], case["T"]
    kept = B * _stored_tokens(case)
    q = 2 * B * T * hq * row
    flops = 7 * B * T * hq * D + 7 * kept * hkv * D
    if op == "append_q4":
        return {"bytes": q + kept * hkv * (2 * row + 2 * 144) + B * T * hkv * 2 * row,
                "flops": flops + 10 * kept * hkv * 2 * D}
    return {"bytes": q + kept * hkv * 4 * row, "flops": flops}


# ------------------------------------------------------------------ the definition, in 64 bits
def _spin(x, w, pos, case):
    """Norm and rotation of x [n, H, D] in 64 bits, the pairs as complex numbers."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
    R = case["rotary_dim"]
    f = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full_like(f, _attn_factor(case)), f * 0)  # modulus
    z = z * torch.exp(1j * (pos.double()[:, None] * f))
    y = x.clone()
    if case["layout"] == "half":
        c = torch.complex(x[..., :R // 2], x[..., R // 2:R]) * z[:, None]
        y[..., :R // 2], y[..., R // 2:R] = c.real, c.imag
    else:
        c = torch.view_as_complex(x[..., :R].contiguous().view(*x.shape[:2], R // 2, 2))
        y[..., :R] = torch.view_as_real(c * z[:, None]).flatten(-2)
    return y


def _exact_grad(x, w, dy, pos, case):
    x = x.double().requires_grad_(True)
    w = w.double().requires_grad_(True) if w is not None else None
    xn = x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w
    R = case["rotary_dim"]
    f = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    a = pos.double()[:, None, None] * f
    c, sn = torch.cos(a) * _attn_factor(case), torch.sin(a) * _attn_factor(case)
    i = torch.arange(R // 2, device="cuda")
    one, two = (i, i + R // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
    dy = dy.double()
    loss = (xn[..., one] * (dy[..., one] * c + dy[..., two] * sn)).sum() \
        + (xn[..., two] * (dy[..., two] * c - dy[..., one] * sn)).sum() \
        + (xn[..., R:] * dy[..., R:]).sum()
    loss.backward()
    return x.grad, None if w is None else w.grad


def _slots(s, rows_k, rows_v):
    """The store after an append, slot by slot: which token of the call each one got."""
    c = s["case"]
    B, T, lp, w, hkv = c["batch"], c["T"], c["lp"], c["w"], c["hkv"]
    p0 = s["pos0"][:, None]
    t_pre = torch.arange(lp, device="cuda") - p0
    slot = torch.arange(w, device="cuda")
    t_ring = T - 1 - torch.remainder(p0 + T - 1 - lp - slot, w)
    out = []
    for t, ok in ((t_pre, (t_pre >= 0) & (t_pre < T)), (t_ring, (t_ring >= 0) & (p0 + t_ring >= lp))):
        for rows in (rows_k, rows_v):
            r = rows.view(B, T, hkv, D)
            got = r.gather(1, t.clamp(0, T - 1)[:, :, None, None].expand(-1, -1, hkv, D))
            out.append(torch.where(ok[:, :, None, None], got, 0.0).transpose(1, 2))
    return out  # k_pre, v_pre, k_ring, v_ring: [B, hkv, rows, D]


def _exact_decode(s):
    c = s["case"]
    hq, hkv, lp, w = c["hq"], c["hkv"], c["lp"], c["w"]
    outs, lses = [], []
    for b, p in enumerate(s["pos"].tolist()):
        first = max(lp, p - w + 1)
        rows = [(s["pre"], torch.arange(min(lp, p + 1), device="cuda"))] if lp else []
        if w and p >= lp:
            rows.append((s["ring"], (torch.arange(first, p + 1, device="cuda") - lp) % w))
        kv = []
        for i in (0, 1):
            parts = []
            for store, r in rows:
                by = store[i][b][:, r].long().unflatten(-1, (8, 2, 4))
                rec = store[2][b][:, r].double()
                val = torch.empty(hkv, len(r), 2, 8, 8, dtype=torch.float64, device="cuda")
                for e in range(8):
                    bit = 4 * (e >> 1) + 16 * (e & 1)
                    code = (by[..., bit // 8] >> (bit % 8)) & 15
                    val[..., e] = code.transpose(-1, -2)
                sc = rec[..., [4 * i, 4 * i + 2]][..., None, None]
                mn = rec[..., [4 * i + 1, 4 * i + 3]][..., None, None]
                parts.append((mn + sc * val).flatten(2))
            kv.append(torch.cat(parts, 1))
        q = s["q"][b].double().view(hkv, hq // hkv, D)
        sc = torch.einsum("hgd,hkd->hgk", q, kv[0]) / math.sqrt(D)
        outs.append(torch.einsum("hgk,hkd->hgd", torch.softmax(sc, -1), kv[1]).reshape(hq, D))
        lses.append(torch.logsumexp(sc, -1).reshape(hq))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "decode_q4":
        return _exact_decode(s)
    if op == "fwd":
        return {"q": _spin(s["q"], s["wq"], s["pos"], case),
                "k": _spin(s["k"], s["wk"], s["pos"], case)}
    if op == "bwd":
        dq, dwq = _exact_grad(s["q"], s["wq"], s["dyq"], s["pos"], case)
        dk, dwk = _exact_grad(s["k"], s["wk"], s["dyk"], s["pos"], case)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    pos = _token_positions(s)
    q = _spin(s["q"], s["wq"], pos, case)
    k = _spin(s["k"], s["wk"], pos, case)
    v = s["v"].double()
    if op == "append_q4":
        pre, ring = _held(s, pos)
        got = {"q": q}
        for name, x in (("k", k.bfloat16()), ("v", v)):
            x = x.double().unflatten(-1, (2, 64))  # the row that the bf16 store would hold
            m, top = x.min(-1, keepdim=True)[0], x.max(-1, keepdim=True)[0]
            sc = ((top - m) / 15).bfloat16().double()
            u = torch.where(sc > 0, ((x - m) / sc).round().clamp(0, 15), 0.0)
            x = torch.where((pre | ring)[:, None, None], (m + sc * u).flatten(-2), 0.0)
            got[name] = x.view(case["batch"], case["T"], case["hkv"], D)
        return got
    k_pre, v_pre, k_ring, v_ring = _slots(s, k, v)
    if op == "append":
        return {"q": q, "k_pre": k_pre, "v_pre": v_pre, "k_ring": k_ring, "v_ring": v_ring}
    got = {"q": q}
    B, hkv, lp, w = case["batch"], case["hkv"], case["lp"], case["w"]
    nb = -(-lp // 64)
    for name, pre, ring in (("k_pool", k_pre, k_ring), ("v_pool", v_pre, v_ring)):
        pad = torch.zeros(B, hkv, nb * 64, D, dtype=torch.float64, device="cuda")
        pad[:, :, :lp] = pre
        blocks = torch.cat((pad, ring), 2).view(B, hkv, -1, 64, D).transpose(1, 2)
        pool = torch.zeros(s["table"].numel(), hkv, 64, D, dtype=torch.float64, device="cuda")
        pool[s["table"].flatten().long()] = blocks.reshape(-1, hkv, 64, D)
        got[name] = pool
    return got
