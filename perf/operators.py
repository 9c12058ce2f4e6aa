"""The microscaled 4-bit operators on real work: quantise and dequantise, the
linear layer forward and backward over a microscaled weight, and a
mixture-of-experts layer for a few tokens.  `own` picks the plain form
(elementary torch operations in 32 bits) or the framework's operators."""
import math

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"mxfp4": 32, "nvfp4": 16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a 7B projection's weight on its way into storage and back
        dict(name="codec_4096x4096_mx", op="codec", fmt="mxfp4", rows=4096, cols=4096, transpose=False),
        # a 65B feed-forward weight, laid out for the backward pass
        dict(name="codec_22016x8192_nv_t", op="codec", fmt="nvfp4", rows=22016, cols=8192, transpose=True),
        # a small ragged matrix: the latency of one call
        dict(name="codec_100x1000_nv", op="codec", fmt="nvfp4", rows=100, cols=1000, transpose=False),
        # one new token through the 65B feed-forward up projection
        dict(name="fwd_22016x8192_m1_mx", op="fwd", fmt="mxfp4", rows=22016, cols=8192, m=1, r=0),
        # sixteen new tokens through the 65B down projection, with an adapter
        dict(name="fwd_8192x22016_m16_nv_r64", op="fwd", fmt="nvfp4", rows=8192, cols=22016, m=16, r=64),
        # a training step's tokens through a 65B projection, with an adapter
        dict(name="fwd_8192x8192_m8192_mx_r64", op="fwd", fmt="mxfp4", rows=8192, cols=8192, m=8192, r=64),
        # a short prompt through a layer of odd sizes
        dict(name="fwd_1001x1999_m77_nv", op="fwd", fmt="nvfp4", rows=1001, cols=1999, m=77, r=0),
        # the input gradient of the 65B up projection for a training step's tokens
        dict(name="bwd_22016x8192_m8192_nv", op="bwd", fmt="nvfp4", rows=22016, cols=8192, m=8192),
        # the input gradient of the 7B up projection for one ragged sequence
        dict(name="bwd_11008x4096_m509_mx", op="bwd", fmt="mxfp4", rows=11008, cols=4096, m=509),
        # one new token over a routed feed-forward layer
        dict(name="moe_e64_k8_2048x1024_m1", op="moe", experts=64, top_k=8, hidden=2048, inner=1024, m=1),
        # sixteen new tokens over a wider one
        dict(name="moe_e32_k4_4096x1536_m16", op="moe", experts=32, top_k=4, hidden=4096, inner=1536, m=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["codec", "codec", "fwd", "fwd", "fwd", "bwd", "bwd", "moe"])
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op == "codec":
        return dict(op=op, fmt=fmt, rows=_log(rng, 1, 13000), cols=_log(rng, 1, 13000), transpose=rng.random() < 0.4)
    if op == "moe":
        return dict(op=op, experts=rng.choice([8, 12, 16, 32, 64]), top_k=rng.randint(1, 8), hidden=128 * _log(rng, 2, 32),
                    inner=128 * _log(rng, 1, 12), m=rng.randint(1, 16))
    m = _log(rng, 1, 8192)
    rows, cols = _log(rng, 64, 22016), _log(rng, 64, 22016)
    r = rng.choice([0, 0, 8, 64, 136]) if op == "fwd" else 0
    if r or rng.random() < 0.4:                      # an adapter needs the layer's usual multiples
        rows, cols = -(-rows // 8) * 8, -(-cols // 64) * 64
    most = 8192 * 22016 * 8192
    m = max(1, min(m, most // (rows * cols)))
    case = dict(op=op, fmt=fmt, rows=rows, cols=cols, m=m)
    return dict(case, r=r) if op == "fwd" else case


# ------------------------------------------------------------------ the formats, plain form
def _round_e2m1(v):
    """Nearest level of |v|, ties to the level with an even code; returns the code 0..7."""
    return ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))


def _pow2(e):
    """2^e for integer e in -149 .. 127, exact (also below the normal range)."""
    return torch.exp2(e.to(torch.float64)).to(torch.float32)


def _encode(x, fmt, per_row):
    """x [rows, cols] -> codes uint8 [rows, padded], scale bytes [rows, blocks], global scale [1] or [rows] (or None)."""
    x = x.to(torch.float32)
    rows, cols = x.shape
    blk = BLOCK[fmt]
    nb = -(-cols // blk)
    xb = torch.nn.functional.pad(x, (0, nb * blk - cols)).view(rows, nb, blk)
    amax = xb.abs().amax(dim=2)
    if fmt == "mxfp4":
        e = ((amax.view(torch.int32) >> 23) - 127 - 2).clamp(min=-127)
        q = xb.abs() * _pow2(-e)[:, :, None]
        sbytes, g = (e + 127).to(torch.uint8), None
    else:
        top = amax.amax(dim=1) if per_row else amax.amax().reshape(1)
        bits = top.view(torch.int32)
        e = (bits >> 23) - 127 - 11 + ((bits & 0x7FFFFF) > 0x280000).to(torch.int32)      # 2688 = 1.3125 * 2^11
        e = torch.where(top == 0, 0, e.clamp(min=-126))
        g = _pow2(e)
        inv = _pow2(-e)[:, None]
        s8 = ((amax * inv) / 6.0).to(torch.float8_e4m3fn)
        s = s8.to(torch.float32)[:, :, None]
        q = torch.where(s > 0, xb.abs() * inv[:, :, None] / s, 0.0)
        sbytes = s8.view(torch.uint8)
    codes = _round_e2m1(q) | (torch.signbit(xb).to(torch.uint8) << 3)
    codes = codes.view(rows, nb * blk)
    pad = -codes.shape[1] % 32
    return torch.nn.functional.pad(codes, (0, pad)), sbytes, g


def _values(codes, sbytes, g, fmt, cols):
    """The float32 values that codes and scales stand for, [rows, cols]."""
    rows = codes.shape[0]
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float32, device=codes.device)
    blk = BLOCK[fmt]
    nb = sbytes.shape[1]
    v = lut[codes[:, : nb * blk].to(torch.int32)].view(rows, nb, blk)
    s = _pow2(sbytes.to(torch.int32) - 127) if fmt == "mxfp4" else sbytes.view(torch.float8_e4m3fn).to(torch.float32)
    v = v * s[:, :, None]
    if g is not None:
        v = v * g[:, None, None]
    return v.view(rows, nb * blk)[:, :cols]


def _pack(codes):
    """Two codes a byte, the earlier one in the low four bits."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), dim=2).view(packed.shape[0], -1)


def _tile(sbytes):
    """Scale bytes [rows, blocks] -> tiles of 128 rows x 4 blocks, 512 bytes each: byte (r % 32) * 16 + (r / 32) * 4 + k."""
    rows, nb = sbytes.shape
    rt, kt = -(-rows // 128), -(-nb // 4)
    p = torch.nn.functional.pad(sbytes, (0, kt * 4 - nb, 0, rt * 128 - rows))
    return p.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile(tiles, rows, nb):
    rt, kt = -(-rows // 128), -(-nb // 4)
    return tiles.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :nb]


def _stored(w, fmt):
    """A weight as a program holds it after loading: packed codes, tiled scales, global scale."""
    codes, sbytes, g = _encode(w, fmt, False)
    return dict(codes=_pack(codes).view(-1), scales=_tile(sbytes), g=g, rows=w.shape[0], cols=w.shape[1], fmt=fmt)


def _weight_values(w):
    rows, cols = w["rows"], w["cols"]
    return _values(_unpack(w["codes"].view(rows, -1)), _untile(w["scales"], rows, -(-cols // BLOCK[w["fmt"]])), w["g"], w["fmt"], cols)


def _round_trip(x, fmt, per_row):
    codes, sbytes, g = _encode(x, fmt, per_row)
    return _values(codes, sbytes, g, fmt, x.shape[1])


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, std):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "codec":
        s["w"] = _normal(gen, (case["rows"], case["cols"]), 0.02)
    elif op == "fwd":
        rows, cols, m, r = case["rows"], case["cols"], case["m"], case["r"]
        s["weight"] = _stored(_normal(gen, (rows, cols), 0.02), case["fmt"])
        s["x"] = _normal(gen, (m, cols), 1.0)
        s["a"] = _normal(gen, (r, cols), 0.02) if r else None
        s["b"] = _normal(gen, (rows, r), 0.02) if r else None
        s["scale"] = 16.0 / r if r else 0.0
    elif op == "bwd":
        rows, cols, m = case["rows"], case["cols"], case["m"]
        s["weight"] = _stored(_normal(gen, (cols, rows), 0.02), case["fmt"])      # W^T, quantised along the rows of W
        s["dy"] = _normal(gen, (m, rows), 1e-3)
    else:
        e, h, f, m = case["experts"], case["hidden"], case["inner"], case["m"]
        s["w13"] = _stored(_normal(gen, (e * 2 * f, h), 0.02), "mxfp4")
        s["w2"] = _stored(_normal(gen, (e * h, f), 0.02), "mxfp4")
        s["router"] = _normal(gen, (e, h), 0.02)
        s["x"] = _normal(gen, (m, h), 1.0)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "codec":
        w = state["w"].t() if state["transpose"] else state["w"]
        return _round_trip(w, state["fmt"], False).to(torch.bfloat16)
    if op == "fwd":
        y = _round_trip(state["x"], state["fmt"], True) @ _weight_values(state["weight"]).t()
        if not state["r"]:
            return y.to(torch.bfloat16)
        xa = state["x"].to(torch.float32) @ state["a"].to(torch.float32).t()
        y = y + (state["scale"] * xa) @ state["b"].to(torch.float32).t()
        return y.to(torch.bfloat16), xa
    if op == "bwd":
        return (_round_trip(state["dy"], state["fmt"], True) @ _weight_values(state["weight"]).t()).to(torch.bfloat16)
    e, h, f, k = state["experts"], state["hidden"], state["inner"], state["top_k"]
    m = state["x"].shape[0]
    logits = state["x"].to(torch.float32) @ state["router"].to(torch.float32).t()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    p = torch.exp(top - top[:, :1])
    p = p / p.sum(dim=1, keepdim=True)
    token = torch.arange(m, device=ids.device)[:, None]
    gu = (_round_trip(state["x"], "mxfp4", True) @ _weight_values(state["w13"]).t()).view(m, e, 2, f)[token, ids]
    gate, up = gu[:, :, 0], gu[:, :, 1]
    inner = gate / (1.0 + torch.exp(-gate)) * up
    inner = _round_trip(inner.reshape(m * k, f), "mxfp4", True).view(m, k, f)
    spread = torch.zeros(m, e, f, device=ids.device).index_put((token, ids), inner)
    out = torch.bmm(spread.transpose(0, 1), _weight_values(state["w2"]).view(e, h, f).transpose(1, 2))
    y = (out.transpose(0, 1)[token, ids] * p[:, :, None]).sum(dim=1)
    return y.to(torch.bfloat16), ids.to(torch.int32), p


def _run_own(state):
    import bit_nf4_quantized_encode_b200 as qb

    def tensor(w):
        return qb.MXTensor(w["codes"], w["scales"], w["g"], w["rows"], w["cols"], w["fmt"])

    op = state["op"]
    if op == "codec":
        return qb.qlora_mx_dequantize(qb.qlora_mx_quantize(state["w"], state["fmt"], transpose=state["transpose"]))
    if op == "fwd":
        y, xa = qb.qlora_mx_linear_fwd(tensor(state["weight"]), state["x"], state["a"], state["b"], state["scale"])
        return (y, xa) if state["r"] else y
    if op == "bwd":
        return qb.qlora_mx_linear_bwd(tensor(state["weight"]), state["dy"])[0]
    return qb.qlora_mx_moe_fwd(tensor(state["w13"]), tensor(state["w2"]), state["router"], state["x"], state["top_k"])


# ------------------------------------------------------------------ what it has to do
def _stored_bytes(n, fmt):
    return n / 2 + n / BLOCK[fmt]


def work(case):
    op = case["op"]
    if op == "codec":
        n = case["rows"] * case["cols"]
        return dict(bytes=2 * n + 2 * _stored_bytes(n, case["fmt"]) + 2 * n, flops=0)
    if op in ("fwd", "bwd"):
        n, k, m, r = case["rows"], case["cols"], case["m"], case.get("r", 0)
        return dict(bytes=2 * m * (n + k) + _stored_bytes(n * k, case["fmt"]) + r * (2 * (n + k) + 4 * m),
                    flops=2 * m * n * k + 2 * m * r * (n + k))
    e, k, h, f, m = (case[x] for x in ("experts", "top_k", "hidden", "inner", "m"))
    k = min(k, e)
    active = e * (1.0 - (1.0 - k / e) ** m)              # experts that m tokens reach, on average
    return dict(bytes=2 * e * h + 4 * m * h + active * _stored_bytes(3 * h * f, "mxfp4") + 8 * m * k,
                flops=2 * m * e * h + 6 * m * k * h * f)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_quant(x, fmt, per_row):
    """Quantise and dequantise in 64 bits: the nearest of the eight levels by distance, ties to an even code."""
    x = x.double()
    rows, cols = x.shape
    blk = BLOCK[fmt]
    out = torch.empty_like(x)
    lv = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    mids, even = (lv[1:] + lv[:-1]) / 2, torch.arange(7, device=x.device) % 2 == 0
    if fmt == "nvfp4":
        whole = x.abs().amax(dim=1, keepdim=True) if per_row else x.abs().amax().reshape(1, 1).expand(rows, 1)
        ratio, ex = torch.frexp(whole / 2688.0)                       # ratio in [0.5, 1): the power of two at or above
        ge = torch.where(ratio == 0.5, ex - 1, ex).clamp(min=-126)
        g = torch.where(whole == 0, torch.ones_like(whole), torch.ldexp(torch.ones_like(whole), ge))
    for lo in range(0, rows, 2048):                                   # a few rows at a time: 64-bit copies are large
        part = x[lo : lo + 2048]
        nb = -(-cols // blk)
        b = torch.cat((part, part.new_zeros(part.shape[0], nb * blk - cols)), dim=1).reshape(-1, nb, blk)
        a = b.abs().amax(dim=2, keepdim=True)
        if fmt == "mxfp4":
            _, ex = torch.frexp(a)
            step = torch.ldexp(torch.ones_like(a), torch.where(a > 0, (ex - 3).clamp(min=-127), -127))
        else:
            want = a / g[lo : lo + 2048, :, None] / 6.0
            _, ex = torch.frexp(want)
            unit = torch.ldexp(torch.ones_like(want), (ex - 4).clamp(min=-9))     # spacing of e4m3 there
            step = (torch.round(want / unit) * unit).clamp(max=448.0) * g[lo : lo + 2048, :, None]
        t = torch.where(step > 0, b.abs() / step, 0.0)
        below = torch.bucketize(t, mids)                              # number of midpoints under t
        tie = (below < 7) & (t == mids[below.clamp(max=6)]) & ~even[below.clamp(max=6)]
        out[lo : lo + 2048] = (torch.sign(b) * lv[below + tie.long()] * step).reshape(-1, nb * blk)[:, :cols]
    return out


def _exact_stored(w):
    rows, cols, fmt = w["rows"], w["cols"], w["fmt"]
    r = torch.arange(rows, device="cuda")[:, None]
    packed = w["codes"].view(rows, -1)
    out = torch.empty(rows, cols, dtype=torch.float64, device="cuda")
    lv = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    tiles_k = -(-(-(-cols // BLOCK[fmt])) // 4)
    for lo in range(0, cols, 512):
        c = torch.arange(lo, min(cols, lo + 512), device="cuda")[None, :]
        nib = (packed[:, lo // 2 : (c[0, -1].item() // 2) + 1].repeat_interleave(2, dim=1)[:, : c.shape[1]].long() >> (4 * (c % 2))) & 15
        blk = c // BLOCK[fmt]
        byte = w["scales"][((r // 128) * tiles_k + blk // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + blk % 4].long()
        if fmt == "mxfp4":
            sc = torch.ldexp(torch.ones_like(byte, dtype=torch.float64), byte - 127)
        else:
            man, ex = byte & 7, byte >> 3
            sc = torch.where(ex > 0, torch.ldexp(1.0 + man.double() / 8, ex - 7), man.double() / 512)
        out[:, lo : lo + 512] = lv[nib & 7] * (1.0 - 2.0 * (nib >> 3)) * sc
    return out if w["g"] is None else out * w["g"].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "codec":
        return _exact_quant(s["w"].t() if case["transpose"] else s["w"], case["fmt"], False)
    if op == "fwd":
        y = _exact_quant(s["x"], case["fmt"], True) @ _exact_stored(s["weight"]).t()
        if not case["r"]:
            return y
        xa = s["x"].double() @ s["a"].double().t()
        return y + s["scale"] * (xa @ s["b"].double().t()), xa
    if op == "bwd":
        return _exact_quant(s["dy"], case["fmt"], True) @ _exact_stored(s["weight"]).t()
    e, h, f, k, m = case["experts"], case["hidden"], case["inner"], case["top_k"], case["m"]
    k = min(k, e)
    x = _exact_quant(s["x"], "mxfp4", True)
    logits = s["x"].double() @ s["router"].double().t()
    w13, w2 = _exact_stored(s["w13"]).view(e, 2, f, h), _exact_stored(s["w2"]).view(e, h, f)
    y = torch.zeros(m, h, dtype=torch.float64, device="cuda")
    p_all = torch.empty(m, k, dtype=torch.float64, device="cuda")
    for t in range(m):
        # the largest k logits, the lowest index first among equal ones
        order = sorted(range(e), key=lambda i, row=logits[t].tolist(): (-row[i], i))[:k]
        p_all[t] = torch.softmax(logits[t, order], dim=0)
        for j, i in enumerate(order):
            gate, up = w13[i, 0] @ x[t], w13[i, 1] @ x[t]
            y[t] += p_all[t, j] * (w2[i] @ _exact_quant((gate * torch.sigmoid(gate) * up)[None], "mxfp4", True)[0])
    return y, None, p_all
