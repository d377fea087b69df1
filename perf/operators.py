"""Cases that measure the serving operators of the dMoE layer: the layer for a few tokens (bf16
and microscaled 4-bit expert weights), the microscaled 4-bit format's two conversions, and the
whole layer in that format over many tokens.

``run`` computes a case in plain PyTorch (``own`` false) or with the library's calls (``own``
true), on the inputs that ``prepare`` makes; ``exact`` gives the same outputs in 64 bits.

The microscaled format (blocks of 32 along a row, 4-bit elements, one power-of-two scale a
block): two elements a byte, the even column in the low four bits; element = sign, two exponent
bits, one mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6); scale byte s = 2^(s - 127), 255 = NaN.  The
scales of a matrix lie in tiles of 128 rows x 128 columns, [row tile, column tile, 32, 4, 4]:
byte [l][q][b] of a tile belongs to its row 32 q + l and its block b.
"""
import math

import torch

own = False

# ---- the cases ---------------------------------------------------------------------------------


def listed():
    return [
        # one token of a decode step, small experts: 19 MB of weights, latency decides
        dict(name="few, 1 token, high granularity", op="few", T=1, h=1536, f=256, E=128, k=8, zipf=False),
        # one token of a decode step, large experts: a pure stream of 0.7 GB of weights
        dict(name="few, 1 token, Mixtral-shaped", op="few", T=1, h=4096, f=14336, E=8, k=2, zipf=False),
        # a small decode batch of an odd size: most experts hold one to four tokens
        dict(name="few, 17 tokens, fine-grained", op="few", T=17, h=2048, f=1024, E=64, k=8, zipf=False),
        # a large decode batch on a skewed router: a few experts hold most of the tokens
        dict(name="few, 96 tokens, skewed", op="few", T=96, h=2048, f=512, E=256, k=8, zipf=True),
        # the 4-bit format of an activation matrix with an odd number of rows, there and back
        dict(name="mx4 there and back, 333 rows", op="quantize", rows=333, cols=1536, scale=1.0),
        # ... and of one projection of 64 experts, as a checkpoint is converted
        dict(name="mx4 there and back, 64 experts", op="quantize", rows=65536, cols=2048, scale=0.02),
        # one token over 4-bit expert weights
        dict(name="mx4 few, 1 token, Mixtral-shaped", op="mx4_few", T=1, h=4096, f=14336, E=8, k=2, zipf=False),
        # a decode batch over 4-bit expert weights
        dict(name="mx4 few, 32 tokens, fine-grained", op="mx4_few", T=32, h=2048, f=1024, E=64, k=8, zipf=False),
        # a short prompt through the 4-bit layer: every expert's block is mostly padding
        dict(name="mx4 layer, 300 tokens", op="mx4_layer", T=300, h=2048, f=512, E=32, k=4, zipf=False),
        # prompts through the 4-bit layer: the fine-grained and the high-granularity workloads
        dict(name="mx4 layer, fine-grained", op="mx4_layer", T=4096, h=2048, f=1024, E=64, k=8, zipf=False),
        dict(name="mx4 layer, high granularity", op="mx4_layer", T=16384, h=1536, f=256, E=128, k=8, zipf=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "quantize", "mx4_few", "mx4_few", "mx4_layer"])
    if op == "quantize":
        cols = 128 * _log(rng, 1, 112)
        return dict(op=op, rows=max(1, min(_log(rng, 1, 65536), 65536 * 2048 // cols)), cols=cols,
                    scale=rng.choice([1.0, 0.02]))
    h = 128 * rng.randint(2, 32)
    E = rng.choice([1, 3, 8, 16, 30, 60, 64, 128, 256])
    k = min(E, rng.randint(1, 8))
    f = 128 * _log(rng, 1, 112)
    if op == "mx4_layer":
        T = _log(rng, 130, 16384)
        f = min(f, 1024)
        E = min(E, 128)
        k = min(E, k)
        # no more work than the largest listed case, and no more blocks of weights to lay out
        while T > 130 and (T * k * h * f > 16384 * 8 * 1536 * 256 or (T * k / 128 + E) * h * f > 1150 * 1536 * 1024):
            T = max(130, T // 2 + rng.randint(0, 3))
        while (T * k / 128 + E) * h * f > 1150 * 1536 * 1024 and f > 128:
            f = 128 * max(1, f // 256)
    else:
        T = _log(rng, 1, 128)
        while E * h * f > 8 * 4096 * 14336 // 2 and f > 128:
            f = 128 * max(1, f // 256)
    return dict(op=op, T=T, h=h, f=f, E=E, k=k, zipf=rng.random() < 0.3)


# ---- inputs ------------------------------------------------------------------------------------


def _normal(gen, shape, scale):
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    t.normal_(0.0, scale, generator=gen)
    return t


def _logits(case, gen, device):
    lg = torch.randn((case["T"], case["E"]), generator=gen, device=device)
    if case["zipf"]:
        lg = lg - 1.5 * torch.log(torch.arange(1, case["E"] + 1, device=device).float())[None, :]
    return lg.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * int(seed) + 17)
    s = dict(case=case)
    if case["op"] == "quantize":
        s["src"] = _normal(gen, (case["rows"], case["cols"]), case["scale"])
        s["back"] = torch.empty_like(s["src"])
        return s
    T, h, f, E, k = (case[n] for n in ("T", "h", "f", "E", "k"))
    s["x"] = _normal(gen, (T, h), 1.0)
    s["logits"] = _logits(case, gen, "cuda")
    s["y"] = torch.empty_like(s["x"])
    for name, rows, cols in (("w1", f, h), ("w3", f, h), ("w2", h, f)):
        w = _normal(gen, (E, rows, cols), 0.02)
        # a checkpoint in the 4-bit format: its codes and scales
        s[name] = w if case["op"] == "few" else _plain_quantize(w)
    return s


# ---- the plain forms ---------------------------------------------------------------------------

_LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _plain_blocks(x):
    """Codes [..., cols] (0..15) and scale bytes [..., cols / 32] of x [..., cols], in int32."""
    v = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = v.abs().amax(-1)
    exp = top.view(torch.int32) >> 23  # biased exponent of the largest magnitude
    s = torch.where(exp == 255, 255, (exp - 2).clamp(0, 254))
    a = v.abs() * ((254 - s.clamp(max=253)) << 23).view(torch.float32)[..., None]
    code = ((a > 0.25).to(torch.int32) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) +
            (a > 5.0) + 8 * (v < 0))
    code = torch.where(s[..., None] == 255, 0, code)
    return code.reshape(x.shape), s


def _plain_quantize(x):
    """(codes [..., rows, cols / 2], scales [..., row tiles, column tiles, 32, 4, 4]) in uint8."""
    code, s = _plain_blocks(x)
    packed = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)
    rows, cols = x.shape[-2:]
    pad = -rows % 128
    s = torch.nn.functional.pad(s, (0, 0, 0, pad)).to(torch.uint8)
    s = s.reshape(*x.shape[:-2], (rows + pad) // 128, 4, 32, cols // 128, 4)
    d = s.dim()
    s = s.permute(*range(d - 5), d - 5, d - 2, d - 3, d - 4, d - 1).contiguous()
    return packed, s


def _scale_value(s):
    """2^(s - 127) in 32 bits (0: the subnormal 2^-127; 255: NaN)."""
    s = s.to(torch.int32)
    bits = torch.where(s == 0, 0x00400000, s << 23)
    return torch.where(s == 255, 0x7FC00000, bits).view(torch.float32)


def _plain_dequantize(packed, scales):
    rows, cols = packed.shape[-2], 2 * packed.shape[-1]
    lut = torch.tensor(_LUT, device=packed.device)
    v = torch.stack((lut[(packed & 15).long()], lut[(packed >> 4).long()]), -1)
    v = v.reshape(*packed.shape[:-1], cols // 32, 32)
    d = scales.dim()
    s = scales.permute(*range(d - 5), d - 5, d - 2, d - 3, d - 4, d - 1)
    s = s.reshape(*packed.shape[:-2], -1, cols // 32)[..., :rows, :]
    return (v * _scale_value(s)[..., None]).reshape(*packed.shape[:-1], cols)


def _plain_values(x):
    """x after the 4-bit format, in 32 bits."""
    code, s = _plain_blocks(x)
    lut = torch.tensor(_LUT, device=x.device)
    v = lut[code.long()].reshape(*s.shape, 32) * _scale_value(s)[..., None]
    return v.reshape(x.shape)


def _plain_route(logits, k):
    lg = logits.float()
    top = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :k]  # ties: lower index
    e = torch.exp(lg - lg.amax(1, keepdim=True))
    return top, torch.gather(e / e.sum(1, keepdim=True), 1, top)


def _weight(w, rows=None):
    """Expert weights in 32 bits: those of the experts `rows`, or all."""
    if isinstance(w, tuple):
        return _plain_dequantize(*(w if rows is None else (w[0][rows], w[1][rows])))
    return (w if rows is None else w[rows]).float()


def _silu(a):
    return a / (1.0 + torch.exp(-a))


def _plain_few(s):
    case = s["case"]
    T, E, k = case["T"], case["E"], case["k"]
    top, wts = _plain_route(s["logits"], k)
    x = s["x"].float()
    if T * k <= E:  # the chosen experts' weights, entry by entry
        rows = top.reshape(-1)
        xr = x.repeat_interleave(k, 0)[:, :, None]
        mid = _silu(torch.bmm(_weight(s["w1"], rows), xr)) * torch.bmm(_weight(s["w3"], rows), xr)
        out = torch.bmm(_weight(s["w2"], rows), mid)[:, :, 0].reshape(T, k, -1)
        y = (out * wts[:, :, None]).sum(1)
    else:  # every expert over every token, the routing weight 0 where it was not chosen
        dense = torch.zeros((T, E), device=x.device).scatter(1, top, wts)
        xe = x[None].expand(E, -1, -1)
        mid = _silu(torch.bmm(xe, _weight(s["w1"]).transpose(1, 2))) * torch.bmm(xe, _weight(s["w3"]).transpose(1, 2))
        y = torch.bmm(mid * dense.t()[:, :, None], _weight(s["w2"]).transpose(1, 2)).sum(0)
    return dict(y=y.to(torch.bfloat16), top_experts=top.to(torch.int32), weights=wts)


def _plain_layer(s):
    case = s["case"]
    T, h, E, k = case["T"], case["h"], case["E"], case["k"]
    top, wts = _plain_route(s["logits"], k)
    flat = top.reshape(-1)
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    ends = torch.cumsum((counts + 127) // 128 * 128, 0)
    order = torch.argsort(flat, stable=True)
    e = flat[order]
    first = torch.cumsum(counts, 0) - counts
    row = (ends - (counts + 127) // 128 * 128)[e] + torch.arange(T * k, device=flat.device) - first[e]
    blocks = (T * k + 127 * E) // 128
    xp = torch.zeros((blocks * 128, h), device=flat.device)
    xp[row] = _plain_values(s["x"])[order // k]
    xp = xp.reshape(blocks, 128, h)
    be = torch.searchsorted(ends, torch.arange(blocks, device=flat.device) * 128, right=True).clamp(max=E - 1)
    mid = _silu(torch.bmm(xp, _weight(s["w1"], be).transpose(1, 2))) * torch.bmm(xp, _weight(s["w3"], be).transpose(1, 2))
    out = torch.bmm(_plain_values(mid), _weight(s["w2"], be).transpose(1, 2)).reshape(blocks * 128, h)
    at = torch.empty_like(row).scatter(0, order, row)
    return (out[at].reshape(T, k, h) * wts[:, :, None]).sum(1).to(torch.bfloat16)


# ---- the library's calls -----------------------------------------------------------------------


def _own_few(s):
    from dropless_mixture_experts_dmoe_b200 import binding as B

    few = s.get("few")
    if few is None:  # what a serving loop keeps: the shape, the call's buffers, the weights' handles
        c = s["case"]
        few = s["few"] = B.FewBuffers(B.make_dims(c["T"], c["h"], c["f"], c["E"], c["k"]))
        s["handles"] = [B.Mx4(*s[n]) if c["op"] == "mx4_few" else s[n] for n in ("w1", "w3", "w2")]
    call = B.dmoe_mx4_forward_few if s["case"]["op"] == "mx4_few" else B.dmoe_forward_few
    call(few.dims, s["x"], s["logits"], *s["handles"], few, s["y"])
    return dict(y=s["y"], top_experts=few.top_experts, weights=few.weights)


def _own_quantize(s):
    from dropless_mixture_experts_dmoe_b200 import binding as B

    q = s.get("mx4")
    if q is None:
        q = s["mx4"] = B.Mx4.empty(*s["src"].shape)
    B.dmoe_mx4_quantize(s["src"], q)
    B.dmoe_mx4_dequantize(q, s["back"])
    return s["back"]


def _own_layer(s):
    from dropless_mixture_experts_dmoe_b200 import binding as B

    b = s.get("bufs")
    if b is None:
        c = s["case"]
        b = s["bufs"] = B.Mx4Buffers(B.make_dims(c["T"], c["h"], c["f"], c["E"], c["k"]))
        s["handles"] = [B.Mx4(*s[n]) for n in ("w1", "w3", "w2")]
    B.dmoe_sparse_map(b.dims, s["logits"], b.map, b.ws_map)
    B.dmoe_mx4_forward(b.dims, s["x"], *s["handles"], b.map, s["y"], b.ws)
    return s["y"]


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_quantize(state) if op == "quantize" else _own_layer(state) if op == "mx4_layer" else _own_few(state)
    if op == "quantize":
        return _plain_dequantize(*_plain_quantize(state["src"])).to(torch.bfloat16)
    return _plain_layer(state) if op == "mx4_layer" else _plain_few(state)


# ---- work and exact values ---------------------------------------------------------------------


def _experts_used(case):
    """Experts that a typical routing of this case uses (a routing of its own, on the CPU)."""
    gen = torch.Generator()
    gen.manual_seed(1)
    lg = _logits(case, gen, "cpu").float()
    return int(torch.unique(torch.topk(lg, case["k"], dim=1).indices).numel())


def work(case):
    if case["op"] == "quantize":  # bf16 in, codes and scales out and in again, bf16 out
        n = case["rows"] * case["cols"]
        return dict(bytes=n * (2 + 17 / 32 + 17 / 32 + 2), flops=0)
    T, h, f, E, k = (case[n] for n in ("T", "h", "f", "E", "k"))
    per = 2.0 if case["op"] == "few" else 17 / 32
    return dict(bytes=_experts_used(case) * 3 * h * f * per + 4 * T * h + 2 * T * E, flops=6 * T * k * h * f)


def _exact_value_of(codes, scales):
    """A matrix in the format, in 64 bits: row r, block c at tile byte [r % 32][r // 32 % 4][c % 4]."""
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=codes.device) / 2
    out = torch.empty((rows, cols), dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes.int() >> (4 * half)) & 15
        out[:, half::2] = torch.where(c >= 8, -1.0, 1.0) * mag[(c & 7).long()]
    r = torch.arange(rows, device=codes.device)[:, None]
    b = torch.arange(cols // 32, device=codes.device)[None, :]
    s = scales[r // 128, b // 4, r % 32, r // 32 % 4, b % 4].double()
    return out * torch.pow(2.0, s - 127).repeat_interleave(32, 1)


def _exact_round(x):
    """x in 64 bits after the format: each block of 32 on the grid of its own power of two."""
    v = x.reshape(-1, 32)
    top = v.abs().amax(1, keepdim=True)
    e = torch.frexp(top)[1].double() - 1 - 2  # floor(log2) less the exponent of the largest element
    e = torch.where(top == 0, -127.0, e.clamp(-127, 127))
    a = v.abs() * torch.pow(2.0, -e)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    q = (torch.round(a / step) * step).clamp(max=6.0)  # ties to the even multiple
    return (torch.sign(v) * q * torch.pow(2.0, e)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_round(s["src"].double())
    T, E, k = case["T"], case["E"], case["k"]
    lg = s["logits"].double()
    top = torch.argsort(lg, dim=1, descending=True, stable=True)[:, :k]
    p = torch.exp(lg - torch.logsumexp(lg, 1, keepdim=True))
    wts = torch.gather(p, 1, top)
    layer = case["op"] == "mx4_layer"
    x = s["x"].double()
    if layer:
        x = _exact_round(x)
    y = torch.zeros_like(x)
    for e in range(E):
        tok, slot = torch.nonzero(top == e, as_tuple=True)
        if not tok.numel():
            continue
        w1, w3, w2 = ((s[n][e].double() if case["op"] == "few" else _exact_value_of(s[n][0][e], s[n][1][e]))
                      for n in ("w1", "w3", "w2"))
        a = x[tok] @ w1.t()
        mid = a * torch.sigmoid(a) * (x[tok] @ w3.t())
        if layer:
            mid = _exact_round(mid)
        y.index_add_(0, tok, wts[tok, slot][:, None] * (mid @ w2.t()))
    return y if layer else dict(y=y, top_experts=None, weights=wts)
