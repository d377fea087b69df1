"""The microscaled 4-bit format and the layer that runs in it, against definitions in 64 bits."""
import time

import numpy as np
import pytest
import torch

from dropless_mixture_experts_dmoe_b200 import binding as B

import serving_ref as R

pytestmark = pytest.mark.gpu


def quantize(x):
    q = B.Mx4.empty(*x.shape)
    q.codes.fill_(0xAA)
    q.scales.fill_(0xAA)
    B.dmoe_mx4_quantize(x, q)
    return q


def check_exact(x, q):
    """Elements and scales as the definition has them, and the padding rows' scales 0."""
    xs = x.reshape(-1, x.shape[-1]).double().cpu().numpy()
    el, e = R.mx4_blocks(xs)
    v, s = R.mx4_decode(q.codes.reshape(-1, q.codes.shape[-1]),
                        q.scales.reshape(-1, *q.scales.shape[-4:]))
    np.testing.assert_array_equal(s, e)
    np.testing.assert_array_equal(v.reshape(el.shape), el)
    rows = xs.shape[0]
    if rows % 128:
        r = np.arange(rows, (rows + 127) // 128 * 128)
        last = q.scales.reshape(-1, *q.scales.shape[-4:])[-1].cpu().numpy()
        assert (last[:, r % 32, r % 128 // 32] == 0).all()


@pytest.mark.parametrize("rows,cols", [(1, 128), (1, 384), (127, 256), (128, 128), (129, 1536),
                                       (333, 1152), (1000, 640), (4096, 2048), (3, 14336)])
def test_quantize_and_back_exact(rows, cols):
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x = (x * torch.exp(4 * torch.randn((rows, 1), generator=g, device="cuda"))).bfloat16()
    x.view(-1)[:: 37] = 0
    q = quantize(x)
    check_exact(x, q)
    back = torch.full((rows + 1, cols), 5.0, dtype=torch.bfloat16, device="cuda")
    B.dmoe_mx4_dequantize(q, back[:-1])
    ref = R.mx4_decode_values(q.codes, q.scales)
    assert torch.equal(back[:-1].double(), ref)  # one mantissa bit: exact in bf16
    assert (back[-1] == 5.0).all()


def test_quantize_every_bf16_value():
    """All 65536 bit patterns, each next to a block maximum that puts it anywhere on the grid:
    subnormals, ties, both zeros, infinities and NaN included."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    val = bits.view(torch.bfloat16).reshape(1, -1)
    rows = []
    for lead in (0.0, 1.0, 1.75, 6.0, 2.0 ** -126, 2.0 ** -133, 3e38):
        blk = val.reshape(-1, 1).expand(-1, 32).clone()
        blk[:, 1:] = lead
        blk[:, 5] = -lead
        rows.append(blk.reshape(-1, 128))
    # ties and their neighbours under a fixed maximum of 6
    t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    t = torch.cat([t, t * (1 + 2 ** -7), t * (1 - 2 ** -8)])
    blk = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    blk[:2, :21] = t.bfloat16()
    blk[2:, :21] = -t.bfloat16()
    blk[:, 31] = torch.tensor([6.0, 4.0, 7.5, -6.0])
    rows.append(blk.reshape(1, 128))
    x = torch.cat(rows).bfloat16().contiguous()
    q = quantize(x)
    check_exact(x, q)


def test_dequantize_every_scale_and_element():
    """16 elements x 256 scale bytes: exact in bf16, NaN for 255, inf past bf16's largest."""
    s = torch.arange(256, dtype=torch.uint8, device="cuda")
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").reshape(1, -1).repeat(256, 1)
    scales = torch.zeros(B.Mx4.scales_shape(256, 512), dtype=torch.uint8, device="cuda")
    r = torch.arange(256, device="cuda")
    for b in range(16):
        scales[r // 128, b // 4, r % 32, r % 128 // 32, b % 4] = s
    q = B.Mx4(codes.contiguous(), scales)
    out = torch.empty((256, 512), dtype=torch.bfloat16, device="cuda")
    B.dmoe_mx4_dequantize(q, out)
    ref = R.mx4_decode_values(q.codes, q.scales).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    assert torch.isnan(out[255]).all()
    assert torch.equal(out[:255], ref[:255])


def test_quantize_a_large_matrix():
    """Offsets past 32 bits: 2.4e9 elements; the last rows against the definition."""
    rows, cols = 150_000, 16384
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[: rows - 300].fill_(1.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    x[rows - 300:] = torch.randn((300, cols), generator=g, device="cuda").bfloat16()
    q = B.Mx4.empty(rows, cols)
    B.dmoe_mx4_quantize(x, q)
    back = torch.empty_like(x)
    B.dmoe_mx4_dequantize(q, back)
    assert (back[: rows - 300].view(-1)[:: 1001] == 1.0).all()
    ref = R.mx4_values(x[rows - 300:].double().cpu().numpy())
    assert torch.equal(back[rows - 300:].double().cpu(), torch.from_numpy(ref))


# (T, h, f, E, k, flags)
SHAPES = [
    (1, 128, 128, 1, 1, 0),
    (5, 256, 128, 8, 2, 0),
    (129, 384, 640, 3, 2, 0),
    (300, 2048, 512, 32, 4, 0),
    (1000, 1536, 256, 128, 8, 0),
    (513, 640, 1152, 5, 3, 0),
    (2000, 256, 384, 16, 4, 0x1),
    (2000, 256, 384, 16, 4, 0x2),      # token rounding: a token-major entry list
    (1024, 512, 256, 256, 8, 0x4 | 0x8),
]


def setup(shape, seed=0):
    T, h, f, E, k, flags = shape
    g = torch.Generator(device="cuda").manual_seed(seed + T)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    dims = B.make_dims(T, h, f, E, k, flags=flags)
    x = n(T, h).bfloat16()
    lg = n(T, E)
    lg = (lg - 0.5 * torch.arange(E, device="cuda") / max(E, 8)).bfloat16()
    w = [quantize((0.05 * n(E, *s)).bfloat16()) for s in ((f, h), (f, h), (h, f))]
    bufs = B.Mx4Buffers(dims)
    bufs.ws.fill_(255)
    return dims, x, lg, w, bufs


def entries(dims, m):
    """(entry's token, padded row, expert, weight) of the listed entries."""
    dest = m.dest_row.long()
    if m.entry_offsets is None:
        tok = torch.arange(dims.T * dims.top_k, device="cuda") // dims.top_k
    else:
        tok = torch.searchsorted(m.entry_offsets.long(), torch.arange(dest.numel(), device="cuda"),
                                 right=True) - 1
    on = dest >= 0
    return tok[on], dest[on], m.top_experts.reshape(-1).long()[on], m.weights.reshape(-1)[on].double()


@pytest.mark.parametrize("shape", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
def test_mx4_forward_parity(shape):
    """H's blocks against the definition on the exact H (an element or scale may differ where H
    lies within the products' error of a border), then y against the kernel's own H."""
    dims, x, lg, w, bufs = setup(shape)
    T, h, f, E, k, flags = shape
    yg = torch.full((T + 1, h), 7.0, dtype=torch.bfloat16, device="cuda")
    yg[:-1] = float("nan")
    B.dmoe_sparse_map(dims, lg, bufs.map, bufs.ws_map)
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, yg[:-1], bufs.ws)
    torch.cuda.synchronize()
    assert int(bufs.map.status.item()) == 0
    tok, row, ex, wt = entries(dims, bufs.map)
    xq = torch.from_numpy(R.mx4_values(x.double().cpu().numpy())).cuda()
    w1, w3, w2 = (R.mx4_decode_values(q.codes, q.scales) for q in w)
    hid = bufs.hidden()
    rows = int(bufs.map.num_blocks.item()) * 128
    tiles = rows // 128
    hv, he = R.mx4_decode(hid.codes[:rows], hid.scales[:tiles])
    hq = torch.from_numpy(hv * np.repeat(np.exp2(he), 32, 1)).cuda()
    # padding rows hold zeros
    pad = torch.ones(rows, dtype=torch.bool, device="cuda")
    pad[row] = False
    assert (hq[pad] == 0).all()
    y = torch.zeros((T, h), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)

    def g(K):  # fp32 accumulation of K products, each step off by 2^-23 of the absolute sum
        return (K / 16 + 32) * 2.0 ** -23

    for e in range(E):
        at = torch.nonzero(ex == e)[:, 0]
        if not at.numel():
            continue
        xe = xq[tok[at]]
        a, b = xe @ w1[e].t(), xe @ w3[e].t()
        da, db = (g(h) * (xe.abs() @ m.abs().t()) for m in (w1[e], w3[e]))
        s = a * torch.sigmoid(a)
        H = s * b
        dH = 1.1 * da * b.abs() + (s.abs() + 1.1 * da) * db + 2.0 ** -18 * H.abs()
        got = hq[row[at]]
        # the format is monotone in x and in the block's scale: the value must lie between the
        # conversions of H - dH and H + dH, each under the smallest and the largest scale that
        # the block's maximum can have
        m = H.abs().reshape(len(at), -1, 32)
        dm = dH.reshape(len(at), -1, 32)
        lo_e, hi_e = (torch.floor(torch.log2(v.amax(-1).clamp(min=2.0 ** -125))) - 2
                      for v in ((m - dm).clamp(min=0), m + dm))
        ok = torch.zeros_like(got, dtype=torch.bool)
        for ee in (lo_e, hi_e):
            sc = torch.exp2(ee)[..., None]
            lo, hi = (grid((v.reshape(len(at), -1, 32) / sc)) * sc for v in (H - dH, H + dH))
            gq = got.reshape(len(at), -1, 32)
            ok |= ((gq >= lo) & (gq <= hi)).reshape(ok.shape)
        assert bool(ok.all()), f"expert {e}: {int((~ok).sum())} elements of H off"
        r = got @ w2[e].t()
        t = (g(f) + 2.0 ** -11 + 2.0 ** -18) * (got.abs() @ w2[e].abs().t())
        y.index_add_(0, tok[at], wt[at][:, None] * r)
        tol.index_add_(0, tok[at], wt[at][:, None] * t)
    R.check(yg[:-1], y, tol, "y")
    assert (yg[-1] == 7.0).all()
    # again in poisoned buffers: bit for bit
    bufs.ws.fill_(0x5A)
    y2 = torch.empty_like(x)
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, y2, bufs.ws)
    assert torch.equal(y2.view(torch.int16), yg[:-1].view(torch.int16))


def grid(v):
    """Nearest e2m1 value, ties to even, saturated (float64 tensor)."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=6.0)


def test_mx4_forward_empty_experts_and_nonfinite_rows():
    """All tokens at one expert of eight; an inf or NaN in a token's x makes that token's y NaN
    and leaves the others as they are without it; weights of unused experts are not used."""
    T, h, f, E, k = 200, 256, 256, 8, 1
    dims, x, lg, w, bufs = setup((T, h, f, E, k, 0))
    lg[:, 5] = 50.0
    for q in w:
        q.scales[:5] = 255
        q.scales[6:] = 255
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    B.dmoe_sparse_map(dims, lg, bufs.map, bufs.ws_map)
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, y0, bufs.ws)
    x[17, 3] = float("nan")
    x[150, 255] = float("-inf")
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, y1, bufs.ws)
    torch.cuda.synchronize()
    assert torch.isfinite(y0.float()).all()
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[17, 150]] = True
    assert torch.isnan(y1[bad].float()).all()
    assert torch.equal(y0[~bad].view(torch.int16), y1[~bad].view(torch.int16))
    assert int(bufs.map.status.item()) == 0


def test_mx4_prompt_then_decode():
    """A checkpoint converted once, a prompt through the 4-bit layer, decode steps through the
    few-token layer over the same weights, on a side stream and replayed from a graph."""
    T, h, f, E, k = 384, 512, 256, 16, 4
    dims, x, lg, w, bufs = setup((T, h, f, E, k, 0), seed=3)
    d2 = B.make_dims(6, h, f, E, k)
    few = B.FewBuffers(d2)
    y, y2 = torch.empty_like(x), torch.empty((6, h), dtype=torch.bfloat16, device="cuda")
    xs, ls = x[:6].clone(), lg[:6].clone()

    def step():
        B.dmoe_sparse_map(dims, lg, bufs.map, bufs.ws_map)
        B.dmoe_mx4_forward(dims, x, *w, bufs.map, y, bufs.ws)
        B.dmoe_mx4_forward_few(d2, xs, ls, *w, few, y2)

    step()
    torch.cuda.synchronize()
    ref = [y.clone(), y2.clone()]
    w1, w3, w2 = (R.mx4_decode_values(q.codes, q.scales) for q in w)
    top, wts = R.route(ls, k)
    yr, tol = R.layer(xs.double(), w1, w3, w2, top, wts, h_rel=2.0 ** -11)
    R.check(y2, yr, tol, "decode")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), ref[0].view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    y.fill_(0)
    y2.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), ref[0].view(torch.int16))
    assert torch.equal(y2.view(torch.int16), ref[1].view(torch.int16))


def test_mx4_forward_given_experts_all_absent():
    """Given experts, every id out of range: no block at all, y is zero, the map says so."""
    dims, x, lg, w, bufs = setup((70, 256, 128, 4, 2, 0))
    bufs.map.top_experts.fill_(-1)
    bufs.map.weights.fill_(1.0)
    y = torch.full_like(x, float("nan"))
    B.dmoe_sparse_map(dims, None, bufs.map, bufs.ws_map)
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, y, bufs.ws)
    torch.cuda.synchronize()
    assert int(bufs.map.num_blocks.item()) == 0
    assert int(bufs.map.status.item()) == B.STATUS_EXPERT_OUT_OF_RANGE
    assert (y == 0).all()


def test_mx4_forward_stall_reports_timeout_and_context_survives():
    """A first stage that is withheld on purpose: the waits run out, the status says so, and the
    next call is right again."""
    dims, x, lg, w, bufs = setup((600, 256, 384, 8, 2, 0))
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    B.dmoe_sparse_map(dims, lg, bufs.map, bufs.ws_map)
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, y, bufs.ws)
    torch.cuda.synchronize()
    assert int(bufs.map.status.item()) == 0
    B.dmoe_debug_inject_stall(True)
    t0 = time.time()
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, y2, bufs.ws)
    torch.cuda.synchronize()
    assert int(bufs.map.status.item()) & B.STATUS_TIMEOUT
    assert time.time() - t0 < 10.0
    B.dmoe_sparse_map(dims, lg, bufs.map, bufs.ws_map)
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, y2, bufs.ws)
    torch.cuda.synchronize()
    assert int(bufs.map.status.item()) == 0
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))


@pytest.mark.parametrize("shape", [(5000, 256, 512, 16, 4, 0), (3001, 384, 1152, 40, 6, 0),
                                   (4100, 128, 128, 100, 3, 0)],
                         ids=lambda s: "-".join(map(str, s)))
def test_mx4_forward_rows_do_not_depend_on_the_batch(shape):
    """Many units per pair of SMs, in whole rounds and shares: every token's row is bit for bit what
    calls over parts of the batch give; the same with two calls in flight on two streams."""
    dims, x, lg, w, bufs = setup(shape)
    T, h, f, E, k, flags = shape
    y = torch.full_like(x, float("nan"))
    B.dmoe_sparse_map(dims, lg, bufs.map, bufs.ws_map)
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, y, bufs.ws)
    step = 700
    parts = torch.full_like(x, float("nan"))
    for a in range(0, T, step):
        n = min(step, T - a)
        d = B.make_dims(n, h, f, E, k, flags=flags)
        b = B.Mx4Buffers(d)
        B.dmoe_sparse_map(d, lg[a:a + n], b.map, b.ws_map)
        B.dmoe_mx4_forward(d, x[a:a + n], *w, b.map, parts[a:a + n], b.ws)
    torch.cuda.synchronize()
    assert int(bufs.map.status.item()) == 0
    assert torch.isfinite(y.float()).all()
    assert torch.equal(y.view(torch.int16), parts.view(torch.int16))
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [(B.Mx4Buffers(dims), torch.full_like(x, float("nan"))) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (b, out) in zip(streams, both):
            B.dmoe_sparse_map(dims, lg, b.map, b.ws_map, stream=s)
            B.dmoe_mx4_forward(dims, x, *w, b.map, out, b.ws, stream=s)
    torch.cuda.synchronize()
    for b, out in both:
        assert int(b.map.status.item()) == 0
        assert torch.equal(y.view(torch.int16), out.view(torch.int16))
