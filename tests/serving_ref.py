"""Plain 64-bit references of the serving operators, with bounds on what the kernels may be off
by.  Nothing here calls the library."""
from __future__ import annotations

import numpy as np
import torch

# Nearest-value rounding is off by at most half a step: bf16 2^-8 of the value.
HALF_BF16 = 2.0 ** -8

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def mx4_blocks(x: np.ndarray):
    """(elements in float64 on the e2m1 grid, scale exponents s) of x [rows, cols] float64, from
    the definition: s = floor(log2 max|x|) - 2 within [-127, 127] (-127 for zeros; NaN marks a
    block with an inf or NaN, whose elements are zero)."""
    v = x.reshape(x.shape[0], -1, 32)
    m = np.abs(v).max(-1)
    bad = ~np.isfinite(m)
    m = np.where(bad, 1.0, m)
    e = np.where(m > 0, np.frexp(m)[1] - 1 - 2, -127)
    e = np.clip(e, -127, 127).astype(np.float64)
    a = np.abs(np.where(bad[..., None], 0.0, v)) / np.exp2(e)[..., None]
    # nearest grid value, ties to the even mantissa bit (grid indices alternate odd / even)
    i = np.clip(np.searchsorted(E2M1, a, side="right") - 1, 0, 6)
    lo, hi = E2M1[i], E2M1[i + 1]
    mid = (lo + hi) / 2
    up = (a > mid) | ((a == mid) & (i % 2 == 1))
    q = np.where(up, hi, lo)
    return np.where(np.signbit(v), -q, q), np.where(bad, np.nan, e)


def mx4_values(x: np.ndarray) -> np.ndarray:
    q, e = mx4_blocks(x)
    return (q * np.exp2(e)[..., None]).reshape(x.shape)


def mx4_decode(codes: torch.Tensor, scales: torch.Tensor):
    """(elements [rows, cols] float64, scale exponents [rows, cols/32], NaN for 255) of a matrix
    in the format, looked up byte by byte."""
    c = codes.cpu().numpy().astype(np.int64)
    s = scales.cpu().numpy()
    rows, cols = c.shape[0], 2 * c.shape[1]
    el = np.empty((rows, cols), np.int64)
    el[:, 0::2] = c & 15
    el[:, 1::2] = c >> 4
    v = np.where(el >= 8, -1.0, 1.0) * E2M1[el & 7]
    r = np.arange(rows)[:, None]
    b = np.arange(cols // 32)[None, :]
    e = s[r // 128, b // 4, r % 32, r % 128 // 32, b % 4].astype(np.float64)
    return v, np.where(e == 255, np.nan, e - 127)


def mx4_decode_values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """float64 values of a matrix or stack, on the codes' device."""
    lead = codes.shape[:-2]
    c2 = codes.reshape(-1, codes.shape[-1])
    s2 = scales.reshape(-1, *scales.shape[len(lead) + 1:])
    v, e = mx4_decode(c2, s2)
    out = v * np.repeat(np.exp2(e), 32, axis=1)
    return torch.from_numpy(out).reshape(*lead, codes.shape[-2], -1).to(codes.device)


def route(logits: torch.Tensor, k: int, renorm: bool = False):
    """Top-k (ties to the lower expert) and weights in 64 bits; finite logits."""
    lg = logits.double()
    top = torch.argsort(lg, dim=1, descending=True, stable=True)[:, :k]
    if renorm:
        return top, torch.softmax(torch.gather(lg, 1, top), 1)
    return top, torch.gather(torch.softmax(lg, 1), 1, top)


def layer(x, w1, w3, w2, top, wts, h_rel=2.0 ** -16):
    """y in 64 bits and an elementwise bound on a kernel's error before its final rounding.

    x [T,h], w1/w3 [E,f,h], w2 [E,h,f] float64; top [T,k] (ids outside [0, E) add nothing),
    wts [T,k].  The bound: an fp32 sum of K products, taken in chains of K/16 steps and joined
    over at most 32 partial sums, each step off by at most 2^-23 of the terms' absolute sum
    (a truncating accumulator), so g(K) = (K/16 + 32) 2^-23 of that sum; silu has a slope below
    1.1 and is evaluated to 2^-18; H is rounded to h_rel of its value (2^-16: a pair of bf16; the
    4-bit weights meet it in fp16, 2^-11) and, in fp16, to 2^-38 of its row's largest value, as
    x is (subnormals under a row scale that puts the largest at 2^14: half of 2^-24 over 2^14,
    rounded up); the routing weights are off by 2^-18 of their value; the k rows add k 2^-24."""
    T, k = top.shape
    E, f, h = w1.shape
    y = torch.zeros((T, h), dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(y)

    def g(K):
        return (K / 16 + 32) * 2.0 ** -23

    for e in range(E):
        tok, slot = torch.nonzero(top == e, as_tuple=True)
        if not tok.numel():
            continue
        xe = x[tok]
        a, b = xe @ w1[e].t(), xe @ w3[e].t()
        tiny = 2.0 ** -38 * xe.abs().amax(1, keepdim=True) if h_rel > 2.0 ** -16 else 0.0
        da, db = (g(h) * (xe.abs() @ w.abs().t()) + tiny * w.abs().sum(1) for w in (w1[e], w3[e]))
        s = a * torch.sigmoid(a)
        H = s * b
        dH = 1.1 * da * b.abs() + (s.abs() + 1.1 * da) * db + (h_rel + 2.0 ** -18) * H.abs()
        if h_rel > 2.0 ** -16:
            dH = dH + 2.0 ** -38 * H.abs().amax(1, keepdim=True)
        w = wts[tok, slot].double()[:, None]
        a2 = w2[e].abs().t()
        yr = H @ w2[e].t()
        t = dH @ a2 + (g(f) + 2.0 ** -18 + k * 2.0 ** -24) * (H.abs() @ a2)
        y.index_put_((tok,), w * yr, accumulate=True)
        tol.index_put_((tok,), w.abs() * t, accumulate=True)
    return y, tol


def check(got, ref, tol, what="", extra=0.0):
    """|got - ref| <= half a bf16 step of ref + (1 + 2^-8) tol (+ extra |ref|), elementwise."""
    got = got.double()
    bound = (HALF_BF16 + extra) * ref.abs() + (1 + HALF_BF16) * tol + 2.0 ** -133
    bad = ~((got - ref).abs() <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
        f"{float(((got - ref).abs() / bound).nan_to_num(1e9).max()):.3g} of the bound")
