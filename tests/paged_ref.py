"""Plain 64-bit forms of rotary positions, the rotating append and attention over a paged cache, for the tests."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def rotate(x, pos, inv_freq, offset=0, interleaved=False, inverse=False, factor=1.0):
    """x [T, H, D] at pos [T] in fp64."""
    y = x.double().clone()
    half = inv_freq.numel()
    ang = pos.double()[:, None, None] * inv_freq.double().to(x.device)
    c, s = factor * torch.cos(ang), factor * torch.sin(ang) * (-1 if inverse else 1)
    if interleaved:
        i, j = slice(offset, offset + 2 * half, 2), slice(offset + 1, offset + 2 * half, 2)
    else:
        i, j = slice(offset, offset + half), slice(offset + half, offset + 2 * half)
    a, b = y[..., i].clone(), y[..., j].clone()
    y[..., i] = a * c - b * s
    y[..., j] = b * c + a * s
    return y


def assert_rotated(got, ref, x, factor=1.0):
    """One rounding to the type (half a step), after fp32 arithmetic: sine and cosine within 2 steps of 2^-23, two products
    and a sum of one half step each, on elements of up to max |x| of the head."""
    top = x.double().abs().amax(-1, keepdim=True) * abs(factor)
    tol = HALF_STEP[got.dtype] * (ref.abs() + 2 ** -18 * top) + 2 ** -19 * top + 2.0 ** -25
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float((got.double() - ref).abs().max())}"


def gather(cache, table, n, scale=1.0):
    """Positions 0..n-1 of one sequence: [n, heads, D] in fp64; scale: what 8-bit codes are divided by."""
    pages = table[: -(-n // 64)].long()
    eight = cache.dtype in (torch.uint8, torch.float8_e4m3fn)
    x = cache.view(torch.uint8)[pages].view(torch.float8_e4m3fn) if eight else cache[pages]
    return x.double().reshape(-1, *cache.shape[2:])[:n] / (scale if eight else 1.0)


def attend(q, k, v, pos, window, sm_scale):
    """q [n, H, D] at pos [n] over k, v [L, Hkv, D]: (out, lse, sum of weights x |v|, sum of |v| seen, score bound)."""
    n, H, D = q.shape
    G = H // k.shape[1]
    out, aout, sv = (torch.zeros(n, H, D, dtype=torch.float64, device=q.device) for _ in range(3))
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    big = torch.zeros(n, H, dtype=torch.float64, device=q.device)
    if k.shape[0] == 0:
        return out, lse, aout, sv, big
    at = torch.arange(k.shape[0], device=q.device)
    seen = at[None] <= pos[:, None]
    if window:
        seen &= at[None] > pos[:, None] - window
    some = seen.any(1)
    for h in range(H):
        qs, ks, vs = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        s = (qs @ ks.T * sm_scale).masked_fill(~seen, -math.inf)
        p = torch.softmax(s[some], -1)
        lse[some, h] = torch.logsumexp(s[some], -1)
        out[some, h], aout[some, h] = p @ vs, p @ vs.abs()
        sv[some, h] = seen[some].double() @ vs.abs()
        big[some, h] = (qs.abs() @ ks.abs().T * abs(sm_scale)).masked_fill(~seen, 0).amax(-1)[some]
    return out, lse, aout, sv, big


def assert_attended(got, ref, lse=None, weight_type=None):
    """Weights are rounded once to `weight_type` (fp16 ones below 2^-14 by up to 2^-25 absolute), the output once to its
    type; scores carry an fp32 dot product's error, at most (D + 4) half steps of 2^-24 of the sum of absolute products,
    which multiplies a weight by e^error."""
    out, rl, aout, sv, big = ref
    D = got.shape[-1]
    w = HALF_STEP[weight_type or got.dtype]
    ds = (D + 4) * 2.0 ** -24 * big[..., None]
    tol = HALF_STEP[got.dtype] * out.abs() + (w + 2 * ds + 2.0 ** -18) * aout * 1.01 + 2.0 ** -25
    if (weight_type or got.dtype) == torch.float16:
        tol = tol + 2.0 ** -25 * sv
    err = (got.double() - out).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float(err.max())}"
    if lse is not None:
        none = rl == -math.inf
        assert torch.equal(lse == -math.inf, none)
        e = (lse.double() - rl).abs()[~none]
        assert (e <= (2 * ds[..., 0] + 2.0 ** -21 * rl.abs() + 2.0 ** -19)[~none]).all(), float(e.max())
