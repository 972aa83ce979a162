"""Plain 64-bit implementations of rotary positions, of the cache in 8 or 4 bits
and of decode attention over it, for the tests, with the tolerances of a
comparison.

Rotary.  An angle's fraction of a half turn is rounded to 24 bits (2^-25 of it: at
most 2^-25 pi), sine and cosine to fp32 (at most 2 steps, 2^-23), and a result is
two products and a sum in fp32: within 2^-21 (|x| + |y|), then half a step of the
type: STEP of the value, and at least half of the type's least step (FLOOR: fp16's
numbers below 2^-14 lie 2^-24 apart, so that rounding is off by up to 2^-25 there).

Reading back.  lo + step code in fp32 (step code is exact there): 2^-24 of
|lo| + step code, then half a step of the type.

Attention.  With V = |lo| + step code and A = sum of softmax V:
  scores   d products and the groups' terms in fp32, sums that the tensor cores may
           cut off instead of rounding: d 2^-23 of sum |q| V; a cap 2^-21 of it
           (dense_ref); an error e of a score is one of 2 e of a weight's share
           With 16-bit outputs the codes are subnormal fp16 numbers whose exponent is a
           code's of 2^10, and the tensor cores cut each of a product's 17 terms off
           2^-24 below the largest: 17 2^-14 |q| step at most, d / 16 times
  weights  11 bits (2^-11 of each) where the output is bf16, else 22, cut off
           (2^-21); 2^x 2^-22, twice
  floor    fp16 loses up to 2^-24 of a part where the largest weight is at least
           2^11 there: two parts, 2^-34 of the largest weight, times a step's codes
  sums     n terms in fp32: n 2^-24 at most; with 16-bit outputs a product over 16
           tokens loses 17 2^-14 of its largest weight times step, all of them at
           most 17 2^-14 of sum softmax step
  output   half a step of its type, as above
"""
import math

import torch

STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FLOOR = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def frequencies(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def axes_of(sections, in_turn):
    left, out, a = list(sections), [], 0
    while sum(left):
        if left[a]:
            out.append(a)
            left[a] -= 1
            if not in_turn:
                continue
        a = (a + 1) % len(left)
    return out


def turn(x, positions, freq, axes, neighbours=False, inverse=False):
    """x [n][heads][d], positions [axes][n]: (rotated in 64 bits, |x| + |y| of the pairs)."""
    y, mag = x.double().clone(), x.double().abs()
    f = torch.tensor(freq, dtype=torch.float64, device=x.device)
    a = positions.double()[torch.tensor(axes, device=x.device)].t() * f
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None] * (-1 if inverse else 1)
    n = len(freq)
    i = torch.arange(n, device=x.device) * (2 if neighbours else 1)
    j = i + (1 if neighbours else n)
    p, q = x[..., i].double(), x[..., j].double()
    y[..., i], y[..., j] = p * c - q * s, p * s + q * c
    mag[..., i] = mag[..., j] = p.abs() + q.abs()
    return y, mag


def quantise(x, bits):
    """x [...][d]: (lo, step, code) per channel in 64 bits; groups that are not
    finite have lo NaN."""
    d = x.shape[-1]
    y = x.double().unflatten(-1, (-1, d if bits == 8 else 32))
    most = 2 ** bits - 1
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    span = hi - lo
    ok = span <= torch.finfo(torch.float32).max  # (False for NaN, too)
    s16 = (torch.where(ok, span, 0.0) / most).to(x.dtype)
    for _ in range(2):
        up = (s16.view(torch.int16) + 1).view(x.dtype)
        s16 = torch.where((s16.double() * most < span) & ok, up, s16)
    step = s16.double()
    code = torch.where(step > 0, torch.round((y - lo) / torch.where(step > 0, step, 1.0)), 0.0)
    lo = torch.where(ok, lo, math.nan).expand_as(y)
    step = step.expand_as(y)
    code = torch.where(ok, code, 0.0)
    return lo.flatten(-2), step.flatten(-2), code.flatten(-2)


def held(x, bits):
    """(values, |lo| + step code) in 64 bits."""
    lo, step, code = quantise(x, bits)
    return lo + step * code, lo.abs() + step * code


def attend(q, k, v, bits, first=0, scale=None, softcap=0.0, slopes=None):
    """One sequence: q [Hq][d], k, v [L][Hkv][d] as they were written.  Returns
    (out [Hq][d], tolerance without the output's own rounding as a function of
    the weights' bits)."""
    hq, d = q.shape
    L, hkv, _ = k.shape
    scale = scale or d ** -0.5
    out = torch.zeros(hq, d, dtype=torch.float64, device=q.device)
    absum, mag, top = torch.zeros_like(out), 0.0, torch.zeros_like(out)
    steps, cut = torch.zeros_like(out), 0.0
    back = torch.arange(L - 1 - first, -1, -1, device=q.device, dtype=torch.float64)
    for g in range(hkv):
        kv, ka = held(k[first:, g], bits)
        vv, va = held(v[first:, g], bits)
        hs = slice(g * hq // hkv, (g + 1) * hq // hkv)
        x = q[hs].double() @ kv.t() * scale
        mag = max(mag, float((q[hs].double().abs() @ ka.t()).max()) * scale)
        ks, vs = (quantise(y[first:, g], bits)[1] for y in (k, v))
        cut = max(cut, float(q[hs].double().abs().max() * ks.max()) * scale * 17 * 2.0 ** -14 * d / 16)
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        if slopes is not None:
            x = x - slopes[hs].double()[:, None] * back
            mag = max(mag, float(slopes[hs].max()) * len(kv) / d)  # (one more fp32 term)
        w = torch.softmax(x, 1)
        out[hs] = w @ vv
        absum[hs] = w @ va
        steps[hs] = w @ vs
        top[hs] = va.sum(0)
    n = L - first

    def tolerance(out_dtype):
        w = 2.0 ** -11 if out_dtype == torch.bfloat16 else 2.0 ** -21
        short = out_dtype != torch.float32
        e = mag * d * 2.0 ** -23 + softcap * 2.0 ** -21 + (cut if short else 0.0)
        return (17 * 2.0 ** -14 * steps if short else 0.0) + absum * (w + 2 * e + n * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -34 * top + \
            STEP[out_dtype] * out.abs() + FLOOR[out_dtype] + 1e-30

    return out, tolerance
