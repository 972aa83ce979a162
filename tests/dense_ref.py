"""Plain 64-bit implementations of the dense attention operators and of
eviction, for the tests, with the tolerances of a comparison.

How far the library may be from these.  With A = sum of softmax |v|:
  weights   rounded to 16 bits once (output in the inputs' type): 2^-8 (bf16) or
            2^-11 (fp16) of each; with fp32 output kept in two parts (fp16),
            2^-22, or three (bf16), 2^-24; two of bf16, 2^-16, over more than
            1,024 keys.  fp16's steps end at 2^-24: whatever a weight is, half a step,
            2^-25, is lost of it too, where the row's largest weight is at least
            1 (the running max is never above the true one), so that
            2^-25 sum |v| over the attended keys bounds it (bf16 has fp32's
            range)
  scores    a product's fp32 sum over d channels is off by at most d 2^-24 of the
            sum of magnitudes; tanh by a polynomial is off by 4 x 2^-24 of the
            score (at most 2^-22 of the cap), beyond |s / cap| = 1 by the
            rounding of 2 / (1 + e^2z) <= 0.24 (2^-22 of it from e^2z, 2^-22
            from the quotient) and of the difference, 2^-23 of the cap in
            all; 2^-21 of the cap covers either.  An error e of a score is one
            of 2 e of a weight's share
  sums      n terms in fp32: n 2^-24 at most
  output    half a step of its type
"""
import math

import torch

STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def score(dot, h, far, scale, softcap, slopes):
    x = dot * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    if slopes is not None:
        x = x - slopes[h].double() * far
    return x


def attend(q, k, v, h, far, seen, scale, softcap, slopes):
    """One head: q [r][d], k, v [t][d], far and seen [r][t].  Returns (out, [A,
    sum |v| over the seen keys], weights, largest sum of |q||k| times the
    scale) in 64 bits; rows that see nothing are 0."""
    q, k, v = q.double(), k.double(), v.double()
    x = score(q @ k.t(), h, far, scale, softcap, slopes)
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    some = seen.any(1)
    w = torch.zeros_like(x)
    w[some] = torch.softmax(x[some], 1)
    mag = float((q.abs() @ k.abs().t()).max()) * scale if x.numel() else 0.0
    return w @ v, torch.stack([w @ v.abs(), seen.double() @ v.abs()]), w, mag


def tolerance(ref, absum, mag, d, n, dtype, out_dtype, softcap):
    step = STEP[dtype]
    w = step
    if out_dtype == torch.float32:
        w = step * step if dtype == torch.float16 or n > 1024 else step ** 3
    absum, plain = absum
    floor = 2.0 ** -25 * plain if dtype == torch.float16 else 0.0
    e = mag * d * 2.0 ** -24 + (softcap or 0.0) * 2.0 ** -21
    return absum * (w + 2 * e + n * 2.0 ** -24 + 2.0 ** -21) + floor + STEP[out_dtype] * ref.abs() + 1e-30


def prompt(q, k, v, begin, end, scale, softcap, slopes):
    """[Lq][Hq][d] in 64 bits, with A and the largest score magnitude."""
    Lq, Hq, d = q.shape
    Lk, Hkv, _ = k.shape
    dev = q.device
    t = torch.arange(Lk, device=dev)
    at = torch.arange(Lk - Lq, Lk, device=dev)
    seen = (t >= begin[:, None]) & (t < end[:, None])
    far = (at[:, None] - t).abs().double()
    out = torch.zeros(Lq, Hq, d, dtype=torch.float64, device=dev)
    ab, mag = torch.zeros(2, Lq, Hq, d, dtype=torch.float64, device=dev), 0.0
    for h in range(Hq):
        o, a, _, m = attend(q[:, h], k[:, h * Hkv // Hq], v[:, h * Hkv // Hq], h, far, seen, scale,
                            softcap, slopes)
        out[:, h], ab[:, :, h], mag = o, a, max(mag, m)
    return out, ab, mag


def shared(q, kp, vp, ko, vo, scale, softcap, slopes):
    """q [n][Hq][d]; kp, vp [Lp][Hkv][d]; ko, vo: per sequence [L_i][Hkv][d].
    Returns out, A, magnitude and per sequence the weights [Hkv][L_i]."""
    n, Hq, d = q.shape
    Hkv = kp.shape[1]
    dev, lp = q.device, kp.shape[0]
    out = torch.zeros(n, Hq, d, dtype=torch.float64, device=dev)
    ab, mag, ws = torch.zeros(2, n, Hq, d, dtype=torch.float64, device=dev), 0.0, []
    for i in range(n):
        k, v = torch.cat([kp, ko[i]]), torch.cat([vp, vo[i]])
        L = k.shape[0]
        far = torch.arange(L - 1, -1, -1, device=dev).double()[None]
        seen = torch.ones(1, L, dtype=torch.bool, device=dev)
        w = torch.zeros(Hkv, L - lp, dtype=torch.float64, device=dev)
        for h in range(Hq):
            g = h * Hkv // Hq
            o, a, p, m = attend(q[i, h][None], k[:, g], v[:, g], h, far, seen, scale, softcap,
                                slopes)
            out[i, h], ab[:, i, h], mag = o[0], a[:, 0], max(mag, m)
            w[g] += p[0, lp:]
        ws.append(w)
    return out, ab, mag, ws


def kept_positions(w, L, keep, recent):
    """Ascending positions that one kv head keeps, by sorting (weight down,
    position up)."""
    m = min(keep, L)
    newest = min(recent, m)
    old = L - newest
    key = [(-math.inf if math.isnan(x) else -x, t) for t, x in enumerate(w[:old].tolist())]
    best = sorted(key)[:m - newest]
    return sorted(t for _, t in best) + list(range(old, L))
