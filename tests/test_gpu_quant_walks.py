"""Decode attention over a quantised cache where every warp of the kernel walks many tiles:
sums that do not drift with the length of a walk, outputs that are the rounding of the exact
value, references of the weights that move in the middle of a walk."""
import math

import pytest
import torch

from quant_ref import STEP, held
from test_gpu_quant import DT, F32, cache, normal

pytestmark = pytest.mark.gpu
WARPS = 12  # of a CTA, one CTA an SM


def tokens_for(tiles_per_warp, hkv):
    """Length of one sequence whose units give every warp that many tiles of 16 tokens."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-tiles_per_warp * WARPS * sms * 16 // hkv)


def filled(L, hq, hkv, d, dtype, bits, seed, n=1, page=1024, piece=1 << 17):
    """A cache of n sequences of L tokens of normal values, and what was written."""
    c = cache(hq, hkv, d, dtype, bits, L, seqs=n, page=page, seed=seed, fill=False)
    ids, ks, vs = [c.seq_create() for _ in range(n)], [], []
    for a in range(0, L, piece):
        m = min(piece, L - a)
        k, v = (normal(seed + 2 * a + i, n, m, hkv, d, dtype=DT[dtype]) for i in range(2))
        c.kv_append(ids, k, v)
        ks.append(k)
        vs.append(v)
    return c, ids, torch.cat(ks, 1), torch.cat(vs, 1)


def exact(q, k, v, bits, scale=None, softcap=0.0, first=0):
    """One sequence in 64 bits: q [Hq][d], k and v [L][Hkv][d] as written."""
    hq, d = q.shape
    g = hq // k.shape[1]
    out = torch.empty(hq, d, dtype=torch.float64, device=q.device)
    for h in range(k.shape[1]):
        x = q[h * g:(h + 1) * g].double() @ held(k[first:, h], bits)[0].t() * (scale or d ** -0.5)
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        out[h * g:(h + 1) * g] = torch.softmax(x, 1) @ held(v[first:, h], bits)[0]
    return out


def rms(x):
    return float(x.double().pow(2).mean().sqrt())


# ---- sums ---------------------------------------------------------------------------
# Relative to the outputs' root mean square, which is s / sqrt(n') for values of deviation s and
# n' = n / e tokens in effect (normal scores).  In a walk of M tokens a product's signed terms
# make partial sums of at most 8.4 s sqrt(m) (a span of values times codes; weights near 1), each
# rounded to 2^-24 of itself when a step is added: 2^-24 8.4 s sqrt(steps M / 6) in all, over M and
# the square root of the walks of a head.  For 1,024 tiles (M = 16,384, 512 steps or 256, 114 walks):
# 3.4e-9 s, of outputs of 1.2e-3 s, 2.8e-6; shorter walks less.  A score's error of e, different for
# every token, is one of e: about 3 2^-24 times sums of 8, 1.4e-6.  MARGIN is several times both.
# The rounding to 16 bits is at most STEP of a value, evenly spread: STEP / sqrt(3).
MARGIN = 2.0 ** -16


@pytest.mark.parametrize("tiles,dtype,bits", [
    (64, "fp16", 8), (64, "fp16", 4), (256, "fp16", 8), (256, "fp16", 4), (256, "bf16", 8),
    (256, "bf16", 4), (1024, "fp16", 8), (1024, "bf16", 4)])
def test_long_walks_do_not_drift(tiles, dtype, bits):
    L = tokens_for(tiles, 16)
    c, ids, k, v = filled(L, 16, 16, 64, dtype, bits, seed=tiles)
    q = normal(5, 1, 16, 64, dtype=DT[dtype])
    ref = exact(q[0], k[0], v[0], bits)
    for od in (DT[dtype], F32):
        got = c.quant_decode_attention(q, ids, out_dtype=od)[0]
        assert rms(got.double() - ref) <= (STEP[od] / math.sqrt(3) + MARGIN) * rms(ref), od
    c.check_status()


@pytest.mark.parametrize("heads,d", [((32, 8), 128), ((64, 8), 128), ((8, 8), 128), ((16, 16), 64)])
@pytest.mark.parametrize("bits", [8, 4])
def test_walks_of_every_layout_do_not_drift(heads, d, bits):
    """Heads that share keys, 128 channels, sixteen sequences."""
    c, ids, k, v = filled(6000, *heads, d, "fp16", bits, seed=7, n=16)
    q = normal(5, 16, heads[0], d, dtype=torch.float16)
    ref = torch.stack([exact(q[i], k[i], v[i], bits) for i in range(16)])
    got = c.quant_decode_attention(q, ids, out_dtype=torch.float16)
    assert rms(got.double() - ref) <= (STEP[torch.float16] / math.sqrt(3) + MARGIN) * rms(ref)
    c.check_status()


# ---- outputs ------------------------------------------------------------------------
# An output that is not the rounding of the exact value lies within its error of the middle
# between two numbers of its type: error / ulp of all, for errors spread evenly.  An error of MARGIN
# of the outputs' root mean square and a bf16 ulp of at least 2^-8 of a value: 2^-8 where values are
# of that size, three times that over a normal distribution, whose smaller values have smaller ulps.
FLIPS = 3 * MARGIN / 2.0 ** -8


@pytest.mark.parametrize("heads,d", [((32, 8), 128), ((64, 8), 128), ((8, 4), 64), ((16, 16), 64)])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rule", [dict(), dict(softcap=50.0, gain=4.0), dict(window=700)])
def test_bf16_outputs_are_the_exact_values_rounded(heads, d, bits, rule):
    n, L = 16, 3000
    c, ids, k, v = filled(L, *heads, d, "bf16", bits, seed=3, n=n)
    q = normal(5, n, heads[0], d, dtype=torch.bfloat16, gain=rule.get("gain", 1.0))
    cap, window = rule.get("softcap", 0.0), rule.get("window", 0)
    ref = torch.stack([exact(q[i], k[i], v[i], bits, softcap=cap, first=L - window if window else 0)
                       for i in range(n)])
    got = c.quant_decode_attention(q, ids, softcap=cap, window=window, out_dtype=torch.bfloat16)
    off = (got != ref.bfloat16()).double().mean()
    assert float(off) <= FLIPS
    c.check_status()
