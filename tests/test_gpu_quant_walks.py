"""Decode attention over a quantised cache where every warp of the kernel walks many tiles:
sums that do not drift with the length of a walk, outputs that are the rounding of the exact
value, references of the weights that move in the middle of a walk."""
import math

import pytest
import torch

from quant_ref import FLOOR, STEP, held, quantise
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


# ---- references that move ------------------------------------------------------------

def step_tiles(d):
    return 4 if d == 64 else 2


def tolerance(q, k, v, bits, scale, steps, d, out_dtype):
    """Of every output of one kv head: q [heads][d], k and v [L][d] as written.  A score's products
    and sums are d + 8 roundings of 2^-23 of sum |q| (|lo| + step code), and with 16-bit outputs 17 terms
    of every product over 16 channels are cut at 2^-14 of the largest |q| step; an error e of the
    scores is one of 2 e of a weight's share.  Weights: 2^-21 cut off, 2^x 2^-21 in all.  Sums:
    2 tiles, one more a step, and at most 24 + 152 + 24 partials, 2^-24 each; with 16-bit outputs 17
    2^-14 of a step, as the weights have them.  What fp16 loses below its range: 2^-34 of the largest
    weight times step codes, all tokens' at most.  Then half a step of the output."""
    short = out_dtype != F32
    q = q.double().abs()
    kv, ka = held(k, bits)
    lo, step, code = quantise(v, bits)
    e = float((q @ ka.t()).max()) * scale * (d + 8) * 2.0 ** -23
    if short:
        e += float(q.max() * quantise(k, bits)[1].max()) * scale * 17 * 2.0 ** -14 * d / 16
    return lambda w, out: (
        w @ (lo.abs() + step * (2 ** bits - 1)) *
        (2.0 ** -20 + 2 * e + 2.0 ** -24 * (2 * step_tiles(d) * steps + steps + 200))
        + (17 * 2.0 ** -14 * (w @ step) if short else 0.0)
        + 2.0 ** -34 * (step * code).sum(0) + STEP[out_dtype] * out.abs() + FLOOR[out_dtype] + 1e-30)


def saw(L, height, period):
    t = torch.arange(L, device="cuda")
    return (t % period).float() / period * height


def scores_of(kind, L):
    """What every key's channels are moved by."""
    return {"noise": lambda: torch.zeros(L, device="cuda"),
            "gently": lambda: saw(L, 8.0, 700),     # 11 bits in 700 tokens
            "rising": lambda: saw(L, 40.0, 700),    # 58 bits
            "falling": lambda: 40.0 - saw(L, 40.0, 700)}[kind]()


def values_of(kind, seed, L, d):
    v = normal(seed, L, d)
    block = torch.arange(L, device="cuda") // 96 % 4
    if kind == "zero":
        return torch.zeros_like(v)
    if kind == "ones":
        return torch.ones_like(v)
    if kind == "blocks":  # nothing, ordinary ones, the same everywhere, tiny ones
        v[block == 0] = 0.0
        v[block == 2] = 1.5
        v[block == 3] *= 2.0 ** -20
    if kind == "sizes":
        v *= torch.exp2((block * 6 - 9).float())[:, None]
    return v


HEADS = [("noise", "normal"), ("rising", "normal"), ("falling", "normal"), ("gently", "zero"),
         ("gently", "ones"), ("rising", "blocks"), ("gently", "blocks"), ("falling", "sizes")]


@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype,out", [("bf16", "same"), ("bf16", "fp32"), ("fp16", "same"),
                                       ("fp16", "fp32")])
def test_references_move_in_the_middle_of_a_walk(g, d, bits, dtype, out):
    """Eight steps and more of every warp, whose scores rise or fall and whose values are ordinary,
    constant, nothing, or change from one to the other."""
    n, dt = len(HEADS), DT[dtype]
    L = tokens_for(9 * step_tiles(d), n)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    steps = -(-L // 16) * n // (WARPS * sms) // step_tiles(d)
    assert steps >= 8
    k = torch.stack([normal(10 + h, L, d) + scores_of(s, L)[:, None] for h, (s, _) in enumerate(HEADS)],
                    1).to(dt)
    v = torch.stack([values_of(x, 30 + h, L, d) for h, (_, x) in enumerate(HEADS)], 1).to(dt)
    c = cache(n * g, n, d, dtype, bits, L, page=256, seed=2)
    s = c.seq_create()
    c.kv_append([s], k[None], v[None])
    q = (1.0 + normal(50, n * g, d, gain=0.1)).to(dt)
    od = F32 if out == "fp32" else dt
    got = c.quant_decode_attention(q[None], [s], scale=1.0 / d, out_dtype=od)[0]
    c.check_status()
    for h, (_, kind) in enumerate(HEADS):
        mine = slice(h * g, (h + 1) * g)
        x = q[mine].double() @ held(k[:, h], bits)[0].t() / d
        w = torch.softmax(x, 1)
        ref = w @ held(v[:, h], bits)[0]
        tol = tolerance(q[mine], k[:, h], v[:, h], bits, 1.0 / d, steps, d, od)(w, ref)
        err = (got[mine].double() - ref).abs()
        assert bool((err <= tol).all()), (HEADS[h], float((err / tol).max()))
        if kind == "zero":
            assert bool((got[mine] == 0).all())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("size", [2.0 ** 80, 2.0 ** -80])
def test_constant_and_vast_values_under_rising_scores(bits, out, size):
    vast_values(bits, out, size, 30.0)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -124])
def test_tiny_values_keep_the_bits_of_their_weights(bits, out, size):
    vast_values(bits, out, size, 0.0)


def vast_values(bits, out, size, height):
    d, hkv = 128, 4
    L = tokens_for(16, hkv)
    k = normal(1, L, hkv, d)
    k = (k + saw(L, height, 500)[:, None, None]).bfloat16()
    v = normal(2, L, hkv, d) * size
    v[:, ::2] = size
    v = v.bfloat16()
    c = cache(hkv * 2, hkv, d, "bf16", bits, L, page=256)
    s = c.seq_create()
    c.kv_append([s], k[None], v[None])
    q = torch.ones(hkv * 2, d, device="cuda").bfloat16()
    od = F32 if out == "fp32" else torch.bfloat16
    got = c.quant_decode_attention(q[None], [s], scale=1.0 / d, out_dtype=od)[0]
    c.check_status()
    for h in range(hkv):
        mine = slice(2 * h, 2 * h + 2)
        w = torch.softmax(q[mine].double() @ held(k[:, h], bits)[0].t() / d, 1)
        ref = w @ held(v[:, h], bits)[0]
        tol = tolerance(q[mine], k[:, h], v[:, h], bits, 1.0 / d, 9, d, od)(w, ref)
        err = (got[mine].double() - ref).abs()
        assert bool((err <= tol).all()), (h, float((err / tol).max()))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype,out", [("bf16", "same"), ("bf16", "fp32"), ("fp16", "same"),
                                       ("fp16", "fp32")])
@pytest.mark.parametrize("at", [0, 40, 1499, 2999])
def test_vast_scores_and_steps(bits, dtype, out, at):
    """Scores near 10^9 (fp32 numbers 64 and more apart) over steps of 2^5 and more: one key's score
    is 2 10^7 above the others', further than what fp32 leaves open (64 2^-23 of 3 10^9), so that
    the output is what is held of its value, rounded."""
    L, d, dt = 3000, 64, DT[dtype]
    k = normal(1, 1, L, 1, d, gain=10.0) + 3e4
    k[:, at] += 6e3
    v = normal(2, 1, L, 1, d, gain=1e4)
    k, v = k.to(dt), v.to(dt)
    c = cache(4, 1, d, dtype, bits, L)
    s = c.seq_create()
    c.kv_append([s], k, v)
    q = torch.full((1, 4, d), 512.0, device="cuda").to(dt)
    x = q[0].double() @ held(k[0, :, 0], bits)[0].t()
    top = x[0].topk(2).values
    assert int(x[0].argmax()) == at and float(top[0] - top[1]) > 2e7 and float(top[0]) > 1e9
    assert float(quantise(v, bits)[1].max()) >= 32
    od = F32 if out == "fp32" else dt
    got = c.quant_decode_attention(q, [s], scale=1.0, out_dtype=od)[0]
    ref, mag = held(v[0, at, 0], bits)
    lo, step, _ = quantise(v[0, at, 0], bits)
    # (its weight is 1, cut off to 22 bits; sums of what is subtracted again: hi and lo)
    tol = 2.0 ** -20 * (lo.abs() + step * (2 ** bits - 1)) + STEP[od] * ref.abs() + FLOOR[od]
    if od != F32:
        tol = tol + 17 * 2.0 ** -14 * step
    assert bool(((got.double() - ref).abs() <= tol).all())
    c.check_status()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("L,g", [(700, 1), (3000, 4), (3000, 8)])
def test_biases_beyond_the_range_leave_the_newest_token(bits, out, L, g):
    """Slopes of 10^36: scores of all but some hundred tokens are -inf in fp32, and whole walks see
    nothing else."""
    d, dt = 128, torch.bfloat16
    c, ids, k, v = filled(L, 2 * g, 2, d, "bf16", bits, seed=9)
    q = normal(1, 1, 2 * g, d, dtype=dt)
    slopes = torch.full((2 * g,), 1e36, device="cuda")
    od = F32 if out == "fp32" else dt
    got = c.quant_decode_attention(q, ids, slopes=slopes, out_dtype=od)[0].unflatten(0, (2, g))
    ref, _ = held(v[0, -1], bits)
    lo, step, _ = quantise(v[0, -1], bits)
    # (a weight of 1, cut off to 22 bits)
    tol = 2.0 ** -20 * (lo.abs() + step * (2 ** bits - 1)) + STEP[od] * ref.abs() + FLOOR[od]
    if od != F32:
        tol = tol + 17 * 2.0 ** -14 * step
    assert bool(((got.double() - ref[:, None]).abs() <= tol[:, None]).all())
    c.check_status()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("out", ["same", "fp32"])
def test_queries_that_are_not_finite_stay_with_their_heads(bits, out):
    """Infinite and NaN queries give NaN in their own heads; the others', in the same columns of the
    products, are as exact as ever."""
    L, hkv, g, d, dt = 3000, 2, 4, 128, torch.float16
    c, ids, k, v = filled(L, hkv * g, hkv, d, "fp16", bits, seed=4)
    q = normal(2, 1, hkv * g, d, dtype=dt)
    q[0, 1, 7], q[0, 2, 9], q[0, 7, 0] = math.inf, math.nan, -math.inf
    od = F32 if out == "fp32" else dt
    got = c.quant_decode_attention(q, ids, out_dtype=od)[0]
    c.check_status()
    for h in range(hkv * g):
        if h in (1, 2, 7):
            assert bool(got[h].isnan().all())
            continue
        kh, vh, row = k[0, :, h // g], v[0, :, h // g], q[0, h:h + 1]
        w = torch.softmax(row.double() @ held(kh, bits)[0].t() * d ** -0.5, 1)
        ref = w @ held(vh, bits)[0]
        tol = tolerance(row, kh, vh, bits, d ** -0.5, 1, d, od)(w, ref)
        assert bool(((got[h:h + 1].double() - ref).abs() <= tol).all()), h
