"""Rotary positions, the cache in 8 or 4 bits and decode attention over it against
the 64-bit implementations in quant_ref.py (which also derives the tolerances)."""
import math

import pytest
import torch

import sparse_paged_decode_logical_gb300 as spd
from quant_ref import FLOOR, STEP, attend, axes_of, frequencies, held, quantise, turn

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
F32 = torch.float32


def normal(seed, *shape, dtype=F32, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * gain).to(dtype)


def places(seed, *shape, lo=0, hi=100000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, device="cuda", generator=g, dtype=torch.int32)


def within(got, ref, tol):
    err = (got.double() - ref).abs()
    ok = bool(((err <= tol) | (got.isnan() & ref.isnan())).all())
    assert ok, float((err / tol).max())


# ---- rotary ----------------------------------------------------------------------

def check_rotary(n, hq, hk, d, dtype="bf16", rot=None, sections=None, in_turn=False, neighbours=False,
                 inverse=False, lo=0, hi=100000, base=10000.0, seed=1):
    dt, rot = DT[dtype], rot or d
    sections = sections or [rot // 2]
    t = spd.Rotary(d, rotary_dim=rot, sections=sections, axes_in_turn=in_turn, neighbours=neighbours,
                   base=base)
    q, k = normal(seed, n, hq, d, dtype=dt), normal(seed + 1, n, max(hk, 1), d, dtype=dt)
    pos = places(seed + 2, len(sections), n, lo=lo, hi=hi)
    got = spd.rotary(t, pos, q, k if hk else None, inverse=inverse)
    for x, y in zip((q, k), got if hk else (got,)):
        ref, mag = turn(x, pos, frequencies(rot, base), axes_of(sections, in_turn), neighbours, inverse)
        assert y.shape == x.shape and y.dtype == dt and y.is_contiguous()
        within(y, ref, mag * 2.0 ** -21 + STEP[dt] * ref.abs() + FLOOR[dt])
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 33, 1500])
@pytest.mark.parametrize("heads", [(8, 2), (1, 1), (5, 0), (3, 7)])
def test_rotary_lengths_and_heads(n, heads):
    check_rotary(n, *heads, 128)
    check_rotary(n, *heads, 64, "fp16")


@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (64, 64), (128, 16), (128, 32), (128, 48),
                                   (128, 80), (128, 96), (128, 112), (128, 128)])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_widths(d, rot, neighbours, inverse):
    for dtype in DT:
        check_rotary(21, 4, 2, d, dtype, rot=rot, neighbours=neighbours, inverse=inverse)


@pytest.mark.parametrize("sections", [[32], [20, 12], [8, 12, 12], [1, 30, 0, 1], [0, 32]])
@pytest.mark.parametrize("in_turn", [False, True])
@pytest.mark.parametrize("neighbours", [False, True])
def test_rotary_axes(sections, in_turn, neighbours):
    check_rotary(40, 4, 1, 64, sections=sections, in_turn=in_turn, neighbours=neighbours)


@pytest.mark.parametrize("lo,hi", [(-5, 5), (1 << 20, 1 << 21), ((1 << 31) - 99, (1 << 31) - 1),
                                   (-(1 << 31), -(1 << 31) + 99)])
def test_rotary_far_positions(lo, hi):
    # (a frequency's own error, 2^-53 of at most 1 radian, grows to 2^-22 at 2^31: both sides)
    n = 50
    t = spd.Rotary(128)
    q = normal(3, n, 4, 128, dtype=torch.float16)
    pos = places(4, 1, n, lo=lo, hi=hi)
    ref, mag = turn(q, pos, frequencies(128), [0] * 64)
    far = max(abs(lo), abs(hi)) * 2.0 ** -51
    within(spd.rotary(t, pos, q), ref, mag * (2.0 ** -21 + far) + STEP[torch.float16] * ref.abs() + 2.0 ** -25)


def test_rotary_given_frequencies():
    f = [0.0, 1.0, 6.0, 1000.0] + [0.01 * i for i in range(28)]
    t = spd.Rotary(64, inv_freq=f)
    q, pos = normal(1, 30, 2, 64, dtype=torch.float16), places(2, 30, hi=5000)
    ref, mag = turn(q, pos[None], f, [0] * 32)
    # (the angle in 64 bits itself is off by 2^-52 of up to 5e6)
    within(spd.rotary(t, pos, q), ref, mag * 2.0 ** -21 + STEP[torch.float16] * ref.abs() + 2.0 ** -25)


def test_rotary_reads_and_writes_strided_rows_and_in_place():
    n, hq, hk, d = 37, 6, 2, 128
    row = normal(1, n, (hq + 2 * hk) * d, dtype=torch.bfloat16)
    q = row[:, :hq * d].unflatten(1, (hq, d))
    k = row[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    t, pos = spd.Rotary(d), places(2, n)
    want = spd.rotary(t, pos, q.contiguous(), k.contiguous())
    got = spd.rotary(t, pos, q, k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    v = row[:, (hq + hk) * d:].clone()
    assert spd.rotary(t, pos, q, k, out=(q, k))[0] is q
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(row[:, (hq + hk) * d:], v)


def test_rotary_inverse_is_the_gradient():
    """<R x, y> = <x, R^T y> in 64 bits of the outputs, and against differences: the
    rotation is linear, so that R (x + e) - R x is R e for any e."""
    n, h, d = 9, 3, 64
    t = spd.Rotary(d, rotary_dim=32, sections=[10, 6], neighbours=True)
    x, y = normal(1, n, h, d, dtype=torch.float16), normal(2, n, h, d, dtype=torch.float16)
    pos = places(3, 2, n)
    rx, ry = spd.rotary(t, pos, x), spd.rotary(t, pos, y, inverse=True)
    a, b = (rx.double() * y.double()).sum(), (x.double() * ry.double()).sum()
    # every product off by half a step of a value of at most sqrt(2) |x|'s pair
    bound = 2.0 ** -10 * float((x.double().norm(dim=-1) * y.double().norm(dim=-1)).sum()) * 2
    assert abs(float(a - b)) <= bound
    i = 5
    e = torch.zeros_like(x)
    e[:, :, i] = 0.5
    diff = (spd.rotary(t, pos, x + e).double() - rx.double()) / 0.5  # column i of R
    col = (diff * y.double()).sum(-1)
    # R^T y at i; differences of rounded values, over 0.5: two half steps of 2^-11 of at most
    # |x| + 0.5 + |its partner|, and x + e itself is rounded
    mag = (x.double().abs().amax(-1) * 2 + 1) * y.double().abs().sum(-1)
    within(col, ry.double()[:, :, i], 6 * 2.0 ** -11 * mag)


def test_rotary_of_nothing_but_zeros_infinities_and_nan():
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 0, 0], x[1, 0, 1], x[1, 0, 63] = math.inf, math.nan, 1.0
    y = spd.rotary(spd.Rotary(64), torch.tensor([7, 0], dtype=torch.int32, device="cuda"), x)
    assert torch.equal(y[0], x[0])
    assert not math.isfinite(float(y[1, 0, 0])) and math.isnan(float(y[1, 0, 1]))
    assert float(y[1, 0, 63]) == 1.0 and bool((y[1, 0, 2:32] == 0).all())


# ---- writing and reading back -----------------------------------------------------

def cache(hq, hkv, d, dtype, bits, tokens, seqs=1, page=64, seed=0, fill=True):
    c = spd.SparsePagedKVCache(
        device="cuda", num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=dtype, logical_page=16,
        physical_page=page, num_physical_pages=seqs * -(-tokens // page) + 2, max_seqs=seqs + 1,
        max_context=tokens, kv_quant=bits, free_list_seed=seed)
    if fill:  # what lies where nothing was written is not finite
        c.buffers["k_pool"].fill_(0xff)
    return c


def rows(seed, n, tokens, hkv, d, dtype):
    """Keys or values: some channels far from 0, one token much larger."""
    x = normal(seed, n, tokens, hkv, d)
    x[..., ::7] += 3.0
    x[:, tokens // 2] *= 20.0
    return x.to(DT[dtype])


def check_held(got, x, bits):
    ref, mag = held(x, bits)
    ref = ref.clamp(max=torch.finfo(x.dtype).max)  # (what is finite is read back finite)
    within(got, ref, STEP[x.dtype] * ref.abs() + 2.0 ** -23 * mag + FLOOR[x.dtype])
    # and no value further than half a step from itself, and then half a step of the type, of
    # what is read: at most |x| + step / 2
    half = quantise(x, bits)[1] * 0.5
    x = x.double()
    within(got, x, half + STEP[got.dtype] * (x.abs() + half) + 2.0 ** -22 * mag + FLOOR[got.dtype])


@pytest.mark.parametrize("tokens", [1, 15, 16, 17, 64, 65, 130])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_written_and_read_back(tokens, d, bits, dtype):
    c = cache(4, 2, d, dtype, bits, tokens, seqs=3, page=48, seed=5)
    ids = [c.seq_create() for _ in range(3)]
    k, v = rows(1, 3, tokens, 2, d, dtype), rows(2, 3, tokens, 2, d, dtype)
    c.kv_append(ids, k, v)
    gk, gv = c.kv_read(ids)
    c.check_status()
    assert gk.shape == k.shape and gk.dtype == k.dtype
    check_held(gk, k, bits)
    check_held(gv, v, bits)


@pytest.mark.parametrize("cuts", [[1] * 40, [3, 13, 16, 1, 31, 7], [16, 1, 15, 16], [33, 1, 1, 30]])
@pytest.mark.parametrize("d,bits", [(64, 8), (128, 4), (64, 4), (128, 8)])
def test_pieces_are_what_a_whole_is(cuts, d, bits):
    """Single tokens, parts of tiles and whole tiles write the same bytes."""
    n = sum(cuts)
    k, v = rows(3, 1, n, 3, d, "bf16"), rows(4, 1, n, 3, d, "bf16")
    c = cache(3, 3, d, "bf16", bits, n, seqs=2, page=16)
    a, b = c.seq_create(), c.seq_create()
    c.kv_append([a], k, v)
    at = 0
    for m in cuts:
        c.kv_append([b], k[:, at:at + m].contiguous(), v[:, at:at + m].contiguous())
        at += m
    whole, pieces = c.kv_read([a]), c.kv_read([b])
    c.check_status()
    assert torch.equal(whole[0], pieces[0]) and torch.equal(whole[1], pieces[1])
    check_held(whole[0], k, bits)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens", [5, 32])
def test_groups_at_the_edges(bits, dtype, tokens):
    """Constant, zero, subnormal and vast groups, infinities and NaN."""
    dt = DT[dtype]
    tiny, big = (2.0 ** -133, 2.0 ** 127) if dtype == "bf16" else (2.0 ** -24, 65504.0)
    x = normal(1, 1, tokens, 1, 128, dtype=dt)
    x[0, 0] = 0.0
    x[0, 1] = -2.5
    x[0, 2] = (torch.arange(128, device="cuda") % 5).to(dt) * tiny
    x[0, 3] = torch.where(torch.arange(128, device="cuda") % 2 == 0, big, -big).to(dt)
    x[0, 4, 0, 3], x[0, 4, 0, 40], x[0, 4, 0, 41] = math.nan, math.inf, -math.inf
    c = cache(1, 1, 128, dtype, bits, tokens)
    s = c.seq_create()
    c.kv_append([s], x, x)
    for y in c.kv_read([s]):
        assert bool((y[0, 0] == 0).all()) and bool((y[0, 1] == -2.5).all())
        check_held(y[:, 2], x[:, 2], bits)
        if dtype == "fp16":
            check_held(y[:, 3], x[:, 3], bits)
        else:
            # (the span, 2^128, exceeds fp32)
            assert bool(y[0, 3].isnan().all())
        bad = torch.zeros(128, dtype=torch.bool, device="cuda")
        bad[:128 if bits == 8 else 64] = True
        assert bool(y[0, 4, 0, bad].isnan().all())
        if bits == 4:
            check_held(y[:, 4, :, 64:], x[:, 4, :, 64:], bits)
        if tokens > 5:
            check_held(y[:, 5:], x[:, 5:], bits)
    c.check_status()


def test_reading_ranges():
    c = cache(2, 2, 64, "fp16", 4, 100, seqs=2, page=32, seed=3)
    ids = [c.seq_create() for _ in range(2)]
    for i, n in zip(ids, (100, 61)):
        c.kv_append([i], rows(i, 1, n, 2, 64, "fp16"), rows(i + 9, 1, n, 2, 64, "fp16"))
    whole = [c.kv_read([i]) for i in ids]
    for begin, n in ((0, 61), (15, 2), (16, 16), (31, 30), (60, 1), (-1, 1), (-61, 61), (-20, 3)):
        k, v = c.kv_read(ids, begin, n)
        for r, L in enumerate((100, 61)):
            a = L + begin if begin < 0 else begin
            assert torch.equal(k[r], whole[r][0][0, a:a + n])
            assert torch.equal(v[r], whole[r][1][0, a:a + n])
    assert c.kv_read(ids, 7)[0].shape[1] == 54 and c.kv_read(ids[::-1], 7)[0].shape[1] == 54
    assert c.kv_read(ids, -9)[0].shape[1] == 9
    for begin, n in ((0, 62), (-62, 1), (61, 1), (-1, 2), (100, 1), (5, 0), (0, 1 << 40)):
        with pytest.raises(spd.SpdError):
            c.kv_read(ids, begin, n)


@pytest.mark.parametrize("n,tokens", [(1, 1), (5, 1), (3, 50), (2, 16), (70, 3)])
@pytest.mark.parametrize("bits,d,dtype", [(8, 128, "bf16"), (4, 64, "fp16"), (4, 128, "bf16")])
@pytest.mark.parametrize("kind", ["halves", "neighbours", "part", "own places"])
def test_rotated_on_the_way(n, tokens, bits, d, dtype, kind):
    """The bits of spd.rotary followed by kv_append, from a fused projection's rows, behind
    a first append of an odd length."""
    hq, hkv, dt = 4, 2, DT[dtype]
    part = kind == "part"
    t = spd.Rotary(d, rotary_dim=48 if part else d, sections=[10, 14] if part else None,
                   neighbours=kind == "neighbours")
    c = cache(hq, hkv, d, dtype, bits, 5 + tokens, seqs=2 * n, page=16)
    a, b = ([c.seq_create() for _ in range(n)] for _ in range(2))
    for ids in (a, b):
        c.kv_append(ids, rows(1, n, 5, hkv, d, dtype), rows(2, n, 5, hkv, d, dtype))
    row = normal(3, n, tokens, (hq + 2 * hkv) * d, dtype=dt)
    q = row[..., :hq * d].unflatten(2, (hq, d))
    k = row[..., hq * d:(hq + hkv) * d].unflatten(2, (hkv, d))
    v = row[..., (hq + hkv) * d:].unflatten(2, (hkv, d))
    pos = places(4, t.axes, n, tokens)
    if kind == "own places":
        pos = torch.arange(5, 5 + tokens, device="cuda", dtype=torch.int32).repeat(1, n, 1)
    wq, wk = spd.rotary(t, pos.flatten(1), q.flatten(0, 1), k.flatten(0, 1))
    c.kv_append(a, wk.view(k.shape), v.contiguous())
    gq = c.kv_append_rotary(b, t, q, k, v, positions=None if kind == "own places" else pos)
    c.check_status()
    assert torch.equal(gq, wq.view(gq.shape))
    for x, y in zip(c.kv_read(a), c.kv_read(b)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("n,tokens", [(2, 2600), (290, 19), (1, 5003)])
@pytest.mark.parametrize("kind", ["places", "positions", "in place"])
def test_rotated_on_the_way_in_long_and_wide_appends(n, tokens, kind):
    """Queries in a launch of their own, and more sequences than a launch holds."""
    hq, hkv, d, dt = 4, 2, 64, torch.bfloat16
    c = cache(hq, hkv, d, "bf16", 4, tokens + 3, seqs=2 * n, page=64)
    t = spd.Rotary(d, neighbours=True)
    a, b = ([c.seq_create() for _ in range(n)] for _ in range(2))
    for ids in (a, b):
        for i, s in enumerate(ids):  # sequences that begin at different places
            if i % 3:
                c.kv_append([s], rows(i, 1, i % 3, hkv, d, "bf16"), rows(i, 1, i % 3, hkv, d, "bf16"))
    q, k, v = (normal(i, n, tokens, h, d, dtype=dt) for i, h in ((1, hq), (2, hkv), (3, hkv)))
    start = torch.tensor([i % 3 for i in range(n)], device="cuda", dtype=torch.int32)[:, None]
    pos = start + torch.arange(tokens, device="cuda", dtype=torch.int32)
    if kind != "places":
        pos = places(4, n, tokens)
    wq, wk = spd.rotary(t, pos.flatten(), q.flatten(0, 1), k.flatten(0, 1))
    c.kv_append(a, wk.view(k.shape), v)
    gq = c.kv_append_rotary(b, t, q, k, v, positions=None if kind == "places" else pos,
                            out=q if kind == "in place" else None)
    c.check_status()
    assert torch.equal(gq, wq.view(gq.shape))
    for x, y in zip(c.kv_read(a, -tokens), c.kv_read(b, -tokens)):
        assert torch.equal(x, y)
    check_held(c.kv_read(b, -tokens)[1], v, 4)


def test_rotated_in_place():
    c = cache(4, 2, 128, "bf16", 8, 40)
    s, t = c.seq_create(), spd.Rotary(128)
    q, k, v = (normal(i, 1, 40, h, 128, dtype=torch.bfloat16) for i, h in ((1, 4), (2, 2), (3, 2)))
    want = spd.rotary(t, torch.arange(40, dtype=torch.int32, device="cuda"), q[0])
    assert c.kv_append_rotary([s], t, q, k, v, out=q) is q
    assert torch.equal(q[0], want)


def test_new_pages_of_every_kind():
    """Pages taken by the append itself, many at once, reserved before (also for others, and in
    an order that does not follow), given back before they were written."""
    c = cache(2, 1, 64, "fp16", 8, 3700, seqs=6, page=16, seed=9)
    k, v = rows(1, 1, 3700, 1, 64, "fp16"), rows(2, 1, 3700, 1, 64, "fp16")
    q = normal(3, 1, 2, 64, dtype=torch.float16)
    ids = [c.seq_create() for _ in range(5)]
    length = dict.fromkeys(ids, 0)

    def put(which, n):
        for i in which:
            assert length[i] == length[which[0]]
        a = length[which[0]]
        c.kv_append(which, k[:, a:a + n].repeat(len(which), 1, 1, 1), v[:, a:a + n].repeat(len(which), 1, 1, 1))
        for i in which:
            length[i] += n

    put(ids[:2], 3)                 # a page each
    put([ids[0]], 1100)             # 69 pages
    c.seq_reserve(ids[2], 100)      # another's, written by the next append of anyone
    put([ids[0]], 2500)             # 156: more than a launch takes along
    put([ids[1]], 40)
    c.seq_reserve(ids[3], 20)
    c.seq_reserve(ids[4], 20)
    c.seq_reserve(ids[3], 60)       # not behind its own first ones
    put(ids[2:5], 90)
    c.seq_reserve(ids[2], 200)
    c.seq_truncate(ids[2], 90)      # given back before anyone wrote them
    put(ids[2:5], 31)
    for i in ids:
        gk, gv = c.kv_read([i])
        check_held(gk, k[:, :length[i]], 8)
        check_held(gv, v[:, :length[i]], 8)
        ref, tol = attend(q[0], k[0, :length[i]], v[0, :length[i]], 8)
        within(c.quant_decode_attention(q, [i])[0], ref, tol(F32))
    c.check_status()


def test_truncated_sequences_go_on():
    c = cache(2, 1, 64, "bf16", 4, 200, page=32)
    s = c.seq_create()
    k, v = rows(1, 1, 200, 1, 64, "bf16"), rows(2, 1, 200, 1, 64, "bf16")
    c.kv_append([s], k[:, :150].contiguous(), v[:, :150].contiguous())
    free = c.free_pages()
    c.seq_truncate(s, 150)
    assert c.free_pages() == free
    c.seq_truncate(s, 70)                      # 5 pages of 32 become 3
    assert c.free_pages() == free + 2 and c.seq_info(s)["length"] == 70
    other = c.seq_create()                     # takes them
    c.kv_append([other], k[:, :64].contiguous(), v[:, :64].contiguous())
    c.kv_append([s], k[:, 100:140].contiguous(), v[:, 100:140].contiguous())
    gk, gv = c.kv_read([s])
    check_held(gk, torch.cat([k[:, :70], k[:, 100:140]], 1), 4)
    check_held(gv, torch.cat([v[:, :70], v[:, 100:140]], 1), 4)
    check_held(c.kv_read([other])[0], k[:, :64], 4)
    c.seq_truncate(s, 0)
    with pytest.raises(spd.SpdError):
        c.quant_decode_attention(normal(1, 1, 2, 64, dtype=torch.bfloat16), [s])
    c.kv_append([s], k[:, :1].contiguous(), v[:, :1].contiguous())
    check_held(c.kv_read([s])[1], v[:, :1], 4)
    c.check_status()


# ---- attention --------------------------------------------------------------------

def check_attend(lens, hq, hkv, d, dtype, bits, out="same", window=0, scale=0.0, softcap=0.0,
                 slopes=False, page=64, gain=1.0, seed=1, fn=rows, kv=None):
    dt = DT[dtype]
    c = cache(hq, hkv, d, dtype, bits, max(lens), seqs=len(lens), page=page, seed=seed)
    ids, ks, vs = [], [], []
    for i, L in enumerate(lens):
        k, v = kv(i, L) if kv else (fn(seed + 2 * i, 1, L, hkv, d, dtype),
                                    fn(seed + 2 * i + 1, 1, L, hkv, d, dtype))
        ids.append(c.seq_create())
        c.kv_append([ids[-1]], k, v)
        ks.append(k[0])
        vs.append(v[0])
    q = normal(seed + 77, len(lens), hq, d, dtype=dt, gain=gain)
    sl = torch.rand(hq, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) \
        * 0.5 if slopes else None
    od = F32 if out == "fp32" else dt
    got = c.quant_decode_attention(q, ids, window=window, scale=scale, softcap=softcap, slopes=sl,
                                   out_dtype=od)
    again = c.quant_decode_attention(q, ids, window=window, scale=scale, softcap=softcap, slopes=sl,
                                     out_dtype=od)
    c.check_status()
    assert got.shape == q.shape and got.dtype == od
    # joined in one order, and tickets are left as they were
    assert torch.equal(got.nan_to_num(7e4), again.nan_to_num(7e4))
    for i, L in enumerate(lens):
        first = max(0, L - window) if window else 0
        ref, tol = attend(q[i], ks[i], vs[i], bits, first, scale or None, softcap, sl)
        within(got[i], ref, tol(od))
    return c, ids, q, got


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 700, 2500])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype,out", [("bf16", "same"), ("bf16", "fp32"), ("fp16", "same")])
def test_attend_lengths(L, bits, dtype, out):
    check_attend([L], 8, 2, 128, dtype, bits, out)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (4, 1), (8, 1), (5, 5), (6, 3), (12, 3), (16, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype,out", [("bf16", "same"), ("bf16", "fp32"), ("fp16", "same"),
                                       ("fp16", "fp32")])
def test_attend_heads_and_types(hq, hkv, d, bits, dtype, out):
    check_attend([37, 200, 1, 64], hq, hkv, d, dtype, bits, out, page=32)


@pytest.mark.parametrize("rule", [dict(softcap=20.0, gain=5.0), dict(slopes=True), dict(scale=0.3),
                                  dict(softcap=50.0, slopes=True), dict(softcap=3e4, gain=9.0),
                                  dict(softcap=1e-3)])
@pytest.mark.parametrize("window", [0, 1, 16, 50, 129, 5000])
def test_attend_rules_and_windows(rule, window):
    check_attend([300, 77, 5], 8, 2, 128, "bf16", 8, window=window, **rule)
    check_attend([300, 77, 5], 8, 2, 64, "fp16", 4, out="fp32", window=window, **rule)


@pytest.mark.parametrize("page", [16, 48, 80, 256, 1024])
def test_attend_pages(page):
    check_attend([333, 1100, 16], 4, 1, 128, "bf16", 4, page=page, seed=3)


@pytest.mark.parametrize("lens,heads", [
    ([4000], (8, 1)), ([30000], (8, 8)), ([9000, 40, 9000, 1], (16, 4)),
    ([70] * 61, (16, 2)), ([33, 500, 1000, 7] * 20, (8, 8))])
@pytest.mark.parametrize("bits", [8, 4])
def test_attend_split_and_shared_warps(lens, heads, bits):
    """Units over many CTAs, units that share a CTA or a warp."""
    check_attend(lens, *heads, 64, "fp16", bits, out="fp32", page=256)


def test_attend_more_sequences_than_a_launch_holds():
    lens = [1 + (37 * i) % 90 for i in range(270)]
    check_attend(lens, 4, 1, 64, "bf16", 4, page=16)


def test_reads_more_sequences_than_a_launch_holds():
    c = cache(1, 1, 64, "fp16", 8, 40, seqs=260, page=16)
    ids = [c.seq_create() for _ in range(260)]
    k, v = rows(1, 260, 33, 1, 64, "fp16"), rows(2, 260, 33, 1, 64, "fp16")
    c.kv_append(ids, k, v)
    gk, gv = c.kv_read(ids)
    check_held(gk, k, 8)
    check_held(gv, v, 8)
    c.check_status()


@pytest.mark.parametrize("bits", [8, 4])
def test_attend_scores_in_rising_and_falling_order(bits):
    """The reference of the weights moves with every tile, or never again."""
    for sign in (1.0, -1.0):
        def kv(i, L):
            ramp = torch.linspace(-1, 1, L, device="cuda")[None, :, None, None] * sign
            k = (ramp * 8 + normal(5, 1, L, 1, 128) * 0.1).bfloat16()
            return k, rows(6, 1, L, 1, 128, "bf16")
        check_attend([900], 4, 1, 128, "bf16", bits, out="fp32", kv=kv, scale=0.2)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bits", [8, 4])
def test_attend_values_of_every_size(dtype, bits):
    """Steps that differ by many powers of two between tokens, groups of zeros, constant rows."""
    def kv(i, L):
        v = normal(7, 1, L, 2, 128)
        v *= torch.exp2((torch.arange(L, device="cuda") * 5 % 23 - 11).float())[None, :, None, None]
        v[:, 3] = 0.0
        v[:, 5, :, 32:64] = 1.5
        k = normal(8, 1, L, 2, 128)
        k[:, 4] = 0.0
        k[:, 9] = 2.0
        return k.to(DT[dtype]), v.to(DT[dtype])
    check_attend([150], 4, 2, 128, dtype, bits, out="fp32", kv=kv)

    def same(i, L):  # every value the same, and none but zeros
        return (torch.full((1, L, 2, 128), x, device="cuda").to(DT[dtype]) for x in (0.5, i * 1.25))
    check_attend([40, 33], 4, 2, 128, dtype, bits, out="fp32", kv=same)


@pytest.mark.parametrize("gain", [0.0, 1e-6, 1e4, 3e4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attend_queries_of_every_size(gain, dtype):
    # (3e4 is beyond fp16 for some: what an infinite query asks for is NaN)
    scale = 1e-5 if gain > 1 else 0.0
    check_attend([90], 4, 1, 64, dtype, 8, out="fp32", gain=gain, scale=scale)
    check_attend([90], 8, 1, 128, dtype, 4, gain=gain, scale=scale)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rule", [dict(), dict(softcap=9.0), dict(slopes=True)])
def test_attend_queries_and_keys_at_the_ends_of_the_range(bits, rule):
    """Scores of ordinary size from queries near 2^110 (whose factor comes in two) and keys near
    2^-110, and the other way round."""
    for up in (2.0 ** 110, 2.0 ** -110):
        def kv(i, L):
            return (rows(11, 1, L, 1, 128, "bf16").double() / up).bfloat16(), rows(12, 1, L, 1, 128, "bf16")
        check_attend([70], 4, 1, 128, "bf16", bits, out="fp32", kv=kv, gain=up, **rule)


def test_attend_what_is_not_finite():
    """NaN in an attended key reaches its heads, in an attended value its group; outside the
    window neither reaches anything."""
    L, hkv, d = 100, 2, 128
    k, v = rows(1, 1, L, hkv, d, "bf16"), rows(2, 1, L, hkv, d, "bf16")
    k[0, 10, 0, 5] = math.nan
    v[0, 20, 1, 40] = math.inf
    c = cache(4, hkv, d, "bf16", 4, L)
    s = c.seq_create()
    c.kv_append([s], k, v)
    q = normal(3, 1, 4, d, dtype=torch.bfloat16)
    out = c.quant_decode_attention(q, [s])[0]
    assert bool(out[:2].isnan().all())
    assert bool(out[2:, 32:64].isnan().all())
    assert bool(out[2:, :32].isfinite().all()) and bool(out[2:, 64:].isfinite().all())
    for window in (79, 64, 70):
        got = c.quant_decode_attention(q, [s], window=window)[0]
        ref, tol = attend(q[0], k[0], v[0], 4, L - window)
        within(got, ref, tol(F32))
    c.check_status()


def test_attend_leaves_rows_behind_alone():
    c, ids, q, got = check_attend([40, 9], 4, 2, 64, "bf16", 8, out="fp32")
    out = torch.full((5, 4, 64), 7.0, device="cuda")
    c.quant_decode_attention(q, ids, out=out[:2])
    assert torch.equal(out[:2], got) and bool((out[2:] == 7).all())
    one = c.quant_decode_attention(q[1:], ids[1:])
    assert torch.equal(one[0], got[1])


# ---- together ---------------------------------------------------------------------

@pytest.mark.parametrize("bits", [8, 4])
def test_a_prompt_in_chunks_and_steps(bits):
    """As a server uses them: chunks are rotated into the cache, each attends what the cache
    holds of the prompt so far; then tokens one by one, one of them taken back."""
    hq, hkv, d, dt = 8, 2, 128, torch.bfloat16
    t = spd.Rotary(d, sections=[24, 20, 20], axes_in_turn=True)
    c = cache(hq, hkv, d, "bf16", bits, 400)
    s = c.seq_create()
    total, pos = 300, places(9, 3, 1, 320, hi=500)
    q, k, v = (normal(i, 1, 320, h, d, dtype=dt) for i, h in ((1, hq), (2, hkv), (3, hkv)))
    rk = turn(k[0], pos[:, 0], frequencies(d), axes_of([24, 20, 20], True))[0].to(dt)
    at = 0
    for n in (130, 1, 169):
        sl = slice(at, at + n)
        gq = c.kv_append_rotary([s], t, q[:, sl], k[:, sl], v[:, sl],
                                positions=pos[:, :, sl].contiguous())
        kk, vv = c.kv_read([s])
        out = spd.prefill_attention(gq[0], kk[0], vv[0])
        at += n
        # the last query of the chunk against the step's kernel: same cache, same query; both
        # are within their own tolerances of the values read back, rounded to bf16 by kv_read
        ref, tol = attend(gq[0, -1], rk[:at], v[0, :at], bits)
        one = c.quant_decode_attention(gq[0, -1:], [s])
        # (a key that the library rounds the other way when it rotates may move a code by one:
        # half a bf16 step of it, in every score at most 2^-7 of |q||k|)
        e = 2 * float((gq[0, -1].double().abs().sum(-1)).max()) * 2.0 ** -7 * d ** -0.5
        slack = e * v[0, :at].double().abs().amax()
        within(one[0], ref, tol(F32) + slack)
        within(out[-1], ref, tol(dt) + slack + 2.0 ** -7 * v[0, :at].double().abs().amax())
    for i in range(total, 305):
        sl = slice(i, i + 1)
        gq = c.kv_append_rotary([s], t, q[:, sl], k[:, sl], v[:, sl],
                                positions=pos[:, :, sl].contiguous())
        got = c.quant_decode_attention(gq[:, 0], [s])
        kk, vv = c.kv_read([s])
        x = torch.einsum("hgd,thd->hgt", gq[0, 0].double().view(hkv, -1, d), kk[0].double()) * d ** -0.5
        ref = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), vv[0].double()).reshape(hq, d)
        # (kv_read rounds to bf16: 2^-8 of every key and value)
        mag = float(torch.einsum("hgd,thd->hgt", gq[0, 0].double().abs().view(hkv, -1, d),
                                 kk[0].double().abs()).max()) * d ** -0.5
        within(got[0], ref, (2.0 ** -8 + 2 * mag * 2.0 ** -8) * float(vv.abs().max()))
        if i == 302:
            c.seq_truncate(s, i)
            again = c.kv_append_rotary([s], t, q[:, sl], k[:, sl], v[:, sl],
                                       positions=pos[:, :, sl].contiguous())
            assert torch.equal(again, gq)
            assert torch.equal(c.quant_decode_attention(gq[:, 0], [s]), got)
    c.check_status()


def test_captured_and_replayed():
    """Rotation, write, read and attention in one graph: replays see new inputs."""
    hq, hkv, d, dt = 8, 2, 64, torch.float16
    t = spd.Rotary(d)
    c = cache(hq, hkv, d, "fp16", 4, 3000, seqs=2)
    ids = [c.seq_create() for _ in range(2)]
    for i, n in zip(ids, (2500, 41)):
        c.kv_append([i], rows(i, 1, n, hkv, d, "fp16"), rows(i + 5, 1, n, hkv, d, "fp16"))
    q, k, v = (normal(i, 2, 1, h, d, dtype=dt) for i, h in ((1, hq), (2, hkv), (3, hkv)))
    pos = places(4, 2, 1)

    def step():
        gq = c.kv_append_rotary(ids, t, q, k, v, positions=pos)
        out = c.quant_decode_attention(gq[:, 0], ids)
        kk, _ = c.kv_read(ids, -1)
        r = spd.rotary(t, pos[:, 0].contiguous(), k[:, 0].contiguous())
        for i, n in zip(ids, (2500, 41)):
            c.seq_truncate(i, n)
        return out, kk, r

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held_ = step()
    for seed in (10, 20):
        for x in (q, k, v):
            x.copy_(normal(seed, *x.shape, dtype=dt))
        pos.copy_(places(seed, 2, 1))
        graph.replay()
        graph.replay()
        got = [x.clone() for x in held_]
        want = step()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    c.check_status()


def test_calls_of_two_caches_and_a_16_bit_one_in_a_row():
    """Nothing of one call is still read or written by the next's."""
    a = check_attend([500, 3], 8, 2, 128, "bf16", 8)
    b = check_attend([64] * 9, 16, 2, 64, "fp16", 4)
    plain = spd.SparsePagedKVCache(device="cuda", num_q_heads=8, num_kv_heads=2, head_dim=128,
                                   dtype="bf16", logical_page=16, physical_page=64,
                                   num_physical_pages=20, max_seqs=2, max_context=600)
    s = plain.seq_create()
    plain.kv_append([s], rows(1, 1, 500, 2, 128, "bf16"), rows(2, 1, 500, 2, 128, "bf16"))
    want = plain.shared_prefix_attention(a[2][:1], None, [s])
    for _ in range(5):
        x = a[0].quant_decode_attention(a[2], a[1], out_dtype=torch.bfloat16)
        y = plain.shared_prefix_attention(a[2][:1], None, [s])
        z = b[0].quant_decode_attention(b[2], b[1], out_dtype=torch.float16)
        assert torch.equal(x, a[3]) and torch.equal(y, want) and torch.equal(z, b[3])


def test_calls_on_a_stream_of_their_own():
    side = torch.cuda.Stream()
    c = cache(4, 2, 64, "bf16", 8, 100)
    s, t = c.seq_create(), spd.Rotary(64)
    q, k, v = (normal(i, 1, 90, h, 64, dtype=torch.bfloat16) for i, h in ((1, 4), (2, 2), (3, 2)))
    side.wait_stream(torch.cuda.current_stream())
    gq = c.kv_append_rotary([s], t, q, k, v, stream=side)
    out = c.quant_decode_attention(gq[0, -1:], [s], stream=side)
    kk, vv = c.kv_read([s], stream=side)
    r = spd.rotary(t, torch.arange(90, device="cuda", dtype=torch.int32), q[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(gq[0], r)
    rk = spd.rotary(t, torch.arange(90, device="cuda", dtype=torch.int32), k[0])
    check_held(kk[0], rk, 8)
    ref, tol = attend(gq[0, -1], rk, v[0], 8)
    within(out[0], ref, tol(F32))
    c.check_status(side)


def test_a_pool_beyond_4_gb():
    """Tiles on pages whose bytes lie beyond 2^32 (and whose tiles beyond 2^31 codes)."""
    page, pages = 4096, 140
    c = spd.SparsePagedKVCache(device="cuda", num_q_heads=32, num_kv_heads=32, head_dim=128,
                               dtype="bf16", logical_page=16, physical_page=page,
                               num_physical_pages=pages, max_seqs=3, max_context=page * pages,
                               kv_quant=8)
    assert c.sizes["k_pool"] > 1 << 32
    s = c.seq_create()
    c.seq_reserve(s, (pages - 1) * page)
    far = c.seq_create()
    k, v = rows(1, 1, 70, 32, 128, "bf16"), rows(2, 1, 70, 32, 128, "bf16")
    c.kv_append([far], k, v)
    assert c.page_table(far) == [pages - 1]
    gk, gv = c.kv_read([far])
    check_held(gk, k, 8)
    check_held(gv, v, 8)
    q = normal(3, 1, 32, 128, dtype=torch.bfloat16)
    ref, tol = attend(q[0], k[0], v[0], 8)
    within(c.quant_decode_attention(q, [far])[0], ref, tol(F32))
    c.check_status()


def test_gpu_refusals():
    c = cache(4, 2, 64, "bf16", 8, 100)
    s, t = c.seq_create(), spd.Rotary(64)
    k = normal(1, 1, 3, 2, 64, dtype=torch.bfloat16)
    q = normal(1, 1, 3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(spd.SpdError):
        c.quant_decode_attention(q[:, 0].contiguous(), [s])
    c.kv_append([s], k, k)
    for bad in (dict(positions=torch.zeros(1, 2, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(1, 3, device="cuda")),
                dict(positions=torch.zeros(1, 3, dtype=torch.int32)),
                dict(out=torch.empty(1, 3, 4, 64, device="cuda"))):
        with pytest.raises(ValueError):
            c.kv_append_rotary([s], t, q, k, k, **bad)
    with pytest.raises(ValueError):
        c.kv_append_rotary([s], t, q.half(), k, k)
    with pytest.raises(ValueError):
        c.kv_append_rotary([s], t, q[:, :2], k, k)
    with pytest.raises(spd.SpdError):
        c.kv_append_rotary([s], spd.Rotary(128), q, k, k)
    for bad in (dict(out_dtype=torch.float16), dict(window=-1), dict(softcap=-1.0),
                dict(slopes=torch.zeros(3, device="cuda"))):
        with pytest.raises((ValueError, spd.SpdError)):
            c.quant_decode_attention(q[:, 0].contiguous(), [s], **bad)
    for bad in (dict(positions=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(3, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            spd.rotary(t, q=q[0], **bad)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        spd.rotary(t, pos, q[0], k[0].half())
    with pytest.raises(ValueError):
        spd.rotary(t, pos, q[0].transpose(1, 2))
    with pytest.raises(ValueError):
        spd.rotary(t, pos, q[0], out=q[0, :2])
    assert c.seq_info(s)["length"] == 3
