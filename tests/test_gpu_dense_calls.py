"""Calls of the dense operators as programs make them: beside one another on
streams, on uneven key intervals, with operands that share a warp or a batch
with others; against the 64-bit implementations of dense_ref.py or against the
same call alone."""
import math

import pytest
import torch

import sparse_paged_decode_logical_gb300 as spd
from dense_ref import attend, prompt, tolerance
from test_gpu_dense import DT, check_shared, new_cache, normal

pytestmark = pytest.mark.gpu


# ---- streams ---------------------------------------------------------------------

def test_cut_prompts_on_two_streams_at_once():
    """Both calls have a workspace of the same size, and their buffers are given
    back and taken again while they run."""
    hq, hkv, d, lk = 16, 8, 128, 20000
    k, v = (normal(i, lk, hkv, d, dtype=torch.bfloat16) for i in (1, 2))
    qs = [normal(10 + i, 40, hq, d, dtype=torch.bfloat16) for i in range(12)]
    want = [spd.prefill_attention(q, k, v, check=True) for q in qs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got, fill = [], []
        for i, q in enumerate(qs):
            got.append(spd.prefill_attention(q, k, v, stream=stream if i % 2 else None))
            # blocks of the workspace's and the output's sizes, written at once
            for n in (want[0].numel() * 4, 1 << 21, 1 << 22, 1 << 23):
                fill.append(torch.full((n // 4,), 7.0, device="cuda"))
            if i % 3 == 2:
                fill.clear()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_cache_calls_on_a_stream_beside_other_work():
    """The cache's calls all on one stream, the caller's stream busy with memory of
    its own; results read there after a wait and given back at once."""
    hq, hkv, d, dt = 8, 2, 128, torch.bfloat16
    c = new_cache(hq, hkv, d, "bf16", 64, 16, 300, 40, 6000)
    doc = c.seq_create()
    c.kv_append([doc], normal(1, 1, 5000, hkv, d, dtype=dt), normal(2, 1, 5000, hkv, d, dtype=dt))
    ids = [c.seq_create() for _ in range(9)]
    c.kv_append(ids, normal(3, 9, 30, hkv, d, dtype=dt), normal(4, 9, 30, hkv, d, dtype=dt))
    q = normal(5, 9, hq, d, dtype=dt)
    w = normal(6, 9, hkv, 30).abs()
    want = c.shared_prefix_attention(q, doc, ids)
    dst = [c.seq_create() for _ in ids]
    kept = c.kv_evict(ids, dst, 12, 3, w)
    kept = kept[0].clone(), kept[1].clone()
    for i in reversed(dst):
        c.seq_free(i)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    here = torch.cuda.current_stream()
    sums = []
    for _ in range(20):
        busy = torch.full((want.numel(),), 3.0, device="cuda") * 2
        x = c.shared_prefix_attention(q, doc, ids, stream=s)
        dst = [c.seq_create() for _ in ids]
        a, b = c.kv_evict(ids, dst, 12, 3, w, stream=s)
        for i in reversed(dst):
            c.seq_free(i)
        here.wait_stream(s)
        sums.append((x - want).abs().max() + (a - kept[0]).abs().max() + (b - kept[1]).abs().max()
                    + (busy - 6).abs().max())
        del x, a, b, busy
    assert float(torch.stack(sums).max()) == 0.0
    c.check_status(stream=s)
    off = torch.tensor([0, 5, 70, 83], dtype=torch.int32, device="cuda")
    b0, e0 = spd.document_key_ranges(off, 90)
    torch.cuda.synchronize()
    b1, e1 = spd.document_key_ranges(off, 90, stream=s)
    here.wait_stream(s)
    assert torch.equal(b0, b1) and torch.equal(e0, e1)


def test_calls_on_a_stream_inside_a_capture_and_on_the_default_stream():
    hq, hkv, d, lk = 16, 8, 128, 20000
    k, v = (normal(i, lk, hkv, d, dtype=torch.bfloat16) for i in (1, 2))
    q, q2 = normal(3, 40, hq, d, dtype=torch.bfloat16), normal(4, 40, hq, d, dtype=torch.bfloat16)
    want = [spd.prefill_attention(x, k, v, check=True) for x in (q, q2)]
    torch.cuda.synchronize()
    got = spd.prefill_attention(q, k, v, stream=0)  # the legacy default stream
    torch.cuda.synchronize()
    assert torch.equal(got, want[0])
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        s.wait_stream(here)
        a = spd.prefill_attention(q, k, v, stream=s)
        b = spd.prefill_attention(q2, k, v)  # beside it: neither has the other's workspace
        c = spd.prefill_attention(q2, k, v, stream=s)
        here.wait_stream(s)
    for _ in range(3):
        for x in (a, b, c):
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, want[1])


# ---- key intervals of one tile's rows far apart ------------------------------------

@pytest.mark.parametrize("near,far", [(64, 40), (700, 1500), (1, 1), (5000, 9000)])
@pytest.mark.parametrize("hq,hkv,d,dtype,out", [(1, 1, 64, "fp16", "same"), (2, 1, 128, "bf16", "fp32"),
                                                (3, 3, 128, "fp16", "fp32"), (2, 2, 64, "bf16", "same")])
@pytest.mark.parametrize("slopes", [False, True])
def test_prompt_rows_that_attend_the_first_keys_beside_rows_that_attend_the_last(near, far, hq, hkv, d,
                                                                                 dtype, out, slopes):
    """Cut prompts with whole cuts between the keys of a tile's two halves; in the
    last rows the halves come the other way round, with rows that attend nothing."""
    lq, lk, dt = 700, 40000, DT[dtype]
    q, k, v = normal(1, lq, hq, d, dtype=dt), normal(2, lk, hkv, d, dtype=dt), normal(3, lk, hkv, d, dtype=dt)
    half = 128 // math.gcd(hq // hkv, 8)
    at = torch.arange(lq, device="cuda")
    first = (at // half % 2 == 0) ^ (at >= 4 * half)
    b = torch.where(first, 0, lk - far)
    e = torch.where(first, near, lk)
    e = torch.where(at % 97 == 5, b, e)
    sl = torch.linspace(0.001, 0.2, hq, device="cuda") if slopes else None
    od = torch.float32 if out == "fp32" else dt
    got = spd.prefill_attention(q, k, v, key_begin=b.int(), key_end=e.int(), slopes=sl, out_dtype=od,
                                check=True)
    ref, ab, mag = prompt(q, k, v, b, e, d ** -0.5, 0.0, sl)
    assert bool(((got.double() - ref).abs() <=
                 tolerance(ref, ab, mag, d, max(near, far, 1025), dt, od, 0.0)).all())
    assert bool((got[b >= e] == 0).all())


# ---- precision ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,d", [(2, 128), (9, 128), (20, 128), (20, 64), (70, 128)])
def test_fp32_outputs_hold_the_weights_over_a_long_prefix(n, d, dtype):
    """As test_fp32_outputs_hold_the_weights_to_22_bits (which derives the bound), where
    a CTA meets more keys than in prompts whose bf16 weights take a third part."""
    dt, lp, hq, hkv = DT[dtype], 60000, 16, 8
    at = torch.randperm(lp, generator=torch.Generator().manual_seed(3))[:16].cuda()
    q = torch.zeros(n, hq, d, device="cuda", dtype=dt)
    q[..., 0], q[..., 1] = normal(1, n, hq).abs().clamp_max(2).to(dt), 1
    k = torch.zeros(lp, hkv, d, device="cuda", dtype=dt)
    k[..., 1] = -1000
    k[at, :, 0], k[at, :, 1] = normal(2, 16, hkv).clamp(-1, 1).to(dt), 0
    v = torch.zeros(lp, hkv, d, device="cuda", dtype=dt)
    v[at, :, torch.arange(16, device="cuda")] = 1
    c = new_cache(hq, hkv, d, dtype, 1024, 16, 59 + n, n + 1, lp)
    pid, ids = c.seq_create(), [c.seq_create() for _ in range(n)]
    c.kv_append([pid], k[None], v[None])
    own = torch.zeros(n, 3, hkv, d, device="cuda", dtype=dt)
    own[..., 1] = -1000
    c.kv_append(ids, own, torch.zeros_like(own))
    got = c.shared_prefix_attention(q, pid, ids, scale=1.0)
    c.check_status()
    x = torch.einsum("rhg,thg->rht", q[..., :1].double(),
                     k[at, :, :1].double().repeat_interleave(hq // hkv, 1))
    want = torch.softmax(x, -1)
    assert float(((got[..., :16].double() - want) / want).abs().max()) < 3.2e-6
    assert bool((got[..., 16:] == 0).all())


@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("n", [5, 20, 40, 200])
def test_kept_weights_over_a_capped_prefix_show_no_rough_cap(n, slopes, out):
    """Every key of the prefix has one score s per query, |s| < 2, an exact product of
    two numbers, the own tokens' scores are 0, and the cap is 170: a form that is off
    by 2^-22 of the cap (1.9e-5 here) shows in every own token's weight,
    1 / (own + Lp e^x).  Allowed, relative: scores 2 x 4 x 2^-24 |s| = 16 x 2^-24, their
    exponents (|x| < 3 in base 2) 6 x 2^-24, 2^x 2 x 2^-22, sums of a thread's 15 equal
    weights, of up to 30 blocks and 19 splits 64 x 2^-24, joins, quotient and product
    8 x 2^-24: 102 x 2^-24 = 6.1e-6."""
    d, lp, own, cap, dt = 128, 4500, 3, 170.0, torch.bfloat16
    c = new_cache(1, 1, d, "bf16", 256, 16, 18 + n + 1, n + 1, 4600)
    k = torch.zeros(lp, 1, d, dtype=dt, device="cuda")
    k[..., 0] = 1.0
    v = normal(2, lp, 1, d, dtype=dt)
    pid, ids = c.seq_create(), [c.seq_create() for _ in range(n)]
    c.kv_append([pid], k[None], v[None])
    c.kv_append(ids, torch.zeros(n, own, 1, d, dtype=dt, device="cuda"),
                normal(3, n, own, 1, d, dtype=dt))
    q = torch.zeros(n, 1, d, dtype=dt, device="cuda")
    q[:, 0, 0] = (torch.rand(n, device="cuda", generator=torch.Generator("cuda").manual_seed(4)) * 4 - 2).to(dt)
    w = torch.zeros(n, 1, own, device="cuda")
    c.shared_prefix_attention(q, pid, ids, scale=1.0, softcap=cap, weights_out=w,
                              slopes=torch.zeros(1, device="cuda") if slopes else None,
                              out_dtype=torch.float32 if out == "fp32" else dt)
    c.check_status()
    x = cap * torch.tanh(q[:, 0, 0].double() / cap)
    want = 1.0 / (own + lp * x.exp())
    assert float(((w[:, 0].double() - want[:, None]) / want[:, None]).abs().max()) < 102 * 2.0 ** -24


# ---- rows that attend nothing --------------------------------------------------------

@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("softcap", [30.0, 300.0])
@pytest.mark.parametrize("lq,lk,hq,hkv", [(300, 300, 4, 2), (300, 300, 8, 1), (60, 3000, 4, 2)])
def test_queries_that_attend_nothing_have_no_say(lq, lk, hq, hkv, d, dtype, out, softcap):
    """Not even in the last bits: padding rows between others hold small numbers, large
    ones or none at all."""
    dt = DT[dtype]
    q, k, v = normal(1, lq, hq, d, dtype=dt, gain=3.0), normal(2, lk, hkv, d, dtype=dt), \
        normal(3, lk, hkv, d, dtype=dt)
    pad = torch.arange(lq, device="cuda") % 7 == 2
    b = torch.zeros(lq, dtype=torch.int32, device="cuda")
    e = torch.where(pad, 0, lk).int()
    got = []
    for what in (1e-3, 300.0, -300.0, math.nan, math.inf):
        q[pad] = what
        got.append(spd.prefill_attention(q, k, v, key_begin=b, key_end=e, softcap=softcap, check=True,
                                         out_dtype=torch.float32 if out == "fp32" else dt))
    for x in got:
        assert torch.equal(x, got[0]) and bool((x[pad] == 0).all())


# ---- a prompt call between a context's own calls -----------------------------------

@pytest.mark.parametrize("lq,lk", [(6, 6), (6, 30000), (6000, 6000)])
def test_early_staging_waits_for_a_prompt_call_in_between(lq, lk):
    """Selection, then a prompt whose output is the decode call's q: streaming heads, which
    may run without a wait behind their context's own selection, have to wait here."""
    hq, hkv, d, dt, n = 8, 2, 128, torch.bfloat16, 6
    c = new_cache(hq, hkv, d, "bf16", 64, 16, 200, n, 2048, streaming=[True, False], sink=16, window=256,
                  token_budget=256)
    ids = [c.seq_create() for _ in range(n)]
    c.kv_append(ids, normal(1, n, 900, hkv, d, dtype=dt), normal(2, n, 900, hkv, d, dtype=dt))
    q0 = normal(3, n, hq, d, dtype=dt)
    k, v = normal(4, lk, hkv, d, dtype=dt), normal(5, lk, hkv, d, dtype=dt)
    qs = [normal(10 + i, lq, hq, d, dtype=dt) for i in range(6)]
    q = torch.zeros(lq, hq, d, dtype=dt, device="cuda")

    def chain(wait):
        outs = []
        for x in qs:
            c.select_pages(q0, ids, force=True)
            spd.prefill_attention(x, k, v, out_dtype=dt, out=q)
            if wait:
                torch.cuda.synchronize()
            outs.append(c.sparse_decode_attention(q[-n:], ids))
        return outs

    want = chain(True)
    c.set_early_kv_staging(True)
    for _ in range(5):
        q.zero_()
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)
    c.check_status()


# ---- distances beyond fp32's integers ---------------------------------------------

@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("lq", [3, 300])
def test_distance_bias_of_keys_far_from_the_query(lq, out):
    """Queries behind 34 million keys (distances of 2^25, where fp32's integers are 4
    apart), that attend a few of the first ones."""
    lk, hq, hkv, d, dt = 34_000_003, 4, 1, 64, torch.float16
    k = torch.zeros(lk, hkv, d, dtype=dt, device="cuda")
    v = torch.zeros(lk, hkv, d, dtype=dt, device="cuda")
    q = normal(1, lq, hq, d, dtype=dt)
    sl = torch.tensor([0.01, 0.3, 1.0, 2.0], device="cuda")
    od = torch.float32 if out == "fp32" else dt
    at = torch.arange(lk - lq, lk, device="cuda")
    for a, n in ((0, 90), (77, 500), (lk - (1 << 25) - 250, 500)):
        k[a:a + n], v[a:a + n] = normal(2, n, hkv, d, dtype=dt), normal(3, n, hkv, d, dtype=dt)
        b, e = torch.full((lq,), a, device="cuda"), torch.full((lq,), a + n, device="cuda")
        e[1::3] -= 7
        got = spd.prefill_attention(q, k, v, key_begin=b.int(), key_end=e.int(), slopes=sl, out_dtype=od,
                                    check=True)
        # the same with the queries right behind their keys: one bias less for a whole row
        ref = torch.zeros(lq, hq, d, dtype=torch.float64, device="cuda")
        t = torch.arange(a, a + n, device="cuda")
        seen = (t >= b[:, None]) & (t < e[:, None])
        far = (at[:, None] - t).double() - (at - e + 1)[:, None].double()
        ab, mag = torch.zeros(2, lq, hq, d, dtype=torch.float64, device="cuda"), 0.0
        for h in range(hq):
            o, x, _, m = attend(q[:, h], k[a:a + n, 0], v[a:a + n, 0], h, far, seen, d ** -0.5, 0.0, sl)
            ref[:, h], ab[:, :, h], mag = o, x, max(mag, m)
        tol = tolerance(ref, ab, mag, d, n, dt, od, 0.0)
        assert bool(((got.double() - ref).abs() <= tol).all())
