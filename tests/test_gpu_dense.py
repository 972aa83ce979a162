"""Dense attention with score rules, shared prefixes and eviction against the
64-bit implementations in dense_ref.py (which also derives the tolerances)."""
import math

import pytest
import torch

import sparse_paged_decode_logical_gb300 as spd
from dense_ref import kept_positions, prompt, shared, tolerance

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def normal(seed, *shape, dtype=torch.float32, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * gain).to(dtype)


def intervals(kind, lq, lk, seed=3):
    """key_begin, key_end int32 [lq] of a kind of mask."""
    at = torch.arange(lk - lq, lk)
    if kind == "causal":
        b, e = torch.zeros(lq), at + 1
    elif kind == "window":
        b, e = (at - 40).clamp_min(0), at + 1
    elif kind == "all":
        b, e = torch.zeros(lq), torch.full((lq,), lk)
    elif kind == "prefix":
        b, e = torch.zeros(lq), (at + 1).clamp_min(min(lk, 70))
    elif kind == "random":  # in no order, some empty or reversed, some outside the keys
        g = torch.Generator().manual_seed(seed)
        b = torch.randint(-9, lk + 9, (lq,), generator=g)
        e = b + torch.randint(-20, max(lk // 2, 30), (lq,), generator=g)
    elif kind == "empty":
        b, e = torch.zeros(lq), torch.zeros(lq)
    elif kind == "far":  # the nearest key lies far back
        b, e = torch.zeros(lq), torch.full((lq,), min(lk, 90))
    return b.int().cuda(), e.int().cuda()


def check_prompt(lq, lk, hq, hkv, d, dtype, out="fp32", softcap=0.0, slopes=False, mask=None,
                 scale=0.0, seed=1, gain=1.0):
    dt = DT[dtype]
    q, k, v = normal(seed, lq, hq, d, dtype=dt, gain=gain), normal(seed + 1, lk, hkv, d, dtype=dt), \
        normal(seed + 2, lk, hkv, d, dtype=dt)
    sl = torch.rand(hq, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) \
        * 0.5 if slopes else None
    od = torch.float32 if out == "fp32" else dt
    b, e = intervals(mask or "causal", lq, lk, seed)
    got = spd.prefill_attention(q, k, v, key_begin=b if mask else None, key_end=e if mask else None,
                                scale=scale, softcap=softcap, slopes=sl, out_dtype=od, check=True)
    assert got.dtype == od and got.shape == (lq, hq, d)
    ref, ab, mag = prompt(q, k, v, b.clamp(0, lk), e.clamp(0, lk), scale or d ** -0.5, softcap, sl)
    tol = tolerance(ref, ab, mag, d, lk, dt, od, softcap)
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    nothing = b.clamp(0, lk) >= e.clamp(0, lk)
    assert bool((got[nothing] == 0).all())


@pytest.mark.parametrize("lq,lk", [(1, 1), (1, 63), (1, 700), (5, 5), (63, 64), (64, 65), (65, 129),
                                   (127, 127), (128, 500), (129, 129), (300, 300), (31, 2100),
                                   (257, 1025)])
@pytest.mark.parametrize("heads", [(8, 2), (4, 4)])
def test_prompt_lengths(lq, lk, heads):
    check_prompt(lq, lk, *heads, 128, "bf16")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 5), (12, 2), (16, 2), (32, 2), (14, 1), (8, 8)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,out", [("bf16", "same"), ("fp16", "same"), ("fp16", "fp32"),
                                       ("bf16", "fp32")])
def test_prompt_heads_and_types(hq, hkv, d, dtype, out):
    check_prompt(150, 210, hq, hkv, d, dtype, out)


@pytest.mark.parametrize("mask", ["window", "all", "prefix", "random", "empty", "far"])
@pytest.mark.parametrize("rule", [dict(), dict(softcap=20.0, gain=5.0), dict(slopes=True),
                                  dict(softcap=50.0, slopes=True, scale=0.2)])
@pytest.mark.parametrize("lq,lk,heads", [(200, 200, (4, 1)), (40, 900, (2, 2)), (333, 333, (3, 3)),
                                         (700, 700, (6, 3))])
def test_prompt_masks_and_rules(mask, rule, lq, lk, heads):
    check_prompt(lq, lk, *heads, 64, "fp16", mask=mask, **rule)
    check_prompt(lq, lk, *heads, 128, "bf16", out="same", mask=mask, **rule)


@pytest.mark.parametrize("mask", [None, "random", "window", "far"])
@pytest.mark.parametrize("lq,lk,heads,d,dtype,out,rule", [
    (2600, 2600, (8, 8), 128, "bf16", "same", dict()),
    (2600, 2600, (8, 8), 64, "fp16", "fp32", dict(slopes=True)),
    (3300, 3300, (4, 2), 128, "fp16", "same", dict(softcap=30.0)),
    (600, 3000, (16, 4), 128, "bf16", "fp32", dict()),
])
def test_prompts_cut_along_the_keys(mask, lq, lk, heads, d, dtype, out, rule):
    """Uneven causal tiles and rows that some cuts hold no key of."""
    check_prompt(lq, lk, *heads, d, dtype, out=out, mask=mask, **rule)


def test_prompt_large_scores_saturate_the_cap():
    check_prompt(90, 90, 4, 2, 128, "bf16", softcap=5.0, gain=300.0)
    check_prompt(90, 90, 4, 2, 128, "bf16", gain=60.0)


@pytest.mark.parametrize("softcap", [1e-6, 1e-3, 300.0, 2e4, 1e6])
@pytest.mark.parametrize("out", ["same", "fp32"])
def test_caps_of_every_size(softcap, out):
    check_prompt(70, 70, 4, 2, 128, "bf16", out=out, softcap=softcap, gain=20.0)
    check_prompt(70, 70, 4, 2, 64, "fp16", out=out, softcap=softcap, slopes=True)
    for n in (2, 4, 20):
        check_shared(n, 150, [9] * n, 8, 2, 128, "fp16", out=out, softcap=softcap, weights=True)


def test_prompt_more_queries_than_keys():
    # queries that stand before the first key attend nothing
    check_prompt(200, 120, 4, 2, 64, "bf16")


def test_prompt_reads_strided_rows():
    hq, hkv, d, n = 8, 2, 128, 300
    row = normal(5, n, (hq + 2 * hkv) * d + 24, dtype=torch.bfloat16)
    q = row[:, :hq * d].unflatten(1, (hq, d))
    k = row[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = row[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    a = spd.prefill_attention(q, k, v, check=True)
    b = spd.prefill_attention(q.contiguous(), k.contiguous(), v.contiguous(), check=True)
    assert torch.equal(a, b)
    one = spd.prefill_attention(q[-1:], k, v, check=True)
    ref, ab, mag = prompt(q[-1:], k, v, torch.zeros(1, device="cuda"),
                          torch.full((1,), n, device="cuda"), d ** -0.5, 0.0, None)
    assert bool(((one.double() - ref).abs() <=
                 tolerance(ref, ab, mag, d, n, torch.bfloat16, torch.float32, 0.0)).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lq,lk", [(300, 300), (20, 1200)])
def test_prompt_unattended_values_that_are_not_finite(bad, lq, lk):
    """Keys and values outside a query's interval never reach it; inside, they
    make it not finite."""
    hq, hkv, d = 4, 2, 128
    q, k, v = normal(1, lq, hq, d, dtype=torch.bfloat16), normal(2, lk, hkv, d, dtype=torch.bfloat16), \
        normal(3, lk, hkv, d, dtype=torch.bfloat16)
    at = torch.arange(lk - lq, lk, device="cuda")
    b = torch.full((lq,), 13, dtype=torch.int32, device="cuda")
    e = torch.minimum(at + 1, torch.tensor(lk - 5, device="cuda")).int()
    clean = spd.prefill_attention(q, k, v, key_begin=b, key_end=e, check=True)
    k2, v2 = k.clone(), v.clone()
    k2[:13], v2[:13], k2[lk - 5:], v2[lk - 5:] = bad, bad, bad, bad
    got = spd.prefill_attention(q, k2, v2, key_begin=b, key_end=e, check=True)
    assert torch.equal(got, clean)
    t = lk - 10  # attended by the queries at or after it
    v2[t, 0, 7] = bad
    got = spd.prefill_attention(q, k2, v2, key_begin=b, key_end=e, check=True)
    hit = (at >= t).nonzero()[:, 0]
    assert not torch.isfinite(got[hit][:, :2, 7]).any()
    got[hit[0]:, :2, 7] = 0
    clean[hit[0]:, :2, 7] = 0
    assert torch.equal(got, clean)


def test_document_key_ranges():
    off = torch.tensor([0, 0, 5, 5, 70, 83], dtype=torch.int32, device="cuda")
    pre = torch.tensor([3, 2, 0, 100, 1], dtype=torch.int32, device="cuda")
    for prefix in (None, pre):
        kb, ke = spd.document_key_ranges(off, 90, prefix)
        for t in range(90):
            doc = [i for i in range(5) if off[i] <= t < off[i + 1]]
            if not doc:
                assert int(kb[t]) >= int(ke[t])
                continue
            a, z = int(off[doc[0]]), int(off[doc[0] + 1])
            seen = 0 if prefix is None else min(int(pre[doc[0]]), z - a)
            assert (int(kb[t]), int(ke[t])) == (a, max(t + 1, a + seen)), t
    # and the attention over them is each document's own
    q, k, v = (normal(i, 90, 4, 64, dtype=torch.float16) for i in (1, 2, 3))
    got = spd.prefill_attention(q, k, v, key_begin=kb, key_end=ke, check=True)
    assert bool((got[83:] == 0).all())
    alone = spd.prefill_attention(q[5:70], k[5:70], v[5:70], *intervals("all", 65, 65), check=True)
    assert (got[5:70] - alone).abs().max() < 1e-5


def test_prompt_on_another_stream_and_in_a_graph():
    q, k, v = (normal(i, 100, 4, 128, dtype=torch.bfloat16) for i in (1, 2, 3))
    ql = normal(4, 3, 4, 128, dtype=torch.bfloat16)
    kl, vl = normal(5, 3000, 4, 128, dtype=torch.bfloat16), normal(6, 3000, 4, 128, dtype=torch.bfloat16)
    a, b = spd.prefill_attention(q, k, v), spd.prefill_attention(ql, kl, vl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a2, b2 = spd.prefill_attention(q, k, v, stream=s), spd.prefill_attention(ql, kl, vl, stream=s)
    s.synchronize()
    assert torch.equal(a, a2) and torch.equal(b, b2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a3, b3 = spd.prefill_attention(q, k, v), spd.prefill_attention(ql, kl, vl)
    want = spd.prefill_attention(k, q, v), spd.prefill_attention(ql.neg(), kl, vl)
    x, ql0 = q.clone(), ql.clone()
    q.copy_(k)
    k.copy_(x)
    ql.copy_(ql0.neg())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a3, want[0]) and torch.equal(b3, want[1])


# ---- shared prefix --------------------------------------------------------------

def new_cache(hq, hkv, d, dtype, page, logical, pages, seqs, longest, **kw):
    c = spd.SparsePagedKVCache(device="cuda", num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                               dtype=dtype, logical_page=logical, physical_page=page,
                               num_physical_pages=pages, max_seqs=seqs, max_context=longest, **kw)
    for f in ("k_pool", "v_pool"):  # rows that hold no token are NaN
        if kw.get("kv_fp8"):
            c.buffers[f].fill_(0x7f)
        else:
            c.buffers[f].view(DT[dtype]).fill_(math.nan)
    return c


def check_shared(n, lp, lens, hq, hkv, d, dtype, page=64, logical=16, out="fp32", softcap=0.0,
                 slopes=False, weights=False, scale=0.0, seed=1, gain=1.0):
    dt = DT[dtype]
    need = -(-lp // page) + sum(-(-x // page) for x in lens) + 1
    c = new_cache(hq, hkv, d, dtype, page, logical, need, n + 1, max([lp, *lens, 1]),
                  free_list_seed=7)
    kp, vp = normal(seed, lp, hkv, d, dtype=dt), normal(seed + 1, lp, hkv, d, dtype=dt)
    ids = [c.seq_create() for _ in lens]
    pid = None
    if lp:
        pid = c.seq_create()
        c.kv_append([pid], kp[None], vp[None])
    ko = [normal(seed + 10 + 2 * i, x, hkv, d, dtype=dt) for i, x in enumerate(lens)]
    vo = [normal(seed + 11 + 2 * i, x, hkv, d, dtype=dt) for i, x in enumerate(lens)]
    for i, x in enumerate(lens):
        if x:
            c.kv_append([ids[i]], ko[i][None], vo[i][None])
    q = normal(seed + 5, n, hq, d, dtype=dt, gain=gain)
    sl = torch.linspace(0.01, 0.6, hq, device="cuda") if slopes else None
    stride = max(lens) + 3
    w_in = normal(seed + 6, n, hkv, stride).abs() if weights else None
    w_out = torch.full((n, hkv, stride), -7.0, device="cuda") if weights else None
    od = torch.float32 if out == "fp32" else dt
    before = [c.seq_info(i) for i in ids]
    got = c.shared_prefix_attention(q, pid, ids, scale=scale, softcap=softcap, slopes=sl,
                                    weights_in=w_in, weights_out=w_out, out_dtype=od)
    c.check_status()
    assert [c.seq_info(i) for i in ids] == before
    ref, ab, mag, ws = shared(q, kp, vp, ko, vo, scale or d ** -0.5, softcap, sl)
    tol = tolerance(ref, ab, mag, d, lp + max(lens), dt, od, softcap)
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    if weights:
        rel = 2 * (mag * d * 2.0 ** -24 + softcap * 2.0 ** -21) + (lp + max(lens)) * 2.0 ** -24 + 2.0 ** -20
        for i, x in enumerate(lens):
            want = w_in[i, :, :x].double() + ws[i]
            assert bool(((w_out[i, :, :x].double() - want).abs() <=
                         ws[i] * rel + want * 2.0 ** -23).all())
            assert bool((w_out[i, :, x:] == -7.0).all())
        # in place, and again from there
        w = w_in.clone()
        c.shared_prefix_attention(q, pid, ids, scale=scale, softcap=softcap, slopes=sl,
                                  weights_in=w, weights_out=w, out_dtype=od)
        for i, x in enumerate(lens):
            assert torch.equal(w[i, :, :x], w_out[i, :, :x])
            assert torch.equal(w[i, :, x:], w_in[i, :, x:])
    return c, q, pid, ids, got


@pytest.mark.parametrize("lp,lens", [(1, [1]), (1, [0]), (17, [0, 5, 16, 17]), (0, [1, 64, 65]),
                                     (64, [3]), (63, [1, 2, 3]), (1000, [130, 1, 0, 700]),
                                     (129, [0, 0, 0])])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (8, 1)])
def test_shared_few_rows(lp, lens, hq, hkv):
    check_shared(len(lens), lp, lens, hq, hkv, 128, "bf16", weights=max(lens) > 0)


@pytest.mark.parametrize("n,hq,hkv", [(5, 8, 2), (16, 8, 1), (17, 8, 1), (33, 4, 1), (128, 2, 2),
                                      (70, 4, 1)])
@pytest.mark.parametrize("lp", [5, 64, 500, 1537])
@pytest.mark.parametrize("page,logical", [(16, 16), (48, 16), (256, 64), (96, 32)])
def test_shared_many_rows(n, hq, hkv, lp, page, logical):
    g = torch.Generator().manual_seed(n + lp)
    lens = torch.randint(0, 90, (n,), generator=g).tolist()
    check_shared(n, lp, lens, hq, hkv, 64, "fp16", page=page, logical=logical, weights=n < 40)


@pytest.mark.parametrize("rule", [dict(softcap=30.0, gain=6.0), dict(slopes=True),
                                  dict(softcap=20.0, slopes=True, scale=0.3)])
@pytest.mark.parametrize("dtype,out,d", [("bf16", "fp32", 128), ("fp16", "same", 128),
                                         ("bf16", "same", 64)])
@pytest.mark.parametrize("n", [3, 20])
def test_shared_rules_and_types(rule, dtype, out, d, n):
    check_shared(n, 777, [11 * i % 200 for i in range(n)], 8, 2, d, dtype, out=out, weights=True,
                 **rule)


def test_shared_more_sequences_than_one_launch_takes():
    check_shared(1030, 300, [i % 7 for i in range(1030)], 1, 1, 64, "bf16", page=16)


def test_shared_long_own_tokens():
    check_shared(2, 0, [5000, 20001], 4, 1, 64, "bf16", page=512, weights=True)


@pytest.mark.parametrize("n,d", [(14, 128), (14, 64), (3, 128), (1, 128)])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("out", ["same", "fp32"])
def test_shared_results_do_not_depend_on_what_ran_before(n, d, softcap, out):
    """Rows behind the prefix's end are whatever shared memory held."""
    c, q, pid, ids, got = check_shared(n, 4937, [9] * n, 8, 1, d, "bf16", page=32, out=out,
                                       softcap=softcap, slopes=True)
    sl = torch.linspace(0.01, 0.6, 8, device="cuda")
    for gain in (1e-3, 1e4):
        k = normal(8, 20000, 8, d, dtype=torch.bfloat16, gain=gain)
        for rows in (1, 512):
            spd.prefill_attention(normal(9, rows, 8, d, dtype=torch.bfloat16), k, k, check=True)
        x = c.shared_prefix_attention(q, pid, ids, softcap=softcap, slopes=sl, out_dtype=got.dtype)
        assert torch.equal(x, got)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind,d", [("prompt", 64), ("prompt", 128), (2, 64), (2, 128), (5, 128),
                                    (20, 64), (20, 128)])
def test_fp32_outputs_hold_the_weights_to_22_bits(kind, d, dtype):
    """16 keys count, each with a channel of V of its own, so that an output is
    one weight.  Scores are exact products of two numbers, |x| < 3 in base 2: the
    exponent (x by a rounded constant, less at most 13 in magnitude) is off by
    2.9 x 2^-24 + 2^-21, e^ln2 of that 4.5e-7, 2^x by 2^-22, fp16's parts by 2^-22;
    numerator and sum 9.3e-7 each, the sum of 16 and the joins 20 x 2^-24, the
    division 2^-23: 3.2e-6.  (Two parts of bf16: 2^-18 = 3.8e-6 more.)"""
    dt = DT[dtype]
    n_keys, hq, hkv = 2000 if kind == "prompt" else 4500, 8, 2
    at = torch.randperm(n_keys, generator=torch.Generator().manual_seed(3))[:16].cuda()
    rows = 30 if kind == "prompt" else kind
    q = torch.zeros(rows, hq, d, device="cuda", dtype=dt)
    q[..., 0], q[..., 1] = normal(1, rows, hq).abs().clamp_max(2).to(dt), 1
    k = torch.zeros(n_keys, hkv, d, device="cuda", dtype=dt)
    k[..., 1] = -1000
    k[at, :, 0], k[at, :, 1] = normal(2, 16, hkv).clamp(-1, 1).to(dt), 0
    v = torch.zeros(n_keys, hkv, d, device="cuda", dtype=dt)
    v[at, :, torch.arange(16, device="cuda")] = 1
    if kind == "prompt":
        b, e = torch.zeros(rows, dtype=torch.int32, device="cuda"), \
            torch.full((rows,), n_keys, dtype=torch.int32, device="cuda")
        got = spd.prefill_attention(q, k, v, key_begin=b, key_end=e, scale=1.0, check=True,
                                    out_dtype=torch.float32)
    else:
        c = new_cache(hq, hkv, d, dtype, 256, 16, 18 + 2 * rows, rows + 1, 4600)
        pid, ids = c.seq_create(), [c.seq_create() for _ in range(rows)]
        c.kv_append([pid], k[None], v[None])
        own = torch.zeros(rows, 3, hkv, d, device="cuda", dtype=dt)
        own[..., 1] = -1000
        c.kv_append(ids, own, torch.zeros_like(own))
        got = c.shared_prefix_attention(q, pid, ids, scale=1.0, out_dtype=torch.float32)
        c.check_status()
    x = torch.einsum("rhg,thg->rht", q[..., :1].double(),
                     k[at, :, :1].double().repeat_interleave(hq // hkv, 1))
    want = torch.softmax(x, -1)
    assert float(((got[..., :16].double() - want) / want).abs().max()) < 3.2e-6
    assert bool((got[..., 16:] == 0).all())


def test_shared_streams_graph_and_another_workspace():
    c, q, pid, ids, got = check_shared(9, 400, [30] * 9, 8, 2, 128, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x = c.shared_prefix_attention(q, pid, ids, stream=s)
    s.synchronize()
    assert torch.equal(x, got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = c.shared_prefix_attention(q, pid, ids)
    want = c.shared_prefix_attention(q.neg(), pid, ids)
    q.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    c.check_status()


def test_shared_refuses_what_it_cannot_hold():
    c, q, pid, ids, _ = check_shared(3, 40, [5, 6, 7], 8, 2, 128, "bf16")
    w = torch.zeros(3, 2, 6, device="cuda")
    with pytest.raises(spd.SpdError) as e:
        c.shared_prefix_attention(q, pid, ids, weights_out=w)
    assert e.value.name == "SPD_ERR_CAPACITY"
    with pytest.raises(spd.SpdError):
        c.shared_prefix_attention(q, ids[0], ids)
    with pytest.raises(ValueError):
        c.shared_prefix_attention(q[:2], pid, ids)
    with pytest.raises(ValueError):
        c.shared_prefix_attention(q, pid, ids, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        c.shared_prefix_attention(q, pid, ids, slopes=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        c.shared_prefix_attention(q, pid, ids, weights_in=w)


# ---- eviction ------------------------------------------------------------------

def cache_rows(c, seq, hkv, d, dtype, page, field="k_pool"):
    """Stored rows of a sequence, [L][Hkv][d], read through its page table."""
    L = c.seq_info(seq)["length"]
    pool = c.buffers[field].view(dtype).view(-1, hkv, page, d)
    rows = pool[torch.tensor(c.page_table(seq), device="cuda")]       # [pages][Hkv][P][d]
    return rows.permute(0, 2, 1, 3).reshape(-1, hkv, d)[:L]


def check_evict(lens, keep, recent, hkv, d, dtype="bf16", page=64, logical=16, seed=1, weights=None,
                fp8=False):
    store = torch.uint8 if fp8 else DT[dtype]
    n, longest = len(lens), max(lens)
    need = sum(-(-x // page) + -(-min(keep, x) // page) for x in lens)
    kw = dict(kv_fp8=True) if fp8 else {}
    c = new_cache(hkv, hkv, d, dtype, page, logical, need, 2 * n, longest, free_list_seed=5, **kw)
    src = [c.seq_create() for _ in lens]
    for i, x in enumerate(lens):
        c.kv_append([src[i]], normal(seed + i, 1, x, hkv, d, dtype=DT[dtype]),
                    normal(seed + 50 + i, 1, x, hkv, d, dtype=DT[dtype]))
    dst = [c.seq_create() for _ in lens]
    w = weights if weights is not None else normal(seed + 99, n, hkv, longest + 2).exp()
    kept, kw_ = c.kv_evict(src, dst, keep, recent, w)
    c.check_status()
    meta = c.buffers["meta"].view(store).view(-1, hkv, page // logical, 2, d)
    for i, x in enumerate(lens):
        m = min(keep, x)
        assert c.seq_info(dst[i]) == dict(length=m, step_counter=0, pages_at_selection=0,
                                          pages_kept=0)
        assert c.seq_info(src[i])["length"] == x
        ks, vs = (cache_rows(c, src[i], hkv, d, store, page, f) for f in ("k_pool", "v_pool"))
        kd, vd = (cache_rows(c, dst[i], hkv, d, store, page, f) for f in ("k_pool", "v_pool"))
        table = c.page_table(dst[i])
        for h in range(hkv):
            at = kept_positions(w[i, h].cpu(), x, keep, recent)
            assert kept[i, h].tolist() == at + [-1] * (keep - m), (i, h)
            idx = torch.tensor(at, device="cuda")
            assert torch.equal(kw_[i, h, :m].view(torch.int32), w[i, h, idx].view(torch.int32))
            assert bool((kw_[i, h, m:] == 0).all())
            assert torch.equal(kd[:, h].view(torch.uint8), ks[idx, h].view(torch.uint8))
            assert torch.equal(vd[:, h].view(torch.uint8), vs[idx, h].view(torch.uint8))
            if fp8:  # codes order by sign and magnitude
                key = kd[:, h].view(torch.float8_e4m3fn).float()
                for j in range(-(-m // logical)):
                    rows = key[j * logical:min(m, (j + 1) * logical)]
                    got = meta[table[j * logical // page], h, j * logical % page // logical]
                    got = got.contiguous().view(torch.float8_e4m3fn).float()
                    assert torch.equal(got[0], rows.amin(0)) and torch.equal(got[1], rows.amax(0))
                continue
            for j in range(-(-m // logical)):
                rows = kd[j * logical:min(m, (j + 1) * logical), h]
                got = meta[table[j * logical // page], h, j * logical % page // logical]
                assert torch.equal(got[0], rows.amin(0)) and torch.equal(got[1], rows.amax(0))
    return c, src, dst, w


@pytest.mark.parametrize("lens,keep,recent", [
    ([1], 1, 0), ([1], 4, 2), ([2], 1, 1), ([2], 1, 0), ([17, 64, 65], 16, 3), ([130], 129, 0),
    ([130, 7], 33, 33), ([500, 1000, 3], 300, 10), ([64], 64, 64), ([2000], 1999, 1)])
@pytest.mark.parametrize("hkv,d,dtype,page,logical", [(2, 128, "bf16", 64, 16), (1, 64, "fp16", 16, 16),
                                                      (3, 128, "fp16", 192, 64),
                                                      (2, 64, "bf16", 96, 32)])
def test_evict(lens, keep, recent, hkv, d, dtype, page, logical):
    check_evict(lens, keep, recent, hkv, d, dtype, page, logical)


@pytest.mark.parametrize("lens", [[9000], [30000, 12345], [70001]])
def test_evict_long(lens):
    check_evict(lens, 2500, 100, 2, 64, page=512, logical=64)


def test_evict_longer_than_the_shared_memory_holds():
    check_evict([450_001], 1200, 64, 1, 64, page=4096, logical=64)


def test_evict_ties_nan_and_signs():
    n, hkv, L = 1, 4, 3000
    w = torch.zeros(n, hkv, L, device="cuda")
    w[0, 1, ::7] = 1.0
    w[0, 2] = normal(3, L)
    w[0, 2, 5::11] = math.nan
    w[0, 2, 6::13] = -0.0
    w[0, 2, 9::17] = math.inf
    w[0, 2, 3::19] = -math.inf
    w[0, 3] = torch.where(torch.arange(L, device="cuda") % 2 == 0, -0.0, 0.0)
    for keep, recent in ((700, 64), (1, 0), (2999, 0), (400, 400)):
        check_evict([L], keep, recent, hkv, 64, page=64, weights=w)


@pytest.mark.parametrize("keep", [16, 100])
def test_evict_fp8_storage(keep):
    check_evict([300, 40], keep, 8, 2, 128, fp8=True)


def test_evict_all_or_nothing_and_states():
    c, src, dst, w = check_evict([200, 100], 64, 8, 2, 64, page=64)
    assert c.free_pages() == 0
    more = c.seq_info(dst[0])
    with pytest.raises(spd.SpdError) as e:
        c.kv_evict(src, dst, 64, 8, w)                 # not empty
    assert e.value.name == "SPD_ERR_STATE"
    c.seq_free(dst[0])
    c.seq_free(dst[1])
    dst = [c.seq_create(), c.seq_create()]
    free = c.free_pages()
    with pytest.raises(spd.SpdError) as e:
        c.kv_evict(src, dst, 100, 8, w)                # two pages too many
    assert e.value.name == "SPD_ERR_NO_PAGES" and c.free_pages() == free
    assert [c.seq_info(i)["length"] for i in dst] == [0, 0]
    with pytest.raises(spd.SpdError) as e:
        c.kv_evict(src, dst, 64, 8, w[:, :, :150].contiguous())
    assert e.value.name == "SPD_ERR_CAPACITY"
    c.kv_evict(src, dst, 64, 8, w)
    assert c.seq_info(dst[0]) == more


# ---- together --------------------------------------------------------------------

def test_prompt_decode_and_eviction_together():
    """A server's run: two requests share a document; each prompt is attended,
    appended and decoded with weights kept; the longer one's own tokens are
    evicted, and decoding goes on over the compacted sequence, densely and with
    page selection."""
    hq, hkv, d, dt, cap = 8, 2, 128, torch.bfloat16, 30.0
    sl = torch.linspace(0.0, 0.05, hq, device="cuda")
    c = new_cache(hq, hkv, d, "bf16", 64, 16, 40, 5, 1024, token_budget=64)
    doc_k, doc_v = normal(1, 600, hkv, d, dtype=dt), normal(2, 600, hkv, d, dtype=dt)
    doc = c.seq_create()
    c.kv_append([doc], doc_k[None], doc_v[None])
    own, ids, lens = [], [], [150, 40]
    for i, x in enumerate(lens):
        q, k, v = (normal(10 * i + j, x, h, d, dtype=dt) for j, h in ((3, hq), (4, hkv), (5, hkv)))
        kk, vv = torch.cat([doc_k, k]), torch.cat([doc_v, v])
        got = spd.prefill_attention(q, kk, vv, softcap=cap, slopes=sl, check=True)
        at = torch.arange(600, 600 + x, device="cuda")
        ref, ab, mag = prompt(q, kk, vv, torch.zeros_like(at), at + 1, d ** -0.5, cap, sl)
        assert bool(((got.double() - ref).abs() <=
                     tolerance(ref, ab, mag, d, 750, dt, torch.float32, cap)).all())
        ids.append(c.seq_create())
        c.kv_append([ids[i]], k[None], v[None])
        own.append([k, v])
    w = torch.zeros(2, hkv, 256, device="cuda")
    want = [torch.zeros(hkv, 256, dtype=torch.float64, device="cuda") for _ in ids]

    def step(i):
        q = normal(100 + i, 2, hq, d, dtype=dt)
        k, v = normal(200 + i, 2, 1, hkv, d, dtype=dt), normal(300 + i, 2, 1, hkv, d, dtype=dt)
        c.kv_append(ids, k, v)
        for j in range(2):
            own[j] = [torch.cat([own[j][0], k[j]]), torch.cat([own[j][1], v[j]])]
        got = c.shared_prefix_attention(q, doc, ids, softcap=cap, slopes=sl, weights_in=w,
                                        weights_out=w)
        ref, ab, mag, ws = shared(q, doc_k, doc_v, [o[0] for o in own], [o[1] for o in own],
                                  d ** -0.5, cap, sl)
        assert bool(((got.double() - ref).abs() <=
                     tolerance(ref, ab, mag, d, 800, dt, torch.float32, cap)).all())
        for j in range(2):
            want[j][:, :ws[j].shape[1]] += ws[j]
            assert (w[j].double() - want[j]).abs().max() < 1e-3

    for i in range(4):
        step(i)
    new = c.seq_create()
    kept, kw = c.kv_evict([ids[0]], [new], 48, 16, w[:1].contiguous())
    L = own[0][0].shape[0]
    for h in range(hkv):
        assert kept[0, h].tolist() == kept_positions(w[0, h].cpu(), L, 48, 16)
    pick = kept[0].long()
    own[0] = [torch.stack([o[pick[h], h] for h in range(hkv)], 1) for o in own[0]]
    c.seq_free(ids[0])
    ids[0] = new
    w[0] = 0
    w[0, :, :48] = kw[0]
    want[0].zero_()
    want[0][:, :48] = kw[0].double()
    for i in range(4, 8):
        step(i)
    c.check_status()
    # the selecting path reads the compacted pages and their metadata
    q = normal(400, 1, hq, d, dtype=dt)
    k, v = normal(401, 1, hkv, d, dtype=dt), normal(402, 1, hkv, d, dtype=dt)
    got = c.decode_step(q, k, v, [ids[0]])
    c.check_status()
    assert c.selection(ids[0], 0) and torch.isfinite(got).all()
    kk = torch.cat([own[0][0], k])
    vv = torch.cat([own[0][1], v])
    for h in range(hkv):  # a budget of 64 of 53 tokens: every page is attended
        assert c.selection(ids[0], h) == list(range(4))
    ref, ab, mag, _ = shared(q, kk[:0], vv[:0], [kk], [vv], d ** -0.5, 0.0, None)
    assert bool(((got.double() - ref).abs() <= 2e-3).all())


# ---- offsets beyond 32 bits ------------------------------------------------------

def test_pools_beyond_four_gigabytes():
    """Sequences whose pages lie behind the first 4 GB of a pool."""
    hq, hkv, d, page, dt = 8, 8, 128, 4096, torch.bfloat16
    pages = 620  # 8 MB of keys each
    c = spd.SparsePagedKVCache(device="cuda", num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                               dtype="bf16", logical_page=64, physical_page=page,
                               num_physical_pages=pages, max_seqs=48, max_context=page * pages)
    low = c.seq_create()
    c.seq_reserve(low, (pages - 46) * page)
    doc = c.seq_create()
    kp, vp = normal(1, 4100, hkv, d, dtype=dt), normal(2, 4100, hkv, d, dtype=dt)
    c.kv_append([doc], kp[None], vp[None])
    assert min(c.page_table(doc)) * page * hkv * d * 2 > 1 << 32
    for n in (2, 12, 40):  # each of the prefix's kernels
        ids = [c.seq_create() for _ in range(n)]
        ko, vo = normal(3, n, 20, hkv, d, dtype=dt), normal(4, n, 20, hkv, d, dtype=dt)
        c.kv_append(ids, ko, vo)
        q = normal(5, n, hq, d, dtype=dt)
        got = c.shared_prefix_attention(q, doc, ids)
        c.check_status()
        ref, ab, mag, _ = shared(q, kp, vp, list(ko), list(vo), d ** -0.5, 0.0, None)
        assert bool(((got.double() - ref).abs() <=
                     tolerance(ref, ab, mag, d, 4120, dt, torch.float32, 0.0)).all())
        for i in ids:
            c.seq_free(i)
    w = normal(6, 1, hkv, 4100).abs()
    dst = c.seq_create()
    kept, _ = c.kv_evict([doc], [dst], 500, 20, w)
    c.check_status()
    for h in range(hkv):
        assert kept[0, h].tolist() == kept_positions(w[0, h].cpu(), 4100, 500, 20)
        assert torch.equal(cache_rows(c, dst, hkv, d, dt, page)[:, h], kp[kept[0, h].long(), h])


def test_keys_beyond_four_gigabytes():
    n, hkv, d = 2_200_000, 8, 128
    k = torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    for a in range(0, n, 200_000):
        k[a:a + 200_000] = normal(a, min(200_000, n - a), hkv, d, dtype=torch.bfloat16)
        v[a:a + 200_000] = normal(a + 1, min(200_000, n - a), hkv, d, dtype=torch.bfloat16)
    q = normal(9, 3, hkv, d, dtype=torch.bfloat16)
    at = [2_199_990, 2_150_000, 17]  # each query's own needle, two of them behind 4 GB
    for i, t in enumerate(at):
        k[t] = q[i] * 4
    got = spd.prefill_attention(q, k, v, check=True)
    for i, t in enumerate(at):
        assert (got[i] - v[t].float()).abs().max() < 1e-2


# ---- calls in a row --------------------------------------------------------------

def test_calls_of_every_kind_in_a_row_on_one_stream():
    """Kernels start before the ones before them have ended: calls whose inputs the
    call before wrote, without a pause, give what they give alone."""
    hq, hkv, d, dt = 8, 2, 128, torch.bfloat16
    c = new_cache(hq, hkv, d, "bf16", 64, 16, 200, 60, 4096)
    doc = c.seq_create()
    c.kv_append([doc], normal(1, 1, 700, hkv, d, dtype=dt), normal(2, 1, 700, hkv, d, dtype=dt))
    sizes = [1, 3, 9]
    groups = [[c.seq_create() for _ in range(n)] for n in sizes]
    for g in groups:
        c.kv_append(g, normal(3, len(g), 40, hkv, d, dtype=dt), normal(4, len(g), 40, hkv, d, dtype=dt))
    long_k, long_v = normal(7, 3000, hkv, d, dtype=dt), normal(8, 3000, hkv, d, dtype=dt)

    def chain(wait):
        outs, x = [], normal(5, 30, hq, d, dtype=dt)
        for r in range(6):
            x = spd.prefill_attention(x, long_k, long_v, out_dtype=dt)
            if wait:
                torch.cuda.synchronize()
            for n, g in zip(sizes, groups):
                y = c.shared_prefix_attention(x[:n], doc, g, out_dtype=dt)
                if wait:
                    torch.cuda.synchronize()
                x[:n] += y
                w = torch.zeros(n, hkv, 64, device="cuda")
                c.shared_prefix_attention(x[:n], doc, g, weights_in=w, weights_out=w, out_dtype=dt)
                dst = [c.seq_create() for _ in g]
                kept, kw = c.kv_evict(g, dst, 24, 4, w)
                y = c.shared_prefix_attention(x[:n], doc, dst, out_dtype=dt)
                if wait:
                    torch.cuda.synchronize()
                x[:n] -= y
                for i in reversed(dst):
                    c.seq_free(i)
                outs += [w, kept, kw]
            outs.append(x.clone())
        return outs

    alone, row = chain(True), chain(False)
    c.check_status()
    for a, b in zip(alone, row):
        assert torch.equal(a, b)


# ---- every kernel of a prefix, by its rows ----------------------------------------

@pytest.mark.parametrize("n,hq,hkv", [(3, 4, 1), (4, 8, 2), (5, 4, 1), (8, 8, 2), (31, 1, 1),
                                      (33, 1, 1), (8, 8, 1), (25, 4, 1), (32, 8, 2), (33, 4, 1),
                                      (65, 4, 1)])
@pytest.mark.parametrize("lp,page", [(4500, 256), (5009, 16), (4160, 48)])
@pytest.mark.parametrize("kind", [dict(), dict(out="same", weights=True),
                                  dict(softcap=25.0, gain=5.0, slopes=True),
                                  dict(softcap=25.0, out="same", gain=5.0)])
def test_shared_prefix_kernels(n, hq, hkv, lp, page, kind):
    lens = [(7 * i) % 40 for i in range(n)]
    check_shared(n, lp, lens, hq, hkv, 128, "bf16" if page == 16 else "fp16", page=page, **kind)


@pytest.mark.parametrize("n", [4, 40])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_shared_rows_behind_the_end_hold_anything(n, bad):
    """Pages are NaN before they are filled; here the rows behind the prefix's end
    are overwritten too."""
    hq, hkv, d, page, dt = 4, 1, 128, 64, torch.bfloat16
    c = new_cache(hq, hkv, d, "bf16", page, 16, 200, n + 1, 8192)
    kp, vp = normal(1, 4501, hkv, d, dtype=dt), normal(2, 4501, hkv, d, dtype=dt)
    doc = c.seq_create()
    c.kv_append([doc], kp[None], vp[None])
    last = c.page_table(doc)[-1]
    for f in ("k_pool", "v_pool"):
        c.buffers[f].view(dt).view(-1, hkv, page, d)[last, :, 4501 % page:] = bad
    ids = [c.seq_create() for _ in range(n)]
    ko, vo = normal(3, n, 3, hkv, d, dtype=dt), normal(4, n, 3, hkv, d, dtype=dt)
    c.kv_append(ids, ko, vo)
    q = normal(5, n, hq, d, dtype=dt)
    got = c.shared_prefix_attention(q, doc, ids)
    c.check_status()
    ref, ab, mag, _ = shared(q, kp, vp, list(ko), list(vo), d ** -0.5, 0.0, None)
    assert bool(((got.double() - ref).abs() <=
                 tolerance(ref, ab, mag, d, 4504, dt, torch.float32, 0.0)).all())


@pytest.mark.parametrize("level", [-1.2, -0.8, -0.26, 0.0, 0.6, 0.74, 0.8, 1.5])
def test_capped_scores_around_every_level(level):
    """All of a row's scores near one part of the cap's curve."""
    d, dt, cap, n = 128, torch.bfloat16, 30.0, 500
    q, k, v = (normal(i, n, h, d, dtype=dt) for i, h in ((1, 4), (2, 2), (3, 2)))
    q[..., 0], k[..., 0] = 16.0, level * cap * d ** 0.5 / 16.0
    b, e = intervals("causal", n, n)
    for out in (dt, torch.float32):
        got = spd.prefill_attention(q, k, v, softcap=cap, out_dtype=out, check=True)
        ref, ab, mag = prompt(q, k, v, b, e, d ** -0.5, cap, None)
        assert bool(((got.double() - ref).abs() <=
                     tolerance(ref, ab, mag, d, n, dt, out, cap)).all())
