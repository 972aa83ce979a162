"""Host-side tests of rotary tables and of the cache in 8 or 4 bits: sizes, what
is refused, and that a refused call changes nothing.  No GPU: device pointers are
fake aligned addresses; every call here is refused before any is used."""
import ctypes
import math

import pytest
import torch

import sparse_paged_decode_logical_gb300 as spd
from test_abi_host import fake_buffers

A = 1 << 41  # an aligned fake device address
INVALID, NO_PAGES, BAD_SEQ, CAPACITY, STATE = 1, 2, 3, 4, 7


def context(**kw):
    base = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, dtype="bf16", logical_page=16,
                physical_page=64, num_physical_pages=6, max_seqs=4, max_context=512, kv_quant=4)
    base.update(kw)
    c = spd.make_config(**base)
    return c, spd.spd_create(c, fake_buffers(spd.spd_query_sizes(c)))


@pytest.mark.parametrize("d,bits,tile", [(128, 8, 4224), (128, 4, 2560), (64, 8, 2176), (64, 4, 1280)])
def test_sizes(d, bits, tile):
    c = spd.make_config(num_q_heads=8, num_kv_heads=2, head_dim=d, dtype="f16", logical_page=16,
                        physical_page=64, num_physical_pages=6, max_seqs=4, max_context=512,
                        kv_quant=bits)
    z = spd.spd_query_sizes(c)
    assert z["k_pool"] == 6 * 2 * 4 * tile
    assert tile == (32 * (d + 4) if bits == 8 else 20 * d)
    assert z["v_pool"] == z["meta"] == z["selection"] == z["stream_k"] == 0
    assert z["page_table"] == 4 * 8 * 4


@pytest.mark.parametrize("bad", [
    dict(kv_quant=1), dict(kv_quant=16), dict(kv_quant=-8), dict(kv_fp8=True),
    dict(streaming=[True, False], sink=4, window=32), dict(head_dim=96), dict(num_q_heads=6)])
def test_configs_refused(bad):
    with pytest.raises(spd.SpdError) as e:
        context(**bad)
    assert e.value.name == "SPD_ERR_INVALID_ARG"


def rule(**kw):
    a = dict(head_dim=128, rotary_dim=128, sections=[64])
    a.update(kw)
    return spd.Rotary(**a)


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=144),
    dict(sections=[63]), dict(sections=[65]), dict(sections=[65, -1]), dict(sections=[32, 16]),
    dict(base=0.5), dict(base=math.nan), dict(base=math.inf), dict(inv_freq=[1.0] * 63 + [-0.1]),
    dict(inv_freq=[1.0] * 63 + [math.nan]), dict(inv_freq=[1001.0] * 64)])
def test_rotary_rules_refused(bad):
    with pytest.raises(spd.SpdError) as e:
        rule(**bad)
    assert e.value.name == "SPD_ERR_INVALID_ARG"


def test_rotary_rules_refused_in_python():
    for bad in (dict(sections=[]), dict(sections=[16, 16, 16, 8, 8]), dict(inv_freq=[1.0] * 63)):
        with pytest.raises(ValueError):
            rule(**bad)
    assert spd.lib().spd_rotary_make(None, None) == INVALID


def test_rotary_tables():
    t = rule(rotary_dim=64, sections=[16, 8, 8], axes_in_turn=True, base=500000.0).table
    assert list(t.axis[:32]) == [0, 1, 2] * 8 + [0] * 8
    for i in range(32):
        want = 500000.0 ** (-2.0 * i / 64) / (2 * math.pi)
        # a double's own error, 2^-52 of it, and half a unit of 2^-64
        assert abs(t.turns[i] / 2.0 ** 64 - want) <= want * 2.0 ** -51 + 2.0 ** -64
    t = rule(sections=[40, 0, 24]).table
    assert list(t.axis[:64]) == [0] * 40 + [2] * 24
    # a frequency of whole turns stands still, one above a turn wraps
    t = rule(inv_freq=[2 * math.pi, 0.0, 4.5 * math.pi] + [1.0] * 61).table
    assert list(t.turns[:2]) == [0, 0] and abs(t.turns[2] / 2.0 ** 64 - 0.25) < 1e-15


def test_sparse_calls_refuse_a_quantised_cache():
    _, ctx = context()
    for _ in range(3):
        spd.spd_seq_create(ctx)
    L, ids = spd.lib(), (ctypes.c_int * 1)(0)
    assert L.spd_select_pages(ctx, A, ids, 1, 0, None) == INVALID
    assert L.spd_sparse_decode_attention(ctx, A, ids, 1, A, None) == INVALID
    assert L.spd_sparse_decode_attention_static(ctx, A, ids, 1, A, None) == INVALID
    assert L.spd_sparse_decode_attention_stats(ctx, A, ids, 1, A, A, A, None) == INVALID
    assert L.spd_sparse_decode_attention_page_mass(ctx, A, ids, 1, A, A, A, A, A, 9, None) == INVALID
    assert L.spd_decode_step(ctx, A, A, A, ids, 1, A, None) == INVALID
    assert b"spd_quant_decode_attention" in L.spd_last_error(ctx)
    ws = ctypes.c_size_t()
    assert L.spd_shared_prefix_sizes(ctx, -1, ids, 1, 0, ctypes.byref(ws)) == INVALID
    assert L.spd_shared_prefix_attention(ctx, A, -1, ids, 1, None, 0, A, None, None, 0, A, 1 << 30,
                                         None) == INVALID
    dst = (ctypes.c_int * 1)(1)
    assert L.spd_kv_evict(ctx, ids, dst, 1, 8, 2, A, 512, A, A, None) == INVALID
    assert spd.spd_free_pages(ctx) == 6
    assert spd.spd_seq_info(ctx, 0)["length"] == 0


def append(ctx, table=None, ids=(0,), n=None, tokens=3, pos=A, q=A, qs=1024, k=A, ks=256, v=A,
           vs=256, out=A):
    t = (table or rule()).table
    return spd.lib().spd_kv_append_rotary(ctx, ctypes.byref(t), (ctypes.c_int * len(ids))(*ids),
                                          len(ids) if n is None else n, tokens, pos, q, qs, k, ks,
                                          v, vs, out, None)


def attend(ctx, q=A, ids=(0,), n=None, window=0, rule=None, out_type=0, out=A):
    r = spd.spd_score_rule(*rule) if rule else None
    return spd.lib().spd_quant_decode_attention(
        ctx, q, (ctypes.c_int * len(ids))(*ids), len(ids) if n is None else n, window,
        ctypes.byref(r) if r else None, out_type, out, None)


def read(ctx, ids=(0,), n=None, begin=0, tokens=1, k=A, v=A):
    return spd.lib().spd_kv_read(ctx, (ctypes.c_int * len(ids))(*ids),
                                 len(ids) if n is None else n, begin, tokens, k, v, None)


def test_quantised_calls_refuse_another_cache():
    for kw in (dict(kv_quant=0), dict(kv_quant=0, kv_fp8=True)):
        _, ctx = context(**kw)
        spd.spd_seq_create(ctx)
        assert append(ctx) == read(ctx) == attend(ctx) == INVALID
        assert spd.lib().spd_seq_truncate(ctx, 0, 0) == INVALID
    L = spd.lib()
    assert L.spd_kv_append_rotary(None, None, None, 1, 1, None, A, 8, A, 8, A, 8, A, None) == INVALID
    assert L.spd_kv_read(None, None, 1, 0, 1, A, A, None) == INVALID
    assert L.spd_seq_truncate(None, 0, 0) == INVALID
    assert L.spd_quant_decode_attention(None, A, None, 1, 0, None, 0, A, None) == INVALID


@pytest.mark.parametrize("bits", [4, 8])
def test_quantised_arguments_refused(bits):
    _, ctx = context(kv_quant=bits)
    for _ in range(2):
        spd.spd_seq_create(ctx)
    for bad in (dict(tokens=0), dict(q=None), dict(q=A + 8), dict(k=None), dict(k=A + 2),
                dict(v=A + 4), dict(v=None), dict(out=None), dict(out=A + 1), dict(pos=A + 2),
                dict(qs=1016), dict(qs=1028), dict(ks=128), dict(vs=-256), dict(vs=1 << 40),
                dict(qs=2048), dict(table=spd.Rotary(64))):
        assert append(ctx, **bad) == INVALID, bad
    blank = spd.Rotary(128)
    blank.table.rotary_dim = 8
    assert append(ctx, table=blank) == INVALID
    blank = spd.Rotary(128)
    blank.table.axis[63] = 1
    assert append(ctx, table=blank) == INVALID
    assert append(ctx, ids=(0, 0)) == append(ctx, ids=(3,)) == append(ctx, ids=(-1,)) == BAD_SEQ
    assert append(ctx, n=0) == INVALID
    assert append(ctx, tokens=513) == CAPACITY
    assert append(ctx, tokens=385) == NO_PAGES
    assert append(ctx, ids=(0, 1), tokens=193) == NO_PAGES
    for bad in (dict(q=None), dict(q=A + 8), dict(out=None), dict(out=A + 2), dict(window=-1),
                dict(out_type=2), dict(rule=(-1.0, 0.0, None)), dict(rule=(0.0, math.nan, None)),
                dict(rule=(0.0, 0.0, A + 1)), dict(n=0)):
        assert attend(ctx, **bad) == INVALID, bad
    assert attend(ctx) == STATE
    assert attend(ctx, ids=(0, 0)) == attend(ctx, ids=(2,)) == BAD_SEQ
    for bad in (dict(tokens=0), dict(k=None), dict(v=A + 8), dict(n=0)):
        assert read(ctx, **bad) == INVALID, bad
    assert read(ctx) == read(ctx, begin=-1) == CAPACITY
    assert read(ctx, begin=(1 << 31) - 1, tokens=(1 << 31) - 1) == CAPACITY
    assert read(ctx, ids=(5,)) == BAD_SEQ
    assert spd.lib().spd_seq_truncate(ctx, 0, -1) == INVALID
    assert spd.lib().spd_seq_truncate(ctx, 0, 1) == CAPACITY
    assert spd.lib().spd_seq_truncate(ctx, 3, 0) == BAD_SEQ
    assert spd.spd_free_pages(ctx) == 6
    with pytest.raises(spd.SpdError):
        spd.spd_seq_truncate(ctx, 0, 1 << 40)


def test_truncation_gives_reserved_pages_back():
    _, ctx = context()
    s = spd.spd_seq_create(ctx)
    spd.spd_seq_reserve(ctx, s, 200)
    assert spd.spd_free_pages(ctx) == 2
    assert spd.lib().spd_seq_truncate(ctx, s, 0) == 0
    assert spd.spd_free_pages(ctx) == 6 and spd.spd_get_page_table(ctx, s) == []
    spd.spd_seq_reserve(ctx, s, 65)
    assert spd.spd_get_page_table(ctx, s) == [0, 1]


def rotary(table=None, dtype=1, n=3, pos=A, q=A, qs=1024, hq=8, k=A, ks=256, hk=2, qo=A + (1 << 30),
           qos=1024, ko=A + (1 << 31), kos=256, inverse=0):
    t = (table or rule()).table
    return spd.lib().spd_rotary(ctypes.byref(t), dtype, n, pos, q, qs, hq, k, ks, hk, qo, qos, ko,
                                kos, inverse, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(n=0), dict(n=-1), dict(pos=None), dict(pos=A + 2), dict(q=None),
    dict(q=A + 8), dict(qs=1000), dict(qs=1028), dict(hq=0), dict(hq=1025), dict(k=None),
    dict(ko=None), dict(k=A + 4), dict(ks=248), dict(hk=0), dict(qo=None), dict(qos=512),
    dict(kos=264 + 4), dict(inverse=2), dict(qo=A, qos=2048), dict(qs=1 << 40)])
def test_rotary_arguments_refused(bad):
    assert rotary(**bad) == INVALID


def test_rotary_outputs_must_be_device_memory():
    assert rotary(n=(1 << 28) + 1) == CAPACITY
    buf = (ctypes.c_char * 4096)()
    at = (ctypes.addressof(buf) + 255) & ~255
    assert rotary(qo=at) == INVALID
    assert spd.lib().spd_rotary(None, 1, 1, A, A, 1024, 8, None, 0, 0, A, 1024, None, 0, 0,
                                None) == INVALID


def test_python_argument_checks_need_no_gpu():
    r = spd.Rotary(128)
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32)
    for a in ((r, pos, q), (r, pos, q.float()), (r, pos, q[0]), (spd.Rotary(64), pos, q)):
        with pytest.raises(ValueError):
            spd.rotary(*a)


def test_rows_at_one_stride():
    c = spd.SparsePagedKVCache.__new__(spd.SparsePagedKVCache)
    c.dtype, c._dev_index, c.device, c.ctx = torch.float16, -1, "cpu", None
    row = torch.zeros(2, 5, 1536, dtype=torch.float16)
    k = row[:, :, 1024:1280].unflatten(2, (2, 128))
    assert c._rows(k, (2, 5, 2, 128), "k") == 1536
    assert c._rows(k[:, :1], (2, 1, 2, 128), "k") == 5 * 1536
    assert c._rows(k[:1, :1], (1, 1, 2, 128), "k") == 256
    with pytest.raises(ValueError):
        c._rows(k[:, :3], (2, 3, 2, 128), "k")       # a gap between the sequences
    with pytest.raises(ValueError):
        c._rows(k.transpose(0, 1), (5, 2, 2, 128), "k")
    with pytest.raises(ValueError):
        c._rows(k.transpose(2, 3), (2, 5, 128, 2), "k")
    with pytest.raises(ValueError):
        c._rows(k.float(), (2, 5, 2, 128), "k")
