"""Host-side tests of the dense attention and eviction entry points: what they
refuse, and that a refused call changes nothing.  No GPU: device pointers are
fake aligned addresses; every call here is refused before any is used."""
import ctypes

import pytest

import sparse_paged_decode_logical_gb300 as spd
from test_abi_host import fake_buffers

A = 1 << 41  # an aligned fake device address


def dense_cfg(hq=8, hkv=2, d=128, dtype=1, out=0, scale=0.0, softcap=0.0, slopes=None):
    return spd.spd_dense_config(hq, hkv, d, dtype, out, spd.spd_score_rule(scale, softcap, slopes))


def sizes(cfg, lq, lk):
    ws = ctypes.c_size_t(7)
    st = spd.lib().spd_prefill_attention_sizes(ctypes.byref(cfg), lq, lk, ctypes.byref(ws))
    return st, ws.value


INVALID, BAD_SEQ, CAPACITY, STATE, NO_PAGES = 1, 3, 4, 7, 2


@pytest.mark.parametrize("bad", [
    dict(hq=7), dict(hq=0), dict(hkv=0), dict(hkv=129, hq=129), dict(d=96), dict(dtype=2),
    dict(out=2), dict(scale=-1.0), dict(scale=float("inf")), dict(softcap=-3.0),
    dict(softcap=float("nan")), dict(scale=float("nan")), dict(slopes=A + 2),
    dict(hq=2048, hkv=128), dict(softcap=1e-7), dict(softcap=2e6), dict(scale=1e-7),
    dict(scale=1e7)])
def test_prompt_configs_refused(bad):
    assert sizes(dense_cfg(**bad), 5, 5)[0] == INVALID


def test_prompt_sizes():
    assert sizes(dense_cfg(), 0, 5)[0] == INVALID
    assert sizes(dense_cfg(), 5, 0)[0] == INVALID
    assert sizes(dense_cfg(), (1 << 28) + 1, 5)[0] == CAPACITY
    assert spd.lib().spd_prefill_attention_sizes(None, 5, 5, None) == INVALID
    # a whole prompt needs no workspace, a token over a long row does
    assert sizes(dense_cfg(hq=32, hkv=8), 8192, 8192) == (0, 0)
    st, ws = sizes(dense_cfg(hq=32, hkv=8), 1, 65536)
    assert st == 0 and ws >= 8 * 128 * 128 * 4


def prompt(cfg=None, lq=64, lk=64, q=A, qs=8 * 128, k=A, ks=2 * 128, v=A, vs=2 * 128, kb=None,
           ke=None, out=A, ws=None, wsb=0):
    cfg = cfg or dense_cfg()
    return spd.lib().spd_prefill_attention(ctypes.byref(cfg), lq, lk, q, qs, k, ks, v, vs, kb, ke,
                                           out, ws, wsb, None)


@pytest.mark.parametrize("bad", [
    dict(lq=0), dict(lk=0), dict(lk=-3), dict(q=None), dict(q=A + 8), dict(k=A + 2), dict(v=None),
    dict(out=A + 4), dict(out=None), dict(qs=8 * 128 - 8), dict(qs=8 * 128 + 4), dict(ks=128),
    dict(vs=-256), dict(vs=2 * 128 + 1), dict(kb=A), dict(ke=A), dict(kb=A + 2, ke=A),
    dict(qs=1 << 40), dict(cfg=dense_cfg(d=32))])
def test_prompt_arguments_refused(bad):
    assert prompt(**bad) == INVALID


def test_prompt_out_must_be_device_memory():
    buf = (ctypes.c_char * 4096)()
    at = (ctypes.addressof(buf) + 255) & ~255
    assert prompt(out=at) == INVALID


@pytest.mark.parametrize("bad", [
    dict(offsets=None), dict(n_docs=0), dict(n_tokens=0), dict(n_tokens=(1 << 28) + 1),
    dict(kb=None), dict(ke=None), dict(offsets=A + 1), dict(prefix=A + 3)])
def test_document_ranges_refused(bad):
    a = dict(offsets=A, prefix=None, n_docs=2, n_tokens=9, kb=A, ke=A)
    a.update(bad)
    assert spd.lib().spd_document_key_ranges(a["offsets"], a["prefix"], a["n_docs"], a["n_tokens"],
                                             a["kb"], a["ke"], None) == INVALID


def context(**kw):
    base = dict(num_q_heads=4, num_kv_heads=2, head_dim=128, dtype="bf16", logical_page=16,
                physical_page=64, num_physical_pages=6, max_seqs=4, max_context=512)
    base.update(kw)
    c = spd.make_config(**base)
    ctx = spd.spd_create(c, fake_buffers(spd.spd_query_sizes(c)))
    return c, ctx


def shared(ctx, q=A, prefix=0, ids=(1, 2), rule=None, out_type=0, out=A, w_in=None, w_out=None,
           stride=0, ws=A, wsb=1 << 30, n=None):
    arr = (ctypes.c_int * max(len(ids), 1))(*ids)
    r = spd.spd_score_rule(*rule) if rule else None
    return spd.lib().spd_shared_prefix_attention(
        ctx, q, prefix, arr, len(ids) if n is None else n, ctypes.byref(r) if r else None, out_type,
        out, w_in, w_out, stride, ws, wsb, None)


def shared_sizes(ctx, prefix, ids, weights=0):
    ws = ctypes.c_size_t()
    arr = (ctypes.c_int * max(len(ids), 1))(*ids)
    return spd.lib().spd_shared_prefix_sizes(ctx, prefix, arr, len(ids), weights,
                                             ctypes.byref(ws)), ws.value


def test_shared_prefix_refusals():
    _, ctx = context()
    for _ in range(3):
        spd.spd_seq_create(ctx)
    L = spd.lib()
    assert L.spd_shared_prefix_attention(None, A, 0, None, 1, None, 0, A, None, None, 0, A, 0,
                                         None) == INVALID
    for bad in (dict(q=A + 8), dict(q=None), dict(out=None), dict(out=A + 2), dict(out_type=2),
                dict(rule=(-1.0, 0.0, None)), dict(rule=(0.0, float("inf"), None)),
                dict(rule=(0.0, 0.0, A + 1)), dict(w_in=A), dict(w_out=A + 2), dict(n=0)):
        assert shared(ctx, **bad) == INVALID, bad
    assert shared(ctx, prefix=-2) == BAD_SEQ
    assert shared(ctx, prefix=3) == BAD_SEQ           # not live
    assert shared(ctx, ids=(1, 1)) == BAD_SEQ         # listed twice
    assert shared(ctx, ids=(1, 9)) == BAD_SEQ
    # empty sequences: no prefix, or a prefix without tokens
    assert shared(ctx, prefix=-1) == STATE
    assert shared(ctx, prefix=0) == STATE
    assert shared_sizes(ctx, -1, (1, 2))[0] == STATE
    assert shared(ctx, prefix=1) in (BAD_SEQ, STATE)
    for i in range(3):
        assert spd.spd_seq_info(ctx, i) == dict(length=0, step_counter=0, pages_at_selection=0,
                                                pages_kept=0)
    assert spd.spd_free_pages(ctx) == 6


def test_shared_prefix_refuses_streaming_and_fp8():
    for kw in (dict(streaming=[True, False], sink=4, window=32), dict(kv_fp8=True)):
        _, ctx = context(**kw)
        for _ in range(3):
            spd.spd_seq_create(ctx)
        assert shared(ctx) == INVALID
        assert shared_sizes(ctx, 0, (1, 2))[0] == INVALID


def evict(ctx, src=(0,), dst=(1,), n=None, keep=8, recent=2, w=A, stride=512, kept=A, kw=A):
    s, t = (ctypes.c_int * len(src))(*src), (ctypes.c_int * len(dst))(*dst)
    return spd.lib().spd_kv_evict(ctx, s, t, len(src) if n is None else n, keep, recent, w, stride,
                                  kept, kw, None)


def test_evict_refusals():
    _, ctx = context()
    for _ in range(4):
        spd.spd_seq_create(ctx)
    assert spd.lib().spd_kv_evict(None, None, None, 1, 8, 2, A, 512, A, A, None) == INVALID
    for bad in (dict(keep=0), dict(keep=-1), dict(recent=-1), dict(recent=9), dict(w=None),
                dict(w=A + 2), dict(kept=None), dict(kept=A + 1), dict(kw=A + 3), dict(n=0)):
        assert evict(ctx, **bad) == INVALID, bad
    assert evict(ctx, src=(0,), dst=(0,)) == BAD_SEQ
    assert evict(ctx, src=(0, 1), dst=(2, 0)) == BAD_SEQ
    assert evict(ctx, src=(0, 0), dst=(1, 2)) == BAD_SEQ
    assert evict(ctx, src=(0, 1), dst=(2, 2)) == BAD_SEQ
    assert evict(ctx, src=(7,)) == BAD_SEQ
    assert evict(ctx) == STATE                        # a source without tokens
    assert spd.spd_free_pages(ctx) == 6
    _, ctx = context(streaming=[True, False], sink=4, window=32)
    for _ in range(2):
        spd.spd_seq_create(ctx)
    assert evict(ctx) == INVALID


def test_error_text_names_the_reason():
    _, ctx = context()
    spd.spd_seq_create(ctx)
    spd.spd_seq_create(ctx)
    assert shared(ctx, prefix=0, ids=(1,)) == STATE
    assert b"prefix" in spd.lib().spd_last_error(ctx)
    with pytest.raises(spd.SpdError) as e:
        spd._check(evict(ctx, keep=3, recent=4), "spd_kv_evict", ctx)
    assert e.value.name == "SPD_ERR_INVALID_ARG" and "recent" in str(e.value)


def test_python_argument_checks_need_no_gpu():
    import torch
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        spd.prefill_attention(q, k, k)                # not on a GPU
    with pytest.raises(ValueError):
        spd.prefill_attention(q.float(), k, k)
    with pytest.raises(ValueError):
        spd.prefill_attention(q[0], k, k)
    with pytest.raises(ValueError):
        spd.document_key_ranges(torch.zeros(3, dtype=torch.int32), 9)
    with pytest.raises(ValueError):
        spd._token_stride(torch.zeros(4, 128, 8).transpose(1, 2), "q")
    row = torch.zeros(4, 12, 128)
    assert spd._token_stride(row[:, :8], "q") == 12 * 128
    assert spd._token_stride(row[:1, :8], "q") == 8 * 128


@pytest.mark.parametrize("keep", [(1 << 28) + 1, (1 << 31) - 64, (1 << 31) - 1])
def test_evict_refuses_a_keep_that_no_sequence_holds(keep):
    """Before anything is looked at (the source is empty here, too), so that no page is taken."""
    _, ctx = context()
    for _ in range(2):
        spd.spd_seq_create(ctx)
    assert evict(ctx, keep=keep, recent=0) == CAPACITY
    assert evict(ctx, keep=1 << 28, recent=0) == STATE
