"""How the Python calls of rotary positions and of the quantised cache handle memory
and numbers, on the CPU: the library's entry points are replaced by recorders."""
import ctypes
import types

import pytest
import torch

import sparse_paged_decode_logical_gb300 as spd
from test_dense_calls import Recorder, Stream, stand_in_cache


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(spd, "lib", lambda: r)
    monkeypatch.setattr(spd, "_rotary_plans", {})
    return r


def cache(rec):
    c = stand_in_cache(rec)
    c._append_plans = {}
    c.cfg = types.SimpleNamespace(max_context=4096)
    c._append_rotary_fn = rec.spd_kv_append_rotary
    c._quant_attend_fn = rec.spd_quant_decode_attention
    c._truncate_fn = rec.spd_seq_truncate
    c._length = ctypes.c_longlong(9)
    c._length_fn = rec.spd_seq_info
    return c


def operands():
    return (torch.zeros(3, 5, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 5, 2, 64, dtype=torch.bfloat16),
            torch.zeros(3, 4, 64, dtype=torch.bfloat16))


TABLE = types.SimpleNamespace(table="table", axes=1, head_dim=64)


@pytest.mark.parametrize("stream", [None, Stream(), 77])
def test_results_come_from_the_pool_of_the_call_s_stream(rec, monkeypatch, stream):
    c, (q, k, one) = cache(rec), operands()
    monkeypatch.setattr(spd, "_raw_stream", lambda *a: 77)
    # a plan as a CUDA tensor's would be
    monkeypatch.setattr(spd, "_rotary_plan", lambda *a: (
        rec.torch, 1, 3, torch.bfloat16, torch.device("cpu"), (3, 4, 64), 256, (3, 2, 64), 128))
    rec.buffers.clear()
    outs = [c.kv_append_rotary([0, 1, 2], TABLE, q, k, k, stream=stream),
            *c.kv_read([0, 1, 2], 2, 4, stream=stream),
            c.quant_decode_attention(one, [0, 1, 2], stream=stream),
            *spd.rotary(TABLE, torch.zeros(3, dtype=torch.int32), one, k[:, 0], stream=stream)]
    calls = {name: held for name, _, held in rec.calls}
    under = "caller" if stream is None else Stream(77)
    for name, n in (("spd_kv_append_rotary", 1), ("spd_kv_read", 2), ("spd_quant_decode_attention", 1),
                    ("spd_rotary", 2)):
        assert len(calls[name]) == n and all(x == (True, under) for x in calls[name]), name
    assert rec.recorded == ({} if stream is None else {t.data_ptr(): {"caller"} for t in outs})


def test_numbers_that_32_bits_would_wrap_are_refused(rec):
    c, (q, k, one) = cache(rec), operands()
    for begin, n in ((0, 2 ** 32 + 4), (2 ** 32, 4), (-2 ** 32 - 4, 4), (0, 4097), (0, 0)):
        with pytest.raises(spd.SpdError) as e:
            c.kv_read([0], begin, n)
        assert e.value.name == "SPD_ERR_CAPACITY"
    assert not rec.calls and not rec.buffers
    c.quant_decode_attention(one, [0, 1, 2], window=2 ** 32 + 5)
    assert rec.calls[-1][1][4] == 2 ** 28  # (as long as any sequence)
    c.seq_truncate(0, 2 ** 32 + 3)
    assert rec.calls[-1][0] == "spd_seq_truncate" and rec.calls[-1][1][2] == 2 ** 28 + 1


def test_sequences_and_places_are_found_by_value(rec):
    """What shapes decide is kept, what tensors hold is not."""
    c, (q, k, one) = cache(rec), operands()
    ids, pos = [torch.tensor(0), torch.tensor(1), torch.tensor(2)], torch.zeros(3, 5, dtype=torch.int32)
    seen = []
    for add in range(3):
        c.kv_append_rotary(ids, TABLE, q, k, k, positions=pos + add)
        args = rec.calls[-1][1]
        seen.append(list(args[2]))
        ids[0] += 5
    assert seen == [[0, 1, 2], [5, 1, 2], [10, 1, 2]] and len(c._append_plans) == 1
    c.kv_append_rotary([0, 1, 2], TABLE, q, k, k)  # no positions: another plan
    assert len(c._append_plans) == 2 and rec.calls[-1][1][5] is None
    for bad in (pos[:, :4], pos.long(), pos.t().contiguous().t(), pos[None].repeat(2, 1, 1)):
        with pytest.raises(ValueError):
            c.kv_append_rotary([0, 1, 2], TABLE, q, k, k, positions=bad)
    for bad in ((q[:, :, :2], k, k), (q, k[:2], k), (q, k, k.float()), (q, k[0], k)):
        with pytest.raises(ValueError):
            c.kv_append_rotary([0, 1, 2], TABLE, *bad)
