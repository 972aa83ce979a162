"""How the dense operators' Python calls handle memory and arguments, on the CPU:
the library's entry points are replaced by recorders, tensors live in host
memory and streams are stand-ins."""
import contextlib
import types
import weakref

import pytest
import torch

import sparse_paged_decode_logical_gb300 as spd


class Recorder:
    """Stands in for torch and for the library: every buffer that a call
    allocates, the stream whose pool it came from and the streams it was
    recorded on, and which of the buffers live when the library is called."""

    def __init__(self):
        self.buffers = {}  # address: (weak reference, stream it was allocated under)
        self.recorded = {}
        self.current = "caller"
        self.calls = []
        self.torch = types.SimpleNamespace(
            empty=self.empty_of(torch.empty), float32=torch.float32, int32=torch.int32, uint8=torch.uint8,
            cuda=types.SimpleNamespace(stream=self.stream, Stream=Stream, ExternalStream=Stream,
                                       current_stream=lambda device=None: self.current))

    def empty_of(self, real):
        """`empty`, from the allocator `real` (to stand in for it)."""
        def empty(shape, dtype=None, device=None):
            t = Buffer(real(shape, dtype=dtype))
            t.recorder = self
            self.buffers[t.data_ptr()] = (weakref.ref(t), self.current)
            return t
        return empty

    @contextlib.contextmanager
    def stream(self, s):
        held, self.current = self.current, s
        yield
        self.current = held

    def __getattr__(self, name):  # a library entry point
        def call(*args):
            addresses = [a for a in args if isinstance(a, int) and a in self.buffers]
            self.calls.append((name, args, [(self.buffers[a][0]() is not None, self.buffers[a][1])
                                            for a in addresses]))
            if name.endswith("_sizes"):
                for a in args:  # (by reference, or the object itself)
                    a = getattr(a, "_obj", a)
                    if hasattr(a, "value"):
                        a.value = 4096
            return 0
        return call


class Stream:
    def __init__(self, address=77, device=None):
        self.cuda_stream = address

    def __hash__(self):
        return self.cuda_stream

    def __eq__(self, other):
        return isinstance(other, Stream) and other.cuda_stream == self.cuda_stream


class Buffer(torch.Tensor):
    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_subclass(cls, t)

    def record_stream(self, s):
        self.recorder.recorded.setdefault(self.data_ptr(), set()).add(s)


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(spd, "lib", lambda: r)
    monkeypatch.setattr(spd, "_prompt_plans", {})
    return r


def prompt_operands(rec, monkeypatch):
    """A prompt call whose plan needs a workspace."""
    cfg = spd.spd_dense_config(4, 2, 64, 1, 0, spd.spd_score_rule(0.0, 0.0, None))
    monkeypatch.setattr(spd, "_prompt_plan", lambda q, k, v, out_dtype, scale, softcap: (
        rec.torch, cfg, 4096, tuple(q.shape), torch.float32, q.shape[0], k.shape[0]))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(9, 2, 64, dtype=torch.bfloat16)
    return q, k


@pytest.mark.parametrize("stream", [None, Stream()])
def test_prompt_workspace_lives_until_the_kernels_are_enqueued(rec, monkeypatch, stream):
    q, k = prompt_operands(rec, monkeypatch)
    monkeypatch.setattr(spd, "_raw_stream", lambda *a: 77)
    spd.prefill_attention(q, k, k, stream=stream)
    (name, args, held), = rec.calls
    work = args[-3]
    assert name == "spd_prefill_attention" and work in rec.buffers and args[-2] == 4096
    assert held and all(alive for alive, _ in held)


def stand_in_cache(rec):
    c = object.__new__(spd.SparsePagedKVCache)
    c.torch, c.ctx, c.device = rec.torch, None, torch.device("cpu")
    c.Hq, c.Hkv, c.d, c.dtype = 4, 2, 64, torch.bfloat16
    c._dev_index, c._raw_stream, c._ids_cache = -1, lambda device: 77, {}
    return c


@pytest.mark.parametrize("stream", [Stream(), 77])
def test_buffers_of_a_call_on_a_stream_come_from_its_pool(rec, monkeypatch, stream):
    """Memory from the caller's pool may still be in use there when the call's
    stream writes it, and the other way round when it is given back."""
    q, k = prompt_operands(rec, monkeypatch)
    c, w = stand_in_cache(rec), torch.zeros(1, 2, 9)
    outs = [spd.prefill_attention(q, k, k, stream=stream),
            c.shared_prefix_attention(q, 5, [0, 1, 2], stream=stream),
            *c.kv_evict([0], [1], 7, 2, w, stream=stream)]
    rec.buffers = {t.data_ptr(): rec.buffers[t.data_ptr()] for t in outs}
    offsets = types.SimpleNamespace(device=types.SimpleNamespace(type="cuda", index=0), shape=(3,),
                                    dtype=torch.int32, dim=lambda: 1, is_contiguous=lambda: True,
                                    data_ptr=lambda: 4096)
    monkeypatch.setattr(torch, "empty", rec.empty_of(torch.empty))
    monkeypatch.setattr(torch, "cuda", rec.torch.cuda)
    outs += spd.document_key_ranges(offsets, 9, stream=stream)
    assert [n for n, _, _ in rec.calls] == ["spd_prefill_attention", "spd_shared_prefix_sizes",
                                            "spd_shared_prefix_attention", "spd_kv_evict",
                                            "spd_document_key_ranges"]
    for name, _, held in rec.calls:
        assert len(held) == (0 if name.endswith("_sizes") else 2), name
        assert all(alive and under == Stream(77) for alive, under in held), name
    # the caller reads the results on its own stream, and nobody but the call a workspace
    assert rec.recorded == {t.data_ptr(): {"caller"} for t in outs}


def test_buffers_of_a_call_without_a_stream(rec, monkeypatch):
    q, k = prompt_operands(rec, monkeypatch)
    monkeypatch.setattr(spd, "_raw_stream", lambda *a: 0)
    c, w = stand_in_cache(rec), torch.zeros(1, 2, 9)
    spd.prefill_attention(q, k, k)
    c.shared_prefix_attention(q, 5, [0, 1, 2])
    c.kv_evict([0], [1], 7, 2, w)
    for _, _, held in rec.calls:
        assert all(alive and under == "caller" for alive, under in held)
    assert not rec.recorded


@pytest.mark.parametrize("stream", [None, Stream(), 77])
def test_sparse_calls_allocate_under_their_stream(rec, monkeypatch, stream):
    c = stand_in_cache(rec)
    c.cfg_dict = {"streaming": [True, False]}
    c._step_fn = rec.spd_decode_step
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    c.sparse_decode_attention(q, [0, 1, 2], stream=stream)
    c.sparse_decode_attention_stats(q, [0, 1, 2], stream=stream)
    c.sparse_decode_attention_page_mass(q, [0, 1, 2], max_pages=4, stream=stream)
    c.decode_step(q, k, k, [0, 1, 2], stream=stream)
    monkeypatch.setattr(torch, "empty", rec.empty_of(torch.empty))
    monkeypatch.setattr(torch, "cuda", rec.torch.cuda)
    monkeypatch.setattr(rec.torch.cuda, "current_stream", lambda device=None: Stream(5))
    q, k, w = torch.zeros(9, 4, 64, dtype=torch.bfloat16), torch.zeros(
        9, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 8)
    rec.buffers.clear()  # (operands may lie where a result given back was)
    spd.prefill_block_sparse_attention(q, k, k, w, w, stream=stream, check=False)
    under = "caller" if stream is None else Stream(77)
    buffers = {name: held for name, _, held in rec.calls}
    for name, n in (("spd_sparse_decode_attention", 1), ("spd_sparse_decode_attention_stats", 3),
                    ("spd_sparse_decode_attention_page_mass", 5), ("spd_decode_step", 1),
                    ("spd_prefill_block_sparse_attention", 3)):
        assert len(buffers[name]) == n and all(x == (True, under) for x in buffers[name]), name


# ---- numbers beyond the ABI's 32 bits --------------------------------------------

def test_numbers_that_32_bits_would_wrap_are_refused(rec):
    """Nothing is allocated and nothing called: as 32 bits, 2^32 + 5 would be 5."""
    c, w = stand_in_cache(rec), torch.zeros(1, 2, 9)
    for keep in (2 ** 28 + 1, 2 ** 31 + 5, 2 ** 32 + 5):
        with pytest.raises(spd.SpdError) as e:
            c.kv_evict([0], [1], keep, 2, w)
        assert e.value.name == "SPD_ERR_CAPACITY"
    for n in (0, -1, 2 ** 28 + 1, 2 ** 32 + 5):
        offsets = types.SimpleNamespace(device=types.SimpleNamespace(type="cuda", index=0), shape=(3,),
                                        dtype=torch.int32, dim=lambda: 1, is_contiguous=lambda: True,
                                        data_ptr=lambda: 4096)
        with pytest.raises(spd.SpdError) as e:
            spd.document_key_ranges(offsets, n, stream=77)
        assert e.value.name == "SPD_ERR_INVALID_ARG"
    assert not rec.calls and not rec.buffers
    for recent in (-1, -2 ** 32 + 2, 2 ** 32, 2 ** 32 + 2):
        c.kv_evict([0], [1], 7, recent, w)
        passed = rec.calls[-1][1][5]
        assert passed == (-1 if recent < 0 else 2 ** 28 + 1)  # (neither is a number that is taken)


def test_a_scale_that_a_tensor_holds_is_read_at_every_call(rec, monkeypatch):
    """The plans of prompt calls are kept by the numbers, not by what held them."""
    made = []

    def plan(q, k, v, out_dtype, scale, softcap):
        cfg = spd.spd_dense_config(4, 2, 64, 1, 0, spd._rule(scale, softcap, None, 4, None))
        made.append((float(scale), float(softcap)))
        return rec.torch, cfg, 0, tuple(q.shape), torch.float32, q.shape[0], k.shape[0]

    monkeypatch.setattr(spd, "_prompt_plan", plan)
    monkeypatch.setattr(spd, "_raw_stream", lambda *a: 0)
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(9, 2, 64, dtype=torch.bfloat16)
    scale, cap = torch.tensor(0.5), torch.tensor(30.0)
    seen = []
    for _ in range(3):
        spd.prefill_attention(q, k, k, scale=scale, softcap=cap)
        rule = rec.calls[-1][1][0].rule
        seen.append((rule.scale, rule.softcap))
        scale *= 0.5
        cap += 1
    assert seen == [(0.5, 30.0), (0.25, 31.0), (0.125, 32.0)]
    spd.prefill_attention(q, k, k, scale=0.5, softcap=30)  # the first again, by its numbers
    assert len(made) == 3
