"""Gradients of rotary positions: against the formula and differences on the GPU; what the
backward pass calls, on the CPU with a recorder in the library's place."""
import types

import pytest
import torch

import sparse_paged_decode_logical_gb300 as spd
from quant_ref import FLOOR, STEP, axes_of, frequencies, turn
from test_dense_calls import Recorder

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
TABLE = types.SimpleNamespace(table="table", axes=1, head_dim=64)


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(spd, "lib", lambda: r)
    monkeypatch.setattr(spd, "_raw_stream", lambda *a: 0)
    # a plan as a CUDA tensor's would be
    monkeypatch.setattr(spd, "_rotary_plan", lambda table, positions, q, k: (
        torch, 1, q.shape[0], q.dtype, torch.device("cpu"), tuple(q.shape), q.stride(0),
        None if k is None else tuple(k.shape), 0 if k is None else k.stride(0)))
    monkeypatch.setattr(spd, "_rotary_plans", {})
    return r


def operands(grad=(True, True)):
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    return torch.zeros(3, dtype=torch.int32), q.requires_grad_(grad[0]), k.requires_grad_(grad[1])


def calls(rec):
    """(rotated rows, whether keys came along, inverse) of every call."""
    return [(a[6], a[7] is not None, a[14]) for name, a, _ in rec.calls if name == "spd_rotary"]


def test_the_backward_pass_rotates_back(rec):
    pos, q, k = operands()
    a, b = spd.rotary(TABLE, pos, q, k)
    assert a.requires_grad and b.requires_grad
    (a.sum() + b.sum()).backward()  # (gradients that are broadcast from one number)
    assert calls(rec) == [(4, True, 0), (4, True, 1)]
    assert q.grad.shape == q.shape and k.grad.shape == k.shape


def test_only_what_asks_for_a_gradient_is_rotated_back(rec):
    pos, q, k = operands((False, True))
    a, b = spd.rotary(TABLE, pos, q, k, inverse=True)
    b.sum().backward()
    assert calls(rec) == [(4, True, 1), (2, False, 0)] and q.grad is None
    pos, q, k = operands()
    a, b = spd.rotary(TABLE, pos, q, k)
    a.sum().backward()  # (the rotated keys go nowhere)
    assert calls(rec)[-1] == (4, False, 1) and k.grad is None
    q = operands()[1]
    spd.rotary(TABLE, pos, q).sum().backward()
    assert calls(rec)[-1] == (4, False, 1) and q.grad.shape == q.shape


def test_what_asks_for_no_gradient_comes_back_without_one(rec):
    for grad in ((True, False), (False, True)):
        pos, q, k = operands(grad)
        assert tuple(y.requires_grad for y in spd.rotary(TABLE, pos, q, k)) == grad
    pos, q, k = operands((False, False))
    assert not any(y.requires_grad for y in spd.rotary(TABLE, pos, q, k))


def test_nothing_is_kept_where_no_gradient_is_asked_for(rec):
    pos, q, k = operands()
    with torch.no_grad():
        a, b = spd.rotary(TABLE, pos, q, k)
    assert not a.requires_grad and not b.requires_grad
    spd.rotary(TABLE, pos, q.detach(), k.detach(), out=(q.detach(), k.detach()))
    n = len(rec.calls)
    for out in (torch.empty_like(q), q):
        with pytest.raises(ValueError):
            spd.rotary(TABLE, pos, q, out=out)
    with pytest.raises(ValueError):
        spd.rotary(TABLE, pos, q.detach(), k, out=(torch.empty_like(q), torch.empty_like(k)))
    assert len(rec.calls) == n


# ---- on the GPU -----------------------------------------------------------------------

def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def rule(neighbours):
    return spd.Rotary(64, rotary_dim=48, sections=[10, 14], neighbours=neighbours), \
        (frequencies(48), axes_of([10, 14], False), neighbours)


def close(got, ref, mag, dt):
    assert got.dtype == dt
    assert bool(((got.double() - ref).abs() <= mag * 2.0 ** -21 + STEP[dt] * ref.abs() + FLOOR[dt]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradients_are_the_rotation_back(dtype, neighbours, inverse):
    """Of rows of a fused projection, whose own gradient is gathered; outputs weighted by hand, so
    that the gradients that come in are strided, broadcast or ordinary."""
    dt, n, hq, hk, d = DT[dtype], 37, 6, 2, 64
    t, how = rule(neighbours)
    pos = torch.randint(0, 1000, (2, n), device="cuda", dtype=torch.int32)
    row = normal(1, n, (hq + hk) * d, dtype=dt).requires_grad_()
    q, k = row[:, :hq * d].unflatten(1, (hq, d)), row[:, hq * d:].unflatten(1, (hk, d))
    a, b = spd.rotary(t, pos, q, k, inverse=inverse)
    for x, y in ((q, a), (k, b)):
        close(y.detach(), *turn(x.detach(), pos, *how, inverse), dt)
    w = normal(2, n, d, hq, dtype=dt).transpose(1, 2)
    one = normal(3, d, dtype=dt)
    ((a * w).sum() + (b * one).sum()).backward()
    got = row.grad.unflatten(1, (hq + hk, d))
    for g, back in ((w, got[:, :hq]), (one.expand(n, hk, d), got[:, hq:])):
        close(back, *turn(g, pos, *how, not inverse), dt)


@pytest.mark.gpu
def test_gradients_against_differences():
    """The rotation is linear: <R(x + e) - R x, y> is <e, gradient>, for every e of one channel."""
    n, h, d = 9, 3, 64
    t, _ = rule(True)
    pos = torch.randint(0, 1000, (2, n), device="cuda", dtype=torch.int32)
    x = normal(1, n, h, d, dtype=torch.float16).requires_grad_()
    y = normal(2, n, h, d, dtype=torch.float16)
    (spd.rotary(t, pos, x).double() * y.double()).sum().backward()
    with torch.no_grad():
        for i in (0, 7, 47, 48, 63):
            e = torch.zeros_like(x)
            e[:, :, i] = 0.5
            diff = ((spd.rotary(t, pos, x + e).double() - spd.rotary(t, pos, x).double()) * y.double()).sum(-1)
            # (three roundings of half a step of at most |x| + 0.5 + |its partner|)
            mag = (x.double().abs().amax(-1) * 2 + 1) * y.double().abs().sum(-1)
            err = (diff / 0.5 - x.grad.double()[:, :, i]).abs()
            assert bool((err <= 6 * 2.0 ** -11 * mag).all())


@pytest.mark.gpu
def test_gradients_of_gradients_and_of_other_streams():
    n, h, d, dt = 21, 4, 64, torch.bfloat16
    t, how = rule(False)
    pos = torch.randint(0, 1000, (2, n), device="cuda", dtype=torch.int32)
    x, y = normal(1, n, h, d, dtype=dt).requires_grad_(), normal(2, n, h, d, dtype=dt).requires_grad_()
    g, = torch.autograd.grad(spd.rotary(t, pos, x), x, y, create_graph=True)
    close(g.detach(), *turn(y.detach(), pos, *how, True), dt)
    z = normal(3, n, h, d, dtype=dt)
    gg, = torch.autograd.grad(g, y, z)
    close(gg, *turn(z, pos, *how), dt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = spd.rotary(t, pos, x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    (out * z).sum().backward()
    close(x.grad, *turn(z, pos, *how, True), dt)
    with torch.cuda.stream(side):
        x.grad = None
        (spd.rotary(t, pos, x) * z).sum().backward()
    torch.cuda.current_stream().wait_stream(side)
    close(x.grad, *turn(z, pos, *how, True), dt)


@pytest.mark.gpu
def test_forward_and_backward_captured_and_replayed():
    n, h, d, dt = 21, 4, 64, torch.bfloat16
    t, how = rule(False)
    pos = torch.randint(0, 1000, (2, n), device="cuda", dtype=torch.int32)
    x, w = normal(1, n, h, d, dtype=dt).requires_grad_(), normal(2, n, h, d, dtype=dt)

    def step():
        return torch.autograd.grad(spd.rotary(t, pos, x), x, w)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (5, 6):
        w.copy_(normal(seed, n, h, d, dtype=dt))
        pos.copy_(torch.randint(0, 1000, (2, n), device="cuda", dtype=torch.int32))
        graph.replay()
        close(held, *turn(w, pos, *how, True), dt)
