"""Steps and codes of a quantised cache where fp32's difference of two values is not exact."""
import pytest
import torch

from quant_ref import FLOOR, STEP, held, quantise
from test_gpu_quant import DT, cache

pytestmark = pytest.mark.gpu


def step_at(levels, dtype):
    """A power of 2 that levels of reach far beyond 2^24 times TINY."""
    return 2.0 ** 24 if dtype == "bf16" else 2.0 ** 7


TINY = 2.0 ** -14


def row_just_beyond(bits, dtype):
    """From -TINY to levels steps of a power of 2: the span rounds to levels steps, and is more."""
    levels, size = 2 ** bits - 1, step_at(bits, dtype)
    x = torch.arange(128) % (levels + 1) * size
    x[::32] = -TINY
    x[1::32] = levels * size
    return x


def row_of_ties(bits, dtype):
    """From TINY to levels steps: distances of values half way between two codes round onto the
    middle, and lie below it."""
    levels, size = 2 ** bits - 1, step_at(bits, dtype)
    n = torch.arange(128) % min(levels, 127)
    x = (n + 0.5) * size
    x[::32] = TINY
    x[1::32] = levels * size
    return x


@pytest.mark.parametrize("row", [row_just_beyond, row_of_ties])
@pytest.mark.parametrize("tokens", [1, 16, 21])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_least_steps_and_nearest_codes(row, tokens, bits, dtype):
    dt = DT[dtype]
    x = row(bits, dtype).to(dt)
    assert torch.equal(x.double(), row(bits, dtype).double())  # (numbers of the type)
    x = torch.stack([x, -x.flip(0)]).cuda()  # (two heads)
    c = cache(2, 2, 128, dtype, bits, tokens)
    s = c.seq_create()
    rows = x[None, None].expand(1, tokens, 2, 128).contiguous()
    c.kv_append([s], rows, rows)
    ref, mag = held(x, bits)
    for y in c.kv_read([s]):
        err = (y[0].double() - ref.clamp(max=torch.finfo(dt).max)).abs()
        assert bool((err <= STEP[dt] * ref.abs() + 2.0 ** -23 * mag + FLOOR[dt]).all())
    # equal rows: the output is the value before its rounding to 16 bits (weights cut off to 22
    # bits, and at most 2 roundings a token of sums of lowest values and steps)
    q = torch.zeros(1, 2, 128, dtype=dt, device="cuda")
    got = c.quant_decode_attention(q, [s])[0].double()
    lo, step, _ = quantise(x, bits)
    assert bool(((got - ref).abs() <= 2.0 ** -18 * (lo.abs() + step * (2 ** bits - 1))).all())
    c.check_status()
