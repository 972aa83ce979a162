"""Numbers beyond 32 bits in rotary rules and configurations: refused, never wrapped."""
import pytest

import sparse_paged_decode_logical_gb300 as spd

WRAP = 1 << 32


@pytest.mark.parametrize("bad", [
    dict(head_dim=128, sections=[WRAP + 64]), dict(head_dim=128, sections=[WRAP + 60, 4]),
    dict(head_dim=128, sections=[60, 4 - WRAP]), dict(head_dim=WRAP + 128, rotary_dim=128),
    dict(head_dim=128 - WRAP, rotary_dim=128), dict(head_dim=128, rotary_dim=WRAP + 64, sections=[32])])
def test_rotary_rules(bad):
    with pytest.raises(spd.SpdError) as e:
        spd.Rotary(**bad)
    assert e.value.name == "SPD_ERR_INVALID_ARG"


@pytest.mark.parametrize("bits", [WRAP + 8, WRAP + 4, 4 - WRAP, WRAP])
def test_bits_of_a_cache(bits):
    c = spd.make_config(num_q_heads=8, num_kv_heads=2, head_dim=128, dtype="bf16", logical_page=16,
                        physical_page=64, num_physical_pages=6, max_seqs=4, max_context=512,
                        kv_quant=bits)
    with pytest.raises(spd.SpdError) as e:
        spd.spd_query_sizes(c)
    assert e.value.name == "SPD_ERR_INVALID_ARG"
