"""4-bit weights in the layer-stack configuration (host only)."""

import json

import pytest

from bit_group_quantized_flexq_b200 import inputs, stack

BLOCK = inputs.LLAMA2_70B_BLOCK
NAMES = [n for n, *_ in BLOCK]


def config(weight4, **act):
    bits = {n: 16 if n in weight4 else 6 for n in NAMES}
    bits.update(act)
    return {"group_size": 128, "weight_bits": {n: 4 for n in weight4}, "act_bits": bits}


def test_layers_default_to_six_bits():
    assert stack.parse_weight_bits(stack.LLAMA2_70B_MIXED, BLOCK) == {n: 6 for n in NAMES}


def test_four_bit_layers_from_a_json_file(tmp_path):
    p = tmp_path / "stack.json"
    p.write_text(json.dumps(config(["gate", "up"])))
    gs, bits = stack.parse_config(str(p), BLOCK)
    assert gs == 128 and [bits[n] for n in NAMES] == [6, 6, 6, 6, 16, 16, 6]
    assert stack.parse_weight_bits(str(p), BLOCK)["gate"] == 4


@pytest.mark.parametrize("cfg, msg", [
    (config(["gate"], gate=8), "4-bit weights take 16"),
    (config([], gate=16), "not 6 or 8"),
    (dict(config([]), weight_bits={"lm_head": 4}), "unknown"),
    (dict(config([]), weight_bits={"gate": 3}), "not 4 or 6"),
    (dict(config([]), weight_bits=[4]), "must map"),
])
def test_invalid_configs_are_rejected(cfg, msg):
    with pytest.raises(ValueError, match=msg):
        stack.parse_config(cfg, BLOCK)


def test_shapes_follow_the_weight_bits():
    layers = [("odd", 200, 8192, "x")]                 # N not a multiple of 128: 4 bits only
    cfg = {"act_bits": {"odd": 16}, "weight_bits": {"odd": 4}}
    assert stack.parse_config(cfg, layers) == (128, {"odd": 16})
    with pytest.raises(ValueError, match="not supported"):
        stack.parse_config(cfg, [("odd", 200, 8200, "x")])
