"""A layer stack with 4- and 6-bit layers, between a token embedding and the
output head that shares its table: the run of a decoder's matrices."""

import numpy as np
import pytest
import torch

from bit_group_quantized_flexq_b200 import flexq, inputs, stack
from tests.w4_util import dequantize, half_step, quantize4, to64

pytestmark = pytest.mark.gpu

# the 70B block with every width divided by 16
SMALL = [(n, N // 16, K // 16, site) for (n, N, K, site) in inputs.LLAMA2_70B_BLOCK]
MIXED = {"group_size": 128, "weight_bits": {"q": 4, "v": 4, "gate": 4, "up": 4, "down": 4},
         "act_bits": {"q": 16, "k": 8, "v": 16, "o": 6, "gate": 16, "up": 16, "down": 16}}
ALL4 = {"group_size": 64, "weight_bits": {n: 4 for n, *_ in SMALL},
        "act_bits": {n: 16 for n, *_ in SMALL}}


def weights():
    # k is 64 rows wide here: 6-bit layers take multiples of 128
    return {n: inputs.weights(N, K, seed=inputs.layer_seed("w4-stack", n)) for n, N, K, _ in SMALL}


def acts(M, dtype=torch.float16):
    ks = {site: K for _, _, K, site in SMALL}
    return {site: inputs.activations(M, K, seed=M + K).to(dtype).cuda() for site, K in ks.items()}


def within(y, x, w16, gs):
    q, s = quantize4(w16.numpy(), gs)
    w64, x64 = dequantize(q, s), to64(x)
    ref, mags = x64 @ w64.T, np.abs(x64) @ np.abs(w64).T
    # FP32 sums as in the linear layers' own test, results and (in larger
    # batches) weights rounded to FP16
    tol = half_step(torch.float16) * (np.abs(ref) + mags) + 2.0 ** -16 * mags + 2.0 ** -20
    assert (np.abs(to64(y) - ref) <= tol).all()


@pytest.mark.parametrize("kw", [{}, {"group_sites": False}, {"fuse_sites": True}])
@pytest.mark.parametrize("M", [1, 7, 40])
def test_all_layers_at_four_bits(M, kw):
    w = weights()
    st = stack.LayerStack(SMALL, ALL4, weights=w, **kw)
    assert st.launches(M) == (7 if kw.get("group_sites") is False else 4)
    x = acts(M)
    out = st.forward(x)
    for name, N, K, site in SMALL:
        assert out[name].shape == (M, N)
        within(out[name], x[site], w[name], 64)


def test_mixed_widths_equal_the_calls_they_are_made_of():
    layers = [(n, max(N, 128), K, site) for n, N, K, site in SMALL]
    w = {n: inputs.weights(N, K, seed=inputs.layer_seed("w4-mix", n)) for n, N, K, _ in layers}
    st = stack.LayerStack(layers, MIXED, weights=w)
    x = acts(5)
    out = st.forward(x)
    q = flexq.linear4_group(x["attn_in"], [st.layer_weights(n) for n in ("q", "v")], 128)
    assert torch.equal(out["q"], q[0]) and torch.equal(out["v"], q[1])
    assert torch.equal(out["k"], flexq.linear_group(x["attn_in"], [st.layer_weights("k")], 128, 8)[0])
    assert torch.equal(out["o"], flexq.linear_group(x["attn_out"], [st.layer_weights("o")], 128, 6)[0])
    assert torch.equal(out["down"], flexq.linear4(x["mlp_act"], *st.layer_weights("down"), 128))
    given = {n: torch.empty_like(t) for n, t in out.items()}
    again = st.forward(x, out=given)
    assert all(again[n] is given[n] and torch.equal(again[n], out[n]) for n in out)
    assert flexq.device_status()[0] == flexq.FLEXQ_OK


@pytest.mark.parametrize("tokens", [1, 6, 70])
def test_from_tokens_through_the_stack_to_the_tied_head(tokens):
    V, K, gs = 503, 512, 64
    table = inputs.weights(V, K, seed=5)
    wp, ws = flexq.quantize_weight4(table.cuda(), gs)
    ids = torch.randint(0, V, (tokens,), generator=torch.Generator().manual_seed(tokens)).cuda()
    w = weights()
    st = stack.LayerStack(SMALL, ALL4, weights=w)
    x = flexq.embedding(ids, wp, ws, V, gs, scale=K ** 0.5)
    out = st.forward({"attn_in": x, "attn_out": x, "mlp_in": x, "mlp_act": acts(tokens)["mlp_act"]})
    within(out["q"], x, w["q"], gs)
    head = flexq.linear4(out["o"], wp, ws, V, gs)
    within(head, out["o"], table, gs)
    # and back: the gradient of the looked-up rows through the head's own dY
    rows, scales = flexq.embedding_backward(x, ids, wp, V, gs, scale=K ** 0.5,
                                            table_dtype=torch.float32)
    assert torch.isfinite(rows).all() and scales.shape == ws.shape
    missing = torch.ones(V, dtype=torch.bool)
    missing[ids.cpu()] = False
    assert (rows.cpu()[missing] == 0).all() and (scales.cpu()[missing] == 0).all()
