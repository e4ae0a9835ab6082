"""The layer with the grouped router, the routed experts, the shared expert
and its adapters together, against the oracle (routed experts) plus the 64-bit
definitions of the rest."""
import numpy as np
import pytest
import torch

import aware_expert_routing_amd as moe
import grouped_ref
import lora_ref
import oracle
import synth
from gpu_util import DEV, bf16_dev, build_layer

pytestmark = pytest.mark.gpu


def _tables(seed, H, I, n, ranks):
    shapes = [(H, I), (H, I), (I, H)]
    host = [lora_ref.make_table(seed + j, n, *s, ranks) for j, s in enumerate(shapes)]
    dev = []
    for t, s in zip(host, shapes):
        d = moe.LoraTable(n, *s, max(ranks), DEV)
        for a, (A, B, sc) in enumerate(t):
            d.publish(a, A.to(DEV), B.to(DEV), sc)
        dev.append(d)
    return host, dev


def _make(seed, N, k, H, I, I_s, n, ranks=(16, 8)):
    layer, host = build_layer(N, k, H, I, seed, "bf16")
    mats = [torch.from_numpy(synth.bf16_bits_to_f32(m)).to(torch.bfloat16)
            for m in synth.expert_weights_bf16(seed, 5000, H, I_s)]
    shared = moe.ExpertTensors.pack(moe.MOE_W_BF16, *[m.to(DEV) for m in mats])
    tabs, loras = _tables(seed, H, I_s, n, ranks)
    bias = synth.normal((seed, 8), N, 0.05)
    g = moe.GroupedRouting("sigmoid", torch.from_numpy(bias).to(DEV), 4, 2, "top2", True, 2.5)
    full = moe.MoELayer(H, I, N, k, layer.w_r, layer.experts, DEV, grouped=g, shared=shared, loras=loras)
    return full, host, mats, tabs, bias


def _expect(layer, host, mats, tabs, bias, logits, x, ids, nv):
    B = x.shape[0]
    ri, rw = grouped_ref.route_grouped(logits, layer.k, "sigmoid", bias, 4, 2, "top2", True, 2.5, nv)
    y = oracle.expert_ffn(host, layer.H, layer.I, x, ri, rw.astype(np.float32)).astype(np.float64)
    sh = lora_ref.shared(torch.from_numpy(x).double(), *mats, tabs, ids).numpy()
    m = B if nv is None else min(nv, B)
    y[:m] += sh[:m]
    return ri, y


@pytest.mark.parametrize("B,nv", [(1, None), (5, None), (16, 9), (64, None), (128, 100)])
def test_layer_together(B, nv):
    N, k, H, I, I_s, n = 32, 4, 256, 128, 160, 6
    layer, host, mats, tabs, bias = _make(40 + B, N, k, H, I, I_s, n)
    xb = synth.to_bf16_bits(synth.activations(B, B, H))
    x = synth.bf16_bits_to_f32(xb)
    logits = synth.logits(B, B, N)
    ids = torch.from_numpy(synth.rng(B, 1).integers(-1, n, B).astype(np.int32))
    n_valid = None if nv is None else torch.tensor([nv], dtype=torch.int32, device=DEV)
    buf = layer.forward(bf16_dev(xb), "grouped", logits=torch.from_numpy(logits).to(DEV), n_valid=n_valid,
                        adapter=ids.to(DEV))
    ri, yref = _expect(layer, host, mats, tabs, bias, logits, x, ids, nv)
    assert np.array_equal(buf.route["idx"].cpu().numpy(), ri)
    for name, ref in grouped_ref.dispatch(ri, N).items():
        assert np.array_equal(buf.disp[name].cpu().numpy(), ref), name
    err = np.abs(buf.y.cpu().numpy() - yref).max()
    assert err <= 1e-2 * np.sqrt(np.mean(yref ** 2))   # the expert FFN's bar


def test_router_on_the_gpu_and_modes_beside_it():
    N, k, H, I, I_s, n, B = 32, 4, 256, 128, 96, 3, 20
    layer, host, mats, tabs, bias = _make(91, N, k, H, I, I_s, n)
    xb = synth.to_bf16_bits(synth.activations(7, B, H))
    x = bf16_dev(xb)
    ids = torch.from_numpy((np.arange(B) % (n + 1) - 1).astype(np.int32)).to(DEV)
    buf = layer.forward(x, "grouped", adapter=ids)
    # (the GPU's own logits route: their rounding is the router GEMV's matter)
    ri, yref = _expect(layer, host, mats, tabs, bias, buf.logits.cpu().numpy(), synth.bf16_bits_to_f32(xb), ids.cpu(),
                       None)
    assert np.array_equal(buf.route["idx"].cpu().numpy(), ri)
    assert np.abs(buf.y.cpu().numpy() - yref).max() <= 1e-2 * np.sqrt(np.mean(yref ** 2))
    # the other modes add the same shared expert to the routed part they always gave
    plain = moe.MoELayer(H, I, N, k, layer.w_r, layer.experts, DEV)
    for mode in ("topk", "oea", "pruned"):
        y0 = plain.forward(x, mode, 2).y.clone()
        y1 = layer.forward(x, mode, 2, adapter=ids).y.clone()
        extra = moe.shared_ffn(x, layer.shared, layer.loras, ids, y_dtype=torch.float32)
        assert torch.equal(y0 + extra, y1)


def test_captured_layer_follows_ids_adapters_and_padding():
    N, k, H, I, I_s, n, B = 32, 4, 256, 128, 128, 4, 24
    layer, host, mats, tabs, bias = _make(77, N, k, H, I, I_s, n)
    x = torch.zeros(B, H, device=DEV, dtype=torch.bfloat16)
    ids = torch.full((B,), -1, device=DEV, dtype=torch.int32)
    n_valid = torch.tensor([B], dtype=torch.int32, device=DEV)
    graph = layer.capture(x, "grouped", n_valid=n_valid, adapter=ids)
    eager = moe.MoELayer(H, I, N, k, layer.w_r, layer.experts, DEV, grouped=layer.grouped, shared=layer.shared,
                         loras=layer.loras)
    for step, nv in enumerate((B, 11, 1, B)):
        x.copy_(bf16_dev(synth.to_bf16_bits(synth.activations(step, B, H))))
        ids.copy_(torch.from_numpy(synth.rng(step, 2).integers(-1, n, B).astype(np.int32)))
        n_valid.fill_(nv)
        if step == 2:   # another adapter under the same handle
            A, Bm, s = lora_ref.make_table(500, 1, H, I_s, (16,))[0]
            layer.loras[0].publish(1, A.to(DEV), Bm.to(DEV), s)
        graph.replay()
        torch.cuda.synchronize()
        got = layer.buffers(B)
        want = eager.forward(x, "grouped", n_valid=n_valid, adapter=ids)
        torch.cuda.synchronize()
        assert torch.equal(got.y, want.y) and torch.equal(got.route["idx"], want.route["idx"])


def test_mode_grouped_needs_its_router():
    layer, _ = build_layer(16, 2, 64, 32, 3, "bf16")
    with pytest.raises(ValueError, match="GroupedRouting"):
        layer.forward(torch.zeros(2, 64, device=DEV, dtype=torch.bfloat16), "grouped")
    with pytest.raises(ValueError, match="adapter"):
        layer.forward(torch.zeros(2, 64, device=DEV, dtype=torch.bfloat16), "topk",
                      adapter=torch.zeros(2, device=DEV, dtype=torch.int32))
