"""CPU-only checks of the grouped-routing entry points' argument validation
(no call here reaches a kernel)."""
import ctypes

import pytest
import torch

import aware_expert_routing_amd as moe

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation


def _route(logits=FAKE, dt=0, bias=None, B=4, N=64, k=4, score=1, G=8, tg=2, gs=1, renorm=1, scale=1.0, idx=FAKE,
           w=FAKE):
    return moe.lib().moe_route_grouped(logits, dt, bias, B, N, k, score, G, tg, gs, renorm, scale, None, idx, w, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), -1), (dict(idx=None), -1), (dict(w=None), -1), (dict(dt=2), -1),
    (dict(logits=ctypes.c_void_p((1 << 20) + 2)), -1), (dict(dt=1, logits=ctypes.c_void_p((1 << 20) + 1)), -1),
    (dict(N=0), -1), (dict(N=513, G=1, tg=1), -2), (dict(k=0), -1), (dict(k=65, G=1, tg=1), -1),
    (dict(k=33, G=1, tg=1), -2), (dict(B=0), -1), (dict(B=-1), -1), (dict(B=(1 << 20) + 1), -2),
    (dict(score=2), -1), (dict(gs=2), -1), (dict(G=0), -1), (dict(G=7), -1), (dict(N=128, G=128), -2),
    (dict(tg=0), -1), (dict(tg=9), -1), (dict(k=17), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1),
])
def test_route_grouped_rejects(kw, status):
    assert _route(**kw) == status
    assert moe.lib().moe_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(N=129, G=1, tg=1), -2), (dict(B=129), -2), (dict(k=17, G=1, tg=1), -2), (dict(cnt=None), -1),
    (dict(sync=None), -1), (dict(T=None), -1),
])
def test_route_grouped_dispatch_rejects(kw, status):
    a = dict(B=4, N=64, k=4, G=8, tg=2, cnt=FAKE, T=FAKE, sync=FAKE)
    a.update(kw)
    assert moe.lib().moe_route_grouped_dispatch(FAKE, 0, None, a["B"], a["N"], a["k"], 1, a["G"], a["tg"], 1, 1, 1.0,
                                                None, FAKE, FAKE, a["cnt"], FAKE, FAKE, FAKE, a["T"], a["sync"],
                                                None) == status


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="GPU"):
        moe.route_grouped(torch.zeros(4, 64), 4)
    with pytest.raises(TypeError):
        moe.route_grouped([[0.0] * 64], 4)
    with pytest.raises(ValueError, match="GPU"):
        moe.route_grouped_dispatch(torch.zeros(4, 64), 4)
