"""Grouped routing (moe_route_grouped, moe_route_grouped_dispatch) against its
definition in 64 bits (grouped_ref): indices and dispatch lists exactly, gate
weights within 1e-6 of themselves (the library's bar for gate weights; one
fp32 rounding is 2^-24, 6e-8, and the scores' own error stays below that)."""
import numpy as np
import pytest
import torch

import aware_expert_routing_amd as moe
import grouped_ref
import synth
from gpu_util import DEV

pytestmark = pytest.mark.gpu


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _check(idx, w, ri, rw):
    assert np.array_equal(idx.cpu().numpy(), ri)
    g = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(g - rw) <= 1e-6 * np.abs(rw) + 1e-38)


def _inputs(seed, B, N, bias):
    favour = synth.normal((seed, 1), N, 0.7)
    logits = synth.normal((seed, 2), (B, N), 1.3) + favour
    return logits.astype(np.float32), ((-0.1 * favour + synth.normal((seed, 3), N, 0.02)).astype(np.float32)
                                       if bias else None)


CASES = [   # B, N, k, groups, topk_group
    (1, 256, 8, 8, 4), (1, 1, 1, 1, 1), (1, 2, 2, 1, 1), (3, 7, 7, 1, 1), (5, 64, 1, 64, 1), (5, 64, 6, 64, 6),
    (17, 65, 16, 1, 1), (33, 160, 6, 8, 3), (64, 128, 8, 2, 1), (130, 512, 32, 16, 5), (129, 511, 10, 1, 1),
    (257, 384, 8, 3, 2), (40, 96, 12, 4, 1), (1000, 256, 8, 8, 4), (9, 66, 4, 33, 2), (31, 20, 20, 10, 10),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("B,N,k,G,tg", CASES)
def test_matches_the_definition(B, N, k, G, tg, group_score, bias, score):
    seed = B * 1000 + N
    logits, b = _inputs(seed, B, N, bias)
    renorm, scale = (seed % 2 == 0), (2.5 if seed % 3 else 1.0)
    idx, w = moe.route_grouped(_dev(logits), k, score=score, bias=_dev(b), n_group=G, topk_group=tg,
                               group_score=group_score, renorm=renorm, scale=scale)
    _check(idx, w, *grouped_ref.route_grouped(logits, k, score, b, G, tg, group_score, renorm, scale))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_bf16_logits_with_ties(score, bias):
    # bf16 logits on a coarse grid: many equal logits, and with a constant bias many equal selection values
    B, N, k, G, tg = 70, 96, 7, 6, 3
    logits = synth.tied_logits(5, B, N, 5)
    b = np.full(N, 0.125, np.float32) if bias else None
    x = torch.from_numpy(logits).to(DEV).to(torch.bfloat16)
    for gs in ("max", "top2"):
        idx, w = moe.route_grouped(x, k, score=score, bias=_dev(b), n_group=G, topk_group=tg, group_score=gs)
        _check(idx, w, *grouped_ref.route_grouped(x.float().cpu().numpy(), k, score, b, G, tg, gs, True, 1.0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B,N", [(1, 64), (50, 128), (300, 250)])
def test_values_closer_than_an_fp32_rounding(score, B, N):
    """Bias values that bring every expert's selection value to the same fp32
    neighbourhood: the order is the 64-bit one."""
    row = synth.normal((B, N, 9), N, 1.0).astype(np.float32)
    logits = np.repeat(row[None], B, 0)
    s = np.exp(row.astype(np.float64) - row.max())
    s = s / s.sum() if score == "softmax" else 1.0 / (1.0 + np.exp(-row.astype(np.float64)))
    b = (0.5 - s).astype(np.float32)   # s + b = 0.5 up to the rounding of b
    # other rows: one logit moved a little, so that each row's order is its own
    for i in range(1, B):
        logits[i, i % N] = np.nextafter(logits[i, i % N], np.float32(10), dtype=np.float32)
    for G, tg, gs in ((1, 1, "max"), (2, 1, "top2"), (2, 1, "max")):
        k = min(8, N // G)
        idx, w = moe.route_grouped(_dev(logits), k, score=score, bias=_dev(b), n_group=G, topk_group=tg,
                                   group_score=gs)
        _check(idx, w, *grouped_ref.route_grouped(logits, k, score, b, G, tg, gs, True, 1.0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_masked_experts_and_empty_rows(score, bias):
    B, N, k, G, tg = 24, 64, 8, 8, 3
    logits, b = _inputs(77, B, N, bias)
    g = synth.rng(78)
    logits[g.random((B, N)) < 0.5] = -np.inf
    logits[g.random((B, N)) < 0.1] = np.nan
    logits[0] = -np.inf            # nothing left
    logits[1] = np.nan
    logits[2] = -np.inf
    logits[2, 13] = 0.25           # one expert left
    logits[3, ::8] = np.finfo(np.float32).min   # the lowest float is not a mask
    logits[4, 5] = np.inf          # counts as the largest float
    logits[5, 5] = logits[5, 40] = np.inf
    logits[6] = np.finfo(np.float32).min
    if bias:
        b[3] = -np.inf
        b[17] = np.nan
        b[30] = np.inf
    for gs in ("max", "top2"):
        for renorm in (True, False):
            idx, w = moe.route_grouped(_dev(logits), k, score=score, bias=_dev(b), n_group=G, topk_group=tg,
                                       group_score=gs, renorm=renorm, scale=2.0)
            _check(idx, w, *grouped_ref.route_grouped(logits, k, score, b, G, tg, gs, renorm, 2.0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_differences_of_logits_past_the_largest_float(score):
    # l - max overflows to -inf: such an expert scores 0 and stays selectable
    low = np.finfo(np.float32).min
    logits, _ = _inputs(79, 4, 32, False)
    logits[0, 7], logits[0, 9:25] = np.inf, low
    logits[1, ::2], logits[1, 1] = low, np.float32(2e38)
    logits[2], logits[2, 3] = low, np.inf
    logits[3, :8] = np.linspace(-3e38, 3e38, 8).astype(np.float32)
    for renorm in (True, False):
        idx, w = moe.route_grouped(_dev(logits), 6, score=score, n_group=4, topk_group=3, group_score="max",
                                   renorm=renorm)
        _check(idx, w, *grouped_ref.route_grouped(logits, 6, score, None, 4, 3, "max", renorm, 1.0))


def test_large_logits_keep_their_order():
    # sigmoid scores that are all 0 or 1 to fp32: without a bias the logits rank the experts
    logits = (synth.normal(3, (6, 40), 1.0) * np.float32(60)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        idx, _ = moe.route_grouped(_dev(logits), 5, score=score, n_group=4, topk_group=2, group_score="max")
        ri, _ = grouped_ref.route_grouped(logits, 5, score, None, 4, 2, "max", True, 1.0)
        assert np.array_equal(idx.cpu().numpy(), ri)


@pytest.mark.parametrize("nv", [0, 1, 6, 9])
def test_padding_tokens(nv):
    logits, b = _inputs(5, 9, 64, True)
    n_valid = torch.tensor([nv], dtype=torch.int32, device=DEV)
    idx, w = moe.route_grouped(_dev(logits), 4, bias=_dev(b), n_group=4, topk_group=2, n_valid=n_valid)
    _check(idx, w, *grouped_ref.route_grouped(logits, 4, "sigmoid", b, 4, 2, "top2", True, 1.0, nv))


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_logits_at_odd_offsets(offset):
    # rows of an odd number of experts inside a larger allocation: element alignment only
    B, N = 21, 33
    for dt in (torch.float32, torch.bfloat16):
        flat = torch.zeros(offset + B * N, device=DEV, dtype=dt)
        x = flat[offset:].view(B, N)
        x.copy_(_dev(synth.normal(8, (B, N))))
        idx, w = moe.route_grouped(x, 5, score="softmax", n_group=3, topk_group=2, group_score="max")
        _check(idx, w, *grouped_ref.route_grouped(x.float().cpu().numpy(), 5, "softmax", None, 3, 2, "max", True, 1.0))


@pytest.mark.parametrize("B,N,k,G,tg,nv", [
    (1, 128, 8, 8, 4, None), (1, 1, 1, 1, 1, None), (16, 128, 8, 8, 4, None), (48, 96, 6, 6, 3, None),
    (49, 127, 16, 1, 1, None), (100, 64, 8, 4, 2, 63), (128, 128, 8, 8, 4, None), (128, 128, 16, 1, 1, 0),
])
def test_dispatch_lists(B, N, k, G, tg, nv):
    logits, b = _inputs(B + N, B, N, True)
    logits[::5, ::3] = -np.inf
    if B > 2:
        logits[2] = -np.inf
    n_valid = None if nv is None else torch.tensor([nv], dtype=torch.int32, device=DEV)
    sync = torch.zeros(1, dtype=torch.int32, device=DEV)
    ri, rw = grouped_ref.route_grouped(logits, k, "sigmoid", b, G, tg, "top2", True, 2.5, nv)
    rd = grouped_ref.dispatch(ri, N)
    for _ in range(2):   # the sync word is left as it was
        route, disp = moe.route_grouped_dispatch(_dev(logits), k, bias=_dev(b), n_group=G, topk_group=tg, scale=2.5,
                                                 n_valid=n_valid, sync=sync)
        _check(route["idx"], route["w"], ri, rw)
        for name, ref in rd.items():
            assert np.array_equal(disp[name].cpu().numpy(), ref), name
        assert int(sync.item()) == 0


def test_graph_replays_follow_the_inputs():
    B, N, k = 96, 128, 8
    x = torch.empty(B, N, device=DEV)
    _, b = _inputs(1, B, N, True)
    bias = _dev(b)
    n_valid = torch.tensor([B], dtype=torch.int32, device=DEV)
    sync = torch.zeros(1, dtype=torch.int32, device=DEV)
    i32 = dict(device=DEV, dtype=torch.int32)
    route = dict(idx=torch.empty(B, k, **i32), w=torch.empty(B, k, device=DEV))
    disp = dict(cnt=torch.empty(N, **i32), offsets=torch.empty(N + 1, **i32), perm=torch.empty(B * k, **i32),
                active=torch.empty(N, **i32), T=torch.empty(1, **i32))

    def call():
        moe.route_grouped_dispatch(x, k, bias=bias, n_group=8, topk_group=4, n_valid=n_valid, route=route, disp=disp,
                                   sync=sync)

    x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed, nv in ((11, B), (12, 50), (13, 0), (14, B)):
        logits, _ = _inputs(seed, B, N, True)
        x.copy_(_dev(logits))
        n_valid.fill_(nv)
        graph.replay()
        torch.cuda.synchronize()
        ri, rw = grouped_ref.route_grouped(logits, k, "sigmoid", b, 8, 4, "top2", True, 1.0, nv)
        _check(route["idx"], route["w"], ri, rw)
        for name, ref in grouped_ref.dispatch(ri, N).items():
            assert np.array_equal(disp[name].cpu().numpy(), ref), (seed, name)


def test_side_stream():
    logits, b = _inputs(4, 200, 256, True)
    ri, rw = grouped_ref.route_grouped(logits, 8, "sigmoid", b, 8, 4, "top2", True, 1.0)
    x, bias = _dev(logits), _dev(b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    idx = torch.empty(200, 8, device=DEV, dtype=torch.int32)
    w = torch.empty(200, 8, device=DEV)
    moe.route_grouped(x, 8, bias=bias, n_group=8, topk_group=4, idx=idx, w=w, stream=st)
    st.synchronize()
    _check(idx, w, ri, rw)


def test_tensors_are_checked():
    x = torch.zeros(4, 64, device=DEV)
    for bad in (torch.zeros(4, 64), torch.zeros(64, 4, device=DEV).t(), torch.zeros(4, 64, device=DEV).double(),
                torch.zeros(64, device=DEV)):
        with pytest.raises((ValueError, TypeError)):
            moe.route_grouped(bad, 4)
    for kw in (dict(bias=torch.zeros(63, device=DEV)), dict(bias=torch.zeros(64)),
               dict(bias=torch.zeros(64, device=DEV).half()), dict(idx=torch.zeros(4, 5, device=DEV, dtype=torch.int32)),
               dict(w=torch.zeros(4, 4, device=DEV).double()), dict(score="tanh"), dict(group_score="sum"),
               dict(n_valid=torch.zeros(1, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            moe.route_grouped(x, 4, **kw)
    with pytest.raises(moe.MoeError):
        moe.route_grouped(x, 65)
    with pytest.raises(moe.MoeError):
        moe.route_grouped(x, 4, n_group=5)


def test_offsets_past_32_bits():
    B, N = 2 ** 20, 512   # the largest call: 2 GiB of fp32 logits
    gen = torch.Generator(device=DEV).manual_seed(7)
    logits = torch.randn(B, N, generator=gen, device=DEV) * 1.5
    _, bias = _inputs(81, 1, N, True)
    idx, w = moe.route_grouped(logits, 32, bias=_dev(bias), n_group=8, topk_group=4, scale=2.5)
    at = torch.cat([torch.arange(20), torch.arange(B // 2 - 20, B // 2 + 20), torch.arange(B - 20, B)]).to(DEV)
    ref = grouped_ref.route_grouped(logits[at].cpu().numpy(), 32, "sigmoid", bias, 8, 4, "top2", True, 2.5)
    _check(idx[at], w[at], *ref)
