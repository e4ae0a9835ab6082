"""The projection with adapters (moe_lora_linear) and the shared expert
(moe_shared_ffn) against their definitions in 64 bits (lora_ref).

Bounds, with u = 2^-23 for an fp32 addition (the matrix units may truncate):
  a sum of n exact products  <= n u sum|products| at each element, and by the
  random walk of its roundings <= 2 sqrt(n) 2^-24 of the result in the 2-norm;
  v = s A x is such a sum with one more rounding; it enters B v exactly (fp32 y)
  or cut to 16 bits, 2^-15 (bf16 y: two terms of 8 bits, the rest dropped);
  a bf16 y adds half a step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import aware_expert_routing_amd as moe
import lora_ref
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _table(entries, H, O, max_rank=None):
    top = max([e[0].shape[0] for e in entries if e is not None], default=1)
    t = moe.LoraTable(len(entries), H, O, top if max_rank is None else max_rank, DEV)
    for a, e in enumerate(entries):
        if e is not None:
            t.publish(a, e[0].to(DEV), e[1].to(DEV), e[2])
    return t


def _weights(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * 0.05).to(torch.bfloat16)


def _acts(seed, B, H, dt):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, H, generator=g).to(DT[dt])


def _ids(seed, B, n, runs=False):
    g = torch.Generator().manual_seed(seed)
    if runs:
        return (torch.arange(B) * (n + 1) // B - 1).to(torch.int32)
    return torch.randint(-1, n, (B,), generator=g).to(torch.int32)


def _pack(W):
    return moe.pack_weights(moe.MOE_W_BF16, W.to(DEV))[0]


def _check_linear(y, x, W, entries, ids, ydt, extra=None):
    ref, mag, lmag = lora_ref.linear(x.double(), W, entries, ids)
    H, R = W.shape[1], max([e[0].shape[0] for e in entries or [] if e is not None], default=0)
    tol = (H + R + 2) * U * mag + (2 * H + R + 4) * U * lmag
    norm = 2 * (H + R + 2) ** 0.5 * 2.0 ** -24
    if ydt == "bf16":
        tol = tol + 2.0 ** -15 * lmag + 2.0 ** -8 * ref.abs()
        norm = 2.0 ** -8
    if extra is not None:
        ref = ref + extra
        tol = tol + U * (ref.abs() + extra.abs())
    err = (y.double().cpu() - ref).abs()
    assert torch.all(err <= tol + 1e-30), float((err - tol).max())
    assert float(err.norm()) <= norm * float(ref.norm()) + 1e-30, (float(err.norm() / ref.norm()), norm)


LINEAR = [   # B, H, O, adapters, ranks, runs
    (1, 32, 16, 1, (1,), False), (1, 2048, 1024, 3, (16,), True), (2, 64, 48, 2, (5,), False),
    (7, 96, 240, 4, (3, 17), False), (15, 256, 32, 20, (16, 8), False), (16, 1056, 528, 3, (64,), False),
    (17, 160, 80, 5, (33, 1), False), (31, 288, 16, 2, (100,), False), (33, 512, 1040, 9, (4, 20), False),
    (64, 2048, 256, 24, (8, 16, 32, 64), False), (65, 96, 48, 30, (256,), False), (100, 352, 112, 6, (24,), True),
    (128, 1024, 768, 16, (16, 48), False), (129, 64, 272, 3, (7,), True), (200, 416, 400, 1, (32,), False),
    (257, 544, 144, 12, (9, 31), False), (300, 2048, 2064, 4, (16, 64), True), (515, 1120, 656, 8, (12,), False),
    (1025, 288, 528, 5, (40, 16), True), (1, 8192, 64, 1, (64,), True), (4, 96, 64, 9, (16,), False),
    (2, 1056, 32, 5, (32, 5), False), (3, 32, 48, 1, (50,), False), (13, 64, 32, 2, (20,), False),
    (256, 160, 96, 300, (3, 18), False), (2500, 64, 48, 2600, (5,), False), (2100, 96, 64, 3, (20,), False),
    (700, 1024, 96, 1, (40,), False), (900, 2048, 128, 2, (16,), True), (2048, 256, 32, 3, (16,), False),
    (1500, 96, 640, 2, (8, 70), True),
]


@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,H,O,n,ranks,runs", LINEAR)
def test_linear_matches_the_definition(B, H, O, n, ranks, runs, xdt, ydt):
    entries = lora_ref.make_table(B + H, n, H, O, ranks)
    W, x, ids = _weights(H + O, O, H), _acts(B, B, H, xdt), _ids(B + O, B, n, runs)
    y = moe.lora_linear(x.to(DEV), _pack(W), _table(entries, H, O), ids.to(DEV), y_dtype=DT[ydt])
    _check_linear(y, x, W, entries, ids, ydt)


@pytest.mark.parametrize("B", [1, 16, 40, 129, 300])
@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("f32", "f32")])
def test_linear_without_adapters(B, xdt, ydt):
    W, x = _weights(1, 208, 320), _acts(2, B, 320, xdt)
    y = moe.lora_linear(x.to(DEV), _pack(W))
    _check_linear(y, x, W, None, None, ydt)
    # A table whose entries are empty, or ids that name none.  (A call with a table may add the same products in
    # another order than one without, as its kernels are chosen for adapters: the bounds hold for any order.)
    t = moe.LoraTable(3, 320, 208, 16, DEV)
    first = None
    for ids in (torch.arange(B) % 3, torch.full((B,), -1), torch.full((B,), 3), torch.full((B,), -2 ** 31),
                torch.full((B,), 2 ** 31 - 1)):
        y = moe.lora_linear(x.to(DEV), _pack(W), t, ids.to(torch.int32).to(DEV))
        first = y if first is None else first
        assert torch.equal(y, first)
    _check_linear(first, x, W, None, None, ydt)


@pytest.mark.parametrize("B", [1, 13, 50, 130, 400])
def test_accumulate_and_padding_rows(B):
    H, O, n = 224, 176, 4
    entries = lora_ref.make_table(7, n, H, O, (16, 3))
    W, x, ids = _weights(8, O, H), _acts(9, B, H, "bf16"), _ids(10, B, n)
    t, w = _table(entries, H, O), _pack(W)
    base = torch.randn(B, O, generator=torch.Generator().manual_seed(3))
    y = base.clone().to(DEV)
    moe.lora_linear(x.to(DEV), w, t, ids.to(DEV), y=y, accumulate=True)
    _check_linear(y, x, W, entries, ids, "f32", extra=base.double())
    for nv in sorted({0, 1, B // 2, B - 1, B, B + 5}):
        xp = x.clone()
        xp[nv:] = float("nan")            # rows behind the last token are not read ...
        y = torch.full((B, O), 7.0, device=DEV)
        n_valid = torch.tensor([nv], dtype=torch.int32, device=DEV)
        moe.lora_linear(xp.to(DEV), w, t, ids.to(DEV), y=y, n_valid=n_valid)
        m = min(nv, B)
        assert torch.all(y[m:] == 7.0)    # ... nor written
        if m:
            _check_linear(y[:m], x[:m], W, entries, ids[:m], "f32")


@pytest.mark.parametrize("B", [5, 20, 48, 160, 300])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_non_finite_values_stay_in_their_rows(B, xdt):
    H, O, n = 128, 96, 5
    entries = lora_ref.make_table(17, n, H, O, (16, 20))
    entries[3] = (torch.full_like(entries[3][0], float("inf")), entries[3][1], 1.0)   # used by no token
    entries[4] = (entries[4][0], torch.full_like(entries[4][1], float("nan")), 1.0)
    W, x, ids = _weights(18, O, H), _acts(19, B, H, xdt), _ids(20, B, n)
    ids[ids >= 3] = 1
    t, w = _table(entries, H, O), _pack(W)
    clean = moe.lora_linear(x.to(DEV), w, t, ids.to(DEV), y_dtype=torch.float32)
    _check_linear(clean, x, W, entries, ids, "f32")
    bad = x.clone()
    bad[1, 3], bad[2, 5] = float("nan"), float("inf")
    ids2 = ids.clone()
    ids2[4], ids2[3] = 3, 4                # one token takes the adapter of infinities, one that of NaN
    y = moe.lora_linear(bad.to(DEV), w, t, ids2.to(DEV), y_dtype=torch.float32)
    rows = [i for i in range(B) if i not in (1, 2, 3, 4)]
    assert torch.equal(y[rows], clean[rows])
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any() and not torch.isfinite(y[4]).any()
    assert torch.isnan(y[3]).all()


@pytest.mark.parametrize("B", [9, 64, 129, 320])
def test_deterministic_and_independent_of_other_tokens_adapters(B):
    H, O, n = 640, 320, 8
    entries = lora_ref.make_table(27, n, H, O, (16, 64))
    W, x, ids = _weights(28, O, H), _acts(29, B, H, "bf16").to(DEV), _ids(30, B, n)
    t, w = _table(entries, H, O), _pack(W)
    ws = torch.empty(moe.lora_workspace_bytes(B, H, O, 64, torch.bfloat16, torch.float32), device=DEV,
                     dtype=torch.uint8)
    ws.fill_(0xFF)                         # NaN: the workspace needs no contents
    y = moe.lora_linear(x, w, t, ids.to(DEV), y_dtype=torch.float32, ws=ws)
    for _ in range(3):
        assert torch.equal(moe.lora_linear(x, w, t, ids.to(DEV), y_dtype=torch.float32, ws=ws), y)
    other = _ids(31, B, n)
    other[3] = ids[3]
    assert torch.equal(moe.lora_linear(x, w, t, other.to(DEV), y_dtype=torch.float32)[3], y[3])


def test_a_wider_adapter_than_the_call_allows_is_left_out():
    H, O = 64, 32
    entries = lora_ref.make_table(37, 2, H, O, (16, 48))
    t, w = _table(entries, H, O, 48), _pack(_weights(38, O, H))
    x = _acts(39, 4, H, "bf16").to(DEV)
    ids = torch.tensor([0, 1, 1, -1], dtype=torch.int32, device=DEV)
    none = moe.lora_linear(x, w)
    full = moe.lora_linear(x, w, t, ids)
    t.max_rank = 16
    y = moe.lora_linear(x, w, t, ids)
    assert torch.equal(y[0], full[0]) and torch.equal(y[1:], none[1:])


def test_publish_replaces_and_clear_removes():
    H, O, B = 96, 64, 20
    entries = lora_ref.make_table(47, 3, H, O, (16, 5))
    W, x, ids = _weights(48, O, H), _acts(49, B, H, "bf16"), _ids(50, B, 3)
    t, w = _table(entries, H, O, 40), _pack(W)
    entries[1] = lora_ref.make_table(51, 1, H, O, (40,))[0]
    t.publish(1, entries[1][0].to(DEV), entries[1][1].to(DEV), entries[1][2])
    _check_linear(moe.lora_linear(x.to(DEV), w, t, ids.to(DEV), y_dtype=torch.float32), x, W, entries, ids, "f32")
    t.clear(0)
    entries[0] = None
    _check_linear(moe.lora_linear(x.to(DEV), w, t, ids.to(DEV), y_dtype=torch.float32), x, W, entries, ids, "f32")


def _shared(seed, B, H, I, n, ranks, xdt):
    ws = [_weights(seed, I, H), _weights(seed + 1, I, H), _weights(seed + 2, H, I)]
    tabs = [lora_ref.make_table(seed + 3 + j, n, *hw, ranks) for j, hw in enumerate([(H, I), (H, I), (I, H)])]
    return ws, tabs, _acts(seed + 7, B, H, xdt), _ids(seed + 8, B, n)


def _check_shared(y, x, ws, tabs, ids, ydt, extra=None):
    ref = lora_ref.shared(x.double(), *ws, tabs, ids)
    H, I = ws[0].shape[1], ws[0].shape[0]
    R = max(e[0].shape[0] for t in tabs for e in t if e is not None) if any(t for t in tabs) else 0
    # g and u as sums of H + R products, twice for each (silu at most doubles a relative error here), then the last sum
    norm = 2.0 ** -24 * (2 * 2 * 2 * (H + R + 2) ** 0.5 + 2 * (I + R + 2) ** 0.5)
    if ydt == "bf16":
        norm = 2.0 ** -7                    # h and y are both rounded to bf16
    if extra is not None:
        ref = ref + extra
    err = float((y.double().cpu() - ref).norm())
    assert err <= norm * float(ref.norm()), (err / float(ref.norm()), norm)


SHARED = [   # B, H, I, adapters, ranks
    (1, 32, 32, 1, (1,)), (1, 2048, 768, 2, (16,)), (3, 96, 160, 4, (5, 16)), (16, 256, 128, 20, (16,)),
    (17, 288, 96, 3, (33,)), (40, 512, 352, 7, (8, 64)), (128, 1024, 512, 24, (16, 32)), (129, 224, 416, 3, (12,)),
    (300, 544, 288, 5, (16, 100)), (600, 1056, 736, 4, (24,)),
]


@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,H,I,n,ranks", SHARED)
def test_shared_expert_matches_the_definition(B, H, I, n, ranks, xdt, ydt):
    ws, tabs, x, ids = _shared(B + H + I, B, H, I, n, ranks, xdt)
    sh = moe.ExpertTensors.pack(moe.MOE_W_BF16, *[w.to(DEV) for w in ws])
    loras = [_table(t, *hw) for t, hw in zip(tabs, [(H, I), (H, I), (I, H)])]
    y = moe.shared_ffn(x.to(DEV), sh, loras, ids.to(DEV), y_dtype=DT[ydt])
    _check_shared(y, x, ws, tabs, ids, ydt)


@pytest.mark.parametrize("B", [1, 30, 200])
def test_shared_expert_with_some_tables_missing(B):
    H, I, n = 192, 160, 3
    ws, tabs, x, ids = _shared(60, B, H, I, n, (16, 9), "bf16")
    sh = moe.ExpertTensors.pack(moe.MOE_W_BF16, *[w.to(DEV) for w in ws])
    loras = [_table(t, *hw) for t, hw in zip(tabs, [(H, I), (H, I), (I, H)])]
    for on in ((0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)):
        y = moe.shared_ffn(x.to(DEV), sh, [t if k else None for t, k in zip(loras, on)], ids.to(DEV),
                           y_dtype=torch.float32)
        _check_shared(y, x, ws, [t if k else [] for t, k in zip(tabs, on)], ids, "f32")


@pytest.mark.parametrize("B", [1, 20, 64, 200])
def test_shared_expert_accumulates_into_real_rows(B):
    H, I, n = 128, 96, 4
    ws, tabs, x, ids = _shared(70, B, H, I, n, (16,), "bf16")
    sh = moe.ExpertTensors.pack(moe.MOE_W_BF16, *[w.to(DEV) for w in ws])
    loras = [_table(t, *hw) for t, hw in zip(tabs, [(H, I), (H, I), (I, H)])]
    nv = max(1, B - 3)
    base = torch.randn(B, H, generator=torch.Generator().manual_seed(4))
    y = base.clone().to(DEV)
    scratch = torch.full((moe.shared_ffn_workspace_bytes(B, H, I, 16, torch.bfloat16, torch.float32),), 255, device=DEV,
                         dtype=torch.uint8)
    moe.shared_ffn(x.to(DEV), sh, loras, ids.to(DEV), y=y, accumulate=True, ws=scratch,
                   n_valid=torch.tensor([nv], dtype=torch.int32, device=DEV))
    _check_shared(y[:nv], x[:nv], ws, tabs, ids[:nv], "f32", extra=base[:nv].double())
    assert torch.equal(y[nv:].cpu(), base[nv:])


def test_side_stream_with_allocated_outputs():
    H, O, B, n = 512, 256, 40, 4
    entries = lora_ref.make_table(80, n, H, O, (16, 32))
    W, x, ids = _weights(81, O, H), _acts(82, B, H, "bf16"), _ids(83, B, n)
    t, w, xd, idd = _table(entries, H, O), _pack(W), x.to(DEV), ids.to(DEV)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for handle in (st, st.cuda_stream):
        y = moe.lora_linear(xd, w, t, idd, y_dtype=torch.float32, stream=handle)
        st.synchronize()
        _check_linear(y, x, W, entries, ids, "f32")


def test_tensors_are_checked():
    H, O, B = 64, 32, 4
    t = moe.LoraTable(2, H, O, 16, DEV)
    w = _pack(_weights(90, O, H))
    x = torch.zeros(B, H, device=DEV, dtype=torch.bfloat16)
    ids = torch.zeros(B, device=DEV, dtype=torch.int32)
    bad = [
        (x.cpu(), w, t, ids, {}), (x.half(), w, t, ids, {}), (x[:, :32], w, t, ids, {}), (x, w.float(), t, ids, {}),
        (x, w, t, ids.long(), {}), (x, w, t, ids[:3], {}), (x, w, t, None, {}), (x, w, t, ids.cpu(), {}),
        (x, w, t, ids, dict(y=torch.zeros(B, O + 1, device=DEV))), (x, w, t, ids, dict(accumulate=True)),
        (x, w, t, ids, dict(y=torch.zeros(B, O, device=DEV).half())),
        (x, w, moe.LoraTable(2, O, H, 16, DEV), ids, {}),
        (x, w, t, ids, dict(n_valid=torch.zeros(1, device=DEV))),
        (x.t().contiguous().t(), w, t, ids, {}),
    ]
    for a, b, c, d, kw in bad:
        with pytest.raises((ValueError, TypeError)):
            moe.lora_linear(a, b, c, d, **kw)
    small = torch.empty(16, device=DEV, dtype=torch.uint8)
    with pytest.raises(moe.MoeError):
        moe.lora_linear(x, w, t, ids, ws=small)
    with pytest.raises(moe.MoeError):   # accumulating in bf16
        moe.lora_linear(x, w, t, ids, y=torch.zeros(B, O, device=DEV, dtype=torch.bfloat16), accumulate=True)
    for args in ((0, torch.zeros(17, H), torch.zeros(O, 17)), (2, torch.zeros(4, H), torch.zeros(O, 4)),
                 (0, torch.zeros(4, H + 32), torch.zeros(O, 4)), (0, torch.zeros(4, H), torch.zeros(O, 5))):
        with pytest.raises(ValueError):
            t.publish(args[0], args[1].to(DEV).bfloat16(), args[2].to(DEV).bfloat16())


def test_packed_adapters_round_trip():
    # the documented layout, element by element
    for rank, H, O in ((1, 32, 16), (20, 96, 48)):
        A, B, _ = lora_ref.make_table(rank, 1, H, O, (rank,))[0]
        pa, pb, R = moe.lora_pack(A.to(DEV), B.to(DEV))
        pa = pa.cpu().view(torch.int16).numpy().reshape(R // 16, H // 32, 64, 8)
        pb = pb.cpu().view(torch.int16).numpy().reshape(O // 16, R // 16, 64, 4)
        a = np.zeros((R, H), np.int16)
        b = np.zeros((O, R), np.int16)
        for l in range(64):
            for j in range(8):
                a[l % 16::16, 8 * (l // 16) + j::32] = pa[:, :, l, j]
            for j in range(4):
                b[l % 16::16, 4 * (l // 16) + j::16] = pb[:, :, l, j]
        assert np.array_equal(a[:rank], A.view(torch.int16).numpy()) and not a[rank:].any()
        assert np.array_equal(b[:, :rank], B.view(torch.int16).numpy()) and not b[:, rank:].any()


@pytest.mark.parametrize("B", [7, 40, 200, 700])
def test_nan_patterns_of_fp32_rows(B):
    # a NaN whose set mantissa bits all lie below the bf16 half is still a NaN, in its row alone
    H, O = 256, 96
    W, x = _weights(95, O, H), _acts(96, B, H, "f32")
    x.view(torch.int32)[3, 17] = 0x7F800001
    y = moe.lora_linear(x.to(DEV), _pack(W))
    rows = [i for i in range(B) if i != 3]
    assert torch.isnan(y[3]).all()
    _check_linear(y[rows], x[rows], W, None, None, "f32")


@pytest.mark.parametrize("B", [1, 24, 300])
def test_graph_replays_follow_table_ids_and_rows(B):
    H, O, n = 512, 272, 5
    entries = lora_ref.make_table(100, n, H, O, (16, 24))
    W = _weights(101, O, H)
    t, w = _table(entries, H, O, 32), _pack(W)
    x = torch.zeros(B, H, device=DEV)
    ids = torch.full((B,), -1, device=DEV, dtype=torch.int32)
    y = torch.zeros(B, O, device=DEV)
    n_valid = torch.tensor([B], device=DEV, dtype=torch.int32)
    ws = torch.empty(moe.lora_workspace_bytes(B, H, O, 32, torch.float32, torch.float32), device=DEV, dtype=torch.uint8)

    def call():
        moe.lora_linear(x, w, t, ids, y=y, ws=ws, n_valid=n_valid)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step, nv in enumerate((B, max(1, B // 2), 0, B)):
        xs, idx = _acts(110 + step, B, H, "f32"), _ids(120 + step, B, n)
        x.copy_(xs)
        ids.copy_(idx)
        n_valid.fill_(nv)
        y.fill_(3.0)
        if step == 3:   # another adapter under the same handle
            entries[2] = lora_ref.make_table(130, 1, H, O, (32,))[0]
            t.publish(2, entries[2][0].to(DEV), entries[2][1].to(DEV), entries[2][2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.all(y[nv:] == 3.0)
        if nv:
            _check_linear(y[:nv], xs[:nv], W, entries, idx[:nv], "f32")


def _far_rows(B):   # the first rows, those round 2^32 bytes of 16 KB rows, and the last
    return torch.cat([torch.arange(20), torch.arange(2 ** 18 - 20, 2 ** 18 + 20), torch.arange(B - 20, B)])


@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("H,O", [(32, 8192), (8192, 32)])
def test_offsets_past_32_bits(H, O, xdt, ydt):
    B = 2 ** 18 + 1001   # rows of 16 KB (bf16): x, its planes or y pass 4 GiB
    g = torch.Generator(device=DEV).manual_seed(B + H)
    x = torch.randn(B, H, generator=g, device=DEV, dtype=DT[xdt])
    entries = lora_ref.make_table(5, 3, H, O, (8, 20))
    W, ids = _weights(H, O, H), _ids(6, B, 3)
    y = moe.lora_linear(x, _pack(W), _table(entries, H, O), ids.to(DEV), y_dtype=DT[ydt])
    at = _far_rows(B)
    _check_linear(y[at.to(DEV)], x[at.to(DEV)].cpu(), W, entries, ids[at], ydt)


@pytest.mark.parametrize("ydt", ["bf16", "f32"])
def test_shared_expert_whose_h_passes_32_bits(ydt):
    B, H, I = 2 ** 18 + 1001, 32, 8192
    ws, tabs, _, _ = _shared(31, 1, H, I, 2, (8,), "bf16")
    g = torch.Generator(device=DEV).manual_seed(32)
    x = torch.randn(B, H, generator=g, device=DEV, dtype=torch.bfloat16)
    ids = _ids(33, B, 2)
    sh = moe.ExpertTensors.pack(moe.MOE_W_BF16, *[w.to(DEV) for w in ws])
    loras = [_table(t, *hw) for t, hw in zip(tabs, [(H, I), (H, I), (I, H)])]
    y = moe.shared_ffn(x, sh, loras, ids.to(DEV), y_dtype=DT[ydt])
    at = _far_rows(B)
    _check_shared(y[at.to(DEV)], x[at.to(DEV)].cpu(), ws, tabs, ids[at], ydt)
