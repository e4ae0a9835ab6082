"""CPU-only checks of the adapter and shared-expert entry points' argument
validation (no call here reaches a kernel)."""
import ctypes

import pytest
import torch

import aware_expert_routing_amd as moe

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p((1 << 20) + 8)


def _linear(**kw):
    a = dict(w=FAKE, table=FAKE, n=2, rank=16, adapter=FAKE, x=FAKE, xdt=1, B=4, H=64, O=32, y=FAKE, ydt=1, acc=0,
             ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return moe.lib().moe_lora_linear(a["w"], a["table"], a["n"], a["rank"], a["adapter"], a["x"], a["xdt"], a["B"],
                                     a["H"], a["O"], None, a["y"], a["ydt"], a["acc"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), -1), (dict(x=None), -1), (dict(y=None), -1), (dict(adapter=None), -1), (dict(n=0), -1),
    (dict(rank=0), -1), (dict(rank=8), -1), (dict(rank=272), -2), (dict(xdt=2), -1), (dict(ydt=-1), -1),
    (dict(acc=1), -1), (dict(B=0), -1), (dict(B=(1 << 20) + 1), -2), (dict(H=0), -1), (dict(H=48), -1),
    (dict(O=8), -1), (dict(O=40), -1), (dict(H=16416), -2), (dict(O=16400), -2), (dict(ws=None), -1),
    (dict(wsb=255), -1), (dict(ws=ctypes.c_void_p((1 << 20) + 128)), -1), (dict(x=ODD), -1), (dict(y=ODD), -1),
    (dict(w=ODD), -1), (dict(table=ODD), -1),
])
def test_lora_linear_rejects(kw, status):
    assert _linear(**kw) == status
    assert moe.lib().moe_last_error()


def _shared(**kw):
    h = moe.ExpertHandle()
    h.fmt, h.w_gate, h.w_up, h.w_down = moe.MOE_W_BF16, 1 << 20, 1 << 20, 1 << 20
    for name in ("fmt", "w_gate", "w_up", "w_down"):
        if name in kw:
            setattr(h, name, kw.pop(name))
    a = dict(tg=FAKE, tu=FAKE, td=FAKE, n=2, rank=16, adapter=FAKE, x=FAKE, xdt=1, B=4, H=64, I=32, y=FAKE, ydt=0,
             acc=1, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return moe.lib().moe_shared_ffn(ctypes.byref(h), a["tg"], a["tu"], a["td"], a["n"], a["rank"], a["adapter"],
                                    a["x"], a["xdt"], a["B"], a["H"], a["I"], None, a["y"], a["ydt"], a["acc"],
                                    a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=moe.MOE_W_F32), -2), (dict(fmt=moe.MOE_W_INT4_G128), -2), (dict(w_gate=None), -1), (dict(w_down=8), -1),
    (dict(x=None), -1), (dict(y=None), -1), (dict(adapter=None), -1), (dict(tg=None, tu=None, td=FAKE, rank=8), -1),
    (dict(td=ODD), -1), (dict(H=48), -1), (dict(I=16), -1), (dict(I=16416), -2), (dict(ydt=1), -1), (dict(ws=None), -1),
    (dict(wsb=1), -1), (dict(B=0), -1), (dict(B=1 << 21), -2), (dict(n=-1), -1),
])
def test_shared_ffn_rejects(kw, status):
    assert _shared(**kw) == status


def test_adapter_pack_and_publish_reject():
    lib = moe.lib()
    ok = (FAKE, FAKE, 16, 64, 32, FAKE, FAKE, None)
    for at, v, status in ((0, None, -1), (1, None, -1), (5, None, -1), (2, 0, -1), (2, 257, -2), (3, 48, -1),
                          (4, 24, -1), (3, 16416, -2), (0, ODD, -1), (6, ODD, -1)):
        a = list(ok)
        a[at] = v
        assert lib.moe_lora_pack(*a) == status, (at, v)
    h = moe.LoraHandle()
    h.rank, h.scale, h.a, h.b = 16, 1.0, 1 << 20, 1 << 20
    assert lib.moe_lora_publish(None, 0, ctypes.byref(h), None) == -1
    assert lib.moe_lora_publish(FAKE, -1, ctypes.byref(h), None) == -1
    assert lib.moe_lora_publish(ODD, 0, ctypes.byref(h), None) == -1
    for name, v, status in (("rank", 8, -1), ("rank", -16, -1), ("rank", 272, -2), ("a", None, -1), ("b", 8, -1),
                            ("scale", float("nan"), -1)):
        old = getattr(h, name)
        setattr(h, name, v)
        assert lib.moe_lora_publish(FAKE, 0, ctypes.byref(h), None) == status, name
        setattr(h, name, old)


def test_handle_record_is_32_bytes():
    assert ctypes.sizeof(moe.LoraHandle) == moe.LORA_HANDLE_BYTES == 32


def test_workspace_sizes():
    bf, f = torch.bfloat16, torch.float32
    assert moe.lora_workspace_bytes(4, 64, 32, 0, bf, bf) == 0
    assert moe.lora_workspace_bytes(0, 64, 32, 16, bf, bf) == 0
    assert moe.lora_workspace_bytes(4, 64, 32, 257, bf, bf) == 0
    assert moe.lora_workspace_bytes(4, 64, 32, 9, bf, bf) >= 4 * 16 * 4
    assert moe.shared_ffn_workspace_bytes(4, 64, 96, 0, bf, f) >= 4 * 96 * 4


def test_binding_refuses_host_tensors_and_bad_tables():
    with pytest.raises(ValueError, match="GPU"):
        moe.lora_linear(torch.zeros(4, 64), torch.zeros(32, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU"):
        moe.lora_pack(torch.zeros(4, 64), torch.zeros(32, 4))
    for args in ((0, 64, 32, 16), (2, 48, 32, 16), (2, 64, 24, 16), (2, 64, 32, 0), (2, 64, 32, 257)):
        with pytest.raises(ValueError):
            moe.LoraTable(*args, device="cpu")
    with pytest.raises(ValueError, match="shared"):
        moe.MoELayer(64, 32, 4, 2, None, [], "cpu", loras=(None, None, None))
