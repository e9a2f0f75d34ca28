"""The binding of the transformer block's operators takes tensors of the current device
only: a launch goes there, and another device's addresses may fault.  The devices here
are names that stand-ins answer with, so one device, or none, is enough."""

import pytest
import torch

dg = pytest.importorskip("moe_grouped_gemm_02_amd", reason="libdg.so not built")
from moe_grouped_gemm_02_amd import block as binding  # noqa: E402


class On:
    def __init__(self, index):
        self.index, self.device = index, f"cuda:{index}"

    def get_device(self):
        return self.index


def test_stream_of_the_tensors_device(monkeypatch):
    monkeypatch.setattr(binding, "_several", True)
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 100 + index)
    assert binding._stream(On(1)) == 101
    assert binding._stream(On(1), None, On(1), None) == 101
    with pytest.raises(ValueError, match="cuda:0, the current device is cuda:1"):
        binding._stream(On(0), On(1))
    with pytest.raises(ValueError, match="cuda:2 beside"):
        binding._stream(On(1), None, On(1), On(2))


@pytest.mark.parametrize("devices", [0, 1, 2, 8])
def test_how_many_devices_there_are_is_asked_once(monkeypatch, devices):
    asked = []
    monkeypatch.setattr(torch.cuda, "device_count", lambda: asked.append(0) or devices)
    monkeypatch.setattr(binding, "_several", None)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 7)
    assert binding._stream(On(0), On(0)) == 7 and binding._stream(On(0)) == 7
    assert len(asked) == 1 and binding._several == (devices > 1)
    if devices > 1:
        with pytest.raises(ValueError, match="beside"):
            binding._stream(On(0), On(1))


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda")


def f32(*shape):
    return torch.zeros(shape, device="cuda")


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def calls():
    """Each entry point with every tensor that it takes: (function, positional tensors, keyword tensors, options)."""
    norm = dict(h=bf16(4, 128), r=bf16(4, 128), x=bf16(4, 128), q=u8(4, 128), weight=f32(128), bias=f32(128), post_weight=f32(128), gate=f32(128))
    bwd = dict(dx=bf16(4, 128), dr=bf16(4, 128), r=bf16(4, 128), y=bf16(4, 128), dh=bf16(4, 128), weight=f32(128), dweight=f32(128), dbias=f32(128),
               post_weight=f32(128), dpost_weight=f32(128), gate=f32(128), dgate=f32(128), workspace=u8(1 << 16))
    bal = dict(seq_offsets=torch.tensor([0, 4], dtype=torch.int32, device="cuda"), workspace=u8(1 << 16))
    epi = lambda: dict(bias=f32(128), residual=bf16(4, 128), pre=bf16(4, 128), dq=u8(4, 128), workspace=u8(1 << 16))
    out = [(dg.dg_block_norm, [bf16(4, 128)], dict(norm, sf=f32(1, 4)), dict(post=True)),
           (dg.dg_block_norm_ue8m0, [bf16(4, 128)], dict(norm, sf=u8(1, 4)), dict(post=True)),
           (dg.dg_block_norm_bwd, [bf16(4, 128)], bwd, dict(post=True)),
           (dg.dg_fp8_gemm_nt_epilogue, [u8(4, 128), f32(1, 4), u8(128, 128), f32(1, 1), bf16(4, 128)], dict(epi(), dsf=f32(1, 4)), {}),
           (dg.dg_fp8_gemm_nt_ue8m0_epilogue, [u8(4, 128), u8(1, 4), u8(128, 128), u8(1, 4), bf16(4, 128)], dict(epi(), dsf=u8(1, 4)), {}),
           (dg.dg_epilogue_bwd, [bf16(4, 128), u8(4, 128), f32(1, 4)],
            dict(pre=bf16(4, 128), dqt=u8(128, 128), dsft=f32(1, 128), dbias=f32(128), workspace=u8(1 << 16)), dict(act="silu"))]
    for fn, back, logits in ((dg.dg_moe_balance, dg.dg_moe_balance_bwd, lambda: f32(4, 8)), (dg.dg_moe_balance_bf16, dg.dg_moe_balance_bwd_bf16, lambda: bf16(4, 8))):
        out.append((fn, [logits(), i32(4, 2), i32(1, 8), i32(1), f32(1)], bal, {}))
        out.append((back, [logits(), i32(1, 8), i32(1), logits()], dict(seq_offsets=bal["seq_offsets"], dloss=f32(1), add=logits()), dict(topk=2)))
    return out


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU visible")
def test_every_entry_point_asks_for_every_tensors_device(monkeypatch):
    """Every tensor of a call is asked, and a call while another device is current is refused."""
    asked = []
    real = binding._stream

    def record(*tensors):
        asked.extend(t.data_ptr() for t in tensors if t is not None)
        return real(*tensors)

    monkeypatch.setattr(binding, "_stream", record)
    for fn, args, kw, options in calls():
        asked.clear()
        fn(*args, **kw, **options)
        assert set(asked) == {t.data_ptr() for t in (*args, *kw.values())}, fn.__name__
        with monkeypatch.context() as m:
            m.setattr(binding, "_several", True)
            m.setattr(binding, "_current_device", lambda: torch.cuda.current_device() + 1)
            with pytest.raises(ValueError, match="current device"):
                fn(*args, **kw, **options)
    torch.cuda.synchronize()
