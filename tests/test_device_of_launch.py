"""Every entry point runs with its tensors' device current, on that device's
current stream (no GPU, no launch: the library, the devices and the tensors'
device are stand-ins). A launch goes to the current device, and a default
stream's null handle means the current device's, so tensors elsewhere would be
read by the wrong one."""
import types

import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tensor_scaled_fp8_amd import binding, block

U8, BF16, I32 = torch.uint8, torch.bfloat16, torch.int32


class Elsewhere(torch.Tensor):
    """A host tensor that claims to be on device 1."""
    is_cuda = True

    def get_device(self):
        return 1


def _t(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Elsewhere)


@pytest.fixture
def calls(monkeypatch):
    """[(entry, current device, stream)] of what is called while device 0 is current."""
    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *e):
            current.pop()

    class Entries:
        def __init__(self, compiled):
            self.compiled = compiled

        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 0
                seen.append((name, current[-1], None if self.compiled else args[-1]))
                return (_t(4), _t(4)) if name == "quantize" else _t(4, 6) if self.compiled else 0
            return call
    lib, compiled = Entries(False), Entries(True)
    for m in (binding, block):
        monkeypatch.setattr(m, "load", lambda: lib)
    monkeypatch.setattr(block, "_binding", lambda: compiled)
    monkeypatch.setattr(block, "_forward_bytes", lambda *a: 0)
    monkeypatch.setattr(block, "_gemm_bytes", lambda *a: 0)
    monkeypatch.setattr(block, "_check_bf16", lambda t, name: None)
    monkeypatch.setattr(binding, "_dev", lambda t, dtype, name: None if t is None else t.data_ptr())
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=0))
    for m in (binding, block):
        monkeypatch.setattr(m, "_raw_stream", lambda device: 100 + device, raising=False)
    monkeypatch.setattr(binding, "_current_device", lambda: current[-1], raising=False)
    return seen


def _ws(M=16, K=32, N=48):
    u = {n: _t(*s, dtype=U8) for n, s in (("x8", (M, K)), ("w8", (K, N)), ("dy8", (M, N)))}
    return types.SimpleNamespace(M=M, K=K, N=N, c=binding.LinearWs(), **u)


def _adam():
    s = types.SimpleNamespace(n=16, step_count=0, alt=None)
    s.m1, s.m2, s.w16 = _t(16, dtype=U8), _t(16, dtype=torch.int16), _t(16, dtype=torch.int16)
    s.s_m1, s.s_m2, s.s_w = (_t(16, dtype=I32) for _ in range(3))
    return s


def _stored(rows, cols):
    return tsf.BlockTensor(torch.zeros(tsf.BlockTensor.empty(rows, cols, "e4m3", "cpu").nbytes, dtype=U8)
                           .as_subclass(Elsewhere), rows, cols, 0)


REC = dict(dtype=I32)
CALLS = {
    "fp8_scale_reset": lambda: tsf.fp8_scale_reset(_t(16, **REC)),
    "fp8_amax": lambda: tsf.fp8_amax(_t(32), _t(16, **REC)),
    "fp8_scale": lambda: tsf.fp8_scale("e4m3", _t(16, **REC)),
    "fp8_amax_scale": lambda: tsf.fp8_amax_scale(_t(32), "e4m3", _t(16, **REC)),
    "fp8_scale_fixed": lambda: tsf.fp8_scale_fixed(_t(16, **REC), 3),
    "fp8_cast": lambda: tsf.fp8_cast(_t(16, 32), "e4m3", _t(16, **REC)),
    "fp8_quantize": lambda: tsf.fp8_quantize(_t(16, 32), "e4m3", _t(16, **REC)),
    "fp8_quantize_spec": lambda: tsf.fp8_quantize_spec(_t(16, 32), "e4m3", _t(16, **REC)),
    "fp8_quantize_batch": lambda: tsf.fp8_quantize_batch([dict(x=_t(16, 32), fmt="e4m3", s=_t(16, **REC))]),
    "fp8_gemm_nt": lambda: tsf.fp8_gemm_nt(_t(16, 32, dtype=U8), 0, _t(16, **REC), _t(16, 32, dtype=U8), 0,
                                           _t(16, **REC)),
    "fp8_gemm": lambda: tsf.fp8_gemm(_t(16, 32, dtype=U8), 0, _t(16, **REC), _t(16, 32, dtype=U8), 0, _t(16, **REC)),
    "fp8_gemm_ws": lambda: tsf.fp8_gemm(_t(16, 32, dtype=U8), 0, _t(16, **REC), _t(16, 32, dtype=U8), 0,
                                        _t(16, **REC), workspace=_t(16, dtype=U8)),
    "fp8_gemm_noalloc": lambda: tsf.fp8_gemm_noalloc(_t(16, 32, dtype=U8), 0, _t(16, **REC), _t(16, 32, dtype=U8), 0,
                                                     _t(16, **REC), _t(16, 16)),
    "fp8_gemm_pair": lambda: tsf.fp8_gemm_pair(*[dict(a=_t(16, 32, dtype=U8), fa=0, sa=_t(16, **REC),
                                                      b=_t(16, 32, dtype=U8), fb=0, sb=_t(16, **REC))] * 2),
    "fp8_linear_fwd": lambda: tsf.fp8_linear_fwd(_t(16, 32), _t(32, 48), _ws()),
    "fp8_linear_bwd": lambda: tsf.fp8_linear_bwd(_t(16, 48), _ws()),
    "fp8_linear_fwd_cached": lambda: tsf.fp8_linear_fwd_cached(_t(16, 32), _t(32, 48, dtype=U8), _t(16, **REC),
                                                               _t(16, 32, dtype=U8), _t(16, **REC)),
    "fp8_wgrad_fp8": lambda: tsf.fp8_wgrad_fp8(_t(32, 16, dtype=U8), _t(16, **REC), _t(48, 16, dtype=U8),
                                               _t(16, **REC), s_dw=_t(16, **REC)),
    "fp8_adam_init_master": lambda: tsf.fp8_adam_init_master(_t(16), _t(16, dtype=torch.int16), _t(16, **REC)),
    "fp8_adam_step": lambda: tsf.fp8_adam_step(_adam(), _t(16, dtype=U8), _t(16, **REC), 0.1),
    "fp8_adam_step_spec": lambda: tsf.fp8_adam_step_spec(_adam(), _t(16, dtype=U8), _t(16, **REC), 0.1),
    "fp8_block_gemm": lambda: tsf.fp8_block_gemm(_stored(4, 8), _stored(6, 8)),
    "fp8_block_linear_fwd": lambda: tsf.block_linear(_t(4, 8), _t(8, 6)),
    "fp8_swiglu_fwd": lambda: tsf.swiglu(_t(4, 8), _t(4, 8)),
    "fp8_block_mlp_fwd": lambda: tsf.block_mlp(_t(4, 8), _t(8, 12), _t(6, 8)),
    "quantize": lambda: tsf.fp8_block_quantize(_t(4, 8)),
    "dequantize": lambda: tsf.fp8_block_dequantize(_stored(4, 8)),
    "serve": lambda: tsf.fp8_block_linear_fwd_cached(_t(4, 8), _stored(6, 8)),
    "linear": lambda: tsf.block_linear(_t(4, 8).requires_grad_(), _t(8, 6)),
    "swiglu": lambda: tsf.swiglu(_t(4, 8).requires_grad_(), _t(4, 8)),
    "mlp": lambda: tsf.block_mlp(_t(4, 8).requires_grad_(), _t(8, 12), _t(6, 8)),
}


@pytest.mark.parametrize("entry", list(CALLS))
def test_runs_on_the_tensors_device(calls, entry):
    CALLS[entry]()
    assert [c[:2] for c in calls] == [(entry, 1)]
    assert calls[0][2] in (None, 101)


def test_nothing_is_switched_where_the_device_is_current(calls, monkeypatch):
    monkeypatch.setattr(Elsewhere, "get_device", lambda self: 0)
    monkeypatch.setattr(torch.cuda, "device", None)
    CALLS["fp8_gemm"]()
    CALLS["serve"]()
    assert [c[:2] for c in calls] == [("fp8_gemm", 0), ("serve", 0)]


def test_every_entry_point_that_takes_a_stream_is_covered():
    """Of the library's entry points with a stream argument, those left are reached from inside the compiled binding."""
    import os
    import re
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8lin.h")).read()
    header = re.sub(r"/\*.*?\*/", "", header, flags=re.S)
    streamed = set(re.findall(r"\b(fp8_\w+)\s*\([^;]*hipStream_t", header))
    inside = {"fp8_block_quantize", "fp8_block_dequantize", "fp8_block_linear_fwd_cached", "fp8_block_linear_fwd_few",
              "fp8_block_linear_bwd", "fp8_swiglu_bwd", "fp8_block_mlp_bwd"}
    assert streamed - set(CALLS) == inside
