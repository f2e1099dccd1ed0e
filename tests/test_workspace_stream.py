"""A workspace that a call allocates itself belongs to the stream that the call runs on.

Torch's pool gives a freed block to the next allocation on the block's own stream, so a block
of the current stream would be handed on (or still be in use) while a kernel on another
stream works in it.
"""
from contextlib import contextmanager

import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv

RS = nv.NVFP4_ROW_SCALED


def _operand(lines, k, device, groups=1):
    return nv.Operand(torch.full((lines, k // 2), 0x21, dtype=torch.uint8, device=device),
                      torch.full((lines, k // 16), 0x38, dtype=torch.uint8, device=device),
                      torch.rand(groups * lines, device=device) + 1, RS, 448.0)


def _calls(device, m=256, n=512, k=2048):
    """Every call that takes a workspace, without one, and the outputs it fills."""
    a, b, bm = _operand(m, k, device), _operand(n, k, device), _operand(2 * n, k, device)
    ag, bg = _operand(m, k, device, 2), _operand(n, k, device, 2)  # an amax per line and group
    g = torch.Generator(device=device)
    g.manual_seed(1)
    x, dd = (torch.randn(m, n, generator=g, device=device) for _ in range(2))
    w, rstd = torch.ones(n, device=device), torch.rand(m, generator=g, device=device) + 0.5
    ends = torch.tensor([128, 256], device=device)
    kends = torch.tensor([256, k], device=device)
    d, d2, dx, dz = (torch.empty(m, n, device=device) for _ in range(4))
    dg = torch.empty(2, m, n, device=device)
    dw, db, ra, ca = (torch.empty(s, device=device) for s in (n, n, m, n))
    norm = torch.empty(1, device=device)
    out = [torch.empty_like(x)]
    return {
        "gemm": ([d], lambda s: nv.nvfp4_gemm(a, b, d, stream=s)),
        "grouped_gemm": ([d], lambda s: nv.nvfp4_grouped_gemm(a, bm, ends, d, stream=s)),
        "grouped_gemm_wgrad": ([dg], lambda s: nv.nvfp4_grouped_gemm_wgrad(ag, bg, kends, dg,
                                                                           stream=s)),
        "gemm_bias_act": ([d2], lambda s: nv.nvfp4_gemm_bias_act(a, b, d2, bias=w, stream=s)),
        "add_rmsnorm_backward": ([dx, dw], lambda s: nv.nvfp4_add_rmsnorm_backward(
            dd, x, w, rstd, dx, dweight=dw, stream=s)),
        "bias_act_backward": ([dz, db, ra, ca], lambda s: nv.nvfp4_bias_act_backward(
            dd, x, nv.NVFP4_ACT_SILU, dz, dbias=db, row_amax=ra, col_amax=ca, stream=s)),
        "grad_norm": ([norm], lambda s: nv.nvfp4_grad_norm([x, dd], norm, stream=s)),
        "clip_grad_norm": ([norm] + out, lambda s: nv.nvfp4_clip_grad_norm(
            [x], 1.0, norm, out=out, stream=s)),
    }


NAMES = ["gemm", "grouped_gemm", "grouped_gemm_wgrad", "gemm_bias_act", "add_rmsnorm_backward",
         "bias_act_backward", "grad_norm", "clip_grad_norm"]


class _Stream:
    cuda_stream = 0x1230


class _Library:
    """Every entry point of the library, doing nothing."""

    def __getattr__(self, name):
        return lambda *args: nv.NVFP4_OK


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("given", ["object", "handle"])
def test_allocated_on_the_given_stream(name, given, monkeypatch):
    calls = _calls("cpu", 8, 16, 64)
    current, allocated = [None], []

    @contextmanager
    def selected(stream):
        current.append(stream)
        yield
        current.pop()

    class External(_Stream):
        def __init__(self, handle):
            self.cuda_stream = handle
    empty = torch.empty

    def recorded(*args, **kw):
        allocated.append(current[-1])
        return empty(*args, **kw)
    monkeypatch.setattr(nv, "_lib", _Library())
    monkeypatch.setattr(nv, "_on_gpu", lambda *tensors: None)
    monkeypatch.setattr(torch.cuda, "stream", selected)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch, "empty", recorded)
    calls[name][1](_Stream() if given == "object" else 0x1230)
    assert len(allocated) == 1
    assert allocated[0] is not None and allocated[0].cuda_stream == 0x1230


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_other_stream_without_a_workspace(name):
    """The call waits on its stream while the current stream takes and fills memory of the
    workspace's size."""
    outs, call = _calls("cuda")[name]
    call(None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    sizes = [nv.nvfp4_gemm_workspace_size(256, 512, 2048),
             nv.nvfp4_gemm_bias_act_workspace_size(256, 512, 2048),
             nv.nvfp4_grouped_gemm_workspace_size(256, 512, 2048, 2),
             nv.nvfp4_add_rmsnorm_backward_workspace_size(256, 512),
             nv.nvfp4_bias_act_backward_workspace_size(256, 512),
             nv.nvfp4_clip_grad_norm_workspace_size()]
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            busy = torch.randn(4096, 4096, device="cuda")
            for _ in range(8):
                busy = busy @ busy * 1e-2
        call(stream)
        filled = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xA5) for n in sizes]
        torch.cuda.synchronize()
        assert all(bool((f == 0xA5).all()) for f in filled)
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_current_stream_without_torchs_inner_call(monkeypatch):
    """A torch that lacks the inner call for the handle is served through its interface."""
    import importlib.util
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: type("S", (), {"cuda_stream": 0x4560 + device}))
    spec = importlib.util.spec_from_file_location("nv_again", nv.__file__)
    again = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(__import__("sys").modules, "nv_again", again)
    spec.loader.exec_module(again)
    assert again._stream(None) == 0x4563
    assert again._stream(0x1230) == 0x1230 and again._stream(_Stream()) == 0x1230


@pytest.mark.gpu
def test_current_stream_is_the_same_by_both_ways():
    s = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), s):
        with torch.cuda.stream(stream):
            assert nv._stream(None) == nv._current_raw_stream(torch.cuda.current_device()) == \
                stream.cuda_stream


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [0, 1, 2])  # the default stream, legacy and per thread
@pytest.mark.parametrize("name", ["gemm_bias_act", "bias_act_backward", "clip_grad_norm"])
def test_default_stream_handles(name, handle):
    outs, call = _calls("cuda")[name]
    call(None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    call(handle)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
