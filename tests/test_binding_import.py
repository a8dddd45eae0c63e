"""The binding on a torch build without the unpublished names by which it asks for a stream's handle cheaply."""

import importlib.util

import pytest
import torch


@pytest.fixture
def bare_lib(monkeypatch):
    """A second copy of the binding, imported where those names do not exist."""
    import fp8_fine_grained_act_amd

    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    path = fp8_fine_grained_act_amd.__path__[0] + "/lib.py"
    spec = importlib.util.spec_from_file_location("bare_lib", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    monkeypatch.undo()                           # torch itself uses them when it makes streams
    return module


def test_imports_and_refuses(bare_lib):
    b = torch.zeros((8, 16), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        bare_lib.fp8bs_epilogue_backward(b, b)
    assert bare_lib.raw.fp8bs_epilogue_backward_workspace(4, 16) == 0


@pytest.mark.gpu
def test_runs_on_the_current_and_on_a_given_stream(gpu_lib, bare_lib):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    dy, z = (torch.randn((40, 512), generator=g, device="cuda").bfloat16() for _ in range(2))
    want = gpu_lib.fp8bs_epilogue_backward(dy, z, act=gpu_lib.FP8BS_ACT_SILU)
    got = [bare_lib.fp8bs_epilogue_backward(dy, z, act=bare_lib.FP8BS_ACT_SILU)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got.append(bare_lib.fp8bs_epilogue_backward(dy, z, act=bare_lib.FP8BS_ACT_SILU, stream=s))
    with torch.cuda.stream(s):
        got.append(bare_lib.fp8bs_epilogue_backward(dy, z, act=bare_lib.FP8BS_ACT_SILU))
        assert bare_lib._raw_stream(0) == s.cuda_stream
    torch.cuda.synchronize()
    for dz, db in got:
        assert torch.equal(dz.view(torch.int16), want[0].view(torch.int16)) and torch.equal(db, want[1])
