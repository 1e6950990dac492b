"""The stream that the linear attention, verification and norms are put on."""

import importlib.util
import sys

import pytest
import torch

import gated_deltanet_03_amd as gdn

pytestmark = pytest.mark.gpu


def without_raw_query(monkeypatch):
    """The binding as it is on a torch without its own stream query."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    spec = importlib.util.spec_from_file_location("gdn_without_raw_query", gdn.__file__,
                                                  submodule_search_locations=list(gdn.__path__))
    module = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, spec.name, module)
    spec.loader.exec_module(module)
    return module


def test_current_stream(monkeypatch):
    other = without_raw_query(monkeypatch)
    side = torch.cuda.Stream()
    y = torch.randn(3, 64, device="cuda")
    want = gdn.gdn_block_norm(y, residual_scale=2.0)[0]
    for stream in (torch.cuda.current_stream(), side):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for m in (gdn, other):
                assert m._on_gpu(y.device) == torch.cuda.current_stream().cuda_stream == stream.cuda_stream
                got = m.gdn_block_norm(y, residual_scale=2.0)[0]
                stream.synchronize()
                assert torch.equal(got, want)
