"""The layer calls through torch's public stream and device calls, where the short ones are absent."""
import importlib.util

import pytest
import torch

from tests.layer_util import DEV

pytestmark = pytest.mark.gpu


def test_same_stream(monkeypatch):
    import fft_causal_long_amd.layers as layers
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    x = torch.randn(40, 96, device=DEV)
    want = layers.layer_norm(x)
    side = torch.cuda.Stream()
    with monkeypatch.context() as m:
        m.delattr(torch._C, "_cuda_getCurrentRawStream")
        m.delattr(torch._C, "_cuda_getDevice")
        spec = importlib.util.spec_from_file_location("fft_causal_long_amd._layers_public", layers.__file__)
        public = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(public)
    assert public._raw_stream is not layers._raw_stream
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            assert public._raw_stream(0) == s.cuda_stream == layers._raw_stream(0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = public.layer_norm(x)
    side.synchronize()
    assert public._get_device() == 0 and torch.equal(want, got)
