"""The handle of the current stream, as every call without a stream takes it."""

import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
from sequence_latent_norm_gb300.checkpoint import on_stream

class Stream:
    cuda_stream = 4711

asked = []
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda device=None: asked.append(device) or Stream
with on_stream(torch.device("cuda", 3), None) as handle:
    assert handle == 4711 and asked == [3], (handle, asked)
"""


def test_a_torch_without_the_short_way():
    """torch's own shorter way to the handle is no public name: without it the
    public one serves."""
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
def test_it_is_the_current_streams():
    from sequence_latent_norm_gb300.checkpoint import on_stream
    dev = torch.device("cuda", 0)
    side = torch.cuda.Stream(dev)
    for stream in (torch.cuda.default_stream(dev), side):
        with torch.cuda.stream(stream):
            with on_stream(dev, None) as handle:
                assert handle == stream.cuda_stream == torch.cuda.current_stream(dev).cuda_stream
    with on_stream(dev, side) as handle:
        assert handle == side.cuda_stream and torch.cuda.current_stream(dev) == side
