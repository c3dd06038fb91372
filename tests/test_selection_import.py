"""What importing the package needs of torch: nothing beyond the names it had
before the selection products. The current stream's raw handle comes from a
private function of torch where there is one, else from the public stream
object. Needs no GPU but for the last test."""

import os
import subprocess
import sys

import pytest
import torch

from helpers import need_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("module", ["sparse_dense_matmul_amd", "sparse_dense_matmul_amd.build"])
def test_import_without_the_private_stream_function(module):
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            f"import {module}\n"
            "from sparse_dense_matmul_amd import CsrMatrix, embedding\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-600:]


@pytest.mark.gpu
def test_stream_handle_without_the_private_function(monkeypatch):
    """The public way names the same stream, and calls through it give the same."""
    need_gpu()
    from sparse_dense_matmul_amd import embedding, selection

    table = torch.arange(12.0, device="cuda").reshape(4, 3)
    ids = torch.tensor([3, -1, 0], device="cuda")
    want = embedding(table, ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            assert selection._public_raw_stream(0) == selection._raw_stream(0) == stream.cuda_stream
    monkeypatch.setattr(selection, "_raw_stream", selection._public_raw_stream)
    with torch.cuda.stream(side):
        got = embedding(table, ids)
    side.synchronize()
    assert torch.equal(got, want)
