"""A stream beside tensors that libfa refuses: its answer stands, as without one."""
import os
import shutil

import pytest

import exact_tiled_attention_forward_gb300 as fa
from exact_tiled_attention_forward_gb300 import build as fa_build


@pytest.mark.parametrize("stream", [None, 0, 1 << 20])
def test_host_tensors_are_refused_by_the_library(stream):
    torch = pytest.importorskip("torch")
    if not os.path.exists(fa.LIB_PATH):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("libfa.so not built and no nvcc")
        fa_build.build()
    if stream is None and not torch.cuda.is_available():
        pytest.skip("no current stream without a GPU")
    q = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(fa.FaError):
        fa.fa_forward(q, q, q, stream=stream)
    with pytest.raises(fa.FaError):
        fa.fa_forward_fp16(q.half(), q.half(), q.half(), stream=stream)
