"""Which memory the training operators take, decided without a device."""
import os
import subprocess

import pytest

from sparse_attention_indexer_bwd_gb300 import _build

PROGRAM = """
#include <cstdio>
#include "train.h"
int main() {
  using ibwd::memory_fits;
  const int own = memory_fits(cudaMemoryTypeDevice, 0, 0) && memory_fits(cudaMemoryTypeDevice, 3, 3);
  const int other = memory_fits(cudaMemoryTypeDevice, 1, 0) || memory_fits(cudaMemoryTypeDevice, 0, 1);
  const int any = memory_fits(cudaMemoryTypeDevice, 1, -1) && memory_fits(cudaMemoryTypeManaged, 1, 0);
  const int host = memory_fits(cudaMemoryTypeHost, 0, 0) || memory_fits(cudaMemoryTypeUnregistered, 0, -1);
  std::printf("%d%d%d%d", own, other, any, host);
}
"""


def test_memory_of_another_device_is_refused(tmp_path):
    source, program = tmp_path / "fits.cpp", tmp_path / "fits"
    source.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-w", "-I", _build.CSRC, "-I", cuda, str(source), "-o", str(program)], check=True)
    assert subprocess.run([str(program)], capture_output=True, text=True, check=True).stdout == "1010"


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused():
    """Tensors that only say where they are: nothing of them can be read."""
    import torch
    from named_tensor import Named
    import sparse_attention_indexer_bwd_gb300 as ibwd
    other = f"cuda:{torch.cuda.current_device() + 1}"
    x, ids, r, t = (Named(shape, dtype, other) for shape, dtype in
                    (((4, 64), torch.float32), ((4, 2), torch.int32), ((4,), torch.float32), ((4, 2), torch.float32)))
    for call in (lambda: ibwd.layer_norm_fwd(x), lambda: ibwd.layer_norm_bwd(x, x, r, r),
                 lambda: ibwd.token_logprobs_fwd(x), lambda: ibwd.token_logprobs_bwd(x, None, r, r, None, r),
                 lambda: ibwd.distill_fwd(x, ids, t), lambda: ibwd.distill_bwd(x, ids, t, r, r),
                 lambda: ibwd.distill_grad(x, ids, t)):
        with pytest.raises(ValueError, match="current device"):
            call()
