"""mxfp8_matmul on the GPU at the edges of its dispatch: short sums in short rows, addends in every
kernel, operands and outputs past 2^31 bytes.  Against float64 with the tolerances of
test_gpu_layer_product.py."""
import pytest
import torch

import layer_reference as R
from gpu_util import DEV, require_gpu
from mxfp8_block_scaled_partial_amd import layer as L
from test_gpu_layer_product import FORMS, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("forms", FORMS, ids="-".join)
@pytest.mark.parametrize("k", [16, 32, 48, 64, 80])
@pytest.mark.parametrize("m,n", [(256, 32), (100, 300), (17, 272), (1040, 2064)])
def test_short_sums(m, n, k, forms, dtype):
    """Rows no longer than a half step, with tiles that end inside and outside the operands."""
    run(m, n, k, forms, (128, 1), (32, 1), dtype, seed=m + k)


def test_own_workspace_outlives_its_description():
    """A split sum on a busy stream, its description dropped at once: memory taken from the allocator
    meanwhile is not the workspace, and the result is right."""
    require_gpu()
    g = torch.Generator(device=DEV).manual_seed(5)
    m, n, k = 40, 512, 16384
    a, b = R.random_mat8(m, k, "cols", 128, 1, g, DEV), R.random_mat8(n, k, "cols", 32, 1, g, DEV)
    out = torch.zeros(m, n, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        p = L.make_product(L.make_operand(*a), L.make_operand(*b, block=32), out)
        at, size = p.workspace, p.workspace_bytes
        assert size >= 2 * m * n * 4
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        L.mxfp8_matmul(p, stream=stream)
        del p
        other = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
        assert other.data_ptr() + size <= at or other.data_ptr() >= at + size
        s.synchronize()
        va, vb = R.decode(*a, 1, 128), R.decode(*b, 1, 32)
        check(out, va @ vb.t(), va.abs() @ vb.abs().t(), k, True)
        out.zero_()
        torch.cuda.synchronize()
