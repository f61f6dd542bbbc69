"""mxfp8_matmul on the GPU at the edges of its dispatch: short sums in short rows, addends in every
kernel, operands and outputs past 2^31 bytes.  Against float64 with the tolerances of
test_gpu_layer_product.py."""
import pytest
import torch

from test_gpu_layer_product import FORMS, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("forms", FORMS, ids="-".join)
@pytest.mark.parametrize("k", [16, 32, 48, 64, 80])
@pytest.mark.parametrize("m,n", [(256, 32), (100, 300), (17, 272), (1040, 2064)])
def test_short_sums(m, n, k, forms, dtype):
    """Rows no longer than a half step, with tiles that end inside and outside the operands."""
    run(m, n, k, forms, (128, 1), (32, 1), dtype, seed=m + k)
