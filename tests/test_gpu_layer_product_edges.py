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


@pytest.mark.parametrize("m,n,k,forms,pad,split", [
    (1, 300, 4096, ("cols", "cols"), 0, False),      # few tokens
    (16, 130, 1000, ("cols", "cols"), 5, False),
    (70, 160, 592, ("cols", "rows"), 5, False),      # rows at any alignment, one part
    (48, 130, 12288, ("rows", "cols"), 5, True),     # .. and a split sum
    (48, 768, 12288, ("cols", "rows"), 0, True),     # aligned rows, split
    (1040, 2064, 720, ("cols", "rows"), 0, False),
], ids=str)
def test_bf16_output_with_addend(m, n, k, forms, pad, split):
    """Each kernel's way of adding before the one rounding to BF16."""
    _, p = run(m, n, k, forms, (128, 1), (32, 1), torch.bfloat16, seed=k, pad=pad, add="apart", ldo=pad)
    if split:
        assert p.workspace_bytes >= 2 * m * n * 4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k,forms", [(1, 512, 16384, ("cols", "rows")), (7, 1536, 8208, ("rows", "rows")),
                                         (48, 768, 12288, ("cols", "cols")), (200, 384, 9000, ("rows", "cols"))],
                         ids=str)
def test_sums_that_are_split(m, n, k, forms, dtype):
    """The workspace shows that these are: it holds the parts."""
    _, p = run(m, n, k, forms, (128, 1), (32, 1), dtype, seed=9)
    assert p.workspace_bytes >= 2 * m * n * 4


def far_operand(rows, cols, ld):
    """Codes [rows, cols] with rows `ld` apart, every row the same ones shifted by 16 times its index;
    scale bytes 127 for blocks of 32 along the columns."""
    g = torch.Generator(device=DEV).manual_seed(8)
    base = torch.randint(0, 256, (cols,), generator=g, device=DEV, dtype=torch.int32)
    base = torch.where((base & 0x7F) == 0x7F, base - 1, base).to(torch.uint8)
    data = torch.full((rows, ld), 0x7F, dtype=torch.uint8, device=DEV)[:, :cols]
    at = torch.arange(cols, device=DEV)
    for i in range(0, rows, 2000):
        r = torch.arange(i, min(rows, i + 2000), device=DEV)
        data[i:i + 2000] = base[(at[None] + 16 * r[:, None]) % cols]
    return data


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 16, 5])
@pytest.mark.parametrize("along", ["cols", "rows"])
def test_operands_past_32_bits(along, pad, dtype):
    """The second operand's last rows start past 2^31 bytes, for the main kernel and, with an odd
    leading dimension, the one for rows at any alignment."""
    require_gpu()
    rows, cols, m = 40000, 57344, 40
    data = far_operand(rows, cols, cols + pad)
    g = torch.Generator(device=DEV).manual_seed(9)
    n, k = (rows, cols) if along == "cols" else (cols, rows)
    shape = (rows, k // 32) if along == "cols" else (k // 32, cols)
    scale = torch.full(shape, 127, dtype=torch.uint8, device=DEV)
    a = R.random_mat8(m, k, "cols", 128, 1, g, DEV, pad)
    out = torch.empty(m, n, dtype=dtype, device=DEV)
    L.mxfp8_matmul(L.make_product(L.make_operand(*a), L.make_operand(data, scale, along=along, block=32), out))
    va = R.decode(*a, 1, 128)
    pick = [0, 1, n // 2, 37449 % n, 37450 % n, n - 2, n - 1]
    v = R.e4m3_value(data[pick] if along == "cols" else data[:, pick].t().contiguous())
    check(out[:, pick], va @ v.t(), va.abs() @ v.abs().t(), k, dtype == torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 5])
def test_outputs_past_32_bits(pad, dtype):
    """More than 2^31 outputs (2^33 bytes in FP32), their last tile ragged in both directions."""
    require_gpu()
    m, n, k = 48008, 46000, 64
    g = torch.Generator(device=DEV).manual_seed(10)
    a, b = R.random_mat8(m, k, "cols", 128, 1, g, DEV, pad), R.random_mat8(n, k, "cols", 32, 1, g, DEV, pad)
    out = torch.empty(m, n, dtype=dtype, device=DEV)
    L.mxfp8_matmul(L.make_product(L.make_operand(*a), L.make_operand(*b, block=32), out))
    va, vb = R.decode(*a, 1, 128), R.decode(*b, 1, 32)
    for rows in (slice(0, 300), slice(46600, 46800), slice(m - 300, m)):
        check(out[rows], va[rows] @ vb.t(), va[rows].abs() @ vb.abs().t(), k, dtype == torch.float32)
