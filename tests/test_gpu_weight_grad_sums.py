"""What a weight gradient adds up and rounds, bit for bit: operands are small
whole numbers, so every sum is exact in fp32 in any order, and what is left is
the one rounding of the result."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def whole_numbers(T, N, K, cuda, seed):
    """dy and a checkpoint of small whole numbers, and their exact product."""
    g = torch.Generator(device=cuda).manual_seed(seed)
    dy = torch.randint(-4, 5, (T, N), generator=g, device=cuda).to(BF16)
    x = torch.randint(-4, 5, (T, K), generator=g, device=cuda).float()
    k = z.new_checkpoint(T, K, cuda)
    z.zero1_checkpoint_pack(x, k)
    out = torch.zeros((N, K), dtype=torch.float64, device=cuda)
    for a in range(0, T, 4096):
        out += (dy[a:a + 4096].double().t() @ x[a:a + 4096].double())
    assert out.abs().max() < 2 ** 24            # each partial sum is a whole number of fp32
    return dy, k, out


def result(N, K, dtype, cuda, off, fill):
    """A [N, K] view at an element offset of a flat buffer, filled with `fill`."""
    flat = torch.full((off + N * K + 8,), 7.0, dtype=dtype, device=cuda)
    dw = flat[off:off + N * K].view(N, K)
    dw.copy_(fill)
    return flat, dw


# rows in one run of the accumulator or several; tiles done whole, split, or both; edges on and off 16 bytes
SIZES = [(100, 300, 260), (777, 771, 1000), (2048, 512, 512), (5000, 2560, 2560), (5000, 2555, 2557), (9000, 300, 200),
         (2200, 70, 130), (4500, 2816, 2600)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("off", [0, 1, 4])
@pytest.mark.parametrize("scaled", [False, True])
def test_added_with_one_rounding(cuda_device, T, N, K, off, scaled):
    """A gradient far larger than what is added to it: the sum is rounded at its
    size once, however many runs of rows there are."""
    dy, k, exact = whole_numbers(T, N, K, cuda_device, T)
    g = torch.Generator(device=cuda_device).manual_seed(1)
    start = torch.randint(-2 ** 20, 2 ** 20, (N, K), generator=g, device=cuda_device).float() * 64 + 2.0 ** 27
    scale = torch.tensor([0.5, 1.0, 2.0, -4.0], device=cuda_device).repeat(-(-K // 4))[:K].contiguous()
    flat, dw = result(N, K, F32, cuda_device, off, start)
    z.zero1_weight_grad(dy, k, dw, col_scale=scale if scaled else None, accumulate=True)
    want = (start.double() + exact * (scale.double() if scaled else 1.0)).float()
    assert torch.equal(dw, want)
    assert (flat[:off] == 7).all() and (flat[off + N * K:] == 7).all()


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_stored_exactly(cuda_device, T, N, K, off, dtype):
    dy, k, exact = whole_numbers(T, N, K, cuda_device, T + 1)
    flat, dw = result(N, K, dtype, cuda_device, off, torch.full((N, K), float("nan")))
    z.zero1_weight_grad(dy, k, dw)
    assert torch.equal(dw, exact.to(dtype))
    assert (flat[:off] == 7).all() and (flat[off + N * K:] == 7).all()


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("off", [0, 1])
def test_bf16_added_with_one_rounding(cuda_device, T, N, K, off):
    dy, k, exact = whole_numbers(T, N, K, cuda_device, T + 2)
    g = torch.Generator(device=cuda_device).manual_seed(2)
    start = (torch.randint(-128, 128, (N, K), generator=g, device=cuda_device) * 2 ** 8).to(BF16)
    flat, dw = result(N, K, BF16, cuda_device, off, start)
    z.zero1_weight_grad(dy, k, dw, accumulate=True)
    assert torch.equal(dw, (start.double() + exact).to(BF16))


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_adding_nothing_changes_nothing(cuda_device, T, N, K, off, dtype):
    """A gradient's own values, subnormal ones and the smallest and largest
    among them, stay bit for bit where the sum is 0."""
    _, k, _ = whole_numbers(T, N, K, cuda_device, T + 3)
    g = torch.Generator(device=cuda_device).manual_seed(3)
    e = torch.randint(-148, 127, (N, K), generator=g, device=cuda_device).double()
    start = (torch.exp2(e) * (1 + torch.rand((N, K), generator=g, device=cuda_device).double())).float().to(dtype)
    flat, dw = result(N, K, dtype, cuda_device, off, start)
    z.zero1_weight_grad(torch.zeros((T, N), dtype=BF16, device=cuda_device), k, dw, accumulate=True)
    bits = torch.int32 if dtype == F32 else torch.int16
    assert torch.equal(dw.reshape(-1).view(bits), start.reshape(-1).view(bits))


@pytest.mark.parametrize("T,N,K", [(5000, 2560, 2560), (9000, 300, 200), (777, 771, 1000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("accumulate", [False, True])
def test_a_workspace_of_the_asked_size_is_enough(cuda_device, T, N, K, dtype, accumulate):
    dy, k, exact = whole_numbers(T, N, K, cuda_device, T + 4)
    need = z.zero1_weight_grad_workspace(dy, K)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=cuda_device)
    _, dw = result(N, K, dtype, cuda_device, 0, torch.zeros((N, K)))
    z.zero1_weight_grad(dy, k, dw, accumulate=accumulate, workspace=ws[:need])
    assert torch.equal(dw, exact.to(dtype)) and (ws[need:] == 0xA5).all()
    if need:
        with pytest.raises(z.Zero1Error, match="workspace"):
            z.zero1_weight_grad(dy, k, dw, accumulate=accumulate, workspace=ws[:need - 1])
