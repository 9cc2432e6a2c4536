"""The 4-bit linear layer around the row counts where its kernels and their shapes change, against the
plain 64-bit form (ops_ref.py) with the bound derived there."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(__file__))

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ops_ref as ref  # noqa: E402
import sparse_moe_transformer_wave_amd as fm  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,K,N", [
    (1, 512, 24576), (64, 256, 24570), (7, 1152, 20479), (33, 640, 18001),        # x read by every workgroup
    (1, 384, 24577), (3, 1280, 24600), (8, 6272, 25001), (16, 3200, 24580),       # staged, in one chunk and several
    (20, 2688, 24577), (40, 2560, 24599), (64, 1408, 24583),
    (2, 1280, 33000), (8, 6272, 32999), (16, 3200, 33000), (5, 256, 65553)])      # K over two waves
def test_linear_row_counts(T, K, N, group):
    print("linear", T, K, N, group, flush=True)
    g = torch.Generator().manual_seed(K + N)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand(N, K // group, generator=g) + 0.5) * 0.01).to(BF)
    x = torch.randn(T, K, generator=g).to(BF)
    y = torch.full((T, N), 7.0, device="cuda")
    fm.linear_int4(fm.Int4Linear(codes.cuda(), scales.cuda()), x.cuda(), y)
    want, bound = ref.linear(codes, scales, x, bf16=False)
    over = (y.cpu().to(torch.float64) - want).abs() - bound
    assert (over <= 0).all(), "over the bound by %g" % over.max()
