"""mq_linear_w4a16 (bf16 activation, NVFP4 weight) against the 64-bit product of
the dequantized weight, element by element: the products are exact, a binary32
sum of K terms in any order, rounded or truncated, is off by at most
2 K 2^-24 sum |x w| (Higham, Lemma 3.1), two factors add 2^-22, and the
output rounds once to bf16 (2^-8)."""
import pytest
import torch

from nvfp4_w4a4_quantized_03_b200 import inputs, mq
from tests import kv_helpers as kv
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


def _check(x, w, y=None):
    N, K = w.shape
    M = x.shape[0]
    q = mq.quantize(w.to(dev()))
    got = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=dev())
    mq.mq_linear_w4a16(x.to(dev()), q.codes, q.scales, q.alpha, N, got)
    torch.cuda.synchronize()
    wv = kv.nvfp4_values(q.codes.cpu(), q.scales.cpu(), None, N, K)
    alpha = float(q.alpha.item())
    want = x.double() @ wv.T * alpha
    bound = (2 * K * 2.0 ** -24 + 2.0 ** -22) * alpha * (x.double().abs() @ wv.abs().T)
    print("worst error / bound:", kv.close_to(got.cpu(), want, bound))
    return got


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("N,K", [(1, 64), (130, 320), (300, 1088), (4096, 128)])
def test_small(M, N, K):
    x = inputs.activation_bf16(M, K, seed=M + K, outlier_channels=2, outlier_scale=50.0)
    _check(x, inputs.weight_bf16(N, K, seed=N))


@pytest.mark.parametrize("M,N,K", [(1, 6144, 4096), (3, 4096, 12288), (40, 1000, 4096), (64, 24576, 1024)])
def test_projections(M, N, K):
    x = inputs.activation_bf16(M, K, seed=M, outlier_channels=inputs.outlier_count(K), outlier_scale=50.0)
    _check(x, inputs.weight_bf16(N, K, seed=N))


def test_every_code_and_scale():
    """All 16 codes under every finite E4M3 scale, the subnormal ones and zero among them, against one-hot rows:
    each output is one exact product."""
    K, N = 256, 128
    codes = torch.arange(16, dtype=torch.uint8).repeat(N, K // 16)
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()
    r, kb = torch.arange(N)[:, None], torch.arange(K // 16)[None, :]
    want_scale = ((r * (K // 16) + kb) % 127).to(torch.uint8)
    at = (r // 128 * (K // 64) + kb // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + kb % 4
    scales = torch.zeros(mq.mq_nvfp4_scales_bytes(N, K), dtype=torch.uint8)
    scales[at.reshape(-1)] = want_scale.reshape(-1)
    alpha = torch.tensor([2.0])
    wv = kv.nvfp4_values(packed, scales, None, N, K)
    for lo in range(0, K, 64):
        x = torch.zeros(64, K)
        x[torch.arange(64), lo + torch.arange(64)] = torch.where(torch.arange(64) % 2 == 0, 1.0, -3.0)
        y = torch.empty(64, N, dtype=torch.bfloat16, device=dev())
        mq.mq_linear_w4a16(x.bfloat16().to(dev()), packed.to(dev()), scales.to(dev()), alpha.to(dev()), N, y)
        assert torch.equal(y.cpu().double(), (x.double() @ wv.T * 2).bfloat16().double())


def test_extreme_activations():
    """Rows of very different sizes, zeros; a NaN or an infinity in x stays in its row."""
    K, N = 512, 200
    x = torch.randn(6, K, generator=torch.Generator().manual_seed(0))
    x *= torch.tensor([1e-30, 1.0, 1e30, 0.0, 1.0, 1.0])[:, None]
    x = x.bfloat16()
    w = inputs.weight_bf16(N, K, seed=1)
    _check(x, w)
    clean = _check(x[:4], w)
    x[4, 7], x[5, 9] = float("nan"), float("inf")
    q = mq.quantize(w.to(dev()))
    y = torch.empty(6, N, dtype=torch.bfloat16, device=dev())
    mq.mq_linear_w4a16(x.to(dev()), q.codes, q.scales, q.alpha, N, y)
    assert torch.equal(y[:4], clean) and torch.isnan(y[4]).all() and not torch.isfinite(y[5]).any()


def test_rows_behind_the_output_stay():
    K, N, M = 128, 50, 3
    q = mq.quantize(inputs.weight_bf16(N, K, seed=1).to(dev()))
    buf = torch.full((M * N + 64,), -7.0, dtype=torch.bfloat16, device=dev())
    mq.mq_linear_w4a16(torch.ones(M, K, dtype=torch.bfloat16, device=dev()), q.codes, q.scales, q.alpha, N,
                       buf[:M * N].view(M, N))
    assert (buf[M * N:] == -7.0).all() and (buf[:M * N] != -7.0).any()
