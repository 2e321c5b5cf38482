"""A linear or an MLP called on another stream than the current one: its output
is not memory that the current stream still works on."""
import pytest
import torch

from nvfp4_w4a4_quantized_03_b200 import inputs, mq
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu
M, N, K = 64, 1024, 512


def _w(n, k, seed):
    return inputs.weight_bf16(n, k, seed=seed).to(dev())


@pytest.mark.parametrize("make", [lambda: mq.LinearW4A4(_w(N, K, 1)), lambda: mq.LinearW4A16(_w(N, K, 1)),
                                  lambda: mq.MLPW4A4(_w(512, K, 1), _w(N, 256, 2))], ids=["w4a4", "w4a16", "mlp"])
def test_an_output_on_another_stream(make):
    call, s = make(), torch.cuda.Stream()
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(0)).bfloat16().to(dev())
    want = call(x)
    call(x, stream=s)
    torch.cuda.synchronize()
    # a tensor that the current stream has yet to read, given back on the host
    torch.cuda.empty_cache()
    t = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=dev())
    read = torch.empty_like(t)
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)                                        # about 25 ms
    read.copy_(t)
    del t
    got = call(x, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert (read == 3.0).all()
    # and the other way: the output, given back while the current stream has yet to read it
    torch.cuda._sleep(50_000_000)
    read.copy_(got)
    del got
    with torch.cuda.stream(s):
        others = [torch.full((M, N), 7.0, dtype=torch.bfloat16, device=dev()) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(read, want) and all((o == 7.0).all() for o in others)


def test_quantize_on_another_stream():
    """Its tensors and its workspace are that stream's: the current one is busy meanwhile."""
    x, s = _w(256, K, 3), torch.cuda.Stream()
    want = mq.quantize(x)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device=dev()) for n in [1 << k for k in range(4, 20)] * 2]
    torch.cuda.synchronize()
    del junk
    torch.cuda._sleep(50_000_000)                                        # about 25 ms
    got = mq.quantize(x, stream=s)
    s.synchronize()
    parts = [(got.codes, want.codes), (got.scales, want.scales), (got.alpha, want.alpha)]
    with torch.cuda.stream(s):
        assert all(torch.equal(a, b) for a, b in parts)
