"""GPU tests of long sums whose result binary32 holds exactly: small integers times a power of two, every partial sum
below 2^24 units whatever the order, so the outputs have to be equal, and one term left out or read twice shows.  A
bound on rounding errors cannot fail there: over 2^21 terms of random sign it is larger than the result."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops  # noqa: E402

BIG = (1 << 21) + 24
SCALE = 2.0 ** -6


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def ints(shape, most, seed, dtype):
    """Integers of [-most, most] without 0, so that every term counts."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(1, most + 1, shape, generator=g, device="cuda", dtype=torch.int8)
    s = torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.int8) * 2 - 1
    return (v * s).to(dtype)


def layer(N, K, most, seed):
    codes = ints((N, K), most, seed, torch.int8)
    return codes, torch.full((N,), SCALE, device="cuda", dtype=torch.float16)


def exact(a, b, scale=SCALE):
    """a @ b.T of integers below 2^53, times scale, as fp32; the products' sizes allow it to be exact."""
    s = a.abs().double() @ b.abs().double().t()
    assert float(s.max()) < 2 ** 24
    want = (a.double() @ b.double().t()) * scale
    cut = (a[:, :-24].double() @ b[:, :-24].double().t()) * scale
    assert not torch.equal(want, cut) and bool(want.any())           # what a lost tail or an empty result would give
    return want.float()


@pytest.mark.parametrize("M", [1, 2, 17, 40, 66])
def test_forward_over_2_to_the_21(M):
    say(f"exact sums: forward {M} tokens, K = 2^21 + 24")
    codes, scales = layer(3, BIG, 3, M)
    x = ints((M, BIG), 2, M + 1, torch.bfloat16)
    y = ops.qlinear(x, codes, scales, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(y, exact(x, codes))


@pytest.mark.parametrize("M,N,K,pad", [(1, 7, 40000, 0), (5, 40, 8192, 0), (16, 64, 6176, 3), (33, 20, 8200, 1), (64, 16, 16384, 8),
                                       (70, 66, 4633, 0), (2076, 70, 6202, 0), (130, 264, 40008, 0), (66, 30, (1 << 21) - 8, 0)])
def test_forward_in_parts(M, N, K, pad):
    say(f"exact sums: forward {M}x{N}x{K}")
    codes, scales = layer(N, K + pad, 3, M)
    x = ints((M, K + pad), 2, M + 1, torch.bfloat16)[:, :K]
    codes = codes[:, :K]
    y = ops.qlinear(x, codes, scales, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(y, exact(x, codes))


@pytest.mark.parametrize("M,K", [(1, 5), (2, 40), (66, 8)])
def test_input_gradient_over_2_to_the_21_outputs(M, K):
    say(f"exact sums: dX of {M} tokens over N = 2^21 + 24")
    codes, scales = layer(BIG, K, 3, K)
    dy = ints((M, BIG), 2, 9, torch.bfloat16)
    x = ints((M, K), 2, 10, torch.bfloat16)
    got = ops.qlinear_backward(dy, codes, scales, x=x, want_dbias=True, dx_dtype=torch.float32, dw_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(got["dx"], exact(dy, codes.t()))
    assert torch.equal(got["dw"].double(), dy.t().double() @ x.double())
    assert torch.equal(got["dbias"].double(), dy.double().sum(0))


@pytest.mark.parametrize("N,K", [(3, 40), (70, 136), (200, 33)])
def test_weight_gradient_over_many_tokens(N, K):
    M = 1_000_000
    say(f"exact sums: dW {N}x{K} over {M} tokens")
    dy, x = ints((M, N), 2, 1, torch.bfloat16), ints((M, K), 3, 2, torch.bfloat16)
    got = ops.qlinear_backward(dy, None, None, x=x, want_dx=False, want_dbias=True, dw_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(got["dw"], exact(dy.t(), x.t(), 1.0))
    assert torch.equal(got["dbias"].double(), dy.double().sum(0))


def test_row_strides_of_2_to_the_21():
    """X, the codes and dY as columns of buffers whose rows are 2^21 + 24 elements apart, with other numbers
    around them."""
    say("exact sums: row strides of 2^21 + 24")
    M, N, K = 70, 40, 64
    x = ints((M, BIG), 2, 3, torch.bfloat16)[:, 8:8 + K]
    dy = ints((M, BIG), 2, 4, torch.bfloat16)[:, 64:64 + N]
    codes = ints((N, BIG), 3, 5, torch.int8)[:, 16:16 + K]
    scales = torch.full((N,), SCALE, device="cuda", dtype=torch.float16)
    y = ops.qlinear(x, codes, scales, out_dtype=torch.float32)
    got = ops.qlinear_backward(dy, codes, scales, x=x, dx_dtype=torch.float32, dw_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(y, exact(x, codes))
    assert torch.equal(got["dx"], exact(dy, codes.t()))
    assert torch.equal(got["dw"], exact(dy.t(), x.t(), 1.0))
