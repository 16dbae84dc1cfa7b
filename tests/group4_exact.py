"""4-bit layers whose sums are whole numbers, for tests that compare to the last bit.

Tokens -16 .. 16, codes -7 .. 7, scales 1, 2, 4 or 8, none equal to its neighbour's: with sum |x w| below 2^24 for every output, every
partial sum in any order is a whole number that binary32 holds, so a right kernel gives the formula's number and nothing else.  A
bound that grows with K hides what one lane or one group adds to a long row; equality does not."""
import torch


def pack(code):
    """Stored bytes [rows, 4 ceil(cols / 8)] of codes in [-7, 7]: byte j of four holds code j and, in its high half, code j + 4."""
    rows, cols = code.shape
    nib = torch.where(code < 0, 8 - code, code).to(torch.uint8)
    nib = torch.nn.functional.pad(nib, (0, -cols % 8)).view(rows, -1, 2, 4)
    return (nib[:, :, 0] | nib[:, :, 1] << 4).view(rows, -1)


def layer(M, N, K, group, seed, device):
    """(x int64 [M, K], codes int8 [N, K], exponents int64 [N, groups])"""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    kw = dict(generator=g, device=device)
    x = torch.randint(-16, 17, (M, K), **kw)
    code = torch.randint(-7, 8, (N, K), dtype=torch.int8, **kw)
    steps = torch.randint(1, 4, (N, -(-K // group)), **kw)          # modulo 4 never 0: a scale differs from the one before it
    return x, code, steps.cumsum(1) % 4


def weights(code, exponents, group):
    """code * 2^e in float64"""
    return code.double() * torch.exp2(exponents.double()).repeat_interleave(group, 1)[:, :code.shape[1]]


def product(x, w):
    """X W^T, after a look at the sums' size."""
    assert float((x.double().abs() @ w.abs().t()).max()) < 2.0 ** 24
    return x.double() @ w.t()
