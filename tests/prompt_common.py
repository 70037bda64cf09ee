"""Plain 64-bit forms of the prompt-side operators, with bounds on how far a kernel may be from them.

Every bound counts roundings. A value stored in bf16 is off by at most 2^-8 of it, in e4m3 by 2^-4 of it
(or 2^-10 of the block's scale, half the step of the smallest codes), in float by 2^-24.
"""
import torch

U = 2.0 ** -24


def bytes_of(top):
    """Scale bytes by the definition: the least e >= -127 with top <= 448 * 2^e, plus 127 (float64 in)."""
    e = torch.full_like(top, -127.0)
    live = top > 448.0 * 2.0 ** -127
    guess = torch.floor(torch.log2(torch.where(live, top, 1.0) / 448.0)) - 1
    for _ in range(3):
        guess = torch.where(top > 448.0 * torch.exp2(guess), guess + 1, guess)
    return torch.where(live, guess, e) + 127


def value_of(codes, scales):
    """float64 values of q8 rows (uint8 tensors)."""
    s = torch.exp2(scales.double() - 127.0)
    s = torch.where(scales == 255, torch.nan, s)
    return codes.view(torch.float8_e4m3fn).double() * torch.repeat_interleave(s, 32, -1)


def check_q8(codes, scales, v, dv):
    """q8 rows against float64 values v that the kernel's own floats are within dv of."""
    rows, K = v.shape
    top = v.abs().reshape(rows, -1, 32).amax(2)
    slack = dv.reshape(rows, -1, 32).amax(2)
    low, high = bytes_of((top - slack).clamp(min=0)), bytes_of(top + slack)
    got = scales.double().reshape(rows, -1)
    assert bool(((got >= low) & (got <= high)).all()), "scale byte"
    s = torch.repeat_interleave(torch.exp2(got - 127.0), 32, 1)
    off = (value_of(codes, scales.reshape(rows, -1)) - v).abs()
    most = 2.0 ** -4 * (v.abs() + dv) + 2.0 ** -10 * s + dv
    assert bool((off <= most).all()), f"code off by {float((off / most).max()):.3f} of its bound"


def check_near(got, v, dv, rounding):
    off = (got.double() - v).abs()
    most = rounding * (v.abs() + dv) + dv + 1e-38
    assert bool((off <= most).all()), f"off by {float((off / most).max()):.3f} of its bound"


def quantize(v):
    """q8 rows of a float tensor [..., K] by the definition (finite values)."""
    b = v.double().reshape(*v.shape[:-1], -1, 32)
    byte = bytes_of(b.abs().amax(-1))
    codes = (b * torch.exp2(127.0 - byte)[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(v.shape), byte.to(torch.uint8)


def products(x64, w64, counts):
    """(sums, bounds) of the rows of every expert, x64 [M, K] sorted, w64 [E, N, K]. The bound of a float
    sum in the tensor cores: every step of 16 (or 32) products is added with an error of at most 2 units in
    the last place of the sum of magnitudes, twice 2^-23 of it, and a few more steps at the ends."""
    M, K = x64.shape
    N = w64.shape[1]
    p = torch.zeros(M, N, dtype=torch.float64, device=x64.device)
    d = torch.zeros_like(p)
    at = 0
    for e, n in enumerate(counts):
        if n:
            p[at:at + n] = x64[at:at + n] @ w64[e].T
            d[at:at + n] = (x64[at:at + n].abs() @ w64[e].abs().T) * ((K / 16 + 8) * 2.0 ** -22)
        at += n
    return p, d


def swiglu(p, d):
    """silu(g) * u of [gate | up] products and its bound: the slope of silu is below 1.1, and the float
    form (exp, sum, quotient, product) adds at most 16 roundings."""
    I = p.shape[1] // 2
    g, u, dg, du = p[:, :I], p[:, I:], d[:, :I], d[:, I:]
    s = g * torch.sigmoid(g)
    return s * u, 1.1 * dg * (u.abs() + du) + s.abs() * du + 16 * U * (s * u).abs()


def offsets_of(counts, device="cuda"):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.cumsum(torch.tensor(counts, dtype=torch.int32), 0)
    return o.to(device)
