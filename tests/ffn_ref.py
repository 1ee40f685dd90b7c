"""Plain 64-bit forms of the int8 and gated feed-forward operators (torch double
tensors, on any device), and the operands their tests feed to the library."""
import math

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def int8_rows(x):
    """(codes, scales) of the row quantizer by its definition in 64 bits."""
    a = x.double().abs().amax(1).clamp_min(2.0 ** -64)
    return torch.round(x.double() * 127 / a[:, None]).to(torch.int8), a / 127


def minifloat(codes, exp_bits, man_bits, bias):
    c = codes.long()
    man, ex = c & ((1 << man_bits) - 1), (c >> man_bits) & ((1 << exp_bits) - 1)
    sign = 1.0 - 2.0 * ((c >> (man_bits + exp_bits)) & 1).double()
    frac = man.double() / (1 << man_bits)
    return sign * torch.where(ex == 0, frac * 2.0 ** (1 - bias),
                              (1 + frac) * 2.0 ** (ex - bias).double())


def mma_layout(s):
    """Row-major scale bytes [R, G] to the MMA layout, byte by byte."""
    R, G = s.shape
    ga = -(-G // 4)
    out = torch.full((-(-R // 128) * ga * 512,), 127, dtype=torch.uint8, device=s.device)
    r = torch.arange(R, device=s.device)[:, None]
    c = torch.arange(G, device=s.device)[None, :]
    at = ((r // 128) * ga + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4
    out[at.reshape(-1)] = s.reshape(-1)
    return out


class Operand:
    """A random operand [R, K] of one format: q and sf as the library takes them, and
    value, its 64-bit values."""

    def __init__(self, kind, R, K, seed, spread=3):
        g = torch.Generator().manual_seed(seed)
        u8 = dict(dtype=torch.uint8, generator=g)
        if kind == "int8":
            self.q = torch.randint(-128, 128, (R, K), dtype=torch.int8, generator=g).cuda()
            self.sf = (torch.rand((R,), generator=g) * 0.02 + 1e-4).cuda()
            self.value = self.q.double() * self.sf.double()[:, None]
            return
        lo, hi = 127 - spread, 127 + spread
        if kind == "fp8blk32":
            s = torch.randint(lo - 6, hi - 5, (-(-R // 32), K // 32), **u8)
            s = s.repeat_interleave(32, 0)[:R]
        else:
            s = torch.randint(lo - 6, hi - 5, (R, K // 32), **u8)
        if kind == "mxfp4":
            self.q = torch.randint(0, 256, (R, K // 2), **u8).cuda()
            nib = torch.stack((self.q & 15, self.q >> 4), -1).reshape(R, K)
            v = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64,
                             device="cuda")[nib.long()]
        else:
            q = torch.randint(0, 254, (R, K), **u8)
            self.q = (q + (q >= 127).to(torch.uint8)).cuda()  # every code but 0x7F, 0xFF
            v = minifloat(self.q, 4, 3, 7)
        self.sf = mma_layout(s.cuda())
        self.value = v * (2.0 ** (s.cuda().double() - 127)).repeat_interleave(32, 1)


def product(a, b):
    """a b^T of two operands in 64 bits.  Int8: the integer sum (exact), then the
    scales, so that a sum of zero stays zero."""
    if a.q.dtype == torch.int8:
        return (a.q.double() @ b.q.double().t()) * a.sf.double()[:, None] * b.sf.double()
    return a.value @ b.value.t()


def gelu(t):
    return t * 0.5 * torch.special.erfc(-t / math.sqrt(2))


def silu(t):
    return t * torch.sigmoid(t)


def gate(t, act):
    return silu(t) if act == 0 else gelu(t)


def gate_slope(t, act):
    if act == 0:
        s = torch.sigmoid(t)
        return s * (1 + t * (1 - s))
    return (0.5 * torch.special.erfc(-t / math.sqrt(2))
            + t * torch.exp(-t * t / 2) / math.sqrt(2 * math.pi))


def close(y, ref, tol, what=""):
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst "
        f"{float((err / tol.clamp_min(1e-300)).max()):.3g} of the tolerance at "
        f"{bad.nonzero()[:4].tolist()}")


# Half a bf16 step, relative; what fp32 arithmetic may add to a value of 1 over a
# chain of a few operations.
BF16, FP32 = 2.0 ** -8, 2.0 ** -24


def int8_tol(p, bias, pre, res, ref, gelu_used):
    """|y - ref| of the int8 product.  p = alpha sa sb acc is off by four fp32 roundings
    (acc to fp32, alpha sb, times sa, times acc); the sum with the bias by one more;
    the GELU multiplies that by its largest slope 1.13 and adds 1.5e-7 / 2 of its
    argument (its erf's error) and two fast operations' 2^-21 of it; the residual's
    sum adds a rounding, and the result is rounded to bf16."""
    d = FP32 * (4.1 * p.abs() + (p + bias).abs() * 1.01)
    if gelu_used:
        d = 1.13 * d + pre.abs() * (1e-7 + 2.0 ** -21)
    d = d + FP32 * ((ref - res).abs() + res.abs() + ref.abs())
    return BF16 * (ref.abs() + d) + d + 1e-38


def gated_tol(g, u, sg, su, h, act):
    """|h' - h| where g and u are off by at most sg and su: the product's first order
    terms with the activation's largest slope 1.13, both errors at once, the
    activation's own error (SiLU: 2^-18 relative for |g| < 30, where e^-g's argument
    takes a rounding of 1.44 |g| 2^-24 and the exponential and division 2^-21; GELU:
    as above), a rounding, and the final one to bf16."""
    a = gate(g, act).abs()
    d = 1.13 * sg * u.abs() + a * su + 1.13 * sg * su
    d = d + h.abs() * 2.0 ** -18 + (g * u).abs() * (1e-7 if act == 1 else 0.0)
    return BF16 * (h.abs() + d) + d + 1e-38
