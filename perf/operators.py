"""Cases of the int8 and gated feed-forward operators, with their plain forms.

Operators, as a program calls them one after another:

* ``int8_quant``  rows of bf16 to int8 codes with one fp32 scale a row (a token's
  activations, or a weight's output channel);
* ``int8_gemm``   the product of two such operands with the scales of its tokens
  and channels, bias, GELU and residual in one pass;
* ``gated``       act(x Wg^T) * (x Wu^T) of a gated feed-forward block, from MXFP8
  or int8 activations; ``keep`` also returns the projections that the backward
  pass reads, ``ffn`` goes on through the MXFP8 hidden row to the down
  projection;
* ``gated_grad``  the block's backward pass: the input's and both weights'
  gradients from the hidden row's gradient.

``own`` chooses between the elementary torch form and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
F448 = torch.tensor(0x3B124925, dtype=torch.int32).view(torch.float32).item()    # fp32(1/448)
F57344 = torch.tensor(0x37924925, dtype=torch.int32).view(torch.float32).item()  # fp32(1/57344)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step's activations, before an int8 projection
        dict(name="int8_quant_decode", op="int8_quant", M=41, K=1536),
        # a whole prompt's activations, or a square weight's rows
        dict(name="int8_quant_prompt", op="int8_quant", M=8192, K=8192),
        # one token through a projection with bias: latency
        dict(name="int8_gemm_token", op="int8_gemm", M=1, N=4608, K=1536, bias=True, res=False,
             gelu=False),
        # a ragged prompt: odd rows, sizes that end inside every tile, all of the epilogue
        dict(name="int8_gemm_ragged", op="int8_gemm", M=1003, N=4104, K=2064, bias=True, res=True,
             gelu=True),
        # a large prompt batch through a square projection
        dict(name="int8_gemm_square", op="int8_gemm", M=8192, N=8192, K=8192, bias=False,
             res=False, gelu=False),
        # decode: 41 rows through an MXFP4 block
        dict(name="gated_decode", op="gated", kind="mxfp4", M=41, F=6144, K=1536, act="silu",
             keep=False, ffn=False),
        # decode against weights far larger than the caches
        dict(name="gated_stream", op="gated", kind="fp8blk32", M=16, F=16384, K=8192, act="silu",
             keep=False, ffn=False),
        # a training step's forward: the projections are kept for the backward pass
        dict(name="gated_train", op="gated", kind="mxfp8", M=4096, F=6144, K=1536, act="silu",
             keep=True, ffn=False),
        # a prompt through an int8 block, GELU-gated
        dict(name="gated_int8", op="gated", kind="int8", M=2048, F=8192, K=4096, act="gelu",
             keep=False, ffn=False),
        # a prompt through the whole block: gate, up, hidden in MXFP8, down projection
        dict(name="gated_ffn", op="gated", kind="mxfp8", M=4096, F=6144, K=1536, act="silu",
             keep=False, ffn=True),
        # a small step's backward pass
        dict(name="gated_grad_small", op="gated_grad", M=512, F=2048, K=1024, act="gelu"),
        # a training step's backward pass
        dict(name="gated_grad_train", op="gated_grad", M=4096, F=6144, K=1536, act="silu"),
    ]


MOST = 2.0 * 8192 ** 3  # operations of the largest listed case


def _size(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(-(-lo // step) * step, int(v) // step * step))


def draw(rng):
    op = rng.choice(["int8_quant", "int8_gemm", "int8_gemm", "gated", "gated", "gated",
                     "gated_grad"])
    if op == "int8_quant":
        while True:
            c = dict(op=op, M=_size(rng, 1, 8192, 1), K=_size(rng, 256, 16384, 16))
            if c["M"] * c["K"] <= 8192 * 8192:
                return c
    if op == "int8_gemm":
        while True:
            c = dict(op=op, M=_size(rng, 1, 8192, 1), N=_size(rng, 256, 16384, 8),
                     K=_size(rng, 256, 16384, 16), bias=rng.random() < 0.5,
                     res=rng.random() < 0.5, gelu=rng.random() < 0.3)
            if 2.0 * c["M"] * c["N"] * c["K"] <= MOST:
                return c
    if op == "gated":
        while True:
            kind = rng.choice(["mxfp4", "fp8blk32", "mxfp8", "int8"])
            ffn = kind == "mxfp8" and rng.random() < 0.5
            c = dict(op=op, kind=kind, M=_size(rng, 1, 8192, 1),
                     F=_size(rng, 256, 16384, 32 if ffn else 8),
                     K=_size(rng, 256, 8192,
                             {"mxfp4": 128, "int8": 16}.get(kind, 32)),
                     act=rng.choice(["silu", "gelu"]), keep=rng.random() < 0.3, ffn=ffn)
            if (6.0 if ffn else 4.0) * c["M"] * c["F"] * c["K"] <= MOST:
                return c
    while True:
        c = dict(op=op, M=_size(rng, 32, 8192, 32), F=_size(rng, 256, 8192, 32),
                 K=_size(rng, 256, 8192, 32), act=rng.choice(["silu", "gelu"]))
        if 8.0 * c["M"] * c["F"] * c["K"] <= MOST:
            return c


def work(case):
    c, op = case, case["op"]
    M, K = c["M"], c["K"]
    if op == "int8_quant":
        return {"bytes": 3 * M * K + 4 * M, "flops": 0}
    if op == "int8_gemm":
        N = c["N"]
        b = M * K + N * K + 4 * (M + N) + 2 * M * N
        return {"bytes": b + 2 * N * c["bias"] + 2 * M * N * c["res"], "flops": 2 * M * N * K}
    F = c["F"]
    if op == "gated":
        if c["kind"] == "int8":
            b = M * K + 4 * M + 2 * (F * K + 4 * F)
        else:
            w = {"mxfp4": F * K // 2 + F * K // 32, "fp8blk32": F * K + F * K // 32,
                 "mxfp8": F * K + F * K // 32}[c["kind"]]
            b = M * K * 33 // 32 + 2 * w
        b += (4 * M * F if c["keep"] else 0)
        f = 4 * M * F * K
        if c["ffn"]:
            return {"bytes": b + 2 * M * K + K * F * 33 // 32, "flops": f + 2 * M * F * K}
        return {"bytes": b + 2 * M * F, "flops": f}
    # the hidden row's gradient and both projections in, x and both weights in, dX and dW out
    b = 6 * M * F + 2 * M * K + 2 * F * K * 33 // 32 + 2 * M * K + 4 * F * K
    return {"bytes": b, "flops": 8 * M * F * K}


# ------------------------------------------------- formats, in plain torch --

def mma_scales(s):
    """Row-major scale bytes [R, G] in the layout that the products read: atoms of
    128 rows x 4 groups, byte (r % 32) * 16 + (r / 32 % 4) * 4 + g % 4, padding 127."""
    R, G = s.shape
    rb, gb = -(-R // 128), -(-G // 4)
    t = torch.full((rb * 128, gb * 4), 127, dtype=torch.uint8, device=s.device)
    t[:R, :G] = s
    return t.view(rb, 4, 32, gb, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def row_scales(sf, R, G):
    """The inverse of mma_scales: bytes [R, G]."""
    rb, gb = -(-R // 128), -(-G // 4)
    return sf.view(rb, gb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, gb * 4)[:R, :G]


def exponents(amax, inv):
    """e = ceil(log2(fp32(max(amax, 1e-4) * inv))) of fp32 group maxima."""
    t = amax.float().clamp_min(1e-4) * inv
    m, e = torch.frexp(t)
    return torch.where(m == 0.5, e - 1, e)


def pow2(e, wide):
    """2^e of integer exponents, by their bits: exact, where pow and ldexp are not
    everywhere."""
    if wide == torch.float64:
        return ((e.long() + 1023) << 52).view(torch.float64)
    return ((e.int() + 127) << 23).view(torch.float32)


def mx_quant(x, inv, top, dtype):
    """Codes and scale bytes of bf16 rows, per 32 of the last dimension."""
    R, C = x.shape
    g = x.float().view(R, C // 32, 32)
    e = exponents(g.abs().amax(-1), inv)
    q = (g * pow2(-e, torch.float32).unsqueeze(-1)).clamp(-top, top).to(dtype)
    return q.view(R, C), (e + 127).to(torch.uint8)


def mx_value(q, s, wide):
    """Codes (float8) times their groups' scales."""
    R, C = q.shape
    v = q.to(wide).view(R, C // 32, 32)
    return (v * pow2(s.int() - 127, wide).unsqueeze(-1)).view(R, C)


def fp4_value(b, s, wide):
    """Packed E2M1 bytes [R, C/2] (low nibble first) times their groups' scales."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=wide, device=b.device)
    R, h = b.shape
    idx = torch.stack((b & 15, b >> 4), -1).view(R, 2 * h).long()
    v = table[idx].view(R, h // 16, 32)
    return (v * pow2(s.int() - 127, wide).unsqueeze(-1)).view(R, 2 * h)


def weight_value(w, kind, rows, K, wide):
    if kind == "int8":
        return w["q"].to(wide) * w["s"].to(wide).unsqueeze(1)
    s = row_scales(w["sf"], rows, K // 32)
    if kind == "mxfp4":
        return fp4_value(w["q"], s, wide)
    return mx_value(w["q"].view(torch.float8_e4m3fn), s, wide)


# ---------------------------------------------------------------- inputs --

def _gen(seed, k):
    return torch.Generator(device=DEV).manual_seed((int(seed) * 64 + k) & 0x7FFFFFFFFFFF)


def _normal(shape, seed, k, std=1.0):
    return (torch.randn(shape, generator=_gen(seed, k), device=DEV) * std).to(torch.bfloat16)


def _int8_rows(x):
    """Int8 codes and fp32 scales of bf16 rows (64-bit quotients: ties are exact)."""
    a = x.double().abs().amax(-1, keepdim=True).clamp_min(2.0 ** -64)
    q = torch.round(x.double() * 127.0 / a).to(torch.int8)
    return q, (a.float() / 127.0).squeeze(1)


def _weight(kind, rows, K, seed, k):
    """A weight [rows, K] of values near N(0, 1/K) in the format `kind`."""
    if kind == "int8":
        q, s = _int8_rows(_normal((rows, K), seed, k, K ** -0.5))
        return {"q": q, "s": s}
    e = round(math.log2(K ** -0.5))
    u8 = dict(dtype=torch.uint8, device=DEV)
    if kind == "mxfp4":
        q = torch.randint(0, 256, (rows, K // 2), generator=_gen(seed, k), **u8)
        s = torch.randint(125 + e, 128 + e, (rows, K // 32), generator=_gen(seed, k + 1), **u8)
        return {"q": q, "sf": mma_scales(s)}
    if kind == "fp8blk32":
        q = (torch.randn((rows, K), generator=_gen(seed, k), device=DEV) * 64).clamp(-448, 448)
        s = torch.randint(120 + e, 123 + e, (-(-rows // 32), K // 32), generator=_gen(seed, k + 1),
                          **u8)
        return {"q": q.to(torch.float8_e4m3fn).view(torch.uint8),
                "sf": mma_scales(s.repeat_interleave(32, 0)[:rows])}
    q, s = mx_quant(_normal((rows, K), seed, k, K ** -0.5), F448, 448.0, torch.float8_e4m3fn)
    return {"q": q.view(torch.uint8), "sf": mma_scales(s)}


def prepare(case, seed):
    c, op = case, case["op"]
    M, K = c["M"], c["K"]
    st = {"c": dict(c)}
    if op == "int8_quant":
        # rows of unequal size, as tokens are, some of whose values stand far out
        x = torch.randn((M, K), generator=_gen(seed, 0), device=DEV)
        x *= torch.exp2(torch.randint(-3, 4, (M, 1), generator=_gen(seed, 1), device=DEV).float())
        far = torch.rand((M, K), generator=_gen(seed, 2), device=DEV) < 1e-3
        st["x"] = torch.where(far, x * 20, x).to(torch.bfloat16)
        return st
    if op == "int8_gemm":
        N = c["N"]
        st["a"], st["sa"] = _int8_rows(_normal((M, K), seed, 0))
        w = _weight("int8", N, K, seed, 1)
        st["b"], st["sb"] = w["q"], w["s"]
        st["bias"] = _normal((N,), seed, 4, 0.02) if c["bias"] else None
        st["res"] = _normal((M, N), seed, 5) if c["res"] else None
        return st
    F = c["F"]
    if op == "gated":
        kind = c["kind"]
        x = _normal((M, K), seed, 0)
        if kind == "int8":
            st["a"], st["sa"] = _int8_rows(x)
        else:
            q, s = mx_quant(x, F448, 448.0, torch.float8_e4m3fn)
            st["a"], st["sa"] = q.view(torch.uint8), mma_scales(s)
        st["wg"] = _weight(kind, F, K, seed, 10)
        st["wu"] = _weight(kind, F, K, seed, 20)
        if c["ffn"]:
            st["wd"] = _weight("mxfp8", K, F, seed, 30)
        return st
    # the projections as the forward pass keeps them, the hidden row's gradient, the
    # input, and both weights transposed in MXFP8 along the stacked output dimension
    st["gu"] = _normal((M, 2 * F), seed, 0)
    st["dh"] = _normal((M, F), seed, 1, 2.0 ** -10)
    st["x"] = _normal((M, K), seed, 2)
    wt = _normal((K, 2 * F), seed, 3, K ** -0.5)
    q, s = mx_quant(wt, F448, 448.0, torch.float8_e4m3fn)
    st["wt"], st["wt_sf"] = q.view(torch.uint8), mma_scales(s)
    return st


# ------------------------------------------------------------ plain forms --

def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _act_grad(g, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(
        2 * math.pi)


def _product(a, b):
    return a @ b.t()


def _compute(st, wide):
    """The operator of st in elementary steps, sums in `wide` (fp32 or 64 bits)."""
    c, op = st["c"], st["c"]["op"]
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731
    if op == "int8_quant":
        return _int8_rows(st["x"])
    M, K = c["M"], c["K"]
    if op == "int8_gemm":
        acc = _product(st["a"].to(wide), st["b"].to(wide))
        y = acc * st["sa"].to(wide).unsqueeze(1) * st["sb"].to(wide)
        if st["bias"] is not None:
            y = y + st["bias"].to(wide)
        if c["gelu"]:
            y = _act(y, "gelu")
        return y + st["res"].to(wide) if st["res"] is not None else y
    F = c["F"]
    if op == "gated":
        if c["kind"] == "int8":
            a = st["a"].to(wide) * st["sa"].to(wide).unsqueeze(1)
        else:
            a = mx_value(st["a"].view(torch.float8_e4m3fn), row_scales(st["sa"], M, K // 32), wide)
        g = _product(a, weight_value(st["wg"], c["kind"], F, K, wide))
        u = _product(a, weight_value(st["wu"], c["kind"], F, K, wide))
        h = _act(g, c["act"]) * u
        if not c["ffn"]:
            return (h, torch.cat((g, u), 1)) if c["keep"] else h
        q, s = mx_quant(bf(h), F448, 448.0, torch.float8_e4m3fn)
        y = _product(mx_value(q, s, wide), weight_value(st["wd"], "mxfp8", K, F, wide))
        return (y, torch.cat((g, u), 1)) if c["keep"] else y
    # rounded to bf16 before they are quantized, as the quantizers take their rows
    g, u = st["gu"][:, :F].to(wide), st["gu"][:, F:].to(wide)
    dh = st["dh"].to(wide)
    d = bf(torch.cat((dh * u * _act_grad(g, c["act"]), dh * _act(g, c["act"])), 1))
    q, s = mx_quant(d, F57344, 57344.0, torch.float8_e5m2)
    wt = mx_value(st["wt"].view(torch.float8_e4m3fn), row_scales(st["wt_sf"], K, 2 * F // 32), wide)
    dx = _product(mx_value(q, s, wide), wt)
    q, s = mx_quant(d.t().contiguous(), F57344, 57344.0, torch.float8_e5m2)
    xq, xs = mx_quant(st["x"].t().contiguous(), F448, 448.0, torch.float8_e4m3fn)
    return dx, _product(mx_value(q, s, wide), mx_value(xq, xs, wide))


def run(state):
    if own:
        return _run_own(state)
    out = _compute(state, torch.float32)
    if state["c"]["op"] == "int8_quant":
        return out
    if isinstance(out, tuple):
        return tuple(t.to(torch.bfloat16) for t in out)
    return out.to(torch.bfloat16)


# ------------------------------------------------------- the library's calls --

def _run_own(st):
    import block_scaled_precision_quant_b200 as bq
    c, op = st["c"], st["c"]["op"]
    M, K = c["M"], c["K"]
    if op == "int8_quant":
        return bq.act_quant_int8(st["x"])
    if op == "int8_gemm":
        return bq.gemm_int8_int8(st["a"], st["sa"], st["b"], st["sb"], M, c["N"], K,
                                 bias=st["bias"], residual=st["res"],
                                 act=bq.BQ_ACT_GELU if c["gelu"] else bq.BQ_ACT_NONE)
    F = c["F"]
    act = bq.BQ_GATE_SILU if c["act"] == "silu" else bq.BQ_GATE_GELU
    if op == "gated":
        kind = {"mxfp4": bq.W_MXFP4, "fp8blk32": bq.W_FP8BLK32, "mxfp8": bq.W_MXFP8,
                "int8": bq.W_INT8}[c["kind"]]
        s = "s" if c["kind"] == "int8" else "sf"
        wg, wu = st["wg"], st["wu"]
        out = bq.gemm_gated(kind, st["a"], st["sa"], wg["q"], wg[s], wu["q"], wu[s], M, F, K,
                            act=act, keep_projections=c["keep"], quantize_out=c["ffn"],
                            write_y=not c["ffn"])
        if not c["ffn"]:
            return out
        y = bq.gemm_mxfp8_mxfp8(out[1], out[2], st["wd"]["q"], st["wd"]["sf"], M, K, F)
        return (y, out[3]) if c["keep"] else y
    xt, xt_sf = bq.quant_transposed(st["x"])
    q, sf, qt, sft = bq.gated_grad_quant(st["dh"], st["gu"], act=act)
    dx = bq.gemm_e5m2_mxfp8(q, sf, st["wt"], st["wt_sf"], M, K, 2 * F)
    return dx, bq.gemm_e5m2_mxfp8(qt, sft, xt, xt_sf, 2 * F, K, M)


# ---------------------------------------------------------- from the definition --
#
# In 64 bits, apart from the plain form: codes are looked up by their bit fields,
# scales by index arithmetic, quantizers search for the scale by comparison.

def _x_two_to(e):
    """2^e for whole numbers e, looked up."""
    table = torch.tensor([2.0 ** k for k in range(-300, 301)], dtype=torch.float64, device=DEV)
    return table[(e + 300).clamp(0, 600).long()]


def _x_scale_bytes(sf, R, G):
    r = torch.arange(R, device=DEV).unsqueeze(1)
    g = torch.arange(G, device=DEV).unsqueeze(0)
    at = (torch.div(r, 128, rounding_mode="floor") * (-(-G // 4))
          + torch.div(g, 4, rounding_mode="floor")) * 512
    at = at + (r % 32) * 16 + (torch.div(r, 32, rounding_mode="floor") % 4) * 4 + g % 4
    return sf[at]


def _x_minifloat(codes, exp_bits, man_bits, bias):
    """Values of the codes by sign, exponent and mantissa fields."""
    c = codes.to(torch.int64)
    man, ex = c & ((1 << man_bits) - 1), (c >> man_bits) & ((1 << exp_bits) - 1)
    sign = 1.0 - 2.0 * ((c >> (man_bits + exp_bits)) & 1).double()
    frac = man.double() / (1 << man_bits)
    mag = torch.where(ex == 0, frac * 2.0 ** (1 - bias),
                      (1 + frac) * _x_two_to(ex - bias))
    return sign * mag


def _x_scaled(v, sb):
    return v * _x_two_to(sb.long() - 127).repeat_interleave(32, 1)


def _x_operand(q, s, kind, R, K):
    if kind == "int8":
        return q.double() * s.double()[:, None]
    sb = _x_scale_bytes(s, R, K // 32)
    if kind == "mxfp4":
        nib = torch.empty((R, K), dtype=torch.uint8, device=DEV)
        nib[:, 0::2], nib[:, 1::2] = q % 16, torch.div(q, 16, rounding_mode="floor")
        return _x_scaled(_x_minifloat(nib, 2, 1, 1), sb)
    return _x_scaled(_x_minifloat(q, 4, 3, 7), sb)


def _x_quantized(x, inv, man_bits, lowest):
    """The values that the codes of x stand for, per 32 of the last dimension: the
    smallest power of two s >= fp32(max(amax, 1e-4) * inv), then x / s to the nearest
    number of man_bits mantissa bits (ties to even), 2^lowest apart at least.  s leaves
    no |x / s| above the format's largest number."""
    x = x.double()
    R, C = x.shape
    g = x.view(R, C // 32, 32)
    floor = torch.tensor(1e-4, dtype=torch.float32).double().item()
    t = (g.abs().max(-1).values.clamp_min(floor).float()
         * torch.tensor(inv, dtype=torch.float32, device=DEV)).double()
    s = _x_two_to(torch.frexp(t).exponent)  # t < s
    s = torch.where(s / 2 >= t, s / 2, s)
    v = g / s[..., None]
    top = torch.frexp(v).exponent - 1
    step = _x_two_to((top - man_bits).clamp_min(lowest))
    return (torch.round(v / step) * step * s[..., None]).view(R, C)


def _x_sigmoid(g):
    e = torch.exp(-g.abs())
    return torch.where(g >= 0, 1 / (1 + e), e / (1 + e))


def _x_phi(g):
    return 0.5 * torch.special.erfc(-g * 0.5 ** 0.5)


def _x_gate(g, act):
    return g * (_x_sigmoid(g) if act == "silu" else _x_phi(g))


def _x_gate_slope(g, act):
    if act == "silu":
        s = _x_sigmoid(g)
        return s + g * s * (1 - s)
    return _x_phi(g) + g * torch.exp(-g * g / 2) * (2 * math.pi) ** -0.5


def exact(case, seed):
    c, op = case, case["op"]
    st = prepare(case, seed)
    M, K = c["M"], c["K"]
    if op == "int8_quant":
        a = st["x"].double().abs().max(1).values
        a = torch.where(a < 2.0 ** -64, torch.full_like(a, 2.0 ** -64), a)
        n = 127 * st["x"].double().abs() / a[:, None]
        lo = torch.floor(n)
        up = ((n - lo) > 0.5) | (((n - lo) == 0.5) & (lo % 2 == 1))
        q = (lo + up.double()) * torch.sign(st["x"].double())
        return q.to(torch.int8), a / 127
    if op == "int8_gemm":
        y = torch.einsum("mk,nk->mn", st["a"].double(), st["b"].double())
        y = y * torch.outer(st["sa"].double(), st["sb"].double())
        if c["bias"]:
            y = y + st["bias"].double()[None, :]
        if c["gelu"]:
            y = _x_gate(y, "gelu")
        return y + st["res"].double() if c["res"] else y
    F = c["F"]
    rounded = lambda t: t.to(torch.bfloat16).double()  # noqa: E731
    if op == "gated":
        kind = c["kind"]
        s = "s" if kind == "int8" else "sf"
        a = _x_operand(st["a"], st["sa"], "int8" if kind == "int8" else "mxfp8", M, K)
        g = torch.einsum("mk,nk->mn", a, _x_operand(st["wg"]["q"], st["wg"][s], kind, F, K))
        u = torch.einsum("mk,nk->mn", a, _x_operand(st["wu"]["q"], st["wu"][s], kind, F, K))
        y = _x_gate(g, c["act"]) * u
        if c["ffn"]:
            y = torch.einsum("mf,kf->mk", _x_quantized(rounded(y), F448, 3, -9),
                             _x_operand(st["wd"]["q"], st["wd"]["sf"], "mxfp8", K, F))
        return (y, torch.cat((g, u), 1)) if c["keep"] else y
    g, u, dh = st["gu"][:, :F].double(), st["gu"][:, F:].double(), st["dh"].double()
    d = rounded(torch.cat((dh * u * _x_gate_slope(g, c["act"]), dh * _x_gate(g, c["act"])), 1))
    dx = torch.einsum("mf,kf->mk", _x_quantized(d, F57344, 2, -16),
                      _x_operand(st["wt"], st["wt_sf"], "mxfp8", K, 2 * F))
    dw = torch.einsum("fm,km->fk", _x_quantized(d.t().contiguous(), F57344, 2, -16),
                      _x_quantized(st["x"].t().contiguous(), F448, 3, -9))
    return dx, dw
