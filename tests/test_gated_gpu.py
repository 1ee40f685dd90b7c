"""The gated feed-forward block and its backward pass against 64-bit forms."""
import numpy as np
import pytest
import torch

import block_scaled_precision_quant_b200 as bq
from ffn_ref import BF16, FP32, Operand, close, gate, gate_slope, gated_tol, product

pytestmark = pytest.mark.gpu

KIND = {"mxfp4": bq.W_MXFP4, "fp8blk32": bq.W_FP8BLK32, "mxfp8": bq.W_MXFP8, "int8": bq.W_INT8}
ACTS = [bq.BQ_GATE_SILU, bq.BQ_GATE_GELU]


def forward(kind, M, N, K, act, seed, alpha=None, config=None, keep=False, quant=False,
            write_y=True):
    a = Operand("int8" if kind == "int8" else "mxfp8", M, K, seed)
    wg, wu = Operand(kind, N, K, seed + 1), Operand(kind, N, K, seed + 2)
    if alpha is None:  # brings g and u to the size of ones
        alpha = float(1.0 / product(a, wg).std().clamp_min(1e-3)) if M * N > 1 else 1.0
        alpha = float(np.float32(alpha))
    out = bq.gemm_gated(KIND[kind], a.q, a.sf, wg.q, wg.sf, wu.q, wu.sf, M, N, K, act=act,
                        alpha=alpha, keep_projections=keep, quantize_out=quant, write_y=write_y,
                        config=config)
    bq.device_status()
    g, u = alpha * product(a, wg), alpha * product(a, wu)
    if kind == "int8":  # four fp32 roundings of the scaled exact sum
        sg, su = 4.1 * FP32 * g.abs(), 4.1 * FP32 * u.abs()
    else:  # the products' bound 2^-20 sum |a b|, and alpha's rounding
        sg = abs(alpha) * (a.value.abs() @ wg.value.abs().t()) * 2.0 ** -20 + FP32 * g.abs()
        su = abs(alpha) * (a.value.abs() @ wu.value.abs().t()) * 2.0 ** -20 + FP32 * u.abs()
    h = gate(g, act) * u
    tol = gated_tol(g, u, sg, su, h, act)
    outs = out if isinstance(out, tuple) else (out,)
    if write_y:
        close(outs[0], h, tol, f"h {kind} {M}x{N}x{K}")
    else:
        assert outs[0] is None
    if keep:
        gu = outs[-1]
        close(gu[:, :N], g, BF16 * (g.abs() + sg) + sg, "g")
        close(gu[:, N:], u, BF16 * (u.abs() + su) + su, "u")
    return outs, h, tol


# one row to many, one K block to several, outputs that end inside a tile
SIZES = [(1, 8, 128), (1, 1536, 512), (3, 136, 256), (17, 520, 128), (32, 128, 1024),
         (41, 1544, 1536), (64, 200, 384), (65, 256, 640), (100, 648, 256), (128, 128, 2048),
         (129, 264, 256), (300, 392, 512), (513, 136, 384)]


@pytest.mark.parametrize("kind", list(KIND))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(kind, M, N, K):
    forward(kind, M, N, K, ACTS[(M + N) % 2], M + N + K, keep=M % 2 == 1)


@pytest.mark.parametrize("kind,K", [("fp8blk32", 32), ("mxfp8", 96), ("mxfp8", 544),
                                    ("fp8blk32", 1184), ("int8", 16), ("int8", 208),
                                    ("int8", 1136)])
@pytest.mark.parametrize("M", [1, 50, 140])
def test_forward_k_tails(kind, K, M):
    for act in ACTS:
        forward(kind, M, 264, K, act, M + K)


@pytest.mark.parametrize("kind", list(KIND))
@pytest.mark.parametrize("bn,split", [(32, 1), (32, 3), (64, 2), (64, 8), (128, 1), (128, 5)])
def test_forward_swap_schedules(kind, bn, split):
    # MX tiles shorter than a scale atom hold all rows; longer operands are refused
    M = 70 if kind == "int8" or bn == 128 else bn - 3
    forward(kind, M, 392, 1152, ACTS[split % 2], bn + split, keep=True,
            config=bq.config(block_n=bn, split_k=split, swap_ab=1))


@pytest.mark.parametrize("kind", list(KIND))
@pytest.mark.parametrize("M,N,K", [(1, 8, 128), (100, 136, 384), (128, 128, 1024),
                                   (129, 264, 1152), (257, 1032, 256), (700, 520, 640)])
def test_forward_pair_tiles(kind, M, N, K):
    forward(kind, M, N, K, ACTS[(M + 1) % 2], M + N, keep=M != 128, config=bq.config(swap_ab=0))


# more tiles than pairs of SMs, K blocks that end anywhere in the rings of operands
# (5 or 6) and scales (4 to a stage)
@pytest.mark.parametrize("kind", list(KIND))
@pytest.mark.parametrize("K", [128, 640, 1408])
def test_forward_pair_tiles_in_several_waves(kind, K):
    forward(kind, 2900, 1672, K, ACTS[K % 3 == 2], K, keep=K == 640, config=bq.config(swap_ab=0))


@pytest.mark.parametrize("kind", ["mxfp4", "int8"])
def test_quantized_hidden_in_several_waves(kind):
    outs, _, _ = forward(kind, 2900, 1696, 384, bq.BQ_GATE_GELU, 3, quant=True)
    q, sf = bq.act_quant(outs[0])
    assert torch.equal(outs[1], q) and torch.equal(outs[2], sf)


@pytest.mark.parametrize("kind", list(KIND))
@pytest.mark.parametrize("M,N,K", [(1, 32, 128), (41, 1536, 512), (70, 160, 384), (130, 96, 256),
                                   (300, 416, 640)])
@pytest.mark.parametrize("write_y", [True, False])
def test_quantized_hidden_is_act_quant_of_h(kind, M, N, K, write_y):
    outs, _, _ = forward(kind, M, N, K, bq.BQ_GATE_SILU, M, quant=True)
    q, sf = bq.act_quant(outs[0])
    assert torch.equal(outs[1], q)
    assert torch.equal(outs[2], sf)  # padding rows and groups included
    if not write_y:
        only, _, _ = forward(kind, M, N, K, bq.BQ_GATE_SILU, M, quant=True, write_y=False,
                             keep=True)
        assert torch.equal(only[1], q) and torch.equal(only[2], sf)


def test_outputs_given_and_rows_behind_them():
    M, N, K = 37, 96, 128
    a, w, v = Operand("mxfp8", M, K, 1), Operand("mxfp8", N, K, 2), Operand("mxfp8", N, K, 3)
    y = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((M + 2, 2 * N), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((M + 2, N), 7, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(bq.sf_bytes(M, N) + 16, dtype=torch.uint8, device="cuda")
    bq.gemm_gated(bq.W_MXFP8, a.q, a.sf, w.q, w.sf, v.q, v.sf, M, N, K, y=y[:M], gu=gu[:M],
                  quantize_out=True, q_out=q[:M], sf_out=sf)
    bq.device_status()
    ref = bq.gemm_gated(bq.W_MXFP8, a.q, a.sf, w.q, w.sf, v.q, v.sf, M, N, K,
                        keep_projections=True)
    assert torch.equal(y[:M], ref[0]) and torch.equal(gu[:M], ref[1])
    assert bool((y[M:] == 7).all()) and bool((gu[M:] == 7).all()) and bool((q[M:] == 7).all())
    assert int(sf[-16:].max()) == 0


def test_nonfinite_hidden_is_reported():
    M, N, K = 4, 32, 128
    a, w = Operand("mxfp8", M, K, 1), Operand("mxfp8", N, K, 2)
    bq.gemm_gated(bq.W_MXFP8, a.q, a.sf, w.q, w.sf, w.q, w.sf, M, N, K, alpha=1e30,
                  quantize_out=True)
    with pytest.raises(bq.BqError) as e:
        bq.device_status()
    assert e.value.status == bq.BQ_ERR_NONFINITE


def test_large_gate_values_saturate():
    """SiLU and GELU far out: act(g) is g or (negative) zero, never a NaN."""
    M, N, K = 8, 64, 128
    a, w, v = Operand("int8", M, K, 1), Operand("int8", N, K, 2), Operand("int8", N, K, 3)
    for act in ACTS:
        y = bq.gemm_gated(bq.W_INT8, a.q, a.sf, w.q, w.sf, v.q, v.sf, M, N, K, act=act,
                          alpha=300.0)
        bq.device_status()
        g, u = 300.0 * product(a, w), 300.0 * product(a, v)
        h = torch.where(g > 0, g, torch.zeros_like(g)) * u
        far = g.abs() > 120
        assert int(far.sum()) > 10 and bool(torch.isfinite(y).all())
        # 2^-20 |g u|: the GELU's erf is off by 1.5e-7 / 2 of g u there
        close(y[far], h[far], (BF16 * 1.01 * h.abs() + (g * u).abs() * 2.0 ** -20)[far])


# -------------------------------------------------------------- backward ----

def grads(M, N, seed, scale=2.0 ** -6):
    g = torch.Generator().manual_seed(seed)
    gu = (torch.randn((M, 2 * N), generator=g) * 2).to(torch.bfloat16).cuda()
    dh = (torch.randn((M, N), generator=g) * scale).to(torch.bfloat16).cuda()
    return dh, gu


def grad_ref(dh, gu, act):
    N = dh.shape[1]
    d, g, u = dh.double(), gu[:, :N].double(), gu[:, N:].double()
    ref = torch.cat((d * u * gate_slope(g, act), d * gate(g, act)), 1)
    # act' in fp32: s and its parts to 2^-20 with factors up to 1 + |g| <= 16 here; act: 2^-18
    # relative (SiLU) or 1e-7 of its argument (GELU); then the roundings
    e = torch.cat(((d * u).abs() * (1 + g.abs()) * 2.0 ** -20,
                   (d * gate(g, act)).abs() * 2.0 ** -18 + (d * g).abs() * 1e-7), 1)
    return ref, BF16 * (ref.abs() + e) + e + 1e-38


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(32, 32), (32, 64), (64, 96), (96, 160), (128, 128), (160, 544),
                                 (512, 1056), (1024, 2048)])
def test_grad_quant(M, N, act):
    dh, gu = grads(M, N, M + N)
    d = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bq.gated_grad_quant(dh, gu, act=act, d=d, status=st)
    ref, tol = grad_ref(dh, gu, act)
    close(d, ref, tol, f"d {M}x{N}")
    assert int(st) == 0
    for x, y in zip(got, bq.grad_quant_dual(d)):
        assert torch.equal(x, y)  # codes and scales, padding included


@pytest.mark.parametrize("act", ACTS)
def test_grad_quant_stochastic(act):
    M, N = 96, 160
    dh, gu = grads(M, N, 5)
    d = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
    for seed in (0, 2 ** 63 + 11):
        got = bq.gated_grad_quant(dh, gu, act=act, stochastic=True, seed=seed, d=d)
        for x, y in zip(got, bq.grad_quant_dual(d, stochastic=True, seed=seed)):
            assert torch.equal(x, y)


def test_grad_quant_strides_and_status():
    M, N = 64, 96
    dh, gu = grads(M, 128, 7)
    wide = torch.cat((gu, gu), 1)
    a, b = dh[:, 16:16 + N], wide[:, 8:8 + 2 * N]
    got = bq.gated_grad_quant(a, b)
    ref = bq.gated_grad_quant(a.contiguous(), b.contiguous())
    for x, y in zip(got, ref):
        assert torch.equal(x, y)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bq.gated_grad_quant(a, b, status=st)
    assert int(st) == 0
    for value in (float("inf"), float("-inf"), float("nan")):
        for r, c in ((M - 1, N - 1), (0, 0), (33, 17)):
            bad = a.contiguous()
            bad[r, c] = value
            st.zero_()
            bq.gated_grad_quant(bad, b, status=st)
            assert int(st) == 1, (value, r, c)


def test_grad_quant_zero_and_signed_zero_groups():
    """Groups of zeros keep the floor scale and the zeros' signs, as grad_quant_dual does."""
    M, N = 64, 96
    dh, gu = grads(M, N, 3)
    dh[:32, :32] = 0.0
    dh[32:, 32:64] = -0.0
    d = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
    got = bq.gated_grad_quant(dh, gu, d=d)
    for x, y in zip(got, bq.grad_quant_dual(d)):
        assert torch.equal(x, y)


def test_grad_far_gates():
    """|g| up to 200: act' is 0 or 1 and nothing overflows to a NaN."""
    M, N = 32, 64
    dh, gu = grads(M, N, 9)
    gu[:, :N] = torch.linspace(-200, 200, M * N).view(M, N).to(torch.bfloat16)
    d = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
    for act in ACTS:
        bq.gated_grad_quant(dh, gu, act=act, d=d)
        assert bool(torch.isfinite(d).all())
        far = gu[:, :N].double().abs() > 60
        one = (gu[:, :N] > 0).double()
        r = dh.double() * gu[:, N:].double() * one
        close(d[:, :N][far], r[far], (BF16 * 1.01 * r.abs() + (dh.double() * gu[:, N:].double())
                                      .abs() * 2.0 ** -20)[far])


@pytest.mark.parametrize("act", ACTS)
def test_block_forward_and_backward(act):
    """A whole gated block: x -> MXFP8, gate and up with the quantized hidden row, down
    projection, and back through the hidden row's gradient to dX and dW, each step's
    output checked against the 64-bit form of its own inputs."""
    M, N, K = 96, 160, 128
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(torch.bfloat16).cuda()  # noqa: E731
    x, wg, wu, wd = rnd(M, K), rnd(N, K, std=K ** -0.5), rnd(N, K, std=K ** -0.5), rnd(
        K, N, std=N ** -0.5)
    qg, qu, qd = bq.act_quant(wg), bq.act_quant(wu), bq.act_quant(wd)
    xq = bq.act_quant(x)
    h, q, sf, gu = bq.gemm_gated(bq.W_MXFP8, *xq, *qg, *qu, M, N, K, act=act, quantize_out=True,
                                 keep_projections=True)
    y = bq.gemm_mxfp8_mxfp8(q, sf, *qd, M, K, N)
    bq.device_status()

    def value(q, sf, R, C, e5m2=False):
        s = bq.unpack_scales(sf, R, C).double()
        v = q.view(torch.float8_e5m2 if e5m2 else torch.float8_e4m3fn).double()
        return v * (2.0 ** (s - 127)).repeat_interleave(32, 1)

    a = value(*xq, M, K)
    gg, uu = a @ value(*qg, N, K).t(), a @ value(*qu, N, K).t()
    # E4M3's half step 2^-4 of each hidden value, and bf16's, over the sum of N terms
    href = gate(gg, act) * uu
    wdv = value(*qd, K, N)
    yref = href @ wdv.t()
    close(y, yref, (href.abs() @ wdv.abs().t()) * (2.0 ** -4 + 2.0 ** -7) + yref.abs() * BF16)

    dh = rnd(M, N, std=2.0 ** -8)
    w = torch.cat((wg, wu), 0)
    wt, xt = bq.quant_transposed(w), bq.quant_transposed(x)
    qr, sr, qt, st = bq.gated_grad_quant(dh, gu, act=act)
    dx = bq.gemm_e5m2_mxfp8(qr, sr, *wt, M, K, 2 * N)
    dw = bq.gemm_e5m2_mxfp8(qt, st, *xt, 2 * N, K, M)
    bq.device_status()
    d, _ = grad_ref(dh, gu, act)
    # the operands' half steps: E5M2 2^-3, E4M3 2^-4, bf16 2^-8 before each, and their products
    rel = (1 + 2.0 ** -3 + 2.0 ** -7) * (1 + 2.0 ** -4) - 1
    for got, p, r in ((dx, d, w.double()), (dw, d.t(), x.double())):
        ref, size = p @ r, p.abs() @ r.abs()
        # values below a group's smallest step: at most 2^-17 (E5M2) and 2^-10 (E4M3) of
        # the group's scale, itself at most 2 amax / 57344 and 2 amax / 448
        small = (p.abs().amax() * 2.0 ** -31 * r.abs().sum(0) + r.abs().amax() * 2.0 ** -17
                 * p.abs().sum(1, keepdim=True))
        close(got, ref, size * rel + small + ref.abs() * BF16)


def test_gradient_formula_against_differences():
    """The 64-bit gradient that the kernel is held to, against differences of the block's
    own formula and autograd."""
    g = torch.linspace(-8, 8, 401, dtype=torch.float64)
    u = torch.linspace(-3, 3, 401, dtype=torch.float64).flip(0)
    for act in ACTS:
        e = 1e-6
        dg = (gate(g + e, act) * u - gate(g - e, act) * u) / (2 * e)
        # e^2 / 6 times third derivatives below 6; both values, up to 24, carry about four
        # 64-bit roundings each: 2 * 4 * 24 * 2^-53 / (2 e) = 1.1e-8
        assert float((dg - u * gate_slope(g, act)).abs().max()) < 1.2e-8
        gr = g.clone().requires_grad_()
        (gate(gr, act) * u).sum().backward()
        assert float((gr.grad - u * gate_slope(g, act)).abs().max()) < 1e-12


def test_training_step_captured_and_replayed():
    """Forward and backward captured in a graph while an eager call's outputs live; replays
    on new inputs equal eager calls bit for bit."""
    M, N, K = 64, 128, 256
    a = Operand("mxfp8", M, K, 1)
    w, v = Operand("mxfp8", N, K, 2), Operand("mxfp8", N, K, 3)
    dh, _ = grads(M, N, 4)
    h = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    gu = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")

    def step():
        bq.gemm_gated(bq.W_MXFP8, a.q, a.sf, w.q, w.sf, v.q, v.sf, M, N, K, alpha=0.01, y=h, gu=gu)
        return bq.gated_grad_quant(dh, gu)

    eager = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (11, 12):
        b = Operand("mxfp8", M, K, seed)
        a.q.copy_(b.q)
        a.sf.copy_(b.sf)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out] + [h.clone(), gu.clone()]
        for x, y in zip(got, list(step()) + [h, gu]):
            assert torch.equal(x, y)
    bq.device_status()
    assert eager[0].shape == (M, 2 * N)


@pytest.mark.parametrize("kind", ["mxfp8", "int8"])
@pytest.mark.parametrize("M", [40, 600])
def test_two_streams_at_once(kind, M):
    N, K = 512, 1024
    a = Operand("int8" if kind == "int8" else "mxfp8", M, K, 1)
    w, v = Operand(kind, N, K, 2), Operand(kind, N, K, 3)

    def call():
        return bq.gemm_gated(KIND[kind], a.q, a.sf, w.q, w.sf, v.q, v.sf, M, N, K, alpha=0.01)

    one = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(20):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(call())
    torch.cuda.synchronize()
    bq.device_status()
    assert all(torch.equal(one, y) for y in outs)


def test_one_weight_as_both():
    """The same operand as gate and up projection."""
    M, N, K = 300, 200, 256
    a, w = Operand("mxfp8", M, K, 1), Operand("mxfp8", N, K, 2)
    b = bq.gemm_gated(bq.W_MXFP8, a.q, a.sf, w.q, w.sf, w.q, w.sf, M, N, K, alpha=0.01,
                      keep_projections=True)
    bq.device_status()
    assert torch.equal(b[1][:, :N], b[1][:, N:])


def test_empty_calls():
    a, w = Operand("mxfp8", 4, 32, 1), Operand("mxfp8", 8, 32, 2)
    y = bq.gemm_gated(bq.W_MXFP8, a.q[:0], a.sf, w.q, w.sf, w.q, w.sf, 0, 8, 32)
    assert y.shape == (0, 8)
    e = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    out = bq.gated_grad_quant(e, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert out[0].shape == (0, 64)


# the nearest form's sizes, and: more columns of F than a block's eight warps hold, a half tile
# of 32 behind them, rows and groups of padding in every number
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(32, 32), (32, 64), (64, 96), (96, 160), (128, 128), (160, 544),
                                 (512, 1056), (1024, 2048), (224, 512), (32, 4128)])
def test_grad_quant_stochastic_sizes(M, N, act):
    dh, gu = grads(M, N, M + N)
    d = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bq.gated_grad_quant(dh, gu, act=act, stochastic=True, seed=M * N, d=d, status=st)
    ref, tol = grad_ref(dh, gu, act)
    close(d, ref, tol, f"d {M}x{N}")
    assert int(st) == 0
    for x, y in zip(got, bq.grad_quant_dual(d, stochastic=True, seed=M * N)):
        assert torch.equal(x, y)  # codes and scales, padding included


def test_grad_quant_stochastic_strides_outputs_and_status():
    M, N = 96, 288
    dh, gu = grads(M, N + 64, 7)
    a, b = dh[:, 16:16 + N], gu[:, 8:8 + 2 * N]
    ref = bq.gated_grad_quant(a.contiguous(), b.contiguous(), stochastic=True, seed=5)
    # buffers that hold other values, with more behind them
    out = [torch.full((t.numel() + 64,), 77, dtype=torch.uint8, device="cuda") for t in ref]
    got = bq.gated_grad_quant(a, b, stochastic=True, seed=5, out=out)
    for x, y in zip(got, ref):
        assert torch.equal(x[:y.numel()], y.reshape(-1)) and bool((x[y.numel():] == 77).all())
    other = bq.gated_grad_quant(a, b, stochastic=True, seed=6)
    assert not torch.equal(other[0], ref[0]) and torch.equal(other[1], ref[1])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for value in (float("inf"), float("nan")):
        for r, c in ((M - 1, N - 1), (0, 0), (33, 257)):
            bad = a.contiguous()
            bad[r, c] = value
            st.zero_()
            bq.gated_grad_quant(bad, b, stochastic=True, status=st)
            assert int(st) == 1, (value, r, c)


@pytest.mark.parametrize("kind", ["mxfp8", "int8"])
def test_offsets_beyond_32_bits(kind):
    """More than 2^31 hidden values and 2^32 projections: the last rows equal those of a
    short call, forward and backward."""
    M, N, K = 65568, 32800, 32
    a = Operand("int8" if kind == "int8" else "mxfp8", M, K, 1)
    w, v = Operand(kind, N, K, 2), Operand(kind, N, K, 3)
    last = torch.arange(M - 32, M)  # a scale atom's last 32 rows
    aq = a.q[M - 32:].contiguous()
    if kind == "int8":
        asf = a.sf[M - 32:].clone()
    else:
        s = bq.unpack_scales(a.sf, M, K)[last.cuda()]
        asf = torch.full((bq.sf_bytes(32, K),), 127, dtype=torch.uint8, device="cuda")
        asf.view(32, 4, 4)[:, 0, 0] = s[:, 0]
    for cfg in (bq.config(swap_ab=0), bq.config(swap_ab=1, block_n=128)):
        h, q, sf, gu = bq.gemm_gated(KIND[kind], a.q, a.sf, w.q, w.sf, v.q, v.sf, M, N, K,
                                     alpha=0.01, keep_projections=True, quantize_out=True,
                                     config=cfg)
        bq.device_status()
        e = bq.gemm_gated(KIND[kind], aq, asf, w.q, w.sf, v.q, v.sf, 32, N, K, alpha=0.01,
                          keep_projections=True, quantize_out=True)
        assert torch.equal(gu[-32:], e[3]) and torch.equal(h[-32:], e[0])
        assert torch.equal(q[-32:], e[1])
        got = bq.unpack_scales(sf, M, N)[-32:]
        assert torch.equal(got, bq.unpack_scales(e[2], 32, N))
        del h, q, sf
    dh = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    dh[-32:], _ = grads(32, N, 5)
    for stochastic in (False, True):
        d_row, d_sf, d_t, d_tsf = bq.gated_grad_quant(dh, gu, stochastic=stochastic)
        # nearest: the last 32 rows alone give the same codes, and so do their columns
        if not stochastic:
            e = bq.gated_grad_quant(dh[-32:], gu[-32:])
            assert torch.equal(d_row[-32:], e[0]) and torch.equal(d_t[:, -32:], e[2])
            assert torch.equal(bq.unpack_scales(d_sf, M, 2 * N)[-32:],
                               bq.unpack_scales(e[1], 32, 2 * N))
            assert torch.equal(bq.unpack_scales(d_tsf, 2 * N, M)[:, -1:],
                               bq.unpack_scales(e[3], 2 * N, 32))
        else:
            d = torch.empty_like(gu)
            got = bq.gated_grad_quant(dh, gu, stochastic=True, out=(d_row, d_sf, d_t, d_tsf), d=d)
            for x, y in zip(bq.grad_quant_dual(d, stochastic=True), got):
                assert torch.equal(x, y)
        del d_row, d_t
    bq.device_status()


@pytest.mark.parametrize("kind", list(KIND))
def test_block_repeats_bit_for_bit(kind):
    """Gate, up, quantized hidden row and down projection over the same inputs, with other
    inputs between and no waits: the same bits every time."""
    M, N, K = 2900, 1696, 640
    a = [Operand("int8" if kind == "int8" else "mxfp8", M, K, s) for s in (1, 2)]
    w, v = Operand(kind, N, K, 3), Operand(kind, N, K, 4)
    d = Operand("mxfp8", K, N, 5)

    def block(a):
        _, q, sf, gu = bq.gemm_gated(KIND[kind], a.q, a.sf, w.q, w.sf, v.q, v.sf, M, N, K,
                                     alpha=0.01, quantize_out=True, write_y=False,
                                     keep_projections=True)
        return bq.gemm_mxfp8_mxfp8(q, sf, d.q, d.sf, M, K, N), q, sf, gu

    first = block(a[0])
    torch.cuda.synchronize()
    for _ in range(20):
        block(a[1])
        assert all(torch.equal(x, y) for x, y in zip(first, block(a[0])))
    bq.device_status()


@pytest.mark.parametrize("alpha", [0.5, -2.0])
def test_gradients_take_alpha_once_more(alpha):
    """g and u hold the forward call's alpha; the products of d with the input and with the
    weights take it as well."""
    M, N, K = 64, 96, 128
    a, w, v = Operand("mxfp8", M, K, 1), Operand("mxfp8", N, K, 2), Operand("mxfp8", N, K, 3)
    small = float(np.float32(alpha / float(product(a, w).std())))
    _, gu = bq.gemm_gated(bq.W_MXFP8, a.q, a.sf, w.q, w.sf, v.q, v.sf, M, N, K, alpha=small,
                          keep_projections=True)
    g = torch.Generator().manual_seed(4)
    dh = (torch.randn((M, N), generator=g) * 2.0 ** -6).to(torch.bfloat16).cuda()
    d = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
    q, sf, _, _ = bq.gated_grad_quant(dh, gu, d=d)
    wt = torch.cat((w.value, v.value), 0)
    wq = bq.quant_transposed(wt.to(torch.bfloat16))
    dx = bq.gemm_e5m2_mxfp8(q, sf, *wq, M, K, 2 * N, alpha=small)
    bq.device_status()
    # autograd in 64 bits through the block's formula
    x, wd, vd = a.value.clone().requires_grad_(), w.value, v.value
    h = torch.nn.functional.silu(small * x @ wd.t()) * (small * x @ vd.t())
    h.backward(dh.double())
    # half steps: bf16's of g, u (each reaches d with a factor up to 1 + |g| or so, 10 here), of d
    # and of the weights, E5M2's of d 2^-3, E4M3's of the weights 2^-4, over the sum's terms; codes
    # below a group's smallest step: as in test_block_forward_and_backward
    size = abs(small) * (d.double().abs() @ wt.abs())
    rel = (1 + 2.0 ** -3 + 2.0 ** -7) * (1 + 2.0 ** -4 + 2.0 ** -8) - 1
    forward = abs(small) * 10 * BF16 * (dh.double().abs() * (gu[:, :N].double().abs() + 1)
                                        * (gu[:, N:].double().abs() + 1)) @ (w.value.abs()
                                                                            + v.value.abs())
    floor = abs(small) * (d.double().abs().amax() * 2.0 ** -31 * wt.abs().sum(0)
                          + wt.abs().amax() * 2.0 ** -17 * d.double().abs().sum(1, keepdim=True))
    close(dx, x.grad, size * rel + forward + floor + x.grad.abs() * BF16)
    # the tolerance tells alpha from alpha squared: without the factor most values lie outside
    off = (dx.double() / small - x.grad).abs() > (size * rel + forward + floor)
    assert float(off.double().mean()) > 0.5
