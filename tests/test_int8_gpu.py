"""The int8 row quantizer (bit-exact) and the int8 product against 64-bit forms."""
import pytest
import torch

import block_scaled_precision_quant_b200 as bq
import ffn_ref
from ffn_ref import Operand, close, gelu, int8_rows, int8_tol

pytestmark = pytest.mark.gpu


def rows(M, K, seed, ld=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, ld or K), generator=g)
    x = x * 2.0 ** torch.randint(-12, 13, (M, 1), generator=g).float()
    return x.to(torch.bfloat16).cuda()


def check_quant(x, q, s):
    rq, rs = int8_rows(x)
    assert torch.equal(q, rq)
    # the scale is one correctly rounded quotient
    assert torch.equal(s, rs.float())


# one row, rows shorter and longer than a block's registers, odd tails of every kind
@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (3, 48), (7, 240), (41, 1536), (130, 2064),
                                 (33, 8192), (5, 8208), (2, 16400), (3, 65552), (1, 131056),
                                 (2500, 272),
                                 # a warp to a row: short rows and longer ones
                                 (595, 16), (1201, 2048), (700, 992), (4740, 2064),
                                 (4737, 4096), (1480, 2064),
                                 # blocks of 128: middling rows, many of them
                                 (444, 16), (590, 1040), (600, 4096), (1481, 4112), (445, 6144),
                                 # and of 256 again
                                 (443, 6144), (444, 6160), (1500, 8192)])
def test_quant_rows(M, K):
    x = rows(M, K, M + K)
    q, s = bq.act_quant_int8(x)
    check_quant(x, q, s)


def test_quant_ties_go_to_even():
    """Every pair of 8-bit significands and the binades a code can span: ties among
    them are decided exactly."""
    big = torch.arange(128, 256).float()
    x = torch.zeros((128, 9 * 256))
    for t in range(9):
        x[:, 256 * t:256 * t + 256] = torch.arange(256).float() * 2.0 ** -t
    x = torch.where(x.abs() > big[:, None], torch.zeros(()), x)
    x[:, 0] = big
    x[::2] *= -1
    x = x.to(torch.bfloat16).cuda()
    q, s = bq.act_quant_int8(x)
    check_quant(x, q, s)
    n = x.double() * 127 / x.double().abs().amax(1, keepdim=True)
    assert int(((n - n.floor()) == 0.5).sum()) == 444  # of these inputs, counted in 64 bits


def test_quant_small_zero_and_large_rows():
    x = torch.zeros((6, 64))
    x[1] = 2.0 ** -64
    x[2, 3] = 2.0 ** -126
    x[3] = torch.linspace(-3, 3, 64) * 1e38  # (the span itself would overflow to an Inf)
    x[4, 0], x[4, 1] = 1e-20, -3e-20
    x[5] = 2.0 ** -133
    x = x.to(torch.bfloat16).cuda()
    q, s = bq.act_quant_int8(x)
    check_quant(x, q, s)
    assert int(q[0].abs().max()) == 0 and int(q[1].min()) == 127


@pytest.mark.parametrize("M,N,K", [(41, 4608, 1536), (300, 8192, 4096)])
def test_weight_quantized_right_before_the_product(M, N, K):
    """The weight's codes come last before the product, into buffers that held others."""
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    ws = [torch.randn((N, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    want = []
    for w in ws:
        q, s = bq.act_quant_int8(x)
        b, sb = bq.act_quant_int8(w)
        torch.cuda.synchronize()
        want.append(bq.gemm_int8_int8(q, s, b, sb, M, N, K))
    torch.cuda.synchronize()
    b, sb = torch.zeros_like(b), torch.zeros_like(sb)
    got = []
    for w in ws * 4:
        q, s = bq.act_quant_int8(x)
        bq.act_quant_int8(w, b, sb)
        got.append(bq.gemm_int8_int8(q, s, b, sb, M, N, K))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 3])


@pytest.mark.parametrize("M", [45, 605])
def test_quant_row_stride_outputs_and_status(M):
    wide = rows(M, 200, 3)
    x = wide[:, :160]
    q = torch.full((M + 1, 160), 77, dtype=torch.int8, device="cuda")
    s = torch.full((M + 1,), 5.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bq.act_quant_int8(x, q=q[:M], scale=s[:M], status=st)
    check_quant(x, q[:M], s[:M])
    assert bool((q[M] == 77).all()) and float(s[M]) == 5.0 and int(st) == 0
    for bad in (float("inf"), float("-inf"), float("nan")):
        y = x.clone()
        y[M - 1, 159] = bad
        st.zero_()
        q2, s2 = bq.act_quant_int8(y, status=st)
        assert int(st) == 1
        check_quant(y[:M - 1], q2[:M - 1], s2[:M - 1])  # the other rows stand


def product(M, N, K, seed, bias=False, res=False, act=0, alpha=1.0, config=None, ldres=None):
    a, b = Operand("int8", M, K, seed), Operand("int8", N, K, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    bv = torch.randn((N,), generator=g).to(torch.bfloat16).cuda() if bias else None
    rv = (torch.randn((M, ldres or N), generator=g) * 3).to(torch.bfloat16).cuda() if res else None
    if res:
        rv = rv[:, :N]
    y = bq.gemm(bq.W_INT8, a.q, a.sf, b.q, b.sf, M, N, K, bias=bv, residual=rv, act=act,
                alpha=alpha, config=config)
    bq.device_status()
    p = alpha * ffn_ref.product(a, b)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    bd, rd = (bv.double() if bias else zero), (rv.double() if res else zero)
    pre = p + bd
    ref = (gelu(pre) if act else pre) + rd
    close(y, ref, int8_tol(p, bd, pre, rd, ref, act), f"{M}x{N}x{K}")
    return y


# from one row to many, sizes that end inside tiles of every kind
@pytest.mark.parametrize("M,N,K", [
    (1, 8, 16), (1, 4608, 1536), (2, 136, 144), (8, 1536, 6144), (31, 128, 128), (32, 264, 2064),
    (33, 512, 496), (41, 4608, 1536), (64, 1000, 1040), (65, 128, 272), (127, 2048, 512),
    (128, 520, 4096), (129, 264, 80), (200, 1032, 1008), (257, 640, 912), (384, 256, 2048),
    (500, 776, 656), (1003, 520, 400)])
def test_product(M, N, K):
    product(M, N, K, M * 7 + N + K)


@pytest.mark.parametrize("M", [1, 41, 100, 300])
@pytest.mark.parametrize("bias,res,act,alpha", [(True, False, 0, 1.0), (False, True, 0, 1.0),
                                                (True, True, 1, 1.0), (False, False, 1, 0.25),
                                                (True, True, 0, -2.0)])
def test_epilogues(M, bias, res, act, alpha):
    product(M, 456, 336, M, bias, res, act, alpha, ldres=472)


@pytest.mark.parametrize("bn", [32, 64, 128])
@pytest.mark.parametrize("split", [1, 2, 3, 5, 8])
def test_swap_schedules(bn, split):
    product(70, 392, 1168, bn + split, bias=True, config=bq.config(block_n=bn, split_k=split,
                                                                   swap_ab=1))


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (100, 136, 400), (128, 256, 128), (129, 264, 1168),
                                   (257, 520, 2064), (513, 1000, 640), (1300, 2056, 272)])
@pytest.mark.parametrize("bias,res,act", [(False, False, 0), (True, True, 1)])
def test_pair_tiles(M, N, K, bias, res, act):
    product(M, N, K, M + K, bias, res, act, 0.5, bq.config(swap_ab=0), ldres=N + 8)


# more tiles than pairs of SMs: every pair works on several, with K blocks that end
# anywhere in the operand ring
@pytest.mark.parametrize("K", [64, 640, 1424])
@pytest.mark.parametrize("bias,res,act", [(False, False, 0), (True, True, 1)])
def test_pair_tiles_in_several_waves(K, bias, res, act):
    product(2900, 3336, K, K, bias, res, act, 0.5, bq.config(swap_ab=0))


# the last column of tiles holds 1 to 8 of its 8 chunks of 32 outputs, so that the epilogue's
# groups have two, one or none of their own; short sums, many tiles a pair: the epilogue is
# what the tiles wait for
@pytest.mark.parametrize("tail", [8, 40, 96, 104, 136, 160, 224, 248, 256])
@pytest.mark.parametrize("full", [0, 2])
def test_pair_tiles_residual_in_narrow_last_columns(tail, full):
    M, N, K = 256 * 150 // (full + 1) - 100, 256 * full + tail, 16
    a, b = Operand("int8", M, K, tail), Operand("int8", N, K, tail + 1)
    res = (torch.randn((M, N), device="cuda") * 3).to(torch.bfloat16)
    want = bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, M, N, K, residual=res,
                             config=bq.config(swap_ab=1, block_n=128))
    got = []
    for _ in range(20):
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        got.append(bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, M, N, K, residual=res, y=y,
                                     config=bq.config(swap_ab=0)))
    bq.device_status()  # no wait gave up
    p = ffn_ref.product(a, b)
    r = res.double()
    close(want, p + r, int8_tol(p, torch.zeros_like(p), p, r, p + r, 0))
    assert all(torch.equal(want, y) for y in got)


def test_pair_tiles_equal_swap_tiles():
    a, b = Operand("int8", 300, 1552, 5), Operand("int8", 776, 1552, 6)
    ys = [bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, 300, 776, 1552, config=c)
          for c in (bq.config(swap_ab=0), bq.config(swap_ab=1), bq.config(split_k=4))]
    bq.device_status()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_sums_are_exact_at_their_largest():
    """The longest K with every code at its end of the range: |sum| = K 2^14 just
    below 2^31; with unit scales the output is that sum rounded to bf16."""
    K = 131056
    a = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((8, K), -128, dtype=torch.int8, device="cuda")
    b[1] = 127
    one = torch.ones(8, device="cuda")
    for cfg in (None, bq.config(split_k=1), bq.config(split_k=8), bq.config(swap_ab=0)):
        y = bq.gemm_int8_int8(a, one[:2].contiguous(), b, one, 2, 8, K, config=cfg)
        bq.device_status()
        ref = (a.double() @ b.double().t()).to(torch.bfloat16)
        assert torch.equal(y, ref)


def test_split_does_not_change_a_bit():
    a, b = Operand("int8", 41, 4096, 5), Operand("int8", 512, 4096, 6)
    ys = [bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, 41, 512, 4096,
                            config=bq.config(split_k=s, block_n=n))
          for s in (1, 2, 7, 8) for n in (32, 64, 128)]
    bq.device_status()
    assert all(torch.equal(ys[0], y) for y in ys[1:])


@pytest.mark.parametrize("M", [20, 64, 300])
def test_batch_with_broadcast_operands(M):
    count, N, K = 3, 200, 272
    a = [Operand("int8", M, K, 10 + i) for i in range(count)]
    b = [Operand("int8", N, K, 20 + i) for i in range(count)]
    res = torch.randn((count, M, N), device="cuda").to(torch.bfloat16)
    aq = torch.stack([t.q for t in a])
    asf = torch.stack([t.sf for t in a])
    bq_, bsf = torch.stack([t.q for t in b]), torch.stack([t.sf for t in b])
    for shared in ("", "a", "b"):
        sa, sb = (0 if shared == "a" else 1), (0 if shared == "b" else 1)
        y = bq.gemm_int8_int8(aq, asf, bq_, bsf, M, N, K, residual=res, batch=dict(
            count=count, stride_a=sa * M * K, stride_a_sf=sa * 4 * M, stride_b=sb * N * K,
            stride_b_sf=sb * 4 * N, stride_y=2 * M * N, stride_res=2 * M * N))
        bq.device_status()
        for i in range(count):
            p = ffn_ref.product(a[i * sa], b[i * sb])
            r = res[i].double()
            z = torch.zeros_like(p)
            close(y[i], p + r, int8_tol(p, z, p, r, p + r, 0), f"{shared} {i}")


@pytest.mark.parametrize("M", [20, 300])
def test_batch_with_gaps_between_the_outputs(M):
    count, N, K = 3, 136, 80
    a = [Operand("int8", M, K, 30 + i) for i in range(count)]
    b = Operand("int8", N, K, 40)
    aq, asf = torch.stack([t.q for t in a]), torch.stack([t.sf for t in a])
    y = torch.full((count, M + 2, N), 9.0, dtype=torch.bfloat16, device="cuda")
    out = bq.gemm_int8_int8(aq, asf, b.q, b.sf, M, N, K, y=y, batch=dict(
        count=count, stride_a=M * K, stride_a_sf=4 * M, stride_y=2 * (M + 2) * N))
    bq.device_status()
    assert out is y and bool((y[:, M:] == 9).all())
    for i in range(count):
        assert torch.equal(y[i, :M], bq.gemm_int8_int8(a[i].q, a[i].sf, b.q, b.sf, M, N, K))


def test_rows_behind_the_last_stay_as_they_were():
    M, N, K = 37, 136, 160
    a, b = Operand("int8", M, K, 1), Operand("int8", N, K, 2)
    y = torch.full((M + 3, N), 9.0, dtype=torch.bfloat16, device="cuda")
    bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, M, N, K, y=y[:M])
    bq.device_status()
    assert bool((y[M:] == 9).all())


def test_linear_layer_chain_captured_and_replayed():
    """Quantizer and product back to back, captured once and replayed on new inputs,
    the weights quantized by the same quantizer."""
    M, N, K = 41, 1536, 512
    w = rows(N, K, 9)
    wq, ws = bq.act_quant_int8(w)
    x = rows(M, K, 1)
    q = torch.empty((M, K), dtype=torch.int8, device="cuda")
    s = torch.empty((M,), device="cuda")
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")

    def step():
        bq.act_quant_int8(x, q=q, scale=s)
        bq.gemm_int8_int8(q, s, wq, ws, M, N, K, y=y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 3, 4):
        x.copy_(rows(M, K, seed))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        rq, rs = int8_rows(x)
        p = (rq.double() @ wq.double().t()) * rs.float().double()[:, None] * ws.double()
        z = torch.zeros_like(p)
        close(got, p, int8_tol(p, z, p, z, p, 0), f"replay {seed}")
    bq.device_status()


@pytest.mark.parametrize("M", [64, 700])
def test_two_streams_at_once(M):
    ops = [(Operand("int8", M, 2048, s), Operand("int8", 1024, 2048, s + 50)) for s in range(2)]
    one = [bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, M, 1024, 2048) for a, b in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    outs = [[], []]
    for _ in range(20):
        for i, (st, (a, b)) in enumerate(zip(streams, ops)):
            with torch.cuda.stream(st):
                outs[i].append(bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, M, 1024, 2048))
    torch.cuda.synchronize()
    bq.device_status()
    for i in range(2):
        assert all(torch.equal(one[i], y) for y in outs[i])


def test_residual_in_place():
    """y may be the residual itself: a chunk's residual is read before it is written."""
    for M in (41, 300):
        a, b = Operand("int8", M, 528, 1), Operand("int8", 648, 528, 2)
        r = (torch.randn((M, 648), device="cuda") * 3).to(torch.bfloat16)
        ref = bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, M, 648, 528, residual=r)
        got = r.clone()
        bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, M, 648, 528, residual=got, y=got)
        bq.device_status()
        assert torch.equal(got, ref)


def test_binding_refuses_what_the_operands_do_not_hold():
    x = rows(8, 64, 1)
    q, s = bq.act_quant_int8(x)
    b, sb = bq.act_quant_int8(rows(16, 64, 2))
    y = torch.empty((8, 16), dtype=torch.bfloat16, device="cuda")
    assert bq.gemm_int8_int8(q, s, b, sb, 8, 16, 64, y=y) is y
    for kw in (dict(y=y[:4]), dict(y=y.float()), dict(y=y.t()), dict(bias=y[0, :8]),
               dict(bias=torch.zeros(16, device="cuda")), dict(residual=y[:4]),
               dict(residual=y.t()), dict(residual=y.cpu())):
        with pytest.raises(ValueError):
            bq.gemm_int8_int8(q, s, b, sb, 8, 16, 64, **kw)
    for M, N, K in ((9, 16, 64), (8, 24, 64), (8, 16, 80)):  # more than the operands have
        with pytest.raises(ValueError):
            bq.gemm_int8_int8(q, s, b, sb, M, N, K)
    for args in ((q.float(), s, b, sb), (q, s.double(), b, sb), (q.t(), s, b, sb),
                 (q, s.cpu(), b, sb)):
        with pytest.raises(ValueError):
            bq.gemm_int8_int8(*args, 8, 16, 64)
    with pytest.raises(ValueError):
        bq.act_quant_int8(x.float())
    with pytest.raises(ValueError):
        bq.act_quant_int8(x.t())
    for M, N, K in ((-1, 16, 64), (8, -8, 64), (8, 16, 0), (8, 12, 64), (8, 16, 24)):
        with pytest.raises(bq.BqError) as e:
            bq.gemm_int8_int8(q, s, b, sb, M, N, K)
        assert e.value.status == bq.BQ_ERR_SHAPE
    torch.cuda.synchronize()


def test_two_host_threads_at_once():
    from concurrent.futures import ThreadPoolExecutor
    x = [rows(41, 512, i) for i in range(2)]
    b, sb = bq.act_quant_int8(rows(768, 512, 9))
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(200):
                q, s = bq.act_quant_int8(x[i])
                y = bq.gemm_int8_int8(q, s, b, sb, 41, 768, 512)
            torch.cuda.current_stream().synchronize()
        return y
    with ThreadPoolExecutor(2) as pool:
        got = list(pool.map(work, range(2)))
    for i in range(2):
        q, s = bq.act_quant_int8(x[i])
        assert torch.equal(got[i], bq.gemm_int8_int8(q, s, b, sb, 41, 768, 512))


def test_empty_calls():
    a, b = Operand("int8", 4, 32, 1), Operand("int8", 8, 32, 2)
    assert bq.gemm_int8_int8(a.q[:0], a.sf[:0], b.q, b.sf, 0, 8, 32).shape == (0, 8)
    q, s = bq.act_quant_int8(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0,)


def test_arch_override_refuses():
    a, b = Operand("int8", 4, 32, 1), Operand("int8", 8, 32, 2)
    bq.lib().bq_debug_override_compute_capability(9, 0)
    try:
        with pytest.raises(bq.BqError) as e:
            bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, 4, 8, 32)
        assert e.value.status == bq.BQ_ERR_ARCH
    finally:
        bq.lib().bq_debug_override_compute_capability(-1, -1)


@pytest.mark.parametrize("M,N,K,config", [
    (1, 4608, 1536, {}), (41, 1536, 6144, {}), (41, 1000, 1040, dict(split_k=1, block_n=64)),
    (130, 2048, 1024, dict(swap_ab=1, block_n=128)), (70, 4096, 512, dict(swap_ab=0)),
    (1000, 4104, 2064, dict(swap_ab=0))])
@pytest.mark.parametrize("gated", [False, True])
def test_weights_quantized_right_before_in_every_schedule(M, N, K, config, gated):
    """Products read their weights after the kernel before has ended: each call's weights
    are written by the kernel just before it, into the buffers that the last call's used, in
    eager order and replayed."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    ws = [torch.randn((N, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    xq, xs = bq.act_quant_int8(x)
    cfg = bq.config(**config)
    b, sb = torch.empty((N, K), dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    ug, us = bq.act_quant_int8(ws[0])  # the other weight of a gated block

    def call(w, wait):
        bq.act_quant_int8(w, b, sb)
        if wait:
            torch.cuda.synchronize()
        if gated:  # written last: the up projection's weight
            return bq.gemm_gated(bq.W_INT8, xq, xs, ug, us, b, sb, M, N, K, config=cfg)
        return bq.gemm_int8_int8(xq, xs, b, sb, M, N, K, config=cfg)

    want = [call(w, True) for w in ws]
    assert not torch.equal(want[0], want[1])
    for _ in range(10):
        got = [call(w, False) for w in ws]
        assert all(torch.equal(a, e) for a, e in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(w, False) for w in ws]
    for _ in range(10):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, e) for a, e in zip(got, want))
    bq.device_status()


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in the rows, the outputs and the residual: the last rows equal
    those of a short call."""
    M, K = 70001, 32768
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-3:] = rows(3, K, 1)
    q, s = bq.act_quant_int8(x)
    check_quant(x[-3:], q[-3:], s[-3:])
    assert int(q[-4].abs().max()) == 0
    del x, q, s
    N, K = 32768, 16
    a, b = Operand("int8", M, K, 2), Operand("int8", N, K, 3)
    res = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    res[-5:] = rows(5, N, 4)
    for cfg in (bq.config(swap_ab=0), bq.config(swap_ab=1, block_n=128)):
        for r in (None, res):
            y = bq.gemm_int8_int8(a.q, a.sf, b.q, b.sf, M, N, K, residual=r, config=cfg)
            for first in (0, 65535, M - 5):  # 65535 N: around 2^31
                t = slice(first, first + 5)
                e = bq.gemm_int8_int8(a.q[t].contiguous(), a.sf[t].clone(), b.q, b.sf, 5, N, K,
                                      residual=None if r is None else r[t])
                assert torch.equal(y[t], e)
            del y
    bq.device_status()
