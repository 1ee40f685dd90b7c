"""Host-side checks of the int8 and gated entry points: what they refuse (nothing is
launched; no device is needed) and the schedules they pick."""
import ctypes

import pytest
import torch

import block_scaled_precision_quant_b200 as bq
from block_scaled_precision_quant_b200 import build


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return bq.lib()


P = 1 << 20  # stands for an aligned address; the checks come before any use of it


def test_quant_refusals(L):
    def call(x=P, M=4, K=32, ldx=32, q=P, s=P):
        return L.bq_act_quant_int8(x, M, K, ldx, q, s, None, None)
    assert call(x=None) == call(q=None) == call(s=None) == bq.BQ_ERR_NULL
    assert call(K=24) == call(K=0) == call(M=-1) == call(ldx=24) == bq.BQ_ERR_SHAPE
    assert call(x=P + 2) == call(ldx=36) == call(q=P + 8) == call(s=P + 2) == bq.BQ_ERR_ALIGN


def product(L, a=P, sa=P, b=P, sb=P, M=4, N=8, K=32, y=P, epi=None, batch=None, cfg=None):
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    return L.bq_gemm_int8_int8_epilogue(a, sa, b, sb, M, N, K, y, ref(epi), ref(batch), ref(cfg),
                                        None)


def test_product_refusals(L):
    for k in ("a", "sa", "b", "sb", "y"):
        assert product(L, **{k: None}) == bq.BQ_ERR_NULL
        assert product(L, **{k: P + 2}) == bq.BQ_ERR_ALIGN
    assert product(L, sb=P + 4) == bq.BQ_ERR_ALIGN
    for kw in (dict(K=24), dict(K=0), dict(N=12), dict(M=-1), dict(K=131072), dict(N=1 << 32),
               dict(M=0x7FFFFF00)):
        assert product(L, **kw) == bq.BQ_ERR_SHAPE
    E = bq.Epilogue
    assert product(L, epi=E(None, None, 0, 1.0, 2, None, None)) == bq.BQ_ERR_INVALID
    assert product(L, epi=E(None, None, 0, 1.0, 0, P, P)) == bq.BQ_ERR_INVALID
    assert product(L, epi=E(P + 2, None, 0, 1.0, 0, None, None)) == bq.BQ_ERR_ALIGN
    assert product(L, epi=E(None, P, 4, 1.0, 0, None, None)) == bq.BQ_ERR_ALIGN
    B = bq.Batch
    assert product(L, batch=B(2, 128, 16, 0, 0, 0, 0)) == bq.BQ_ERR_SHAPE  # outputs on top
    assert product(L, batch=B(2, 128, 2, 0, 0, 64, 0)) == bq.BQ_ERR_ALIGN
    assert product(L, batch=B(-1, 0, 0, 0, 0, 0, 0)) == bq.BQ_ERR_SHAPE
    for c in (dict(block_n=48), dict(split_k=9), dict(split_mode=bq.BQ_SPLIT_WORKSPACE),
              dict(k_chunks=2), dict(split_k=-1), dict(swap_ab=2), dict(cta_pair=3),
              dict(swap_ab=0, split_k=2), dict(swap_ab=1, block_n=256),
              dict(cta_pair=2, block_n=64), dict(cta_pair=1, swap_ab=0)):
        assert product(L, cfg=bq.config(**c)) == bq.BQ_ERR_INVALID


def gated(L, kind=2, a=P, sa=P, g=P, sg=P, u=P, su=P, M=4, N=32, K=128, h=P, epi=None, cfg=None):
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    return L.bq_gemm_gated(kind, a, sa, g, sg, u, su, M, N, K, h, ref(epi), ref(cfg), None)


def test_gated_refusals(L):
    for kind in (3, 4, 5, 7, -1):
        assert gated(L, kind=kind) == bq.BQ_ERR_INVALID
    for kind in (0, 1, 2, 6):
        for k in ("a", "sa", "g", "sg", "u", "su", "h"):
            assert gated(L, kind=kind, **{k: None}) == bq.BQ_ERR_NULL
            assert gated(L, kind=kind, **{k: P + 2}) == bq.BQ_ERR_ALIGN
    assert gated(L, kind=0, g=P + 16) == bq.BQ_ERR_ALIGN  # packed codes: 32 bytes
    assert gated(L, kind=0, K=96) == gated(L, K=48) == gated(L, N=36) == bq.BQ_ERR_SHAPE
    assert gated(L, kind=6, K=131072) == bq.BQ_ERR_SHAPE
    E = bq.GatedEpilogue
    assert gated(L, epi=E(1.0, 2, None, None, None)) == bq.BQ_ERR_INVALID
    assert gated(L, epi=E(1.0, 0, None, P, None)) == bq.BQ_ERR_NULL
    assert gated(L, N=40, epi=E(1.0, 0, None, P, P)) == bq.BQ_ERR_SHAPE
    assert gated(L, epi=E(1.0, 0, P + 2, None, None)) == bq.BQ_ERR_ALIGN
    assert gated(L, epi=E(1.0, 0, None, P + 8, P)) == bq.BQ_ERR_ALIGN
    assert gated(L, cfg=bq.config(block_n=16)) == bq.BQ_ERR_INVALID


def test_grad_refusals(L):
    def call(dh=P, ld=64, gu=P, ldg=128, M=32, N=64, act=0, rnd=0, q=P, sf=P, qt=P, st=P, d=None):
        return L.bq_gated_grad_quant(dh, ld, gu, ldg, M, N, act, rnd, 0, q, sf, qt, st, d, None,
                                     None)
    for k in ("dh", "gu", "q", "sf", "qt", "st"):
        assert call(**{k: None}) == bq.BQ_ERR_NULL
    for k in ("dh", "gu", "q", "qt", "d"):
        assert call(**{k: P + 2}) == bq.BQ_ERR_ALIGN
    assert call(act=2) == call(rnd=2) == bq.BQ_ERR_INVALID
    assert call(M=33) == call(N=48) == call(N=0) == call(M=-32) == bq.BQ_ERR_SHAPE
    assert call(ld=32) == call(ldg=120) == bq.BQ_ERR_SHAPE
    assert call(ld=68) == call(ldg=132) == bq.BQ_ERR_ALIGN


def test_binding_refusals():
    i8 = torch.zeros((4, 32), dtype=torch.int8)
    f = torch.zeros(32)
    with pytest.raises(ValueError):
        bq.act_quant_int8(torch.zeros((4, 32), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        bq.gemm_int8_int8(i8, f, i8, f, 4, 4, 32)
    with pytest.raises(ValueError):
        bq.gemm(bq.W_INT8, i8, f, i8, f, 4, 4, 32, quantize_out=True)
    with pytest.raises(ValueError):
        bq.gemm_gated(bq.W_INT8, i8, f, i8, f, i8, f, 4, 4, 32)
    with pytest.raises(ValueError):
        bq.gated_grad_quant(torch.zeros((32, 32), dtype=torch.bfloat16),
                            torch.zeros((32, 64), dtype=torch.bfloat16))


def test_binding_argument_types():
    i8, f = torch.zeros((4, 32), dtype=torch.int8), torch.zeros(32)
    for bad in (None, 3, [1.0]):
        with pytest.raises(TypeError):
            bq.act_quant_int8(bad)
        with pytest.raises(TypeError):
            bq.gemm_int8_int8(i8, bad, i8, f, 4, 4, 32)
        with pytest.raises(TypeError):
            bq.gemm_gated(bq.W_INT8, i8, f, bad, f, i8, f, 4, 4, 32)
        with pytest.raises(TypeError):
            bq.gated_grad_quant(f, bad)
    with pytest.raises(TypeError):
        bq.gemm_int8_int8(i8, f, i8, f, 4.0, 4, 32)
    with pytest.raises(TypeError):
        bq.gemm_int8_int8(i8, f, i8, f, 4, 4, 32, alpha="1")


def batched_product(M, N, K, count, residual, stride_res):
    z = torch.zeros
    return bq.gemm_int8_int8(
        z((count, M, K), dtype=torch.int8), z(count * M), z((count, N, K), dtype=torch.int8),
        z(count * N), M, N, K, residual=residual,
        batch=dict(count=count, stride_a=M * K, stride_a_sf=4 * M, stride_b=N * K,
                   stride_b_sf=4 * N, stride_y=2 * M * N, stride_res=stride_res))


def test_binding_refuses_a_batched_residual_that_ends_early():
    """The kernels go by the strides alone: the residual's storage has to reach the last
    problem's last row.  (What passes this check is refused for being on the CPU.)"""
    M, N, K, count = 5, 16, 32, 3
    bf = dict(dtype=torch.bfloat16)
    step = 2 * M * N
    whole = torch.zeros((count, M, N), **bf)
    wide = torch.zeros((count, M, 24), **bf)
    fits = [(whole, step), (whole.view(count * M, N), step), (whole[0], 0), (whole[1], step // 2),
            (wide, 2 * M * 24), (wide[:, :, :N], 2 * M * 24), (wide[:, :, 8:], 2 * M * 24),
            (torch.zeros((M, 1, N), **bf).transpose(0, 1), 0)]
    for res, stride in fits:
        with pytest.raises(ValueError, match="CUDA tensors only"):
            batched_product(M, N, K, count, res, stride)
    short = [(whole[:2].clone(), step, "last row"), (whole, step + 16, "last row"),
             (whole[1], step, "last row"), (whole[0].clone(), step, "last row"),
             (wide[1:, :, 8:], 2 * M * 24, "last row"),
             (torch.zeros((count, M - 1, N), **bf), step, "unit column"),
             (torch.zeros((count, M, N - 8), **bf), step, "unit column"),
             (torch.zeros((M, count, N), **bf), step, "unit column"),
             (torch.zeros((count, N, M), **bf).transpose(1, 2), step, "unit column"),
             (torch.zeros((M * N,), **bf), 0, "unit column"),
             (whole.float(), step, "unit column")]
    for res, stride, why in short:
        with pytest.raises(ValueError, match=why):
            batched_product(M, N, K, count, res, stride)
    # one row has no stride of its own
    one = torch.zeros((count, 2, N), **bf)[:, :1]
    with pytest.raises(ValueError, match="CUDA tensors only"):
        batched_product(1, N, K, count, one, 4 * N)


def test_status_is_an_int32_word(L):
    x = torch.zeros((32, 32), dtype=torch.bfloat16)
    gu = torch.zeros((32, 64), dtype=torch.bfloat16)
    for bad in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64),
                torch.zeros(0, dtype=torch.int32), torch.zeros(4)):
        with pytest.raises(ValueError, match="status must be a torch.int32"):
            bq.act_quant_int8(x, status=bad)
        with pytest.raises(ValueError, match="status must be a torch.int32"):
            bq.gated_grad_quant(x, gu, status=bad)
    for good in (torch.zeros((), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)[1::2]):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            bq.act_quant_int8(x, status=good)
        with pytest.raises(ValueError, match="CUDA tensors only"):
            bq.gated_grad_quant(x, gu, status=good)
    assert L.bq_act_quant_int8(P, 4, 32, 32, P, P, P + 2, None) == bq.BQ_ERR_ALIGN
    for rounding in (0, 1):
        assert L.bq_gated_grad_quant(P, 64, P, 128, 32, 64, 0, rounding, 0, P, P, P, P, None,
                                     P + 2, None) == bq.BQ_ERR_ALIGN


@pytest.mark.parametrize("rounding", [0, 1])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_grad_scale_buffers_are_aligned(L, rounding, off):
    """The scales leave as words."""
    for sf, st in ((P + off, P), (P, P + off)):
        assert L.bq_gated_grad_quant(P, 64, P, 128, 32, 64, 0, rounding, 0, P, sf, P, st, None,
                                     None, None) == bq.BQ_ERR_ALIGN


def test_batched_outputs_keep_apart(L):
    """Problems' outputs (2 M N bytes each) may have gaps between them, in a y that the
    caller brings, but not overlap."""
    B = bq.Batch
    for stride in (16, 48):
        assert product(L, batch=B(2, 128, 16, 0, 0, stride, 0)) == bq.BQ_ERR_SHAPE
    # (as far as the alignment that is checked next)
    assert product(L, batch=B(2, 128, 16, 0, 0, 72, 0)) == bq.BQ_ERR_ALIGN
    assert product(L, M=0x7FFFFE00, N=0x7FFFFE00, batch=B(2, 0, 0, 0, 0, 1 << 61, 0)) \
        == bq.BQ_ERR_SHAPE
    M, N, K, count = 4, 8, 32, 3
    i8, f = torch.zeros(count * M * K + N * K, dtype=torch.int8), torch.zeros(64)

    def call(stride_y, y=None):
        bq.gemm_int8_int8(i8, f, i8, f, M, N, K, y=y, batch=dict(
            count=count, stride_a=M * K, stride_a_sf=4 * M, stride_y=stride_y))
    dense, gaps = 2 * M * N, 2 * M * N + 64
    with pytest.raises(ValueError, match="needs y"):
        call(gaps)
    held = torch.zeros(2 * (gaps // 2) + M * N, dtype=torch.bfloat16)
    for stride, y in ((dense, None), (gaps, held)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call(stride, y)


@pytest.mark.parametrize("kind", [bq.W_MXFP4, bq.W_FP8BLK32, bq.W_MXFP8, bq.W_A4W4, bq.W_GRAD,
                                  bq.W_NVFP4])
def test_block_scaled_batch_with_gaps_needs_its_outputs(kind):
    """The tensors made for a batch's outputs have no room for gaps."""
    M, N, K, count = 4, 32, 128, 2
    u8 = torch.zeros(1 << 16, dtype=torch.uint8)
    y, q = torch.zeros(1024, dtype=torch.bfloat16), torch.zeros(1024, dtype=torch.uint8)

    def call(stride_y, **kw):
        bq.gemm(kind, u8, u8, u8, u8, M, N, K, batch=dict(count=count, stride_y=stride_y), **kw)
    gaps = 2 * M * N + 64
    for kw in (dict(), dict(quantize_out=True, y=y), dict(quantize_out=True, write_y=False),
               dict(quantize_out=True, q_out=q)):
        with pytest.raises(ValueError, match="needs them given"):
            call(gaps, **kw)
    for stride, kw in ((2 * M * N, {}), (gaps, dict(y=y)),
                       (gaps, dict(quantize_out=True, y=y, q_out=q))):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call(stride, **kw)


def test_plans():
    def p(M, N, K, **kw):
        c = bq.ffn_plan(M, N, K, **kw)
        return c.swap_ab, c.block_n, c.split_k

    # decode: one tile of rows, split where K is long and SMs are left
    assert p(1, 4608, 1536)[:2] == (1, 32)
    assert p(41, 1536, 6144) == (1, 64, 8)
    assert p(41, 6144, 1536, weight_kind=bq.W_MXFP4, gated=True)[:2] == (1, 64)
    # large weights: every SM streams
    assert p(16, 16384, 8192)[2] * 128 >= 128
    assert p(16, 16384, 8192, weight_kind=bq.W_FP8BLK32, gated=True) == (1, 32, 1)
    # between: tiles of one SM while pairs would leave most of them idle
    assert p(512, 1024, 1024) == (1, 64, 1)
    assert p(200, 512, 8192) == (1, 64, 8)
    # many rows: pairs of SMs
    for kw in (dict(), dict(gated=True), dict(gated=True, weight_kind=bq.W_MXFP8)):
        assert p(8192, 8192, 8192, **kw) == (0, 256, 1)
    for kind in (bq.W_MXFP4, bq.W_FP8BLK32, bq.W_MXFP8):  # short MX tiles hold all rows
        for M in range(1, 400, 7):
            sw, bn, _ = p(M, 768, 2048, weight_kind=kind, gated=True)
            assert sw == 0 or bn == 128 or M <= bn
    # an MX tile shorter than a scale atom holds all rows
    for M, bn, ok in ((32, 32, True), (33, 32, False), (64, 64, True), (65, 64, False),
                      (300, 128, True)):
        for kind in (bq.W_MXFP4, bq.W_FP8BLK32, bq.W_MXFP8, bq.W_INT8):
            kw = dict(config=bq.config(block_n=bn, swap_ab=1), weight_kind=kind, gated=True)
            if ok or kind == bq.W_INT8:
                assert bq.ffn_plan(M, 256, 256, **kw).block_n == bn
            else:
                with pytest.raises(bq.BqError) as e:
                    bq.ffn_plan(M, 256, 256, **kw)
                assert e.value.status == bq.BQ_ERR_INVALID
    for kind, gate in ((bq.W_MXFP8, False), (bq.W_A4W4, True), (bq.W_NVFP4, True)):
        with pytest.raises(bq.BqError):
            bq.ffn_plan(41, 4608, 1536, weight_kind=kind, gated=gate)


def test_plans_of_large_weights_fill_the_device():
    """Products that read their weights once keep at least 85 % of the SMs streaming."""
    for M, N, K in ((1, 16384, 8192), (16, 16384, 8192), (41, 18944, 4096)):
        for kw in (dict(), dict(gated=True), dict(gated=True, weight_kind=bq.W_FP8BLK32)):
            c = bq.ffn_plan(M, N, K, **kw)
            assert (c.swap_ab, c.block_n) == (1, 32 if M <= 32 else 64)
            assert N // 128 * c.split_k >= 0.85 * 148


def test_block_scaled_gemm_refuses_a_second_32_row_tile():
    """32-row decode tiles hold all activation rows: a second one would begin in the
    middle of a scale atom."""
    for kind in (bq.W_MXFP4, bq.W_FP8BLK32, bq.W_MXFP8, bq.W_A4W4, bq.W_GRAD, bq.W_NVFP4):
        assert bq.plan(32, 512, 1024, weight_kind=kind,
                       config=bq.config(block_n=32, swap_ab=1)).block_n == 32
        for M in (33, 64):
            with pytest.raises(bq.BqError) as e:
                bq.plan(M, 512, 1024, weight_kind=kind, config=bq.config(block_n=32, swap_ab=1))
            assert e.value.status == bq.BQ_ERR_INVALID
