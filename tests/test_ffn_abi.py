"""The C ABI of the operators of a feed-forward block on the CPU: exports, sizes, and refusals, which
are decided before any device work (no kernel is launched; there is no GPU here)."""
import ctypes
import os
import re

import pytest
import torch

import tile_scheduled_dense_amd as tg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tile_gemm_ffn.h")
P = [0x100000000 + (i << 36) for i in range(12)]     # never dereferenced, far apart
INVALID, UNSUPPORTED, OK = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED, tg.TG_OK


def header_text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_exports_every_declared_symbol():
    declared = set(re.findall(r"\b(tile_gemm_[a-z0-9_]*)\s*\(", header_text()))
    assert declared == set(tg.EXPORTED_FFN)
    lib = ctypes.CDLL(tg.library_path())
    for name in declared:
        assert hasattr(lib, name), name


def test_version_matches_the_header():
    assert int(re.search(r"TILE_GEMM_FFN_VERSION (\d+)", header_text()).group(1)) == tg.ffn_version() == tg.FFN_VERSION


def call(fn, defaults, **kw):
    return tg.tile_gemm_status(fn, *{**defaults, **kw}.values())


GATED = dict(experts=4, rows=64, N=32, K=48, dtype=1, A=P[0], lda=48, B=P[1], B_up=P[1] + 64, ldb=64, strideB=48 * 64,
             transposed=0, activation=3, H=P[2], ldh=32, U=P[3], V=P[3] + 64, ldu=64, offsets=P[4], workspace=None,
             workspace_bytes=0, stream=0)
GRAD = dict(experts=4, rows=64, N=32, K=48, dtype=1, D=P[0], ldd=48, B=P[1], ldb=48, strideB=32 * 48, transposed=1,
            activation=3, U=P[2], V=P[2] + 64, ldu=64, dU=P[3], dV=P[3] + 64, lddu=64, H=P[4], ldh=32, offsets=P[5],
            stream=0)
ADAPT = dict(adapters=4, rows=64, N=32, K=48, rank=8, dtype=1, X=P[0], ldx=48, W=P[1], ldw=32, A=P[2], lda=8, strideA=384,
             B=P[3], ldb=32, strideB=256, transposed=0, scales=P[4], Y=P[5], ldy=32, T=P[6], ldt=8, offsets=P[7],
             order=P[8], workspace=P[9], workspace_bytes=1 << 30, stream=0)
WGRAD = dict(adapters=4, rows=300, N=32, K=48, rank=8, dtype=1, X=P[0], ldx=48, dY=P[1], ldy=32, T=P[2], ldt=8, dT=P[3],
             lddt=8, dA=P[4], lda=8, strideA=384, dB=P[5], ldb=32, strideB=256, transposed=0, c_dtype=0, offsets=P[6],
             order=P[7], workspace=P[8], workspace_bytes=1 << 30, stream=0)
GATE = dict(rows=64, N=32, dtype=1, activation=3, U=P[0], V=P[0] + 64, ldu=64, H=P[1], ldh=32, stream=0)
GATE_GRAD = dict(rows=64, N=32, dtype=1, activation=3, D=P[0], ldd=32, U=P[1], V=P[1] + 64, ldu=64, dU=P[2], dV=P[2] + 64,
                 lddu=64, H=P[3], ldh=32, stream=0)
ALL = [("tile_gemm_gate", GATE), ("tile_gemm_gate_grad", GATE_GRAD), ("tile_gemm_gated", GATED), ("tile_gemm_gated_grad", GRAD), ("tile_gemm_adapters", ADAPT),
       ("tile_gemm_adapters_wgrad", WGRAD)]


@pytest.mark.parametrize("fn,base", ALL, ids=[f for f, _ in ALL])
def test_valid_arguments_only_lack_the_device(fn, base):
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible")
    assert call(fn, base) == UNSUPPORTED


@pytest.mark.parametrize("fn,base,kw", [
    ("tile_gemm_gated", GATED, dict(U=None, V=None)), ("tile_gemm_gated", GATED, dict(experts=1, offsets=None)),
    ("tile_gemm_gated", GATED, dict(B_up=P[1])), ("tile_gemm_gated", GATED, dict(V=P[10], ldu=32)),
    ("tile_gemm_gated", GATED, dict(transposed=1, B_up=P[1] + 32 * 48 * 2, ldb=48)),
    ("tile_gemm_gated", GATED, dict(workspace=P[0], workspace_bytes=0)),        # too small: not used, so not looked at
    ("tile_gemm_gated_grad", GRAD, dict(H=None)), ("tile_gemm_gate_grad", GATE_GRAD, dict(H=None)), ("tile_gemm_gated_grad", GRAD, dict(dV=P[10], lddu=33)),
    ("tile_gemm_adapters", ADAPT, dict(order=None, scales=None, T=None)), ("tile_gemm_adapters", ADAPT, dict(rank=0)),
    ("tile_gemm_adapters", ADAPT, dict(transposed=1, ldw=48, lda=48, ldb=8)),
    ("tile_gemm_adapters_wgrad", WGRAD, dict(transposed=1, lda=48, ldb=8)),
    ("tile_gemm_adapters_wgrad", WGRAD, dict(rows=256, workspace=None, workspace_bytes=0)),     # no sums to add up
    ("tile_gemm_adapters_wgrad", WGRAD, dict(rows=0)), ("tile_gemm_adapters_wgrad", WGRAD, dict(order=None, c_dtype=1)),
], ids=lambda v: str(v) if isinstance(v, dict) and len(v) < 6 else "")
def test_forms_that_are_taken(fn, base, kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible")
    assert call(fn, base, **kw) == UNSUPPORTED       # for want of a device, after every check


REFUSED = [
    ("tile_gemm_gated", GATED, [
        dict(experts=0), dict(rows=-1), dict(N=-1), dict(K=-1), dict(dtype=3), dict(transposed=2), dict(activation=-1),
        dict(activation=4), dict(offsets=None), dict(offsets=P[4] + 2), dict(A=None), dict(B=None), dict(B_up=None),
        dict(H=None), dict(U=None), dict(V=None), dict(lda=47), dict(ldb=31), dict(ldh=31), dict(ldu=31), dict(strideB=-1),
        dict(A=P[0] + 1), dict(B_up=P[1] + 1), dict(H=P[0]), dict(H=P[1] + 64), dict(H=P[3]), dict(H=P[4]),
        dict(V=P[3] + 62), dict(V=P[3]), dict(U=P[0], V=P[0] + 64), dict(U=P[1], V=P[10]), dict(V=P[2]),
        dict(workspace=P[5] + 8), dict(workspace_bytes=-1), dict(transposed=1, ldb=47)]),
    ("tile_gemm_gated_grad", GRAD, [
        dict(experts=0), dict(rows=-1), dict(dtype=-1), dict(transposed=-1), dict(activation=9), dict(offsets=None),
        dict(D=None), dict(B=None), dict(U=None), dict(V=None), dict(dU=None), dict(dV=None), dict(ldd=47), dict(ldb=47),
        dict(ldu=31), dict(lddu=31), dict(ldh=31), dict(strideB=-1), dict(dU=P[2], dV=P[2] + 64), dict(dV=P[3] + 62),
        dict(H=P[0]), dict(H=P[2]), dict(H=P[3]), dict(H=P[5]), dict(dU=P[0]), dict(dV=P[1]), dict(D=P[0] + 1)]),
    ("tile_gemm_gate", GATE, [
        dict(rows=-1), dict(N=-1), dict(dtype=3), dict(activation=4), dict(U=None), dict(V=None), dict(H=None), dict(ldu=31),
        dict(ldh=31), dict(H=P[0]), dict(H=P[0] + 64), dict(U=P[0] + 1)]),
    ("tile_gemm_gate_grad", GATE_GRAD, [
        dict(rows=-1), dict(N=-1), dict(dtype=-1), dict(activation=-1), dict(D=None), dict(U=None), dict(V=None), dict(dU=None),
        dict(dV=None), dict(ldd=31), dict(ldu=31), dict(lddu=31), dict(ldh=31), dict(dU=P[0]), dict(dV=P[1]), dict(H=P[2]),
        dict(dV=P[2] + 32), dict(H=P[0]), dict(D=P[0] + 1)]),
    ("tile_gemm_adapters", ADAPT, [
        dict(adapters=0), dict(rows=-1), dict(N=-1), dict(K=-1), dict(rank=-1), dict(dtype=3), dict(transposed=2),
        dict(X=None), dict(W=None), dict(A=None), dict(B=None), dict(Y=None), dict(offsets=None), dict(workspace=None),
        dict(workspace_bytes=16), dict(workspace=P[9] + 8), dict(ldx=47), dict(ldw=31), dict(lda=7), dict(ldb=31),
        dict(ldy=31), dict(ldt=7), dict(strideA=-1), dict(strideB=-1), dict(scales=P[4] + 2), dict(order=P[8] + 2),
        dict(offsets=P[7] + 1), dict(X=P[0] + 1), dict(Y=P[0]), dict(Y=P[1]), dict(Y=P[2]), dict(Y=P[3]), dict(Y=P[4]),
        dict(Y=P[7]), dict(Y=P[8]), dict(T=P[5]), dict(T=P[0]), dict(workspace=P[5]), dict(workspace=P[0]),
        dict(transposed=1, lda=48, ldb=8), dict(transposed=1, ldw=48, ldb=8)]),
    ("tile_gemm_adapters_wgrad", WGRAD, [
        dict(adapters=0), dict(rows=-1), dict(rank=-1), dict(dtype=3), dict(c_dtype=2), dict(transposed=2), dict(X=None),
        dict(dY=None), dict(T=None), dict(dT=None), dict(dA=None), dict(dB=None), dict(offsets=None), dict(workspace=None),
        dict(workspace_bytes=100), dict(workspace=P[8] + 4), dict(ldx=47), dict(ldy=31), dict(ldt=7), dict(lddt=7),
        dict(lda=7), dict(ldb=31), dict(strideA=383), dict(strideB=255), dict(dA=P[0]), dict(dB=P[2]), dict(dB=P[4]),
        dict(dA=P[3]), dict(dB=P[6]), dict(dB=P[7]), dict(workspace=P[4]), dict(workspace=P[1]), dict(dA=P[4] + 2)]),
]
REFUSED = [(f, b, kw) for f, b, kws in REFUSED for kw in kws]


@pytest.mark.parametrize("fn,base,kw", REFUSED, ids=lambda v: str(v)[:40] if not isinstance(v, dict) or len(v) < 4 else "")
def test_invalid_arguments(fn, base, kw):
    assert call(fn, base, **kw) == INVALID


@pytest.mark.parametrize("fn,base,kw", [
    ("tile_gemm_gated", GATED, dict(experts=2049)), ("tile_gemm_gated", GATED, dict(rows=(1 << 30) + 1)),
    ("tile_gemm_gated", GATED, dict(lda=1 << 22)), ("tile_gemm_gated", GATED, dict(ldb=1 << 22)),
    ("tile_gemm_gated", GATED, dict(ldh=1 << 22)), ("tile_gemm_gated", GATED, dict(ldu=1 << 22)),
    ("tile_gemm_gated_grad", GRAD, dict(experts=2049)), ("tile_gemm_gated_grad", GRAD, dict(ldd=1 << 22)),
    ("tile_gemm_gated_grad", GRAD, dict(lddu=1 << 22)), ("tile_gemm_gated_grad", GRAD, dict(ldh=1 << 22)),
    ("tile_gemm_adapters", ADAPT, dict(adapters=2049)), ("tile_gemm_adapters", ADAPT, dict(ldx=1 << 22)),
    ("tile_gemm_adapters", ADAPT, dict(ldw=1 << 22)), ("tile_gemm_adapters", ADAPT, dict(ldy=1 << 22)),
    ("tile_gemm_adapters", ADAPT, dict(rows=1 << 14, ldx=1 << 16)),                         # with an order: 2^31 bytes of x
    ("tile_gemm_adapters_wgrad", WGRAD, dict(adapters=2049)), ("tile_gemm_gate", GATE, dict(ldu=1 << 22)),
    ("tile_gemm_gate_grad", GATE_GRAD, dict(rows=(1 << 30) + 1)),
], ids=lambda v: str(v) if isinstance(v, dict) and len(v) < 4 else "")
def test_unsupported(fn, base, kw):
    assert call(fn, base, **kw) == UNSUPPORTED


@pytest.mark.parametrize("fn,base,kw", [
    ("tile_gemm_gated", GATED, dict(rows=0, A=None, H=None, U=None, V=None)), ("tile_gemm_gated", GATED, dict(N=0)),
    ("tile_gemm_gated_grad", GRAD, dict(rows=0, D=None, U=None, V=None, dU=None, dV=None, H=None)),
    ("tile_gemm_gated_grad", GRAD, dict(N=0)), ("tile_gemm_gate", GATE, dict(rows=0, U=None, V=None, H=None)),
    ("tile_gemm_gate_grad", GATE_GRAD, dict(N=0)),
    ("tile_gemm_adapters", ADAPT, dict(rows=0, X=None, Y=None, T=None, offsets=None, workspace=None)),
    ("tile_gemm_adapters", ADAPT, dict(N=0)), ("tile_gemm_adapters_wgrad", WGRAD, dict(rank=0)),
    ("tile_gemm_adapters_wgrad", WGRAD, dict(N=0, K=0)),
], ids=lambda v: str(v) if isinstance(v, dict) and len(v) < 4 else "")
def test_nothing_to_write_is_ok_without_a_device(fn, base, kw):
    assert call(fn, base, **kw) == OK


def test_workspace_sizes():
    assert tg.tile_gemm_gated_workspace_size(8, 16384, 2048, 2048, "bf16") == 0          # tiles
    n = tg.tile_gemm_gated_workspace_size(1, 1, 2816, 1024, "bf16")
    assert n % (2 * 2816 * 4) == 0                                                       # u and v of each split
    assert tg.tile_gemm_gated_workspace_size(1, 0, 2816, 1024, "bf16") == 0
    assert tg.tile_gemm_adapters_workspace_size(4, 8192, 4096, 4096, 60, "f16") >= 8192 * 64 * 2 + 8192 * 60 * 4
    assert tg.tile_gemm_adapters_workspace_size(4, 8192, 4096, 4096, 0, "f16") == 0
    assert tg.tile_gemm_adapters_workspace_size(4, 16, 4096, 4096, 16, "f16") > 16 * 4096 * 4
    assert tg.tile_gemm_adapters_wgrad_workspace_size(2, 0, 64, 64, 8, "f16") == 0
    for bad in (lambda: tg.tile_gemm_gated_workspace_size(1, -1, 8, 8, "f16"),
                lambda: tg.tile_gemm_adapters_workspace_size(0, 1, 8, 8, 8, "f16"),
                lambda: tg.tile_gemm_adapters_wgrad_workspace_size(1, 1, 8, 8, -8, "f16")):
        with pytest.raises(tg.TileGemmError):
            bad()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_workspace_that_no_memory_holds_is_refused(dt):
    """Extents of 2^30 are taken, but not their product, which passes 64 bits."""
    big = 1 << 30
    for ask in (lambda: tg.tile_gemm_adapters_workspace_size(1, big, big, 64, big, dt),
                lambda: tg.tile_gemm_adapters_workspace_size(1, big, 4, 64, big, dt),
                lambda: tg.tile_gemm_adapters_wgrad_workspace_size(1, big, big, big, big, dt),
                lambda: tg.tile_gemm_adapters_wgrad_workspace_size(1, big, 1 << 10, 0, big, dt)):
        with pytest.raises(tg.TileGemmError):
            ask()
    assert tg.tile_gemm_adapters_workspace_size(1, 64, 1 << 20, 64, 1 << 10, dt) > 0
