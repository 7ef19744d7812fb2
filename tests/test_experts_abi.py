"""The C ABI of the mixture-of-experts operators on the CPU: exports, sizes, and refusals, which
are decided before any device work (no kernel is launched; there is no GPU here)."""
import ctypes
import os
import re

import pytest
import torch

import tile_scheduled_dense_amd as tg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tile_gemm_experts.h")
P = [0x100000000 + (i << 36) for i in range(8)]     # never dereferenced, far apart
INVALID, UNSUPPORTED, OK = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED, tg.TG_OK


def header_text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_exports_every_declared_symbol():
    declared = set(re.findall(r"\b(tile_gemm_[a-z0-9_]*)\s*\(", header_text()))
    assert declared == set(tg.EXPORTED_EXPERTS)
    lib = ctypes.CDLL(tg.library_path())
    for name in declared:
        assert hasattr(lib, name), name


def test_version_and_limits_match_the_header():
    text = header_text()
    assert int(re.search(r"TILE_GEMM_EXPERTS_VERSION (\d+)", text).group(1)) == tg.experts_version() == tg.EXPERTS_VERSION
    assert int(re.search(r"TILE_GEMM_MAX_EXPERTS (\d+)", text).group(1)) == tg.MAX_EXPERTS


def call(fn, defaults, **kw):
    return tg.tile_gemm_status(fn, *{**defaults, **kw}.values())


SORT = dict(tokens=64, top_k=2, experts=8, ids=P[0], ld_ids=2, offsets=P[1], entry_of_row=P[2], row_of_entry=P[3],
            workspace=None, workspace_bytes=0, stream=0)
GATHER = dict(tokens=64, top_k=2, cols=32, dtype=1, x=P[0], ldx=32, row_of_entry=P[1], rows=P[2], ldr=32, stream=0)
COMBINE = dict(tokens=64, top_k=2, cols=32, dtype=1, y=P[0], ldy=32, row_of_entry=P[1], weights=P[2], ld_w=2, out=P[3],
               ldo=32, stream=0)
GRAD = dict(tokens=64, top_k=2, cols=32, dtype=1, d_out=P[0], ldo=32, y=P[1], ldy=32, row_of_entry=P[2], weights=P[3],
            ld_w=2, d_y=P[4], ldd=32, d_w=P[5], ld_dw=2, stream=0)
GROUPED = dict(experts=4, rows=64, N=32, K=48, dtype=1, A=P[0], lda=48, B=P[1], ldb=32, strideB=48 * 32, transposed=0,
               C=P[2], ldc=32, c_dtype=1, offsets=P[3], stream=0)
WGRAD = dict(experts=4, rows=64, M=48, N=32, dtype=1, A=P[0], lda=48, D=P[1], ldd=32, C=P[2], ldc=32, strideC=48 * 32,
             c_dtype=1, offsets=P[3], stream=0)
PACK = dict(experts=4, N=32, K=48, group=32, dtype=1, codes=P[0], ld_codes=24, stride_codes=32 * 24, scales=P[1],
            ld_scales=2, stride_scales=64, packed=P[2], packed_bytes=1 << 30, stream=0)
Q4 = dict(experts=4, rows=64, N=32, K=48, group=32, dtype=1, A=P[0], lda=48, packed=P[1], C=P[2], ldc=32, c_dtype=1,
          offsets=P[3], stream=0)
ALL = [("tile_gemm_expert_sort", SORT), ("tile_gemm_expert_gather", GATHER), ("tile_gemm_expert_combine", COMBINE),
       ("tile_gemm_expert_combine_grad", GRAD), ("tile_gemm_grouped", GROUPED), ("tile_gemm_grouped_wgrad", WGRAD),
       ("tile_gemm_pack_q4", PACK), ("tile_gemm_q4", Q4)]


@pytest.mark.parametrize("fn,base", ALL, ids=[f for f, _ in ALL])
def test_valid_arguments_only_lack_the_device(fn, base):
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible")
    assert call(fn, base) == UNSUPPORTED


REFUSED = [
    ("tile_gemm_expert_sort", SORT, [dict(tokens=-1), dict(top_k=-1), dict(experts=0), dict(ids=None),
                                     dict(offsets=None), dict(entry_of_row=None), dict(row_of_entry=None),
                                     dict(ld_ids=1), dict(ids=P[0] + 2), dict(offsets=P[1] + 1),
                                     dict(tokens=8192),                          # needs a workspace
                                     dict(tokens=8192, workspace=P[4], workspace_bytes=16),
                                     dict(tokens=8192, workspace=P[4] + 2, workspace_bytes=1 << 20),
                                     dict(tokens=8192, workspace=P[2] + 4, workspace_bytes=1 << 20),
                                     dict(row_of_entry=P[2] + 4), dict(offsets=P[0] + 8)]),
    ("tile_gemm_expert_gather", GATHER, [dict(tokens=-1), dict(cols=-1), dict(dtype=3), dict(x=None), dict(rows=None),
                                         dict(row_of_entry=None), dict(ldx=31), dict(ldr=31), dict(x=P[0] + 1),
                                         dict(row_of_entry=P[1] + 2), dict(rows=P[0] + 64), dict(rows=P[1])]),
    ("tile_gemm_expert_combine", COMBINE, [dict(top_k=-1), dict(cols=-1), dict(dtype=-1), dict(y=None), dict(out=None),
                                           dict(row_of_entry=None), dict(ldy=31), dict(ldo=31), dict(ld_w=1),
                                           dict(weights=P[2] + 2), dict(out=P[0] + 64), dict(out=P[2]), dict(out=P[1])]),
    ("tile_gemm_expert_combine_grad", GRAD, [dict(tokens=-1), dict(dtype=9), dict(d_out=None), dict(y=None),
                                             dict(weights=None), dict(d_y=None), dict(d_w=None), dict(ldo=31),
                                             dict(ldd=31), dict(ld_w=1), dict(ld_dw=1), dict(d_y=P[1]), dict(d_y=P[0]),
                                             dict(d_w=P[3]), dict(d_w=P[4] + 64), dict(d_w=P[5] + 2)]),
    ("tile_gemm_grouped", GROUPED, [dict(experts=0), dict(rows=-1), dict(N=-1), dict(K=-1), dict(dtype=4),
                                    dict(c_dtype=2), dict(dtype=0, c_dtype=1), dict(offsets=None), dict(A=None),
                                    dict(B=None), dict(C=None), dict(lda=47), dict(ldb=31), dict(ldc=31),
                                    dict(transposed=2), dict(transposed=1, ldb=47), dict(strideB=-1), dict(C=P[0]),
                                    dict(C=P[1] + 3 * 48 * 32 * 2), dict(C=P[3]), dict(A=P[0] + 1),
                                    dict(c_dtype=0, C=P[2] + 2), dict(offsets=P[3] + 1)]),
    ("tile_gemm_grouped_wgrad", WGRAD, [dict(experts=-1), dict(rows=-1), dict(M=-1), dict(N=-1), dict(c_dtype=2),
                                        dict(offsets=None), dict(A=None), dict(D=None), dict(C=None), dict(lda=47),
                                        dict(ldd=31), dict(ldc=31), dict(strideC=48 * 32 - 1), dict(strideC=-1),
                                        dict(C=P[0]), dict(C=P[1]), dict(C=P[3])]),
    ("tile_gemm_pack_q4", PACK, [dict(experts=0), dict(N=-1), dict(K=-1), dict(group=0), dict(dtype=3),
                                 dict(codes=None), dict(scales=None), dict(packed=None), dict(ld_codes=23),
                                 dict(ld_scales=1), dict(stride_codes=-1), dict(stride_scales=-1),
                                 dict(packed=P[2] + 8), dict(packed_bytes=100), dict(packed=P[0]), dict(packed=P[1]),
                                 dict(scales=P[1] + 1)]),
    ("tile_gemm_q4", Q4, [dict(experts=0), dict(rows=-1), dict(N=-1), dict(K=-1), dict(group=-32), dict(dtype=3),
                          dict(c_dtype=2), dict(offsets=None), dict(A=None), dict(packed=None), dict(C=None),
                          dict(lda=47), dict(ldc=31), dict(packed=P[1] + 8), dict(C=P[0]), dict(C=P[1]), dict(C=P[3])]),
]
REFUSED = [(f, b, kw) for f, b, kws in REFUSED for kw in kws]


@pytest.mark.parametrize("fn,base,kw", REFUSED, ids=lambda v: str(v)[:40] if not isinstance(v, dict) or len(v) < 4 else "")
def test_invalid_arguments(fn, base, kw):
    assert call(fn, base, **kw) == INVALID


@pytest.mark.parametrize("fn,base,kw", [
    ("tile_gemm_expert_sort", SORT, dict(tokens=1 << 30)), ("tile_gemm_expert_sort", SORT, dict(experts=2049)),
    ("tile_gemm_expert_gather", GATHER, dict(tokens=1 << 31)),
    ("tile_gemm_grouped", GROUPED, dict(experts=2049)), ("tile_gemm_grouped", GROUPED, dict(lda=1 << 22)),
    ("tile_gemm_grouped", GROUPED, dict(ldc=1 << 22, c_dtype=0)), ("tile_gemm_grouped", GROUPED, dict(ldb=1 << 22)),
    ("tile_gemm_grouped_wgrad", WGRAD, dict(ldd=1 << 22)),
    ("tile_gemm_pack_q4", PACK, dict(group=48)), ("tile_gemm_q4", Q4, dict(group=256)),
    ("tile_gemm_q4", Q4, dict(experts=5000)),
], ids=lambda v: str(v) if isinstance(v, dict) and len(v) < 4 else "")
def test_unsupported(fn, base, kw):
    assert call(fn, base, **kw) == UNSUPPORTED


@pytest.mark.parametrize("fn,base,kw", [
    ("tile_gemm_expert_gather", GATHER, dict(tokens=0, x=None, rows=None)),
    ("tile_gemm_expert_gather", GATHER, dict(cols=0)),
    ("tile_gemm_expert_combine", COMBINE, dict(tokens=0, y=None, out=None)),
    ("tile_gemm_expert_combine_grad", GRAD, dict(top_k=0)),
    ("tile_gemm_grouped", GROUPED, dict(rows=0, A=None, C=None)), ("tile_gemm_grouped", GROUPED, dict(N=0)),
    ("tile_gemm_grouped_wgrad", WGRAD, dict(M=0)),
    ("tile_gemm_pack_q4", PACK, dict(N=0)), ("tile_gemm_q4", Q4, dict(rows=0)),
], ids=lambda v: str(v) if isinstance(v, dict) and len(v) < 4 else "")
def test_nothing_to_write_is_ok_without_a_device(fn, base, kw):
    assert call(fn, base, **kw) == OK


def test_sizes():
    assert tg.tile_gemm_expert_sort_workspace_size(16, 2, 8) == 0
    n = tg.tile_gemm_expert_sort_workspace_size(8192, 2, 8)
    assert n > 0 and n % (9 * 4) == 0
    # one block's counts for 64 blocks at most, whatever the number of entries
    assert tg.tile_gemm_expert_sort_workspace_size(1 << 26, 8, 2048) <= 2049 * 64 * 4
    # 16-byte codes of 16 n x 128 k, then 16 scales a group
    assert tg.tile_gemm_q4_packed_size(1, 4096, 4096, 128, "bf16") == 4096 * 2048 + 4096 * 32 * 2
    assert tg.tile_gemm_q4_packed_size(3, 17, 130, 32, "f32") == 3 * (2 * 2 * 1024 + 2 * 8 * 16 * 4)
    assert tg.tile_gemm_q4_packed_size(1, 0, 0, 64, "f16") == 0
    with pytest.raises(tg.TileGemmError):
        tg.tile_gemm_q4_packed_size(1, 16, 16, 16, "bf16")
    with pytest.raises(tg.TileGemmError):
        tg.tile_gemm_expert_sort_workspace_size(-1, 2, 8)
