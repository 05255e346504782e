"""Prefill calls over 8-bit caches on both sides of the rules that choose between the tiles (which expand what the call
sees to bf16 in the workspace) and the cluster kernel, against the float64 oracle and against the single-query calls."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_maxpool_b200 as msa
from oracle import cache_ops as C
from tests import parity_window as PW
from tests.test_gpu_fp8_cache import random_sel

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_attention_maxpool_b200 import build as msa_build
    msa_build.build()
    msa.msa_get_device_error()


def caches(S, G, cap, gen, rows=None):
    """K and V in 8 bits: [(codes, scales, float64 rows)] * 2; ``rows`` of each stream are filled, the rest is NaN codes
    (scales 1)."""
    rows = cap if rows is None else rows
    out = []
    for _ in range(2):
        x = torch.randn((S, G, rows, 128), generator=gen)
        x = (x.view(S, G, rows // 128, 128, 128) * torch.exp2(torch.randint(-3, 4, (S, G, rows // 128, 1, 1), generator=gen).float()
                                                              )).view(S, G, rows, 128)
        q8, sc = PW.quantise(x)
        codes = torch.full((S, G, cap, 128), 0x7f, dtype=torch.uint8)
        codes[:, :, :rows] = q8.view(torch.uint8)
        scale = torch.ones((S, G, cap // 128))
        scale[:, :, :rows // 128] = sc
        out.append((codes, scale, C.fp8_values(q8, sc)))
    return out


def raw_sparse(shape, q, kv, sel, stream, pos, scale, out, ws=None, pages=None):
    """The C call with the given workspace (None: NULL, no bytes)."""
    t = [x.data_ptr() for x in (q, *kv, sel, stream, pos)]
    return msa.library().msa_sparse_attn_prefill_fp8(
        shape.c(), None if pages is None else pages.c(shape), *t, pos.numel(), ctypes.c_float(scale), out.data_ptr(),
        0 if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("cap,scale", [(16384, 128 ** -0.5), (2048, -0.05), (2048, 0.0)])
def test_selection_without_tiles_needs_no_workspace(cap, scale):
    """256 queries x 4 groups: few of them over a long cache, and scales that are not positive, take the cluster kernel,
    which asks for no workspace."""
    gen = torch.Generator().manual_seed(cap)
    G, n, rows = 4, 256, 2048
    shape = msa.Shape(1, cap, 16 * G, G)
    kv = caches(1, G, cap, gen, rows)
    pos = torch.arange(rows - n, rows).int()
    stream = torch.zeros(n, dtype=torch.int32)
    sel = random_sel(n, G, pos, gen, cap // 128)
    q = torch.randn((n, 16 * G, 128), generator=gen).bfloat16()
    dev = [x.cuda() for x in (kv[0][0], kv[1][0], kv[0][1], kv[1][1])]
    out = torch.full((n, 16 * G, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    args = (q.cuda(), dev, sel.cuda(), stream.cuda(), pos.cuda(), scale)
    assert msa.msa_attn_workspace_bytes(shape, n, msa.MODE_PREFILL, True) > 0
    assert raw_sparse(shape, *args, out) == 0
    PW.device_error()
    some = torch.arange(0, n, 5)
    want = C.selected_attention(q[some], kv[0][2], kv[1][2], sel[some], stream[some], pos[some], scale)
    PW.check_attention(out[some.cuda()], *want, PW.P_FP16, 0.0, PW.P_FP16)
    # the binding's call, and the single-query call: the same kernel, the same bits
    for fn in (msa.msa_sparse_attn_prefill_fp8, msa.msa_sparse_attn_decode_fp8):
        got = fn(shape, args[0], dev[0].view(F8), dev[1].view(F8), dev[2], dev[3], *args[2:5], softmax_scale=scale)
        assert torch.equal(got, out)
