"""Host-side checks (no GPU): arguments of the rotating append, 8-bit and window attention calls are refused with the
documented status before any device work, the binding refuses what the library cannot check, and the oracle's own
rounding and rotation agree with independent forms."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_maxpool_b200 as msa
from block_sparse_attention_maxpool_b200 import build as msa_build
from oracle import cache_ops as C

FAKE = 0x10000
GOOD = msa.Shape(2, 1024)
BAD = msa.Shape(2, 1000)


@pytest.fixture(scope="module")
def lib():
    msa_build.build()
    return msa.library()


def rope_call(lib, shape=GOOD, pages=None, rope=(FAKE, 64, 0), kv=(FAKE,) * 4, idx=(FAKE, 0, FAKE), tok=(FAKE, FAKE),
              nt=2, q=(FAKE, FAKE), iq=(FAKE, FAKE), qp=FAKE, nq=2):
    r = None if rope is None else msa.CRope(*rope)
    return lib.msa_rope_append(shape.c(), pages, r, *kv, *idx, *tok, nt, *q, *iq, qp, nq, None)


def test_rope_append_refusals(lib):
    assert rope_call(lib, shape=BAD) == -3
    assert rope_call(lib, rope=None) == -1
    assert rope_call(lib, rope=(0, 64, 0)) == -1
    assert rope_call(lib, rope=(FAKE + 4, 64, 0)) == -2
    for rot in (0, 8, 24, 144, -16):
        assert rope_call(lib, rope=(FAKE, rot, 0)) == -3
    for i in range(4):
        assert rope_call(lib, kv=tuple(0 if j == i else FAKE for j in range(4))) == -1
        assert rope_call(lib, kv=tuple(FAKE + 8 if j == i else FAKE for j in range(4))) == -2
    assert rope_call(lib, idx=(FAKE, 0, 0)) == -1
    assert rope_call(lib, idx=(FAKE + 4, 1, FAKE)) == -2
    assert rope_call(lib, kv=(0,) * 4, idx=(0, 0, 0)) == -1
    assert rope_call(lib, tok=(FAKE, 0)) == -1
    assert rope_call(lib, nt=-1) == -4
    assert rope_call(lib, nq=-1) == -4
    assert rope_call(lib, q=(FAKE, 0)) == -1
    assert rope_call(lib, iq=(0, FAKE)) == -1
    assert rope_call(lib, q=(0, 0), iq=(0, 0)) == -1
    assert rope_call(lib, q=(FAKE + 2, FAKE)) == -2
    assert rope_call(lib, qp=0) == -1
    assert rope_call(lib, pages=msa.CPages(0, 4)) == -1
    assert rope_call(lib, pages=msa.CPages(FAKE, 0)) == -4
    assert rope_call(lib, nt=0, nq=0, kv=(0,) * 4, idx=(0, 0, 0), q=(0, 0), iq=(0, 0), qp=0, tok=(0, 0)) == 0


def test_fp8_append_refusals(lib):
    need = lib.msa_kv_append_fp8_workspace_bytes(GOOD.c(), 257)
    assert need == 2 * 8 * 4 * 16
    assert lib.msa_kv_append_fp8_workspace_bytes(GOOD.c(), 256) == 0
    assert lib.msa_kv_append_fp8_workspace_bytes(GOOD.c(), 0) == 0
    assert lib.msa_kv_append_fp8_workspace_bytes(BAD.c(), 2) == ctypes.c_size_t(-1).value
    assert lib.msa_kv_append_fp8_workspace_bytes(GOOD.c(), -1) == ctypes.c_size_t(-1).value

    def call(shape=GOOD, rope=None, p=(FAKE,) * 6, tok=(FAKE, FAKE), n=257, ws=FAKE, wb=need, pages=None):
        return lib.msa_kv_append_fp8(shape.c(), pages, rope, *p, *tok, n, ws, wb, None)
    assert call(shape=BAD) == -3
    assert call(n=-1) == -4
    assert call(n=0, p=(0,) * 6, tok=(0, 0), ws=0, wb=0) == 0
    for i in range(6):
        assert call(p=tuple(0 if j == i else FAKE for j in range(6))) == -1
        assert call(p=tuple(FAKE + 8 if j == i else FAKE for j in range(6))) == -2
    assert call(tok=(0, FAKE)) == -1
    assert call(ws=0) == -5
    assert call(wb=need - 1) == -5
    assert call(ws=FAKE + 8) == -2
    assert call(rope=msa.CRope(FAKE, 40, 0)) == -3
    assert call(pages=msa.CPages(FAKE + 1, 4)) == -2


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_attention_refusals(lib, mode):
    m = msa.MODE_PREFILL if mode == "prefill" else msa.MODE_DECODE
    need = lib.msa_attn_workspace_bytes(GOOD.c(), None, 2, m, 1)
    assert need == lib.msa_attn_workspace_bytes(GOOD.c(), None, 200, m, 0) == 0
    assert lib.msa_attn_workspace_bytes(BAD.c(), None, 2, m, 0) == ctypes.c_size_t(-1).value
    assert lib.msa_attn_workspace_bytes(GOOD.c(), None, -2, m, 0) == ctypes.c_size_t(-1).value
    assert lib.msa_attn_workspace_bytes(GOOD.c(), None, 2, 2, 1) == ctypes.c_size_t(-1).value
    scale = ctypes.c_float(0.1)
    for f8 in (False, True):
        fn = getattr(lib, f"msa_window_attn_{mode}" + ("_fp8" if f8 else ""))
        nkv = 4 if f8 else 2

        def call(shape=GOOD, pages=None, q=FAKE, kv=(FAKE,) * nkv, qs=FAKE, qp=FAKE, n=2, w=5, sink=0, sc=scale,
                 out=FAKE, ws=FAKE, wb=need):
            return fn(shape.c(), pages, q, *kv, qs, qp, n, w, sink, sc, out, ws, wb, None)
        assert call(shape=BAD) == -3
        assert call(w=0) == -4
        assert call(w=-1) == -4
        assert call(sink=-1) == -4
        assert call(n=-1) == -4
        assert call(n=0, q=0, out=0) == 0
        assert call(q=0) == -1
        assert call(qp=0) == -1
        assert call(out=0) == -1
        assert call(q=FAKE + 8) == -2
        assert call(out=FAKE + 2) == -2
        assert call(sc=ctypes.c_float(math.inf)) == -4
        for i in range(nkv):
            assert call(kv=tuple(0 if j == i else FAKE for j in range(nkv))) == -1
            assert call(kv=tuple(FAKE + 4 if j == i else FAKE for j in range(nkv))) == -2
        assert call(pages=msa.CPages(FAKE, -1)) == -4
        assert call(n=1 << 26, shape=msa.Shape(1, 128, 256, 16)) == -4
        if f8 and mode == "prefill":           # many queries: the cache is expanded to bf16
            big = lib.msa_attn_workspace_bytes(GOOD.c(), None, 256, m, 1)
            assert big >= 2 * 4 * 1024 * 512
            assert lib.msa_attn_workspace_bytes(GOOD.c(), None, 255, m, 1) == 0
            assert lib.msa_attn_workspace_bytes(msa.Shape(64, 1024).c(), None, 1023, m, 1) == 0
            assert 5 * 4 * 128 * 512 <= lib.msa_attn_workspace_bytes(GOOD.c(), msa.CPages(0, 5), 256, m, 1) < big
            assert lib.msa_attn_workspace_bytes(GOOD.c(), msa.CPages(0, 0), 256, m, 1) == ctypes.c_size_t(-1).value
            assert call(n=256, ws=0, wb=big) == -5
            assert call(n=256, wb=big - 1) == -5
            assert call(n=256, ws=FAKE + 128, wb=big) == -2
    fn = getattr(lib, f"msa_sparse_attn_{mode}_fp8")

    def sparse(shape=GOOD, q=FAKE, kv=(FAKE,) * 4, sel=FAKE, n=2, sc=scale, ws=FAKE, wb=need):
        return fn(shape.c(), None, q, *kv, sel, FAKE, FAKE, n, sc, FAKE, ws, wb, None)
    assert sparse(shape=BAD) == -3
    assert sparse(sel=0) == -1
    assert sparse(sel=FAKE + 4) == -2
    assert sparse(kv=(FAKE, FAKE, 0, FAKE)) == -1
    assert sparse(n=0, sel=0) == 0
    assert sparse(sc=ctypes.c_float(math.nan)) == -4


def test_binding_refuses_cpu_tensors_and_mixed_caches():
    t = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((1, 64, 128), dtype=torch.bfloat16)
    kv = torch.zeros((2, 4, 1024, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        msa.msa_window_attn_decode(GOOD, q, kv, kv, t, t, 5)
    with pytest.raises(ValueError):
        msa.msa_sparse_attn_decode_fp8(GOOD, q, kv, kv, None, None, t, t, t)
    with pytest.raises(ValueError):
        msa.msa_kv_append_fp8(GOOD, kv, kv, None, None, kv, kv, t, t)
    with pytest.raises(ValueError):
        msa.msa_rope_append(GOOD, msa.Rope(torch.zeros(32, dtype=torch.float64)), q=q, q_pos=t)
    with pytest.raises(ValueError):
        msa.msa_rope_append(GOOD, msa.Rope(torch.zeros(32, dtype=torch.float64)))


def test_oracle_rounding_and_scales():
    x = torch.linspace(-460, 460, 20001, dtype=torch.float64)
    x = torch.cat((x, torch.linspace(-0.03, 0.03, 4001, dtype=torch.float64), C._VALUES,
                   (C._VALUES[1:] + C._VALUES[:-1]) / 2))
    want = x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    assert torch.equal(C.round_e4m3(x), want)
    for a in (0.0, 1e-45, 1.0, 447.9, 448.0, 448.1, 3.3e38, 1.75, 1.7500001, 2.0 ** -95):
        s = C.needed_scale(a)
        assert math.log2(s) == int(math.log2(s)) and a <= 448 * s
        assert s == 2.0 ** -100 or a > 448 * s / 2


def test_oracle_rotation():
    x = torch.randn((3, 128))
    f = torch.tensor([1.0, 0.25, 0.5], dtype=torch.float64)
    y = C.rotate_row(x, 7, f, True)
    z = torch.view_as_complex(x[:, :6].double().reshape(3, 3, 2).contiguous()) * torch.exp(1j * 7 * f)
    assert torch.allclose(y[:, :6], torch.view_as_real(z).reshape(3, 6), atol=1e-14)
    assert torch.equal(y[:, 6:], x[:, 6:].double())
    assert torch.allclose((y ** 2).sum(1), (x.double() ** 2).sum(1))
    y2 = C.rotate_row(x, 7, f, False)
    assert torch.allclose(y2[:, 0], x[:, 0].double() * math.cos(7) - x[:, 3].double() * math.sin(7))


def test_oracle_window_is_dense_attention_with_a_mask():
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn((1, 1, 256, 128), generator=gen) for _ in range(2))
    q = torch.randn((2, 16, 128), generator=gen)
    pos = torch.tensor([200, 3])
    out, _, _ = C.window_attention(q, k, v, torch.zeros(2), pos, 50, 10, 0.1)
    for i in range(2):
        s = q[i].double() @ k[0, 0].double().T * 0.1
        j, p = torch.arange(256), int(pos[i])
        s[:, ~((j <= p) & ((p - j < 50) | (j < 10)))] = -math.inf
        assert torch.allclose(out[i], torch.softmax(s, 1) @ v[0, 0].double())
