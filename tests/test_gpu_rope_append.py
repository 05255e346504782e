"""msa_rope_append on the GPU against the float64 oracle: rotated keys and queries, copied values, untouched rows,
contiguous and paged caches, skipped tokens, and a whole decode step with the rotation on the way."""
import math

import pytest
import torch

import block_sparse_attention_maxpool_b200 as msa
from tests import parity_window as PW

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_attention_maxpool_b200 import build as msa_build
    msa_build.build()
    msa.msa_get_device_error()


def freqs(rot, theta=1.0e6):
    return theta ** -(torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)


@pytest.mark.parametrize("G,cap,rot,inter,paged,idx,positions", [
    (4, 512, 64, False, False, "f32", [(0, 0), (1, 127), (0, 128), (1, 511), (0, 300)]),
    (1, 256, 128, True, False, "f16", [(1, 255)]),
    (16, 128, 16, False, True, None, [(0, 5), (1, 5), (0, 6)]),
    (2, 1 << 20, 128, False, True, "f32", [(0, 1048575), (1, 786431), (0, 131072)]),
    (4, 1 << 20, 64, True, True, "f16", [(1, 1000003), (0, 999999)]),
    (3, 384, 96, False, False, "f32", [(s, p) for s in (0, 1) for p in range(3, 380, 5)]),
])
def test_append_and_queries(G, cap, rot, inter, paged, idx, positions):
    gen = torch.Generator().manual_seed(G * cap + rot)
    S, nblk, n = 2, cap // 128, len(positions)
    shape = msa.Shape(S, cap, 16 * G, G)
    stream = torch.tensor([s for s, _ in positions], dtype=torch.int32)
    pos = torch.tensor([p for _, p in positions], dtype=torch.int32)
    k_new, v_new = (torch.randn((n, G, 128), generator=gen).bfloat16() for _ in range(2))
    q = torch.randn((n, 16 * G, 128), generator=gen).bfloat16()
    idx_k, idx_q = (torch.randn((n, G, 128), generator=gen) for _ in range(2))
    f = freqs(rot)
    pages = None
    if paged:
        used = sorted({(s, p // 128) for s, p in positions})
        table = torch.full((S, nblk), -1, dtype=torch.int32)
        order = torch.randperm(len(used) + 2, generator=gen)
        for i, (s, b) in enumerate(used):
            table[s, b] = int(order[i])
        pages = msa.Pages(table.cuda(), len(used) + 2)
        rows = (len(used) + 2, G, 128)
        at = [(int(table[s, p // 128]), p % 128) for s, p in positions]
    else:
        rows, at = (S, G, cap), positions
    before = {c: torch.randn(rows + (128,), generator=gen).to(t) for c, t in
              (("k", torch.bfloat16), ("v", torch.bfloat16), ("i", torch.float16 if idx == "f16" else torch.float32))}
    dev = {c: t.cuda() for c, t in before.items()}
    more = {} if idx is None else dict(idx_k_cache=dev["i"], idx_k_new=idx_k.cuda(), idx_q=idx_q.cuda())
    q_out, iq_out = msa.msa_rope_append(shape, msa.Rope(f.cuda(), inter), dev["k"], dev["v"], k_new.cuda(),
                                        v_new.cuda(), stream.cuda(), pos.cuda(), q=q.cuda(), q_pos=pos.cuda(),
                                        pages=pages, **more)
    PW.device_error()
    a, b = torch.tensor(at).T
    PW.check_rotated(dev["k"].cpu()[a, :, b], k_new, pos, f, inter, 2.0 ** -8)
    assert torch.equal(dev["v"].cpu()[a, :, b], v_new)
    PW.check_rotated(q_out.cpu(), q, pos, f, inter, 2.0 ** -8)
    if idx is not None:
        PW.check_rotated(dev["i"].cpu()[a, :, b], idx_k, pos, f, inter, 2.0 ** -11 if idx == "f16" else 2.0 ** -24)
        PW.check_rotated(iq_out.cpu(), idx_q, pos, f, inter, 2.0 ** -24)
    else:
        assert iq_out is None
    for c in "kv" + ("i" if idx else ""):
        now, was = dev[c].cpu(), before[c].clone()
        now[a, :, b] = 0
        was[a, :, b] = 0
        assert torch.equal(now, was), "a row that no token names changed"


def test_parts_alone_in_place_and_empty():
    """K/V without queries, queries without K/V (rotated in place), and calls with nothing to do."""
    gen = torch.Generator().manual_seed(5)
    shape, f = msa.Shape(1, 256, 32, 2), freqs(64, 1.0e4)
    rope = msa.Rope(f.cuda())
    k_new, v_new = (torch.randn((3, 2, 128), generator=gen).bfloat16() for _ in range(2))
    pos = torch.tensor([7, 8, 200], dtype=torch.int32)
    kc, vc = (torch.zeros((1, 2, 256, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tok = (torch.zeros(3, dtype=torch.int32, device="cuda"), pos.cuda())
    assert msa.msa_rope_append(shape, rope, kc, vc, k_new.cuda(), v_new.cuda(), *tok) == (None, None)
    PW.check_rotated(kc.cpu()[0][:, pos.long()].transpose(0, 1), k_new, pos, f, False, 2.0 ** -8)
    q = torch.randn((3, 32, 128), generator=gen).bfloat16()
    qd = q.cuda()
    out, _ = msa.msa_rope_append(shape, rope, q=qd, q_pos=pos.cuda(), q_out=qd)
    assert out is qd
    PW.check_rotated(qd.cpu(), q, pos, f, False, 2.0 ** -8)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, _ = msa.msa_rope_append(shape, rope, kc, vc, k_new[:0].cuda(), v_new[:0].cuda(), none, none, q=q[:0].cuda(),
                                 q_pos=none)
    assert out.shape == (0, 32, 128)
    PW.device_error()


def test_skipped_tokens_and_queries():
    shape, f = msa.Shape(2, 256, 16, 1), freqs(64)
    rope = msa.Rope(f.cuda())
    table = torch.tensor([[0, -1], [7, 1]], dtype=torch.int32)
    pages = msa.Pages(table.cuda(), 2)
    ts = torch.tensor([0, 0, 1, 1, 2, -1, 0, 1], dtype=torch.int32)
    tp = torch.tensor([3, 130, 5, 255, 1, 1, 256, -1], dtype=torch.int32)
    new = torch.randn((8, 1, 128)).bfloat16()
    kc, vc = (torch.zeros((2, 1, 128, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.randn((3, 16, 128)).bfloat16().cuda()
    q_out = torch.full_like(q, 9.0)
    qp = torch.tensor([256, 10, -1], dtype=torch.int32, device="cuda")
    msa.msa_rope_append(shape, rope, kc, vc, new.cuda(), new.cuda(), ts.cuda(), tp.cuda(), q=q, q_pos=qp, q_out=q_out,
                        pages=pages)
    PW.device_error(0x1 | 0x2 | 0x10)
    v = vc.cpu()
    assert torch.equal(v[0, 0, 3], new[0, 0]) and torch.equal(v[1, 0, 127], new[3, 0])
    v[0, 0, 3] = v[1, 0, 127] = 0
    assert not v.any()
    assert bool((q_out[0] == 9).all()) and bool((q_out[2] == 9).all()) and not bool((q_out[1] == 9).all())


@pytest.mark.parametrize("paged,f16", [(False, False), (True, True)])
def test_decode_step_with_rotation(paged, f16):
    """decode_step with the rotation on the way equals decode_step on rows rotated beforehand, bit for bit."""
    gen = torch.Generator().manual_seed(11)
    S, G, cap = 3, 2, 2560
    shape = msa.Shape(S, cap, 32, G)
    rope = msa.Rope(freqs(64).cuda())
    rows = (S * cap // 128 + 1, G, 128) if paged else (S, G, cap)
    pages = None
    if paged:
        table, n = PW.random_pages(S, cap // 128, 1, gen)
        pages = msa.Pages(table.cuda(), n)
    base = dict(idx_k_cache=torch.randn(rows + (128,), generator=gen).to(torch.float16 if f16 else torch.float32),
                k_cache=torch.randn(rows + (128,), generator=gen).bfloat16(),
                v_cache=torch.randn(rows + (128,), generator=gen).bfloat16())
    pos = torch.tensor([2400, 100, 2559], dtype=torch.int32, device="cuda")
    stream = torch.arange(3, dtype=torch.int32, device="cuda")
    new = dict(tok_stream=stream, tok_pos=pos, q_stream=stream, q_pos=pos,
               idx_k_new=torch.randn((3, G, 128), generator=gen).cuda() / math.sqrt(128),
               k_new=torch.randn((3, G, 128), generator=gen).bfloat16().cuda(),
               v_new=torch.randn((3, G, 128), generator=gen).bfloat16().cuda(),
               idx_q=torch.randn((3, G, 128), generator=gen).cuda() / math.sqrt(128),
               q=torch.randn((3, 32, 128), generator=gen).bfloat16().cuda())
    c1, c2 = ({k: v.cuda() for k, v in base.items()} for _ in range(2))
    got = msa.decode_step(shape, c1, new, pages=pages, rope=rope)
    # the rows rotated beforehand: through one-token caches
    flat = msa.Shape(3, cap, 32, G)
    kc, vc = (torch.zeros((3, G, cap, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ic = torch.zeros((3, G, cap, 128), device="cuda")
    q, iq = msa.msa_rope_append(flat, rope, kc, vc, new["k_new"], new["v_new"], stream, pos, q=new["q"], q_pos=pos,
                                idx_k_cache=ic, idx_k_new=new["idx_k_new"], idx_q=new["idx_q"])
    at = (stream.long(), slice(None), pos.long())
    turned = dict(new, k_new=kc[at].contiguous(), idx_k_new=ic[at].contiguous(), q=q, idx_q=iq)
    want = msa.decode_step(shape, c2, turned, pages=pages)
    PW.device_error()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for k in c1:
        assert torch.equal(c1[k], c2[k])
    # captured and replayed
    c3 = {k: v.cuda() for k, v in base.items()}
    graph = msa.DecodeGraph(shape, c3, new, pages=pages, rope=rope)
    assert torch.equal(graph.replay(), want[0])
    PW.device_error()
