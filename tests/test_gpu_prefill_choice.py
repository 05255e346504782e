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


# ---- caches whose expansion is larger than the workspace's 1 GiB: 2^21 slots of one group -----------------------------
def codes(gen, *rows):
    """Random e4m3 codes (no NaN) and scales of [..][rows][128] caches, on the GPU."""
    x = torch.randint(0, 254, (*rows, 128), generator=gen, device="cuda", dtype=torch.uint8)
    return torch.where(x >= 127, x + 1, x)


def large_and_small(S, G, small, large, gen):
    """Contiguous caches of the same rows in capacities ``small`` and ``large`` (NaN codes and scales behind them)."""
    out = ([], [])
    for _ in range(2):
        x, sc = codes(gen, S, G, small), torch.exp2(torch.randint(-9, -5, (S, G, small // 128), generator=gen, device="cuda").float())
        big = torch.full((S, G, large, 128), 0x7f, dtype=torch.uint8, device="cuda")
        big[:, :, :small] = x
        bsc = torch.full((S, G, large // 128), math.nan, device="cuda")
        bsc[:, :, :small // 128] = sc
        out[0].append((x.view(F8), sc))
        out[1].append((big.view(F8), bsc))
    return out


def call(form, mode, shape, q, kv, stream, pos, sel, pages=None, window=1000, sink=130):
    if form == "window":
        fn = msa.msa_window_attn_prefill if mode == "prefill" else msa.msa_window_attn_decode
        return fn(shape, q, kv[0][0], kv[1][0], stream, pos, window, sink, pages=pages, k_scale=kv[0][1], v_scale=kv[1][1])
    fn = msa.msa_sparse_attn_prefill_fp8 if mode == "prefill" else msa.msa_sparse_attn_decode_fp8
    return fn(shape, q, kv[0][0], kv[1][0], kv[0][1], kv[1][1], sel, stream, pos, pages=pages)


def selections(n, G, pos, gen):
    """16 visible blocks (or all) of each (query, group), the local one among them."""
    nblk = int(pos.max()) // 128 + 1
    b = torch.arange(nblk, device="cuda")
    score = torch.rand((n, G, nblk), generator=gen, device="cuda")
    local = (pos // 128)[:, None, None]
    score = torch.where(b == local, 2.0, torch.where(b < local, score, -1.0))
    best = score.topk(min(16, nblk), 2)
    sel = torch.where(best.values >= 0, best.indices, -1).int()
    return torch.nn.functional.pad(sel, (0, 16 - sel.shape[2]), value=-1).contiguous()


@pytest.mark.parametrize("form", ["window", "selection"])
def test_large_cache_expands_what_the_call_sees(form):
    """2112 queries of 33 streams near the front of caches of 33 x 16384: the same bits as in caches of 33 x 2048, which
    expand in place, with a workspace of little more than 1 GiB."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    S, G, small, large, per = 33, 4, 2048, 16384, 64
    assert S * G * large * 512 > 1 << 30 > S * G * small * 512
    kv = large_and_small(S, G, small, large, gen)
    stream = torch.arange(S, device="cuda").repeat_interleave(per).int()
    pos = (torch.arange(S, device="cuda")[:, None] * 53 % (small - per) + torch.arange(per, device="cuda")).flatten().int()
    n = S * per
    q = torch.randn((n, 16 * G, 128), generator=gen, device="cuda").bfloat16()
    sel = selections(n, G, pos, gen)
    assert (1 << 30) < msa.msa_attn_workspace_bytes(msa.Shape(S, large), n, msa.MODE_PREFILL, True) < 1.1 * (1 << 30)
    want = call(form, "prefill", msa.Shape(S, small), q, kv[0], stream, pos, sel)
    for _ in range(2):
        assert torch.equal(call(form, "prefill", msa.Shape(S, large), q, kv[1], stream, pos, sel), want)
    one = call(form, "decode", msa.Shape(S, small), q, kv[0], stream, pos, sel)
    assert bool((want != one).any())          # (the kernels round differently: it was the tiles that ran)
    PW.device_error()


@pytest.mark.parametrize("form", ["window", "selection"])
def test_large_cache_that_sees_too_much(form):
    """More visible blocks than the workspace holds: the single-query kernel answers, bit for bit, also captured, and
    next to a call that fits."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    S, G, cap, per = 33, 4, 16384, 64
    shape = msa.Shape(S, cap)
    kv = [(codes(gen, S, G, cap).view(F8), torch.exp2(torch.randint(-9, -5, (S, G, cap // 128), generator=gen, device="cuda").float()))
          for _ in range(2)]
    stream = torch.arange(S, device="cuda").repeat_interleave(per).int()
    n = S * per
    far = (cap - per + torch.arange(per, device="cuda")).repeat(S).int()
    near = far - cap + 3000
    pos = far.clone()
    q = torch.randn((n, 16 * G, 128), generator=gen, device="cuda").bfloat16()
    sel = torch.empty((n, G, 16), dtype=torch.int32, device="cuda")
    ws = torch.empty(msa.msa_attn_workspace_bytes(shape, n, msa.MODE_PREFILL, True), dtype=torch.uint8, device="cuda")

    def run(mode):
        extra = dict(window=cap, sink=0) if form == "window" else {}
        return call(form, mode, shape, q, kv, stream, pos, sel, **extra)
    want = {}
    for name, p in (("far", far), ("near", near)):
        pos.copy_(p)
        sel.copy_(selections(n, G, p, gen))
        want[name] = (run("prefill"), run("decode"), sel.clone())
    assert torch.equal(want["far"][0], want["far"][1])
    assert bool((want["near"][0] != want["near"][1]).any())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run("prefill")
    for name, p in (("near", near), ("far", far), ("near", near)):
        pos.copy_(p)
        sel.copy_(want[name][2])
        graph.replay()
        assert torch.equal(out, want[name][0])
    PW.device_error()
    del ws


@pytest.mark.parametrize("form", ["window", "selection"])
def test_large_pool_with_unmapped_and_shared_pages(form):
    """Two streams over a pool of 4200 pages (more than the workspace's), one page of both, one missing, one out of
    range: as over a pool of 40."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    G, per, nblk = 4, 700, 16
    kv = [(codes(gen, 40, G, 128).view(F8), torch.exp2(torch.randint(-9, -5, (40, G), generator=gen, device="cuda").float()))
          for _ in range(2)]
    at = torch.randperm(4200, generator=gen, device="cuda")[:40]
    big = []
    for x, sc in kv:
        y = torch.full((4200, G, 128, 128), 0x7f, dtype=torch.uint8, device="cuda")
        y[at] = x.view(torch.uint8)
        s = torch.full((4200, G), math.nan, device="cuda")
        s[at] = sc
        big.append((y.view(F8), s))
    table = torch.randperm(40, generator=gen, device="cuda")[:2 * nblk].view(2, nblk).int()
    table[1, 2] = table[0, 2]
    far = at[table.long()].int()
    for t, n_pages in ((table, 40), (far, 4200)):
        t[0, 9] = -1
        t[1, 11] = n_pages
    stream = torch.tensor([0, 1], device="cuda").repeat_interleave(per).int()
    pos = torch.cat((torch.arange(1300, 1300 + per, device="cuda"), torch.arange(1100, 1100 + per, device="cuda"))).int()
    q = torch.randn((2 * per, 16 * G, 128), generator=gen, device="cuda").bfloat16()
    sel = selections(2 * per, G, pos, gen)
    shape = msa.Shape(2, nblk * 128)
    want = call(form, "prefill", shape, q, kv, stream, pos, sel, msa.Pages(table, 40))
    PW.device_error(0x10)
    got = call(form, "prefill", shape, q, big, stream, pos, sel, msa.Pages(far, 4200))
    PW.device_error(0x10)
    assert torch.equal(got, want) and bool(want.isfinite().all())
    # the workspace holds what the table can name, not the pool
    assert msa.msa_attn_workspace_bytes(shape, 2 * per, msa.MODE_PREFILL, True, msa.Pages(far, 4200)) < 2 * nblk * G * 128 * 512 + (4 << 20)


@pytest.mark.parametrize("S,per,cap", [(1, 2048, 131072), (16, 128, 16384)])
def test_selection_chooses_by_what_the_queries_see(S, per, cap):
    """2048 queries of one stream or of 16, near the front (the tiles answer) and far behind (the cluster kernel
    does): the bits of each kernel, in one captured call whose positions change."""
    gen = torch.Generator(device="cuda").manual_seed(11 + S)
    G, small = 4, 4096
    shape, n = msa.Shape(S, cap), S * per
    kv = [(codes(gen, S, G, cap).view(F8), torch.exp2(torch.randint(-9, -5, (S, G, cap // 128), generator=gen, device="cuda").float()))
          for _ in range(2)]
    front = [(x.view(torch.uint8)[:, :, :small].contiguous().view(F8), s[:, :, :small // 128].contiguous()) for x, s in kv]
    stream = torch.arange(S, device="cuda").repeat_interleave(per).int()
    near = (1900 + torch.arange(per, device="cuda")).repeat(S).int()
    far = near + (cap - 1900 - per)
    q = torch.randn((n, 16 * G, 128), generator=gen, device="cuda").bfloat16()
    pos, sel = near.clone(), selections(n, G, near, gen)
    want = {}
    for name, p in (("near", near), ("far", far)):
        pos.copy_(p)
        sel.copy_(selections(n, G, p, gen))
        one = call("selection", "decode", shape, q, kv, stream, pos, sel)
        got = call("selection", "prefill", shape, q, kv, stream, pos, sel)
        want[name] = (got, sel.clone())
        assert torch.equal(got, one) == (name == "far")
    sel.copy_(want["near"][1])
    # the same rows in a cache of the context's size, where the host is sure of the tiles
    assert torch.equal(call("selection", "prefill", msa.Shape(S, small), q, front, stream, near, sel), want["near"][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call("selection", "prefill", shape, q, kv, stream, pos, sel)
    for name, p in (("near", near), ("far", far), ("near", near)):
        pos.copy_(p)
        sel.copy_(want[name][1])
        graph.replay()
        assert torch.equal(out, want[name][0])
    PW.device_error()


def one_prompt_in_many_slots(slots, cap, per, gen, f8):
    """The queries of one prompt in a pool that ``slots`` streams share, and as the only stream of a small one: (shape,
    pages, stream) of both, and the caches, positions and queries."""
    G, nblk, n_pages = 4, cap // 128, cap // 128 + 3
    kv = []
    for _ in range(2):
        if f8:
            kv.append((codes(gen, n_pages, G, 128).view(F8), torch.exp2(torch.randint(-9, -5, (n_pages, G), generator=gen,
                                                                                      device="cuda").float())))
        else:
            kv.append((torch.randn((n_pages, G, 128, 128), generator=gen, device="cuda").bfloat16(), None))
    table = torch.full((slots, nblk), -1, dtype=torch.int32, device="cuda")
    mine = slots * 2 // 3
    table[mine] = torch.randperm(n_pages, generator=gen, device="cuda")[:nblk].int()
    alone = msa.Pages(table[mine:mine + 1].contiguous(), n_pages)
    pos = (cap - per + torch.arange(per, device="cuda")).int()
    q = torch.randn((per, 16 * G, 128), generator=gen, device="cuda").bfloat16()
    zero = torch.zeros(per, dtype=torch.int32, device="cuda")
    return ((msa.Shape(slots, cap), msa.Pages(table, n_pages), zero + mine), (msa.Shape(1, cap), alone, zero)), kv, pos, q


def test_one_prompt_in_a_cache_of_many_slots():
    """1024 queries of one stream, window over bf16: the tiles answer, however many slots the cache has."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    (many, alone), kv, pos, q = one_prompt_in_many_slots(512, 2048, 1024, gen, False)
    run = lambda mode, at: call("window", mode, at[0], q, kv, at[2], pos, None, at[1])
    want = run("prefill", alone)
    assert torch.equal(run("prefill", many), want)
    assert bool((run("decode", alone) != want).any())
    PW.device_error()


@pytest.mark.parametrize("form", ["window", "selection"])
def test_8bit_prompts_in_a_cache_of_many_slots(form):
    """1024 queries over 8-bit pages of 256 slots, 4 per slot: those of one stream take the tiles, those of all streams
    the cluster kernel, in one captured call; without a workspace the cluster kernel answers."""
    gen = torch.Generator(device="cuda").manual_seed(22)
    slots, cap, n = 256, 2048, 1024
    (many, alone), kv, pos, q = one_prompt_in_many_slots(slots, cap, n, gen, True)
    shape, pages, stream = many
    pages.block_table[:] = pages.block_table[slots * 2 // 3]               # the other slots share its pages
    sel = selections(n, 4, pos, gen)
    run = lambda mode, at: call(form, mode, at[0], q, kv, at[2], pos, sel, at[1])
    want, one = run("prefill", alone), run("decode", alone)
    assert bool((want != one).any())
    scattered = (torch.arange(n, device="cuda") % slots).int()
    mine = stream.clone()
    graph = torch.cuda.CUDAGraph()
    assert torch.equal(run("prefill", many), want)
    with torch.cuda.graph(graph):
        out = run("prefill", many)
    for s, result in ((mine, want), (scattered, one), (mine, want)):
        stream.copy_(s)
        graph.replay()
        assert torch.equal(out, result)
    if form == "selection":
        need = msa.msa_attn_workspace_bytes(shape, n, msa.MODE_PREFILL, True, pages)
        large = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
        for ws, result in ((None, one), (large[:need - 1], one), (large[16:], one), (large[:need], want)):
            out.fill_(math.nan)
            assert raw_sparse(shape, q, [kv[0][0], kv[1][0], kv[0][1], kv[1][1]], sel, stream, pos, 128 ** -0.5, out, ws, pages) == 0
            assert torch.equal(out, result)
    PW.device_error()


def test_a_nan_that_one_of_two_streams_sees():
    """Two streams share a page, only one of them sees the row whose V is NaN: its queries say so, in every call, and the
    other's are as without it (window over 8-bit pages, expanded in place)."""
    gen = torch.Generator(device="cuda").manual_seed(31)
    G, n = 4, 512
    shape = msa.Shape(2, 512)
    kv = [(codes(gen, 6, G, 128).view(F8), torch.full((6, G), 2.0 ** -8, device="cuda")) for _ in range(2)]
    table = torch.tensor([[3, 1, -1, -1], [3, 1, 5, 0]], dtype=torch.int32, device="cuda")
    stream = (torch.arange(n, device="cuda") // 256).int()
    i = torch.arange(256, device="cuda")
    pos = torch.cat((i % 60 + 130, 384 + i % 120)).int()                  # stream 0 ends inside the second page
    q = torch.randn((n, 16 * G, 128), generator=gen, device="cuda").bfloat16()
    run = lambda: call("window", "prefill", shape, q, kv, stream, pos, None, msa.Pages(table, 6), window=512, sink=0)
    clean = run()
    kv[1][0].view(torch.uint8)[1, 2, 100, 7] = 0x7f                         # slot 228 of both, group 2
    for _ in range(20):
        out = run()
        bad = out.isnan()
        assert bool(bad[256:, 32:48, 7].all())
        bad[256:, 32:48, 7] = False
        assert not bool(bad.any())
        assert torch.equal(out[:256], clean[:256])
    PW.device_error()


def test_a_block_named_twice_counts_once():
    """Selections that name a block several times, in single-query and prompt calls, of the tiles and of the cluster
    kernel: the rows of the blocks in sel, each once."""
    gen = torch.Generator().manual_seed(41)
    G, cap, n = 4, 2048, 256
    shape = msa.Shape(1, cap)
    kv = caches(1, G, cap, gen)
    pos = (1500 + torch.arange(n)).int()
    stream = torch.zeros(n, dtype=torch.int32)
    sel = torch.randint(-1, 11, (n, G, 16), generator=gen).int()
    sel[::3, :, 5] = sel[::3, :, 9]
    sel[1] = 7
    q = torch.randn((n, 16 * G, 128), generator=gen).bfloat16()
    once = sel.clone()
    for i in range(n):
        for g in range(G):
            seen = set()
            for j in range(16):
                b = int(sel[i, g, j])
                once[i, g, j] = -1 if b in seen else b
                seen.add(b)
    dev = [x.cuda() for x in (kv[0][0], kv[1][0], kv[0][1], kv[1][1])]
    some = torch.arange(0, n, 9)
    want = C.selected_attention(q[some], kv[0][2], kv[1][2], once[some], stream[some], pos[some], 128 ** -0.5)
    for fn in (msa.msa_sparse_attn_decode_fp8, msa.msa_sparse_attn_prefill_fp8):
        a, b = (fn(shape, q.cuda(), dev[0].view(F8), dev[1].view(F8), dev[2], dev[3], x.cuda(), stream.cuda(), pos.cuda())
                for x in (sel, once))
        PW.check_attention(a[some.cuda()], *want, PW.P_BF16, 0.0, PW.P_FP16)
        PW.check_attention(b[some.cuda()], *want, PW.P_BF16, 0.0, PW.P_FP16)
    PW.device_error()
