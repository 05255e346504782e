"""Sliding-window attention with sinks on the GPU against the float64 oracle: bf16 and 8-bit caches, contiguous and
paged, single queries and batches, windows from one token to the whole cache, sinks before and inside the window."""
import math

import pytest
import torch

import block_sparse_attention_maxpool_b200 as msa
from oracle import cache_ops as C
from tests import parity_window as PW
from tests.test_gpu_rope_append import freqs

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_attention_maxpool_b200 import build as msa_build
    msa_build.build()
    msa.msa_get_device_error()


def attend(mode, *a, **k):
    return (msa.msa_window_attn_prefill if mode == "prefill" else msa.msa_window_attn_decode)(*a, **k)


def make(S, G, cap, f8, gen):
    """K and V: (as stored, scales or None, the float64 rows they stand for)."""
    out = []
    for _ in range(2):
        x = torch.randn((S, G, cap, 128), generator=gen)
        if f8:
            x = x * torch.exp2(torch.randint(-3, 4, (S, G, cap // 128, 1, 1), generator=gen).float()).expand(
                -1, -1, -1, 128, 1).reshape(S, G, cap, 1)
            q8, sc = PW.quantise(x)
            out.append((q8, sc, C.fp8_values(q8, sc)))
        else:
            out.append((x.bfloat16(), None, x.bfloat16().double()))
    return out


def run(mode, shape, q, kv, stream, pos, window, sink, table=None, n_pages=0, poison=True, scale=None, out=None):
    """The call on device copies; every row that no query sees is NaN there."""
    f8 = kv[0][1] is not None
    args, scales = [], {}
    for name, (x, sc, _) in zip("kv", kv):
        raw = (x.view(torch.uint8) if f8 else x).clone()
        if poison:
            seen = torch.zeros(raw.shape[0], raw.shape[2], dtype=torch.bool)
            for i in range(pos.numel()):
                s, p = int(stream[i]), int(pos[i])
                if 0 <= s < raw.shape[0] and 0 <= p < raw.shape[2]:
                    seen[s, C.visible_slots(p, window, sink)] = True
            raw.permute(0, 2, 1, 3)[~seen] = 0x7f if f8 else math.nan
        if table is not None:
            raw = PW.to_pool(raw, table, n_pages, 0x7f if f8 else math.nan)
        args.append(raw.cuda().view(F8) if f8 else raw.cuda())
        if f8:
            scales[name + "_scale"] = (sc if table is None else PW.scale_pool(sc, table, n_pages)).cuda()
    pages = None if table is None else msa.Pages(table.cuda(), n_pages)
    return attend(mode, shape, q.cuda(), *args, stream.cuda(), pos.cuda(), window, sink, softmax_scale=scale, out=out,
                  pages=pages, **scales)


CASES = [
    # S, G, cap, positions (stream, position), window, sink
    (1, 4, 128, [(0, 0)], 1, 0),
    (1, 1, 128, [(0, 127)], 1, 1),
    (1, 4, 256, [(0, 200)], 64, 4),
    (2, 4, 1024, [(0, 1023), (1, 511), (0, 63), (1, 64)], 300, 4),
    (1, 2, 4096, [(0, 4095)], 4096, 0),
    (1, 2, 2048, [(0, 2047), (0, 2000)], 1 << 30, 0),
    (3, 1, 1536, [(2, 1500), (0, 7), (1, 900)], 129, 300),
    (2, 16, 640, [(0, 600), (1, 601)], 100, 128),
    (1, 4, 1024, [(0, p) for p in range(480, 560)], 200, 3),
    (2, 2, 2048, [(s, p) for s in (0, 1) for p in range(900 + 7 * s, 1041)], 257, 129),
    (4, 1, 768, [(s, p) for p in (5, 700, 300) for s in (3, 1, 2, 0)], 65, 0),
    (2, 3, 896, [(i % 2, (37 * i) % 896) for i in range(70)], 150, 64),
    (2, 2, 896, [(i % 2, (37 * i) % 896) for i in range(150)], 150, 64),
    # enough queries for the tiles: in order, over two streams, scattered (windows with gaps between them)
    (1, 4, 1024, [(0, p) for p in range(480, 779)], 200, 3),
    (2, 4, 1408, [(s, p) for s in (0, 1) for p in range(900 + 7 * s, 1041)], 257, 129),
    (2, 4, 896, [(i % 2, (37 * i) % 896) for i in range(300)], 10, 64),
    (3, 4, 1280, [(i % 3, (97 * i) % 1280) for i in range(333)], 700, 0),
]


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_oracle(mode, f8, paged, case):
    S, G, cap, at, window, sink = CASES[case]
    gen = torch.Generator().manual_seed(1000 + case)
    shape = msa.Shape(S, cap, 16 * G, G)
    kv = make(S, G, cap, f8, gen)
    stream, pos = (torch.tensor(x, dtype=torch.int32) for x in zip(*at))
    q = (2 * torch.randn((len(at), 16 * G, 128), generator=gen)).bfloat16()
    table, n_pages = PW.random_pages(S, cap // 128, 2, gen) if paged else (None, 0)
    want, spread, reach = C.window_attention(q, kv[0][2], kv[1][2], stream, pos, window, sink, 128 ** -0.5)
    got = run(mode, shape, q, kv, stream, pos, window, sink, table, n_pages)
    PW.device_error()
    PW.check_attention(got, want, spread, reach, PW.P_BF16, 0.0, PW.norm_of(f8))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("S,G,cap,window,sink", [(1, 1, 16384, 16000, 4), (2, 4, 8192, 5000, 100), (40, 4, 1024, 700, 4)])
def test_long_windows_split_over_ctas(f8, S, G, cap, window, sink):
    """One query per stream at odd places: every cluster size the host picks."""
    gen = torch.Generator().manual_seed(S + cap)
    shape = msa.Shape(S, cap, 16 * G, G)
    kv = make(S, G, cap, f8, gen)
    stream = torch.arange(S, dtype=torch.int32)
    pos = torch.randint(cap // 2, cap, (S,), generator=gen).int()
    q = torch.randn((S, 16 * G, 128), generator=gen).bfloat16()
    want, spread, reach = C.window_attention(q, kv[0][2], kv[1][2], stream, pos, window, sink, 128 ** -0.5)
    got = run("decode", shape, q, kv, stream, pos, window, sink)
    again = run("decode", shape, q, kv, stream, pos, window, sink)
    PW.device_error()
    PW.check_attention(got, want, spread, reach, PW.P_BF16, 0.0, PW.norm_of(f8))
    assert torch.equal(got, again)


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("f8", [False, True])
def test_steep_scores(mode, f8):
    """Scores hundreds apart, the largest early, late and in the sinks, and a negative and a zero scale."""
    gen = torch.Generator().manual_seed(77)
    G = 4
    shape = msa.Shape(1, 1024, 16 * G, G)
    kv = make(1, G, 1024, f8, gen)
    n = 259 if mode == "prefill" else 3
    pos = torch.cat((torch.tensor([1023, 600, 300]), torch.arange(700, 700 + n - 3))).int()
    stream = torch.zeros(n, dtype=torch.int32)
    q = (40 * torch.randn((n, 16 * G, 128), generator=gen)).bfloat16()
    for scale in (128 ** -0.5, -0.05, 0.0):
        want, spread, reach = C.window_attention(q, kv[0][2], kv[1][2], stream, pos, 500, 10, scale)
        got = run(mode, shape, q, kv, stream, pos, 500, 10, scale=scale)
        PW.check_attention(got, want, spread, reach, PW.P_BF16, 0.0, PW.norm_of(f8))
    PW.device_error()


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("f8", [False, True])
def test_invalid_queries_and_unmapped_pages(mode, f8):
    gen = torch.Generator().manual_seed(9)
    S, G, cap = 2, 4, 640
    shape = msa.Shape(S, cap, 64, G)
    kv = make(S, G, cap, f8, gen)
    table, n_pages = PW.random_pages(S, 5, 1, gen)
    bad = table.clone()
    bad[0, 3] = -1                   # inside the window of query 0
    bad[1, 0] = n_pages              # the sinks of stream 1
    bad[1, 1] = 1 << 30              # the window's first rows of query 5: 500 - 250 < j, j in block 1 is 251 .. 255
    times = 40 if mode == "prefill" else 1
    stream = torch.tensor([0, 2, -1, 0, 1, 1, 0] * times, dtype=torch.int32)
    pos = torch.tensor([600, 5, 5, 640, -7, 500, 3] * times, dtype=torch.int32)
    n = 7 * times
    q = torch.randn((n, 64, 128), generator=gen).bfloat16()
    window, sink = 250, 70
    hidden = [(0, j) for j in range(384, 512)] + [(1, j) for j in range(0, 256)]
    want, spread, reach = C.window_attention(q, kv[0][2], kv[1][2], stream, pos, window, sink, 128 ** -0.5, hidden)
    out = torch.full((n, 64, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    args = []
    for x, sc, _ in kv:
        raw = x.view(torch.uint8) if f8 else x
        pool = PW.to_pool(raw, table, n_pages, 0x7f if f8 else math.nan).cuda()
        args.append((pool.view(F8) if f8 else pool, PW.scale_pool(sc, table, n_pages).cuda() if f8 else None))
    attend(mode, shape, q.cuda(), args[0][0], args[1][0], stream.cuda(), pos.cuda(), window, sink, out=out,
           pages=msa.Pages(bad.cuda(), n_pages), k_scale=args[0][1], v_scale=args[1][1])
    PW.device_error(0x1 | 0x10)
    PW.check_attention(out, want, spread, reach, PW.P_BF16, 0.0, PW.norm_of(f8))
    assert not bool(out[(stream < 0) | (stream > 1) | (pos < 0) | (pos >= cap)].any())


@pytest.mark.parametrize("prefill,f8", [(False, False), (True, False), (False, True), (True, True)])
def test_window_steps_in_a_row(prefill, f8):
    """Several steps of a local layer (append with rotation, then attention), on a stream of their own, and the last
    one captured and replayed: each against the oracle on the caches it left."""
    gen = torch.Generator().manual_seed(31)
    S, G, cap, n_new = 3, 4, 1024, 90 if prefill else 1
    shape = msa.Shape(S, cap, 64, G)
    rope = msa.Rope(freqs(128, 1.0e4).cuda(), True)
    table, n_pages = PW.random_pages(S, cap // 128, 1, gen)
    pages = msa.Pages(table.cuda(), n_pages)
    if f8:
        c = msa.fp8_caches(shape, "cuda", n_pages)
    else:
        c = {k: torch.zeros((n_pages, G, 128, 128), dtype=torch.bfloat16, device="cuda") for k in ("k_cache", "v_cache")}
    side = torch.cuda.Stream()
    at = [0, 100, 500]

    def logical():
        out = []
        for x in "kv":
            pool = c[x + "_cache"].cpu()
            pool = pool.double() * (c[x + "_scale"].cpu().double()[..., None, None] if f8 else 1.0)
            out.append(torch.stack([torch.cat([pool[int(table[s, b])] for b in range(cap // 128)], 1) for s in range(S)]))
        return out

    def inputs():
        stream = torch.arange(S).repeat_interleave(n_new).int()
        pos = torch.cat([torch.arange(p, p + n_new) for p in at]).int()
        n = S * n_new
        d = dict(tok_stream=stream, tok_pos=pos, q_stream=stream, q_pos=pos,
                 k_new=torch.randn((n, G, 128), generator=gen).bfloat16(),
                 v_new=torch.randn((n, G, 128), generator=gen).bfloat16(),
                 q=torch.randn((n, 64, 128), generator=gen).bfloat16())
        return {k: v.cuda() for k, v in d.items()}

    def check(out, new):
        q, _ = msa.msa_rope_append(shape, rope, q=new["q"], q_pos=new["q_pos"])
        k, v = logical()
        want = C.window_attention(q.cpu(), k, v, new["q_stream"].cpu(), new["q_pos"].cpu(), 150, 20, 128 ** -0.5)
        PW.check_attention(out, *want, PW.P_BF16, 0.0, PW.norm_of(f8))
    for _ in range(3):
        new = inputs()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out = msa.window_step(shape, c, new, 150, 20, prefill=prefill, pages=pages, rope=rope)
        torch.cuda.current_stream().wait_stream(side)
        check(out, new)
        at = [p + n_new for p in at]
    new = inputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = msa.window_step(shape, c, new, 150, 20, prefill=prefill, pages=pages, rope=rope)
    for _ in range(2):                       # the second replay appends the same rows again
        graph.replay()
        check(out, new)
    # new contents in the captured buffers
    at = [p + n_new for p in at]
    for k, v in inputs().items():
        new[k].copy_(v)
    graph.replay()
    check(out, new)
    PW.device_error()


def test_two_calls_at_once():
    """Two decode calls on two streams share nothing."""
    gen = torch.Generator().manual_seed(2)
    shape = msa.Shape(1, 4096, 64, 4)
    kv = make(1, 4, 4096, False, gen)
    k, v = kv[0][0].cuda(), kv[1][0].cuda()
    q = torch.randn((1, 64, 128), generator=gen).bfloat16().cuda()
    zero, pos = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 4000, dtype=torch.int32, device="cuda")
    want = msa.msa_window_attn_decode(shape, q, k, v, zero, pos, 3000, 4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(msa.msa_window_attn_decode(shape, q, k, v, zero, pos, 3000, 4))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got[0] + got[1])


@pytest.mark.parametrize("form", ["window", "append", "rope", "decode_step"])
def test_memory_of_a_call_on_another_stream(form):
    """A call launched on another stream than the current one: memory that it allocated for itself is not handed out
    again while its kernels are still waiting there."""
    S, G, cap, n = 2, 4, 2048, 2048
    shape = msa.Shape(S, cap, 64, G)
    gen = torch.Generator(device="cuda").manual_seed(8)
    stream = (torch.arange(n, device="cuda") * S // n).int()
    pos = (torch.arange(n, device="cuda") % (n // S) + 500).int()
    randn = lambda *d, t=torch.bfloat16: torch.randn(d, device="cuda", generator=gen).to(t)
    new = dict(tok_stream=stream, tok_pos=pos, q_stream=stream, q_pos=pos, k_new=randn(n, G, 128), v_new=randn(n, G, 128),
               q=randn(n, 64, 128), idx_k_new=randn(n, G, 128, t=torch.float32), idx_q=randn(n, G, 128, t=torch.float32))
    rope = msa.Rope(10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64))

    def call(side):
        caches = msa.fp8_caches(shape, "cuda")
        for c, size in (("k", 0x60), ("v", 0x48)):
            caches[c + "_cache"].view(torch.uint8).copy_(torch.arange(S * G * cap * 128, device="cuda").view(S, G, cap, 128)
                                                         * 37 % size)
            caches[c + "_scale"].fill_(2.0 ** -6)
        caches["idx_k_cache"] = torch.zeros((S, G, cap, 128), device="cuda")
        torch.cuda.synchronize()
        if side is not None:
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
        out = torch.zeros_like(new["q"])
        bufs = {"out": out, "workspace": torch.zeros(msa.msa_workspace_bytes(shape, n, msa.MODE_PREFILL), dtype=torch.uint8,
                                                     device="cuda"),
                "block_scores": torch.zeros((n, G, cap // 128), device="cuda")}
        torch.cuda.synchronize() if side is None else torch.cuda.current_stream().synchronize()
        if form == "window":
            msa.msa_window_attn_prefill(shape, new["q"], caches["k_cache"], caches["v_cache"], stream, pos, 300, 4, out=out,
                                        stream=side, k_scale=caches["k_scale"], v_scale=caches["v_scale"])
        elif form == "append":
            msa.msa_kv_append_fp8(shape, caches["k_cache"], caches["v_cache"], caches["k_scale"], caches["v_scale"],
                                  new["k_new"], new["v_new"], stream, pos, rope, stream=side)
        elif form == "rope":
            msa.window_step(shape, caches, new, 300, 4, {"out": out}, side, True, None, rope)
        else:
            kept = msa.decode_step(shape, caches, new, bufs, side, True, None, rope)     # noqa: F841 (sel, n_sel)
        # everything that the call let go of, taken again and overwritten at once
        junk = [torch.full((m,), 1, dtype=torch.uint8, device="cuda") for k in range(8, 27) for m in (1 << k,) * 3]
        torch.cuda.synchronize()
        PW.device_error()
        del junk
        return [out] + [caches[c].view(torch.uint8) for c in ("k_cache", "v_cache")] + [caches["k_scale"], caches["v_scale"]]

    want = call(None)
    got = call(torch.cuda.Stream())
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("f8", [False, True])
def test_windows_past_32_bits(mode, f8):
    """A window or a count of sinks larger than the capacity means the capacity, however large it is."""
    S, G, cap, n = 1, 4, 384, 300
    shape = msa.Shape(S, cap, 64, G)
    gen = torch.Generator().manual_seed(9)
    kv = make(S, G, cap, f8, gen)
    q = torch.randn((n, 64, 128), generator=gen).bfloat16()
    stream, pos = torch.zeros(n, dtype=torch.int32), (torch.arange(n) + cap - n).int()
    for huge, same in (((2 ** 31 - 1, 0), (cap, 0)), ((2 ** 32, 0), (cap, 0)), ((2 ** 32 + 5, 2 ** 40), (cap, cap)),
                       ((5, 2 ** 32), (5, cap))):
        want = run(mode, shape, q, kv, stream, pos, *same, poison=False)
        assert torch.equal(run(mode, shape, q, kv, stream, pos, *huge, poison=False), want)


def test_large_offsets():
    """A pool of more than 2^31 bytes: pages beyond 32-bit byte offsets."""
    gen = torch.Generator().manual_seed(4)
    G, n_pages = 16, 4500                               # 4500 * 16 * 128 * 256 B = 2.4 GB a cache
    shape = msa.Shape(1, 512, 256, G)
    k, v = (torch.zeros((n_pages, G, 128, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.tensor([[n_pages - 1, 4400, 3, n_pages - 2]], dtype=torch.int32)
    kl, vl = (torch.randn((1, G, 512, 128), generator=gen).bfloat16() for _ in range(2))
    for b in range(4):
        k[int(ids[0, b])], v[int(ids[0, b])] = kl[0, :, b * 128:b * 128 + 128].cuda(), vl[0, :, b * 128:b * 128 + 128].cuda()
    for mode in ("decode", "prefill"):
        n = 2 if mode == "decode" else 40
        q = torch.randn((n, 256, 128), generator=gen).bfloat16()
        stream, pos = torch.zeros(n, dtype=torch.int32), torch.linspace(511, 400, n).int()
        want = C.window_attention(q, kl, vl, stream, pos, 300, 4, 128 ** -0.5)
        got = attend(mode, shape, q.cuda(), k, v, stream.cuda(), pos.cuda(), 300, 4, pages=msa.Pages(ids.cuda(), n_pages))
        PW.check_attention(got, *want, PW.P_BF16)
    PW.device_error()


@pytest.mark.parametrize("spread_v", [False, True])
def test_far_apart_scales(spread_v):
    """8-bit blocks whose K and V scales differ by up to 2^60 (a block of zeros, a block with a zero scale among them),
    so that the block with the largest values and the one with the largest weights are different ones."""
    gen = torch.Generator().manual_seed(15)
    shape = msa.Shape(1, 1280, 16, 1)
    S = [1.0, 2.0 ** -40, 2.0 ** 20, 0.0, 2.0 ** -20, 2.0 ** -100, 3.0, 2.0 ** 10, 0.7, 1.3]
    kv = []
    for i in range(2):
        q8, _ = PW.quantise(torch.randn((1, 1, 1280, 128), generator=gen))
        q8 = q8.view(torch.uint8).clone()
        q8[:, :, 640:768] = 0                                   # block 5: zeros
        q8 = q8.view(F8)
        sc = torch.tensor(S if i == 1 or not spread_v else [1.0 / 448] * 10).view(1, 1, 10)
        sc = sc / (448 if i else 2.0 ** 24)                     # scores up to a few hundred where K has the scales
        kv.append((q8, sc, C.fp8_values(q8, sc)))
    q = torch.randn((4, 16, 128), generator=gen).bfloat16()
    stream, pos = torch.zeros(4, dtype=torch.int32), torch.tensor([1279, 700, 500, 130], dtype=torch.int32)
    for window in (2000, 300, 100):
        want, spread, reach = C.window_attention(q, kv[0][2], kv[1][2], stream, pos, window, 4, 128 ** -0.5)
        got = run("decode", shape, q, kv, stream, pos, window, 4, poison=False)
        PW.check_attention(got, want, spread, reach, PW.P_BF16, 0.0, PW.P_FP16)
    PW.device_error()


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("f8", [False, True])
def test_streams_that_share_pages(mode, f8):
    """Two streams on the same prefix pages, one of them ending inside a shared page: each sees its own rows, also where
    an 8-bit pool is expanded by both."""
    gen = torch.Generator().manual_seed(19)
    G, cap = 4, 512
    shape = msa.Shape(2, cap, 16 * G, G)
    kv = make(1, G, cap, f8, gen)                                    # one sequence's rows; both streams map its pages
    table = torch.tensor([[2, 0, -1, -1], [2, 0, 3, 1]], dtype=torch.int32)
    args = []
    for x, sc, _ in kv:
        raw = (x.view(torch.uint8) if f8 else x)
        pool = torch.full((4, G, 128, 128), 0x7f if f8 else math.nan, dtype=raw.dtype)
        scp = torch.full((4, G), math.nan)
        for b in range(4):
            pool[int(table[1, b])] = raw[0, :, b * 128:b * 128 + 128]
            if f8:
                scp[int(table[1, b])] = sc[0, :, b]
        args.append((pool.cuda().view(F8) if f8 else pool.cuda(), scp.cuda() if f8 else None))
    n = 300 if mode == "prefill" else 2
    stream = (torch.arange(n) * 2 // n).int()
    pos = torch.where(stream == 0, 30 + torch.arange(n) % 150, 511 - torch.arange(n) % 400).int()
    q = torch.randn((n, 16 * G, 128), generator=gen).bfloat16()
    both = [torch.cat((x, x)) for _, _, x in kv]
    want = C.window_attention(q, *both, stream, pos, 100, 4, 128 ** -0.5)
    for _ in range(3):
        got = attend(mode, shape, q.cuda(), args[0][0], args[1][0], stream.cuda(), pos.cuda(), 100, 4,
                     pages=msa.Pages(table.cuda(), 4), k_scale=args[0][1], v_scale=args[1][1])
        PW.check_attention(got, *want, PW.P_BF16, 0.0, PW.norm_of(f8))
    PW.device_error()


def test_wrong_arguments_are_refused():
    shape = msa.Shape(1, 256, 16, 1)
    q = torch.zeros((1, 16, 128), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((1, 1, 256, 128), dtype=torch.bfloat16, device="cuda")
    k8 = torch.zeros((1, 1, 256, 128), dtype=torch.uint8, device="cuda").view(F8)
    sc = torch.ones((1, 1, 2), device="cuda")
    t = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = dict(window=4)
    for fn in (msa.msa_window_attn_decode, msa.msa_window_attn_prefill):
        fn(shape, q, kv, kv, t, t, **good)
        for bad in (dict(q=q[:, :8].contiguous()), dict(k=kv[:, :, :128].contiguous()), dict(v=kv.float()),
                    dict(k=kv.transpose(2, 3)), dict(s=t.long()), dict(p=t.cpu()), dict(k=k8), dict(k=k8, v=k8),
                    dict(scales=(sc, sc)), dict(k=k8, v=k8, scales=(sc[..., :1].contiguous(), sc)),
                    dict(k=k8, v=kv, scales=(sc, sc))):
            a = dict(q=q, k=kv, v=kv, s=t, p=t, scales=(None, None))
            a.update(bad)
            with pytest.raises(ValueError):
                fn(shape, a["q"], a["k"], a["v"], a["s"], a["p"], 4, k_scale=a["scales"][0], v_scale=a["scales"][1])
        for w, s in ((0, 0), (-3, 0), (4, -1)):
            with pytest.raises(msa.MsaError):
                fn(shape, q, kv, kv, t, t, w, s)
        for a in ((q, None, kv, t, t), (q, kv, None, t, t), (q, kv, kv, None, t), (q, kv, kv, t, None)):
            with pytest.raises((ValueError, AttributeError)):
                fn(shape, *a, 4)
    assert msa.msa_window_attn_decode(shape, q[:0], kv, kv, t[:0], t[:0], 4).shape == (0, 16, 128)
    PW.device_error()
