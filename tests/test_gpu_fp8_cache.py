"""The 8-bit cache on the GPU: the quantising append against the float64 oracle (scales, requantised rows, order of
tokens), block-selected attention over it, and a decode step on 8-bit caches."""
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


def caches(S, G, cap, gen, spread=True):
    """Random 8-bit caches whose blocks differ in size: codes and scales, K and V."""
    out = {}
    for n in "kv":
        x = torch.randn((S, G, cap, 128), generator=gen)
        if spread:
            x = x * torch.exp2(torch.randint(-6, 7, (S, G, cap // 128, 1, 1), generator=gen).float()).expand(
                S, G, cap // 128, 128, 1).reshape(S, G, cap, 1)
        out[n], out[n + "s"] = PW.quantise(x)
    return out


def tokens(pattern, S, cap, gen):
    if pattern == "decode":                       # one per stream, in the middle of a block, first and last slots
        return [(s, p) for s, p in zip(range(S), (77, 128, cap - 1, 0))]
    if pattern == "chunk":                        # runs over several blocks, both ends inside one
        return [(s, p) for s in range(S) for p in range(100 + 3 * s, 100 + 3 * s + 300)]
    if pattern == "shuffled":
        t = [(s, p) for s in range(S) for p in range(50, 250)]
        return [t[i] for i in torch.randperm(len(t), generator=gen)]
    if pattern == "draft":                        # a few consecutive slots per stream
        return [(s, p) for s in range(S) for p in range(126, 131)]
    if pattern == "mixed":                        # a short list in any order, several tokens of a block apart in it
        t = [(s, p) for s in range(S) for p in range(90, 160, 1 + s)]
        return [t[i] for i in torch.randperm(len(t), generator=gen)]
    raise ValueError(pattern)


@pytest.mark.parametrize("pattern", ["decode", "chunk", "shuffled", "draft", "mixed"])
@pytest.mark.parametrize("G,paged,rope", [(4, False, None), (2, True, (64, False)), (1, True, (128, True)), (16, False, None)])
def test_append(pattern, G, paged, rope):
    gen = torch.Generator().manual_seed(G + len(pattern))
    S, cap = 3, 640
    shape = msa.Shape(S, cap, 16 * G, G)
    had = caches(S, G, cap, gen)
    toks = tokens(pattern, S, cap, gen)
    n = len(toks)
    stream = torch.tensor([s for s, _ in toks], dtype=torch.int32)
    pos = torch.tensor([p for _, p in toks], dtype=torch.int32)
    size = torch.exp2(torch.randint(-12, 13, (n, G, 1), generator=gen).float())
    k_new, v_new = ((torch.randn((n, G, 128), generator=gen) * size).bfloat16() for _ in range(2))
    f = None if rope is None else freqs(rope[0])
    krows = k_new.double() if rope is None else C.rotate_rows(k_new, pos, f, rope[1])
    want = {}
    for name, x in (("k", krows), ("v", v_new.double())):
        want[name], want[name + "s"] = C.fp8_append(had[name].double(), had[name + "s"], x, stream, pos)
    pages, dev = None, {}
    if paged:
        table, n_pages = PW.random_pages(S, cap // 128, 2, gen)
        pages = msa.Pages(table.cuda(), n_pages)
    for c in "kv":
        x, sc = had[c].view(torch.uint8), had[c + "s"]
        dev[c] = (PW.to_pool(x, table, n_pages, 127) if paged else x).cuda().view(F8)
        dev[c + "s"] = (PW.scale_pool(sc, table, n_pages) if paged else sc).cuda()
    r = None if rope is None else msa.Rope(f.cuda(), rope[1])
    msa.msa_kv_append_fp8(shape, dev["k"], dev["v"], dev["ks"], dev["vs"], k_new.cuda(), v_new.cuda(), stream.cuda(),
                          pos.cuda(), rope=r, pages=pages)
    PW.device_error()
    for c in "kv":
        got = dev[c].cpu().view(torch.uint8)
        gs = dev[c + "s"].cpu()
        if paged:
            got = torch.stack([torch.cat([got[int(table[s, b])] for b in range(cap // 128)], 1) for s in range(S)])
            gs = torch.stack([torch.stack([gs[int(table[s, b])] for b in range(cap // 128)], 1) for s in range(S)])
        assert torch.equal(gs.double(), want[c + "s"]), f"{c} scales"
        got = got.view(F8).double()
        if c == "v" or rope is None:
            assert torch.equal(got, want[c]), f"{c} rows"
        else:
            # a turned value may fall on the other side of a tie: then it is off by one step at most, and only there
            same = got == want[c]
            mine = torch.zeros_like(same)
            mine[stream.long(), :, pos.long()] = True
            assert bool((same | mine).all()), "a row that no token names differs"
            assert float((~same).double().mean()) < 1e-4
            rows, sc = got[stream.long(), :, pos.long()], gs.double()[stream.long(), :, pos.long() // 128]
            err = (rows * sc[..., None] - krows).abs()
            tol = 2.0 ** -4 * krows.abs() + 2.0 ** -10 * sc[..., None] + 2.0 ** -19 * krows.abs().amax(-1, keepdim=True)
            assert bool((err <= tol).all())


def test_order_of_tokens_does_not_matter():
    gen = torch.Generator().manual_seed(3)
    S, G, cap, n = 2, 4, 512, 700
    shape = msa.Shape(S, cap, 64, G)
    had = caches(S, G, cap, gen)
    slots = torch.randperm(S * cap, generator=gen)[:n]
    stream, pos = (slots // cap).int(), (slots % cap).int()
    k_new, v_new = ((torch.randn((n, G, 128), generator=gen) * 2.0 ** float(i)).bfloat16() for i in (0, 9))
    out = []
    for perm in (torch.arange(n), torch.randperm(n, generator=gen)):
        d = {c: had[c].cuda() for c in had}
        msa.msa_kv_append_fp8(shape, d["k"], d["v"], d["ks"], d["vs"], k_new[perm].cuda(), v_new[perm].cuda(),
                              stream[perm].cuda(), pos[perm].cuda())
        out.append({c: d[c].cpu().view(torch.uint8) for c in d})
    PW.device_error()
    for c in had:
        assert torch.equal(out[0][c], out[1][c])


def test_extreme_values():
    """Zeros, infinities, NaN, the largest and smallest bf16 values, and blocks that held nothing valid."""
    shape = msa.Shape(1, 256, 16, 1)
    rows = torch.zeros((7, 1, 128))
    rows[1, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 1.0])
    rows[2] = 3.0e38
    rows[3] = 1e-38
    rows[4, 0, 0] = math.inf
    rows[5] = 448.0
    rows[6] = 449.0                     # bf16: 448 rounds to 448, 449 to 448 or 450
    rows = rows.bfloat16()
    for i in range(7):
        for slot, held in ((0, float("nan")), (5, float("nan")), (5, -1.0), (5, 0.0)):
            d = msa.fp8_caches(shape, "cuda")
            d["k_scale"].fill_(held)
            d["v_scale"].fill_(held)
            one = torch.zeros(1, dtype=torch.int32, device="cuda")
            msa.msa_kv_append_fp8(shape, d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"], rows[i:i + 1].cuda(),
                                  rows[i:i + 1].cuda(), one, one + slot)
            x = rows[i].double()
            fin = x[x.isfinite()].abs()
            need = C.needed_scale(float(fin.max()) if fin.numel() else 0.0)
            assert float(d["v_scale"][0, 0, 0]) == need
            want = C.round_e4m3((x / need)[0])
            got = d["v_cache"][0, 0, slot].cpu().double()
            assert torch.equal(got.nan_to_num(1e6), want.nan_to_num(1e6))
            assert torch.equal(d["k_cache"].view(torch.uint8), d["v_cache"].view(torch.uint8))
    PW.device_error()


@pytest.mark.parametrize("n", [1, 300])
def test_scale_growing_past_float32(n):
    """The old scale over the new one is below any float32: the older rows become zeros, not values of the new scale."""
    G, cap = 2, 512
    shape = msa.Shape(1, cap, 32, G)
    had = {"k": torch.zeros((1, G, cap, 128), dtype=torch.uint8), "ks": torch.zeros((1, G, 4))}
    had["k"][0, :, 1:5] = torch.tensor([0x7e, 0xfe, 0x38, 0x01], dtype=torch.uint8)[:, None]
    had["ks"][0, :, 0] = 2.0 ** -90
    pos = torch.arange(5, 5 + n, dtype=torch.int32)
    stream = torch.zeros(n, dtype=torch.int32)
    new = torch.full((n, G, 128), 2.0 ** 120).bfloat16()
    want, ws = C.fp8_append(had["k"].view(F8).double(), had["ks"], new.double(), stream, pos)
    assert not bool(want[0, :, 1:5].any()) and bool((ws[0, :, 0] == 2.0 ** 112).all())
    k, v = had["k"].cuda().view(F8), had["k"].cuda().view(F8)
    ks, vs = had["ks"].cuda(), had["ks"].cuda()
    msa.msa_kv_append_fp8(shape, k, v, ks, vs, new.cuda(), new.cuda(), stream.cuda(), pos.cuda())
    PW.device_error()
    for got, scale in ((k, ks), (v, vs)):
        assert torch.equal(scale.cpu().double(), ws)
        assert torch.equal(got.cpu().double(), want)


def test_skipped_tokens():
    shape = msa.Shape(2, 256, 16, 1)
    table = torch.tensor([[0, -1], [9, 1]], dtype=torch.int32)
    d = msa.fp8_caches(shape, "cuda", 2)
    ts = torch.tensor([0, 0, 1, 1, 2, 0], dtype=torch.int32, device="cuda")
    tp = torch.tensor([3, 130, 5, 255, 1, 256], dtype=torch.int32, device="cuda")
    new = torch.randn((6, 1, 128)).bfloat16().cuda()
    msa.msa_kv_append_fp8(shape, d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"], new, new, ts, tp,
                          pages=msa.Pages(table.cuda(), 2))
    PW.device_error(0x2 | 0x10)
    raw = d["v_cache"].view(torch.uint8).cpu()
    assert raw[0, 0, 3].any() and raw[1, 0, 127].any()
    raw[0, 0, 3] = raw[1, 0, 127] = 0
    assert not raw.any()
    assert bool((d["v_scale"] > 0).all())


def random_sel(n, G, pos, gen, nblk):
    """Random selections: local block included or not, fewer than 16, in any order, with -1 anywhere."""
    sel = torch.full((n, G, 16), -1, dtype=torch.int32)
    for i in range(n):
        vis = int(pos[i]) // 128 + 1
        for g in range(G):
            k = min(vis, 16 if i % 3 else int(torch.randint(1, 17, (1,), generator=gen)))
            blocks = torch.randperm(vis, generator=gen)[:k].int()
            at = torch.randperm(16, generator=gen)[:k] if i % 4 == 3 else torch.arange(k)
            sel[i, g, at] = blocks if i % 2 else blocks.sort().values
    return sel


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("S,G,cap,n,paged,pow2", [
    (1, 4, 128, 1, False, True),
    (1, 1, 4096, 1, False, True),
    (3, 4, 3328, 3, True, False),
    (5, 2, 2176, 37, False, False),
    (2, 16, 640, 9, True, True),
    (1, 4, 2944, 150, True, True),
    (2, 4, 2560, 400, False, False),
    (3, 4, 1024, 500, True, True),
])
def test_selected_attention(mode, S, G, cap, n, paged, pow2):
    gen = torch.Generator().manual_seed(S * cap + n)
    shape = msa.Shape(S, cap, 16 * G, G)
    size = torch.exp2(torch.randint(-4, 5, (S, G, cap // 128, 1, 1), generator=gen).float()).expand(
        -1, -1, -1, 128, 1).reshape(S, G, cap, 1)
    k8, ks = PW.quantise(torch.randn((S, G, cap, 128), generator=gen) * size, pow2)
    v8, vs = PW.quantise(torch.randn((S, G, cap, 128), generator=gen) * size.flip(2), pow2)
    q = torch.randn((n, 16 * G, 128), generator=gen).bfloat16()
    stream = (torch.arange(n) * S // n).int()
    pos = torch.randint(0, cap, (n,), generator=gen).int()
    if mode == "prefill":
        pos = pos.sort().values
    sel = random_sel(n, G, pos, gen, cap // 128)
    want, spread, reach = C.selected_attention(q, C.fp8_values(k8, ks), C.fp8_values(v8, vs), sel, stream, pos,
                                               128 ** -0.5)
    # rows past every query of their stream hold NaN codes
    kd, vd = k8.view(torch.uint8).clone(), v8.view(torch.uint8).clone()
    for s in range(S):
        mine = pos[stream == s]
        end = int(mine.max()) + 1 if mine.numel() else 0
        kd[s, :, end:] = 0x7f
        vd[s, :, end:] = 0xff
    pages = None
    if paged:
        table, n_pages = PW.random_pages(S, cap // 128, 2, gen)
        pages = msa.Pages(table.cuda(), n_pages)
        kd, vd = PW.to_pool(kd, table, n_pages, 0x7f), PW.to_pool(vd, table, n_pages, 0x7f)
        ks, vs = PW.scale_pool(ks, table, n_pages), PW.scale_pool(vs, table, n_pages)
    fn = msa.msa_sparse_attn_prefill_fp8 if mode == "prefill" else msa.msa_sparse_attn_decode_fp8
    out = torch.full((n, 16 * G, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    got = fn(shape, q.cuda(), kd.cuda().view(F8), vd.cuda().view(F8), ks.cuda(), vs.cuda(), sel.cuda(), stream.cuda(),
             pos.cuda(), out=out, pages=pages)
    assert got is out
    PW.device_error()
    kv_round = 2.0 ** -8 if mode == "prefill" and not pow2 else 0.0
    print(f"\n[fp8 {mode}] of its bound: {PW.check_attention(got, want, spread, reach, PW.P_BF16, kv_round, PW.norm_of(True)):.2f}")


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_nothing_to_attend(mode):
    """Queries outside the caches, empty selections, invisible and unmapped blocks: zeros, and the error bits."""
    gen = torch.Generator().manual_seed(8)
    shape = msa.Shape(2, 512, 16, 1)
    k8, ks = PW.quantise(torch.randn((3, 1, 128, 128), generator=gen))
    table = torch.tensor([[0, -1, 1, 2], [3, -2, 0, 1]], dtype=torch.int32)
    pages = msa.Pages(table.cuda(), 3)
    times = 700 if mode == "prefill" else 1
    stream = torch.tensor([0, 2, -1, 0, 0, 0, 1] * times, dtype=torch.int32)
    pos = torch.tensor([511, 5, 5, 512, -1, 200, 130] * times, dtype=torch.int32)
    sel = torch.full((7, 1, 16), -1, dtype=torch.int32)
    sel[1:5, 0, 0] = 0
    sel[5, 0, :2] = torch.tensor([1, 3])            # unmapped, and past the query
    sel[6, 0, :2] = torch.tensor([0, 1])            # page 3 of 3, and -2
    sel = sel.repeat(times, 1, 1)
    fn = msa.msa_sparse_attn_prefill_fp8 if mode == "prefill" else msa.msa_sparse_attn_decode_fp8
    out = torch.full((7 * times, 16, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    q = torch.randn((7 * times, 16, 128), generator=gen).bfloat16().cuda()
    fn(shape, q, k8.cuda(), k8.cuda(), ks.view(3, 1).cuda(), ks.view(3, 1).cuda(), sel.cuda(), stream.cuda(),
       pos.cuda(), out=out, pages=pages)
    PW.device_error(0x1 | 0x4 | 0x10)
    assert not bool(out.any())


@pytest.mark.parametrize("prefill", [False, True])
def test_decode_step_on_8bit_caches(prefill):
    """decode_step with 8-bit caches and rotation: the selection of the bf16 step's scores, attention within the bound
    of the oracle on the caches the step left; captured and replayed it gives the same bits."""
    gen = torch.Generator().manual_seed(21)
    S, G, cap, new_n = 2, 2, 2560, 400 if prefill else 1
    shape = msa.Shape(S, cap, 32, G)
    rope = msa.Rope(freqs(64).cuda())
    had = caches(S, G, cap, gen, spread=False)
    n = S * new_n
    stream = torch.arange(S).repeat_interleave(new_n).int()
    pos = torch.cat([torch.arange(e - new_n, e) for e in (2500, 1800)]).int()
    new = dict(tok_stream=stream.cuda(), tok_pos=pos.cuda(), q_stream=stream.cuda(), q_pos=pos.cuda(),
               idx_k_new=torch.randn((n, G, 128), generator=gen).cuda() / math.sqrt(128),
               k_new=torch.randn((n, G, 128), generator=gen).bfloat16().cuda(),
               v_new=torch.randn((n, G, 128), generator=gen).bfloat16().cuda(),
               idx_q=torch.randn((n, G, 128), generator=gen).cuda() / math.sqrt(128),
               q=torch.randn((n, 32, 128), generator=gen).bfloat16().cuda())
    idx = torch.randn((S, G, cap, 128), generator=gen) / math.sqrt(128)

    def fresh():
        return dict(idx_k_cache=idx.cuda(), k_cache=had["k"].cuda(), v_cache=had["v"].cuda(),
                    k_scale=had["ks"].cuda(), v_scale=had["vs"].cuda())
    c = fresh()
    out, sel, n_sel, bs = msa.decode_step(shape, c, new, prefill=prefill, rope=rope)
    PW.device_error()
    q, _ = msa.msa_rope_append(shape, rope, q=new["q"], q_pos=new["q_pos"])
    k, v = (C.fp8_values(c[x + "_cache"].cpu(), c[x + "_scale"].cpu()) for x in "kv")
    some = torch.arange(0, n, 17 if prefill else 1)                 # every query of a decode step, some of a prompt
    want, spread, reach = C.selected_attention(q.cpu()[some], k, v, sel.cpu()[some], stream[some], pos[some], 128 ** -0.5)
    PW.check_attention(out[some.cuda()], want, spread, reach, PW.P_BF16, 0.0, PW.norm_of(True))
    assert bool((n_sel >= 1).all())
    graph = msa.DecodeGraph(shape, fresh(), new, prefill=prefill, rope=rope)
    assert torch.equal(graph.replay(), out)
    PW.device_error()
