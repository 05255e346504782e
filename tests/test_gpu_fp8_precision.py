"""What single queries over an 8-bit cache keep: p times the V scale is held in fp16 (11 bits), not in bf16 as in the
prompt's tiles.  The bound counts that rounding and nothing looser."""
import math

import pytest
import torch

import block_sparse_attention_maxpool_b200 as msa
from oracle import cache_ops as C
from tests import parity_window as PW
from tests.test_gpu_fp8_cache import random_sel
from tests.test_gpu_window import CASES, F8, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from block_sparse_attention_maxpool_b200 import build as msa_build
    msa_build.build()
    msa.msa_get_device_error()


def largest_weight(q, k, v_scale, stream, pos, rows_of, scale):
    """max_j w_j |vs_j| and the number of rows, [n][Hq][1] in float64 (w the softmax weights, vs the V scale of j's block)."""
    n, Hq, _ = q.shape
    S, G, cap, _ = k.shape
    top, rows = torch.zeros((n, Hq, 1), dtype=torch.float64), torch.zeros((n, Hq, 1), dtype=torch.float64)
    for i in range(n):
        s, p = int(stream[i]), int(pos[i])
        if not (0 <= s < S and 0 <= p < cap):
            continue
        for g in range(G):
            idx = torch.as_tensor(rows_of(i, g, s, p), dtype=torch.long)
            if idx.numel() == 0:
                continue
            h = slice(g * (Hq // G), (g + 1) * (Hq // G))
            w = torch.softmax(q[i, h].double() @ k[s, g, idx].double().T * scale, 1)
            top[i, h, 0] = (w * v_scale[s, g, idx // 128].double().abs()).amax(1)
            rows[i, h] = idx.numel()
    return top, rows


def check(got, want, spread, reach, top, rows):
    """out = sum_j w_j (1 + d_j) v_j, where the p in the sum below are not rounded: off by d sum_j w_j |v_j| <= d (spread +
    |out|).  d: half a step of fp16 (2^-11); the score's error in the exponent (as in parity_window); log2 of the V scale
    (at most 127 in magnitude) and the reference in the exponent, four roundings of at most 2^7 u each (below 2^-15 after
    the factor ln 2); ex2 and the float32 sums 2^-18.  Where 2^10 p vs (over the reference, which is no larger than the
    largest p vs) is subnormal in fp16, half a step is 2^-25 instead: each row is off by at most 2^-35 times the largest
    w vs, times the e4m3 value (at most 448)."""
    d = 2.0 ** -11 + 2.0 ** -15 + 2 * 138 * PW.U * reach + 2.0 ** -18
    tol = d / (1 - d).clamp_min(0.5) * (spread + want.abs()) + 2.0 ** -8 * want.abs() * (1 + 2.0 ** -7)
    tol = tol + rows * 2.0 ** -35 * 448 * top + 1e-30
    err = (got.double().cpu() - want).abs()
    assert bool(got.isfinite().all()) and bool((err <= tol).all()), f"{float((err / tol).max()):.2f} of the bound"


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_window(paged, case):
    S, G, cap, at, window, sink = CASES[case]
    gen = torch.Generator().manual_seed(3000 + case)
    shape = msa.Shape(S, cap, 16 * G, G)
    kv = make(S, G, cap, True, gen)
    at = at[::max(1, len(at) // 40)]
    stream, pos = (torch.tensor(x, dtype=torch.int32) for x in zip(*at))
    q = (2 * torch.randn((len(at), 16 * G, 128), generator=gen)).bfloat16()
    table, n_pages = PW.random_pages(S, cap // 128, 2, gen) if paged else (None, 0)
    rows_of = lambda i, g, s, p: C.visible_slots(p, window, sink)
    want = C.window_attention(q, kv[0][2], kv[1][2], stream, pos, window, sink, 128 ** -0.5)
    top = largest_weight(q, kv[0][2], kv[1][1], stream, pos, rows_of, 128 ** -0.5)
    modes = ("decode", "prefill") if len(at) * G < 1024 else ("decode",)      # prompts too short for the tiles
    for mode in modes:
        check(run(mode, shape, q, kv, stream, pos, window, sink, table, n_pages), *want, *top)
    PW.device_error()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("S,G,cap,n", [(1, 4, 128, 1), (1, 1, 4096, 5), (3, 4, 3328, 9), (2, 16, 640, 12)])
def test_selection(S, G, cap, n, pow2):
    gen = torch.Generator().manual_seed(S * cap + n + 7)
    shape = msa.Shape(S, cap, 16 * G, G)
    size = torch.exp2(torch.randint(-4, 5, (S, G, cap // 128, 1, 1), generator=gen).float()).expand(
        -1, -1, -1, 128, 1).reshape(S, G, cap, 1)
    k8, ks = PW.quantise(torch.randn((S, G, cap, 128), generator=gen) * size, pow2)
    v8, vs = PW.quantise(torch.randn((S, G, cap, 128), generator=gen) * size.flip(2), pow2)
    q = torch.randn((n, 16 * G, 128), generator=gen).bfloat16()
    stream = (torch.arange(n) * S // n).int()
    pos = torch.randint(0, cap, (n,), generator=gen).int()
    sel = random_sel(n, G, pos, gen, cap // 128)
    k, v = C.fp8_values(k8, ks), C.fp8_values(v8, vs)
    rows_of = lambda i, g, s, p: [j for b in sel[i, g].tolist() if 0 <= b <= p // 128
                                  for j in range(b * 128, min(b * 128 + 128, p + 1))]
    want = C.selected_attention(q, k, v, sel, stream, pos, 128 ** -0.5)
    top = largest_weight(q, k, vs, stream, pos, rows_of, 128 ** -0.5)
    for fn in (msa.msa_sparse_attn_decode_fp8, msa.msa_sparse_attn_prefill_fp8):
        got = fn(shape, q.cuda(), k8.cuda(), v8.cuda(), ks.cuda(), vs.cuda(), sel.cuda(), stream.cuda(), pos.cuda())
        check(got, *want, *top)
    PW.device_error()


@pytest.mark.parametrize("spread_v", [False, True])
def test_far_apart_scales(spread_v):
    """Blocks whose scales differ by up to 2^60: the block with the largest values and the one with the largest weights
    are different ones."""
    gen = torch.Generator().manual_seed(16)
    shape = msa.Shape(1, 1280, 16, 1)
    sizes = [1.0, 2.0 ** -40, 2.0 ** 20, 0.0, 2.0 ** -20, 2.0 ** -100, 3.0, 2.0 ** 10, 0.7, 1.3]
    kv = []
    for i in range(2):
        q8, _ = PW.quantise(torch.randn((1, 1, 1280, 128), generator=gen))
        sc = torch.tensor(sizes if i == 1 or not spread_v else [1.0 / 448] * 10).view(1, 1, 10) / (448 if i else 2.0 ** 24)
        kv.append((q8.to(F8), sc, C.fp8_values(q8, sc)))
    q = torch.randn((4, 16, 128), generator=gen).bfloat16()
    stream, pos = torch.zeros(4, dtype=torch.int32), torch.tensor([1279, 700, 500, 130], dtype=torch.int32)
    for window in (2000, 300, 100):
        want = C.window_attention(q, kv[0][2], kv[1][2], stream, pos, window, 4, 128 ** -0.5)
        top = largest_weight(q, kv[0][2], kv[1][1], stream, pos, lambda i, g, s, p: C.visible_slots(p, window, 4), 128 ** -0.5)
        check(run("decode", shape, q, kv, stream, pos, window, 4, poison=False), *want, *top)
    PW.device_error()


def test_tiny_weights_beside_a_dominating_one():
    """The stated range: rows whose p vs is down to 2^-24 of the largest keep 11 bits; below that they are off by at most
    2^-35 of the largest, times their value (the dominating row's V is zero, so nothing else shows; a warp's reference
    is the largest of its own rows, so rows of the other warps lose less)."""
    shape = msa.Shape(1, 128, 16, 1)
    for e in (20, 24, 30, 37, 60):
        k8 = torch.zeros((1, 1, 128, 128))
        v8 = torch.zeros((1, 1, 128, 128))
        k8[0, 0, 0, 0] = 1.0                                  # the dominating row: score e ln 2 above the others'
        v8[0, 0, 1:64] = 1.0
        q = torch.zeros((1, 16, 128))
        q[..., 0] = 1.0
        one = torch.ones((1, 1, 1))
        scale = e * math.log(2.0)
        kv = [(x.to(F8), one, x.double()) for x in (k8, v8)]
        stream, pos = torch.zeros(1, dtype=torch.int32), torch.tensor([127], dtype=torch.int32)
        got = run("decode", shape, q.bfloat16(), kv, stream, pos, 128, 0, scale=scale, poison=False).double().cpu()
        want = 63 * 2.0 ** -e / (1 + 127 * 2.0 ** -e)
        lost = 63 * 2.0 ** -35 if e > 24 else 0.0
        assert bool(((got - want).abs() <= (2.0 ** -11 + 2.0 ** -8 + 2.0 ** -16) * want + lost).all()), (e, got.flatten()[0], want)
    PW.device_error()


EXPANDED = [c for c in range(len(CASES)) if len(CASES[c][3]) * CASES[c][1] >= 1024 and len(CASES[c][3]) >= 16 * CASES[c][0]]


@pytest.mark.parametrize("case", EXPANDED)
def test_expanded_window_prompts(case):
    """Where the cache is expanded (scales that are powers of two: exactly), the row sum adds the rounded p, so rounding p
    to bf16 moves out by 2^-8 of the spread and nothing else."""
    S, G, cap, at, window, sink = CASES[case]
    gen = torch.Generator().manual_seed(5000 + case)
    shape = msa.Shape(S, cap, 16 * G, G)
    kv = make(S, G, cap, True, gen)
    stream, pos = (torch.tensor(x, dtype=torch.int32) for x in zip(*at))
    assert msa.msa_attn_workspace_bytes(shape, len(at), msa.MODE_PREFILL, True) > 0
    q = torch.randn((len(at), 16 * G, 128), generator=gen).bfloat16()
    want = C.window_attention(q, kv[0][2], kv[1][2], stream, pos, window, sink, 128 ** -0.5)
    PW.check_attention(run("prefill", shape, q, kv, stream, pos, window, sink), *want, PW.P_BF16, 0.0, 0.0)
    PW.device_error()


def test_every_query_of_an_8bit_prompt_step():
    """decode_step over 8-bit caches, 600 new tokens with rotation: every query of the prompt."""
    gen = torch.Generator().manual_seed(23)
    S, G, cap, per = 2, 2, 2304, 300
    shape, n = msa.Shape(S, cap, 32, G), 600
    stream = torch.arange(S).repeat_interleave(per).int()
    pos = torch.cat([torch.arange(e - per, e) for e in (2200, 1500)]).int()
    caches = {"idx_k_cache": (torch.randn((S, G, cap, 128), generator=gen) / math.sqrt(128)).cuda()}
    for c in "kv":
        q8, sc = PW.quantise(torch.randn((S, G, cap, 128), generator=gen))
        caches[c + "_cache"], caches[c + "_scale"] = q8.cuda(), sc.cuda()
    rope = msa.Rope((10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda(), True)
    rows = lambda *d, f=1.0: (torch.randn(d, generator=gen) * f).cuda()
    new = dict(tok_stream=stream.cuda(), tok_pos=pos.cuda(), q_stream=stream.cuda(), q_pos=pos.cuda(),
               idx_k_new=rows(n, G, 128, f=128 ** -0.5), idx_q=rows(n, G, 128, f=128 ** -0.5),
               k_new=rows(n, G, 128).bfloat16(), v_new=rows(n, G, 128).bfloat16(), q=rows(n, 32, 128).bfloat16())
    out, sel, _, _ = msa.decode_step(shape, caches, new, prefill=True, rope=rope)
    PW.device_error()
    q, _ = msa.msa_rope_append(shape, rope, q=new["q"], q_pos=new["q_pos"])
    k, v = (C.fp8_values(caches[x + "_cache"].cpu(), caches[x + "_scale"].cpu()) for x in "kv")
    want = C.selected_attention(q.cpu(), k, v, sel.cpu(), stream, pos, 128 ** -0.5)
    PW.check_attention(out, *want, PW.P_BF16, 0.0, 0.0)
