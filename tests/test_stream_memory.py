"""Calls launched on another stream than the current one: every piece of memory that a call allocates for itself (its
outputs and workspaces) is tied to the stream it launches on.  On the CPU the allocations are watched and the library
is a stand-in; on the GPU what the calls let go of is taken again and overwritten while their kernels still wait."""
import ctypes

import pytest
import torch

import block_sparse_attention_maxpool_b200 as msa

SIDE = 0x5150
S, G, CAP = 2, 4, 1024
SHAPE = msa.Shape(S, CAP, 64, G)
DSHAPE = msa.DsaShape(S, CAP)
F8 = torch.float8_e4m3fn


class _Library:
    """Every call succeeds, every workspace query asks for some bytes."""
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("workspace_bytes") else 0


@pytest.fixture
def watched(monkeypatch):
    """(tensors allocated, tensors tied to SIDE) during a call on CPU tensors."""
    made, held = [], []

    def keep(fn):
        def f(*a, **k):
            made.append(fn(*a, **k))
            return made[-1]
        return f

    def hold(t, *rest):
        assert rest[-1] == SIDE
        held.append(t)
        return t
    monkeypatch.setattr(msa, "_lib", _Library())
    monkeypatch.setattr(msa, "_ptr", lambda t, *a: 0 if t is None else 0x10000)
    monkeypatch.setattr(msa, "_dptr", lambda *a: 0x10000)
    monkeypatch.setattr(msa, "_device_of", lambda *a: "cpu")
    monkeypatch.setattr(msa, "_launch", lambda *a: None)
    monkeypatch.setattr(msa, "_held", hold)
    monkeypatch.setattr(torch, "empty", keep(torch.empty))
    monkeypatch.setattr(torch, "empty_like", keep(torch.empty_like))
    monkeypatch.setattr(ctypes, "byref", lambda x: x)
    return made, held


def inputs(n):
    z = lambda *d, t=torch.bfloat16: torch.zeros(d, dtype=t)
    i = torch.zeros(n, dtype=torch.int32)
    return dict(tok_stream=i, tok_pos=i, q_stream=i, q_pos=i, k_new=z(n, G, 128), v_new=z(n, G, 128), q=z(n, 64, 128),
                idx_k_new=z(n, G, 128, t=torch.float32), idx_q=z(n, G, 128, t=torch.float32),
                k_idx_new=z(n, 128, t=torch.float32), q_idx=z(n, 64, 128, t=torch.float16),
                weights=z(n, 64, t=torch.float32))


def kv(dtype, idx=torch.float32):
    c = {k: torch.zeros((S, G, CAP, 128), dtype=torch.uint8 if dtype is F8 else dtype) for k in ("k_cache", "v_cache")}
    if dtype is F8:
        c = {k: v.view(F8) for k, v in c.items()}
        c.update({k: torch.ones((S, G, CAP // 128)) for k in ("k_scale", "v_scale")})
    c["idx_k_cache"] = torch.zeros((S, G, CAP, 128), dtype=idx)
    c["k_idx_cache"] = torch.zeros((S, CAP, 128), dtype=torch.float16)
    return c


ROPE = msa.Rope(torch.zeros(32, dtype=torch.float64))
STEPS = [(dt, prefill, rope, idx) for dt in (torch.bfloat16, F8) for prefill in (False, True) for rope in (None, ROPE)
         for idx in (torch.float32, torch.float16)]


@pytest.mark.parametrize("dt,prefill,rope,idx", STEPS)
def test_decode_step_ties_its_memory(watched, dt, prefill, rope, idx):
    made, held = watched
    msa.decode_step(SHAPE, kv(dt, idx), inputs(3), None, SIDE, prefill, None, rope)
    assert len(made) >= 5
    assert {id(t) for t in made} == {id(t) for t in held}


def test_every_call_ties_its_memory(watched):
    made, held = watched
    d, c, c8 = inputs(3), kv(torch.bfloat16), kv(F8)
    sel = torch.zeros((3, G, 16), dtype=torch.int32)
    at = (d["q_stream"], d["q_pos"])
    bs = msa.msa_block_scores(SHAPE, d["idx_q"], c["idx_k_cache"], *at, stream=SIDE)
    msa.msa_select_topk(SHAPE, bs, d["q_pos"], stream=SIDE)
    msa.msa_sparse_attn_decode(SHAPE, d["q"], c["k_cache"], c["v_cache"], sel, *at, stream=SIDE)
    msa.msa_sparse_attn_prefill(SHAPE, d["q"], c["k_cache"], c["v_cache"], sel, *at, stream=SIDE)
    msa.msa_sparse_attn_decode_noalloc(SHAPE, d["q"], c["k_cache"], c["v_cache"], sel, *at, stream=SIDE)
    msa.msa_select_attn_decode(SHAPE, bs, d["q"], c["k_cache"], c["v_cache"], *at, stream=SIDE)
    msa.msa_decode_step_fused(SHAPE, c, d, stream=SIDE)
    msa.dsa_decode_step(SHAPE, DSHAPE, c, d, stream=SIDE)
    for prefill in (False, True):
        for caches in (c, c8):
            msa.window_step(SHAPE, caches, d, 100, 4, None, SIDE, prefill, None, ROPE)
    assert len(made) >= 20
    assert {id(t) for t in made} == {id(t) for t in held}


def test_calls_on_the_current_stream_tie_nothing(monkeypatch):
    t = torch.zeros(4)
    assert msa._held(t, None) is t


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefill", [False, True])
def test_steps_on_another_stream(fp8, prefill):
    """decode_step with nothing preallocated but its output, and every other result dropped at once: the same output
    and caches as on the current stream."""
    s, cap, n = 2, 2048, 2048 if prefill else 64
    shape = msa.Shape(s, cap, 64, G)
    gen = torch.Generator(device="cuda").manual_seed(18)
    stream = (torch.arange(n, device="cuda") * s // n).int()
    pos = (torch.arange(n, device="cuda") % (n // s) + 900).int()
    randn = lambda *d, t=torch.bfloat16: torch.randn(d, device="cuda", generator=gen).to(t)
    new = dict(tok_stream=stream, tok_pos=pos, q_stream=stream, q_pos=pos, k_new=randn(n, G, 128), v_new=randn(n, G, 128),
               q=randn(n, 64, 128), idx_k_new=randn(n, G, 128, t=torch.float32), idx_q=randn(n, G, 128, t=torch.float32))
    rope = msa.Rope(10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64))
    start = dict(idx_k_cache=randn(s, G, cap, 128, t=torch.float32))
    if fp8:
        start.update(msa.fp8_caches(shape, "cuda"))
        for c in ("k_cache", "v_cache"):
            start[c].view(torch.uint8).copy_(torch.arange(s * G * cap * 128, device="cuda").view(s, G, cap, 128) * 37 % 96)
        start["k_scale"].fill_(2.0 ** -6)
        start["v_scale"].fill_(2.0 ** -6)
    else:
        start.update(k_cache=randn(s, G, cap, 128), v_cache=randn(s, G, cap, 128))

    def call(side):
        caches = {k: v.clone() for k, v in start.items()}
        out = torch.zeros_like(new["q"])
        torch.cuda.synchronize()
        if side is not None:
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
        msa.decode_step(shape, caches, new, {"out": out}, side, prefill, None, rope)
        junk = [torch.full((m,), 1, dtype=torch.uint8, device="cuda") for k in range(8, 27) for m in (1 << k,) * 3]
        torch.cuda.synchronize()
        assert msa.msa_get_device_error() == 0
        del junk
        return [out] + [caches[k].view(torch.uint8) for k in sorted(caches)]

    want = call(None)
    for got in (call(torch.cuda.Stream()) for _ in range(2)):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
