"""How the binding's step functions pass their arguments on (no GPU: the calls below them are stand-ins), and the same
steps on the GPU."""
import copy
import pickle

import pytest
import torch

import block_sparse_attention_maxpool_b200 as msa
from block_sparse_attention_maxpool_b200 import build as msa_build

F8 = torch.float8_e4m3fn
SHAPE = msa.Shape(2, 1024)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    msa_build.build()


def test_shape_hands_out_its_own_copy():
    """What a caller does to the C structure does not reach the frozen Shape, nor what the library gets of it."""
    shape = msa.Shape(2, 1024, 64, 4)
    want = msa.msa_attn_workspace_bytes(shape, 400, msa.MODE_PREFILL, True)
    c = shape.c()
    c.capacity, c.n_streams = 128, 1
    assert (shape.c().capacity, shape.c().n_streams) == (1024, 2)
    assert msa.msa_attn_workspace_bytes(shape, 400, msa.MODE_PREFILL, True) == want
    for twin in (copy.copy(shape), copy.deepcopy(shape), pickle.loads(pickle.dumps(shape))):
        assert twin == shape and msa.msa_attn_workspace_bytes(twin, 400, msa.MODE_PREFILL, True) == want


def step_inputs(n):
    i = torch.zeros(n, dtype=torch.int32)
    return dict(tok_stream=i, tok_pos=i, q_stream=i, q_pos=i, k_new=None, v_new=None, q=torch.zeros(1))


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("f8", [False, True])
def test_window_step_takes_the_bufs_of_decode_step(monkeypatch, prefill, f8):
    """One bufs dict for the layers of a model: ``workspace`` is the scoring workspace there, often too small for the
    attention of an 8-bit prompt."""
    n = 300
    need = msa.msa_attn_workspace_bytes(SHAPE, n, msa.MODE_PREFILL if prefill else msa.MODE_DECODE, f8)
    seen = []
    monkeypatch.setattr(msa, "_append_step", lambda *a: (None, None))
    for name in ("msa_window_attn_prefill", "msa_window_attn_decode"):
        monkeypatch.setattr(msa, name, lambda *a: seen.append(a[10]))
    caches = dict(k_cache=torch.zeros(1).to(F8 if f8 else torch.bfloat16), v_cache=None)
    if f8:
        caches.update(k_scale=1, v_scale=1)
    small, large, own = (torch.zeros(m, dtype=torch.uint8) for m in (64, need + 64, need + 32))
    for bufs in ({"workspace": small}, {"workspace": small, "workspace_attn": own}, {"workspace": large}, {}, None):
        msa.window_step(SHAPE, caches, step_inputs(n), 100, 4, bufs, prefill=prefill)
    assert seen[0] is None or need <= 64 and seen[0] is small
    assert seen[1] is own
    assert seen[2] is (large if f8 and prefill else None)
    assert seen[3] is None and seen[4] is None


class _OnDevice1:
    """Stands for a tensor on cuda:1."""
    is_cuda, device, dtype, shape = True, torch.device("cuda", 1), torch.bfloat16, (1,)

    def get_device(self):
        return 1


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("step", ["decode_step", "window_step"])
def test_steps_launch_on_the_device_of_their_tensors(monkeypatch, step, prefill, f8):
    """With another device current, every call of a step runs with the tensors' device current, and the old one is
    current again afterwards."""
    current, seen = [0], []

    class use:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *a):
            current[0] = self.before
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", use)

    def stand_in(result):
        return lambda *a, **k: (seen.append(current[0]), result)[1]
    for name in ("msa_kv_append", "msa_step_append", "msa_block_scores", "msa_kv_append_fp8", "msa_indexer_append",
                 "msa_sparse_attn_prefill", "msa_sparse_attn_prefill_fp8", "msa_sparse_attn_decode_fp8",
                 "msa_window_attn_decode", "msa_window_attn_prefill"):
        monkeypatch.setattr(msa, name, stand_in(None))
    monkeypatch.setattr(msa, "msa_select_topk", stand_in((None, None)))
    monkeypatch.setattr(msa, "msa_select_attn_decode", stand_in((None, None, None)))
    monkeypatch.setattr(msa, "msa_workspace_bytes", lambda *a: 0)
    new = dict(step_inputs(3), q=_OnDevice1(), idx_q=None, idx_k_new=None)
    caches = dict(k_cache=torch.zeros(1).to(F8 if f8 else torch.bfloat16), v_cache=None, idx_k_cache=torch.zeros(1))
    if f8:
        caches.update(k_scale=1, v_scale=1)
    args = (100, 4) if step == "window_step" else ()
    getattr(msa, step)(SHAPE, caches, new, *args, prefill=prefill)
    assert len(seen) >= 2 and set(seen) == {1} and current == [0]


@pytest.mark.gpu
def test_one_bufs_for_both_kinds_of_layers():
    """A selection layer and a window layer of one model share their bufs over an 8-bit prompt."""
    shape, n = msa.Shape(1, 1024), 300
    gen = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *d, t=torch.bfloat16: torch.randn(d, device="cuda", generator=gen).to(t)
    at = dict(stream=torch.zeros(n, dtype=torch.int32, device="cuda"), pos=torch.arange(n, dtype=torch.int32, device="cuda"))
    new = dict(tok_stream=at["stream"], tok_pos=at["pos"], q_stream=at["stream"], q_pos=at["pos"], k_new=randn(n, 4, 128),
               v_new=randn(n, 4, 128), q=randn(n, 64, 128), idx_k_new=randn(n, 4, 128, t=torch.float32),
               idx_q=randn(n, 4, 128, t=torch.float32))
    bufs = {"workspace": torch.zeros(msa.msa_workspace_bytes(shape, n, msa.MODE_PREFILL), dtype=torch.uint8, device="cuda")}
    out = []
    for b in (None, bufs):
        c = dict(msa.fp8_caches(shape, "cuda"), idx_k_cache=torch.zeros((1, 4, 1024, 128), device="cuda"))
        out.append((msa.decode_step(shape, c, new, b, prefill=True)[0], msa.window_step(shape, c, new, 100, 4, b, prefill=True)))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert msa.msa_get_device_error() == 0


def test_attention_workspace_of_large_caches_is_bounded(monkeypatch):
    """The workspace of an 8-bit prompt grows with the cache up to 1 GiB of expanded rows, then stays (plus four bytes a
    block of the table): a pool that fills the GPU needs no second one."""
    G, n = 4, 2048
    for shape, pages in ((msa.Shape(8, 131072), None), (msa.Shape(1, 131072 * 8), msa.CPages(0, 300000)),
                         (msa.Shape(16, 131072), msa.CPages(0, 100000))):
        blocks = shape.n_streams * shape.n_blocks
        got = msa.library().msa_attn_workspace_bytes(shape.c(), pages, n, msa.MODE_PREFILL, 1)
        room = min(blocks, (1 << 30) // (G * 128 * 512))
        assert room * G * 128 * 512 <= got <= (1 << 30) + 4 * blocks + (8 << 20)
    tiny = msa.Shape(2, 4096)
    need = msa.msa_attn_workspace_bytes(tiny, n, msa.MODE_PREFILL, True)
    assert 0 <= need - 2 * G * 4096 * 512 < 8 << 20
