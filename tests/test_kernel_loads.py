"""What one of the library's kernels writes for the next, the next does not read through the non-coherent path: a grid
may start (programmatic launch) while the one before it still writes, and that path wants its data unchanged for as
long as the reading grid lives."""
import glob
import os
import re

import pytest
import torch

import block_sparse_attention_maxpool_b200 as msa
from tests import parity_window as PW
from tests.test_gpu_fp8_cache import F8

CSRC = os.path.join(os.path.dirname(os.path.abspath(msa.__file__)), "csrc")
# what the caller's own kernels wrote before the call: tokens and queries, frequencies, head weights
INPUTS = {"a", "c", "idx_src", "src", "tok_stream", "tok_pos", "P.q_stream", "P.q_pos", "r.inv_freq", "wp"}


def test_only_inputs_are_read_non_coherently():
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        for m in re.finditer(r"__ldg\((?:reinterpret_cast<[^>]*>\()?([A-Za-z_][\w.]*)", open(path).read()):
            found += 1
            assert m.group(1) in INPUTS, f"{os.path.basename(path)}: {m.group(0)}"
    assert found >= 10


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 300])
def test_attention_sees_the_scales_of_the_append_before(n):
    """Appends that grow a block's scales, each with the attention over that block behind it, queued without a pause
    and captured: the same bits as with a synchronisation between them."""
    G, cap, steps = 4, 512, 40
    shape = msa.Shape(1, cap, 16 * G, G)
    gen = torch.Generator().manual_seed(n)
    zero = torch.zeros(n, dtype=torch.int32, device="cuda")
    q = torch.randn((n, 16 * G, 128), generator=gen).bfloat16().cuda()
    rows = [(torch.randn((n, G, 128), generator=gen) * 2.0 ** (i % 20 - 10)).bfloat16().cuda() for i in range(steps)]
    pos = [torch.arange(3 + i % 100, 3 + i % 100 + n, dtype=torch.int32, device="cuda") for i in range(steps)]
    attend = msa.msa_window_attn_prefill if n > 1 else msa.msa_window_attn_decode
    ws = [torch.zeros(max(1, f), dtype=torch.uint8, device="cuda") for f in
          (msa.msa_kv_append_fp8_workspace_bytes(shape, n), msa.msa_attn_workspace_bytes(shape, n, msa.MODE_PREFILL, True))]

    def run(wait):
        out = []
        for x, p in zip(rows, pos):
            msa.msa_kv_append_fp8(shape, d["k_cache"], d["v_cache"], d["k_scale"], d["v_scale"], x, x, zero, p,
                                  workspace=ws[0])
            if wait:
                torch.cuda.synchronize()
            out.append(attend(shape, q, d["k_cache"], d["v_cache"], zero, p, cap, 0, k_scale=d["k_scale"],
                              v_scale=d["v_scale"], workspace=ws[1]))
        return out

    def clear():
        for c in d.values():
            c.view(torch.uint8).zero_()
        torch.cuda.synchronize()
    d = msa.fp8_caches(shape, "cuda")
    want = run(True)
    clear()
    got = run(False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(False)
    for result in (got, captured):
        if result is captured:
            clear()
            graph.replay()
            torch.cuda.synchronize()
        for a, b in zip(result, want):
            assert torch.equal(a, b)
    assert d["k_cache"].dtype is F8
    PW.device_error()
