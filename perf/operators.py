"""Cases of the cache-append and attention operators: inputs, plain forms and the framework's calls.

Four operators share one cache geometry (G groups of 16 query heads, head_dim 128, 128-token blocks, contiguous
``[S][G][capacity][128]`` caches or pools of pages ``[n_pages][G][128][128]`` behind a block table):

  rope_append  new K, V and indexer rows written at their slots with the position rotation applied on the way, and the
               step's queries rotated in the same call;
  fp8_append   new K and V rows (K rotated) written to an e4m3 cache with one power-of-two scale for each block of 128
               tokens and group; a block whose scale grows has its older rows requantised;
  sparse_fp8   attention over the blocks selected for each query and group, read from the e4m3 cache;
  window       attention over the last ``window`` tokens and the first ``sink`` ones, from a bf16 or e4m3 cache.

Where ``own`` is false ``run`` computes an operator in elementary torch operations in 32 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128            # head_dim, indexer dim and block size
HPG = 16           # query heads of a group
TOP_K = 16
E_MIN = -100       # exponent of the scale of a block that holds only zeros
DEV = "cuda"


# ---- cases -------------------------------------------------------------------------------------------------------
def _case(op, streams, ctx, new, groups=4, paged=False, ragged=False, fp8=False, window=0, sink=0, rot=64,
          interleaved=False, indexer=False, theta=1.0e6, name=None):
    c = dict(op=op, streams=streams, ctx=ctx, new=new, groups=groups, paged=paged, ragged=ragged, fp8=fp8,
             window=window, sink=sink, rot=rot, interleaved=interleaved, indexer=indexer, theta=theta)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # one decode step of 32 sequences far into their contexts: one row for each group, latency alone
        _case("rope_append", 32, 131072, 1, paged=True, ragged=True, indexer=True, name="rope_append_decode_32x128k"),
        # a prompt of 16384 tokens written to an empty cache, all 64 query heads rotated: bytes alone
        _case("rope_append", 1, 16384, 16384, indexer=True, name="rope_append_prefill_1x16k"),
        # one decode step of 32 sequences into the 8-bit cache, each in the middle of a block
        _case("fp8_append", 32, 32768, 1, paged=True, ragged=True, fp8=True, name="fp8_append_decode_32x32k"),
        # chunks of 2048 tokens for four sequences at odd places: blocks that are full, begun and left open
        _case("fp8_append", 4, 67000, 2048, paged=True, ragged=True, fp8=True, rot=128, interleaved=True,
              name="fp8_append_chunk_4x2k"),
        # a single sequence with a short context: the smallest attention call
        _case("sparse_fp8", 1, 4096, 1, fp8=True, name="sparse_fp8_decode_1x4k"),
        # the decode batch of the benchmark, from the 8-bit cache
        _case("sparse_fp8", 32, 32768, 1, fp8=True, name="sparse_fp8_decode_32x32k"),
        # a prompt chunk over a long paged context: every token selects its own blocks
        _case("sparse_fp8", 1, 16384, 2048, paged=True, fp8=True, name="sparse_fp8_prefill_2k_on_16k"),
        # decode batch of a local layer: 4096 tokens and four sinks from shuffled pages, lengths apart
        _case("window", 32, 32768, 1, paged=True, ragged=True, window=4096, sink=4, name="window_decode_32x4096"),
        # one sequence, a short window: latency alone
        _case("window", 1, 9001, 1, window=512, sink=4, name="window_decode_1x512"),
        # few sequences with a long window in 8 bits: the work of each has to be split over the chip
        _case("window", 8, 131072, 1, fp8=True, window=32768, sink=128, name="window_fp8_decode_8x32k"),
        # a prompt through a local layer
        _case("window", 1, 8192, 8192, window=4096, sink=4, name="window_prefill_1x8k"),
        # prompt chunks of odd length over 8-bit pages
        _case("window", 2, 6001, 2001, groups=2, paged=True, fp8=True, window=1000, sink=130,
              name="window_fp8_prefill_2x2001"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["rope_append", "fp8_append", "sparse_fp8", "sparse_fp8", "window", "window"])
    groups = rng.choice([1, 2, 4, 4, 8])
    paged = rng.random() < 0.5
    prefill = rng.random() < 0.4
    rot, inter = rng.choice([32, 64, 64, 128]), rng.random() < 0.3
    theta = rng.choice([1.0e4, 5.0e5, 1.0e6])
    if op in ("rope_append", "fp8_append"):
        streams = _log(rng, 1, 64)
        new = min(_log(rng, 2, 8192), 32768 // (streams * groups)) if prefill else rng.choice([1, 1, 1, 2, 5])
        new = max(1, new)
        ctx = new + _log(rng, 1, 131072 if paged else 4096)
        return _case(op, streams, ctx, new, groups, paged, rng.random() < 0.5, op == "fp8_append", rot=rot,
                     interleaved=inter, indexer=op == "rope_append" and rng.random() < 0.5, theta=theta)
    if op == "sparse_fp8":
        if prefill:
            streams = rng.choice([1, 1, 2, 3])
            new = max(1, _log(rng, 16, 8192) // (streams * groups))
            return _case(op, streams, new + _log(rng, 1, 16384), new, groups, paged, False, True)
        streams = max(1, _log(rng, 1, 256) // groups)
        return _case(op, streams, _log(rng, 100, 32768), 1, groups, paged, rng.random() < 0.5, True)
    fp8, sink = rng.random() < 0.5, rng.choice([0, 1, 4, 4, 64, 200])
    if prefill:
        streams = rng.choice([1, 1, 2, 3])
        new = max(1, _log(rng, 64, 8192) // (streams * groups))
        return _case(op, streams, new + _log(rng, 1, 8192), new, groups, paged, False, fp8,
                     window=_log(rng, 16, 8192), sink=sink)
    streams = max(1, _log(rng, 1, 256) // groups)
    return _case(op, streams, _log(rng, 100, 32768), 1, groups, paged, rng.random() < 0.5, fp8,
                 window=_log(rng, 16, 4096), sink=sink)


# ---- inputs ------------------------------------------------------------------------------------------------------
def _capacity(c):
    return -(-c["ctx"] // D) * D


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _quantised_cache(gen, blocks):
    """e4m3 rows [blocks][128][128] and their power-of-two scales [blocks], of keys or values whose size differs
    from block to block."""
    x = torch.empty((blocks, D, D), device=DEV, dtype=torch.float32)
    x.normal_(generator=gen)
    size = torch.randint(-2, 3, (blocks,), generator=gen, device=DEV)
    x.mul_(torch.exp2(size.float())[:, None, None])
    scale = _scale_of(x.abs().amax((1, 2)))
    return (x.div_(scale[:, None, None])).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = {k: v for k, v in case.items() if k != "name"}
    gen = torch.Generator(DEV).manual_seed(seed)
    rng = random.Random(seed)
    S, G, new, ctx = c["streams"], c["groups"], c["new"], c["ctx"]
    cap, n = _capacity(c), S * new
    nblk = cap // D
    last = [rng.randint(max(new - 1, ctx // 4), ctx - 1) if c["ragged"] else ctx - 1 for _ in range(S)]
    pos = [p - new + 1 + i for p in last for i in range(new)]
    st = dict(case=c, capacity=cap, table=None, n_pages=0,
              stream=torch.arange(S, device=DEV, dtype=torch.int32).repeat_interleave(new),
              pos=torch.tensor(pos, device=DEV, dtype=torch.int32))
    append = c["op"] in ("rope_append", "fp8_append")
    if c["paged"]:
        # appends: only the blocks of the step are in the pool, reads: every block, each at a random page
        used = [(s, b) for s in range(S)
                for b in range((last[s] - new + 1) // D if append else 0, (last[s] // D if append else nblk - 1) + 1)]
        st["n_pages"] = len(used) + 3
        page = torch.randperm(st["n_pages"], generator=gen, device=DEV)[:len(used)].to(torch.int32)
        table = torch.full((S, nblk), -1, device=DEV, dtype=torch.int32)
        at = torch.tensor(used, device=DEV)
        table[at[:, 0], at[:, 1]] = page
        st["table"] = table
        rows = (st["n_pages"], G, D)
    else:
        rows = (S, G, cap)
    n_rows = rows[0] * rows[1] * rows[2]
    if c["fp8"]:
        for name in ("k", "v"):
            q8, scale = _quantised_cache(gen, n_rows // D)
            st[name + "_cache"] = q8.view(*rows, D)
            st[name + "_scale"] = scale.view(rows[0], G) if c["paged"] else scale.view(S, G, nblk)
    else:
        for name in ("k", "v"):
            st[name + "_cache"] = _randn(gen, *rows, D).to(torch.bfloat16)
    st["q"] = _randn(gen, n, G * HPG, D).to(torch.bfloat16)
    if append:
        st["inv_freq"] = c["theta"] ** -(torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64) * 2 / c["rot"])
        for name in ("k", "v"):
            size = torch.exp2(torch.randint(-1, 2, (n, G, 1), generator=gen, device=DEV).float())
            st[name + "_new"] = (_randn(gen, n, G, D) * size).to(torch.bfloat16)
        if c["indexer"]:
            st["idx_k_cache"] = _randn(gen, *rows, D) / math.sqrt(D)
            st["idx_k_new"] = _randn(gen, n, G, D) / math.sqrt(D)
            st["idx_q"] = _randn(gen, n, G, D) / math.sqrt(D)
        if c["fp8"]:
            # the blocks (rows of the scale tensor, all groups) that the step writes, and each token's place in them
            blocks = sorted({(s, b) for s in range(S) for b in range((last[s] - new + 1) // D, last[s] // D + 1)})
            where = {sb: i for i, sb in enumerate(blocks)}
            token = [where[s, pos[s * new + i] // D] for s in range(S) for i in range(new)]
            fresh = [last[s] - new + 1 <= b * D for s, b in blocks]
            st["blocks"] = torch.tensor(blocks, device=DEV)
            st["token_block"] = torch.tensor(token, device=DEV)
            st["fresh"] = torch.tensor(fresh, device=DEV)
    if c["op"] == "sparse_fp8":
        score = torch.rand((n, G, nblk), generator=gen, device=DEV)
        local = (st["pos"].long() // D)[:, None, None]
        b = torch.arange(nblk, device=DEV)
        score = torch.where(b == local, 2.0, torch.where(b < local, score, -1.0))
        best = score.topk(min(TOP_K, nblk), dim=2)
        sel = torch.where(best.values >= 0, best.indices, nblk).sort(2).values
        sel = torch.where(sel < nblk, sel, -1).to(torch.int32)
        st["sel"] = torch.nn.functional.pad(sel, (0, TOP_K - sel.shape[2]), value=-1).contiguous()
    return st


# ---- plain forms -------------------------------------------------------------------------------------------------
def _scale_of(amax):
    """The smallest power of two 2^e, e >= E_MIN, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)                                   # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, E_MIN).clamp_min(E_MIN))


def _row_ids(st, stream, slot):
    """Rows of the cache viewed as [rows][128] for slots [...] of streams [...]: [...][G]."""
    c = st["case"]
    g = torch.arange(c["groups"], device=DEV)
    if st["table"] is None:
        return (stream.long()[..., None] * c["groups"] + g) * st["capacity"] + slot.long()[..., None]
    page = st["table"][stream.long(), slot.long() // D].long()
    return (page[..., None] * c["groups"] + g) * D + (slot.long() % D)[..., None]


def _rotate(st, x, pos):
    """x [n][heads][128] rotated at its positions, in 32 bits (the angles in 64)."""
    r = st["case"]["rot"]
    angle = pos.double()[:, None] * st["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    if st["case"]["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _rope_append_plain(st):
    rows = _row_ids(st, st["stream"], st["pos"]).flatten()
    st["k_cache"].view(-1, D)[rows] = _rotate(st, st["k_new"], st["pos"]).to(torch.bfloat16).view(-1, D)
    st["v_cache"].view(-1, D)[rows] = st["v_new"].view(-1, D)
    out = dict(k=st["k_cache"], v=st["v_cache"], q=_rotate(st, st["q"], st["pos"]).to(torch.bfloat16))
    if st["case"]["indexer"]:
        st["idx_k_cache"].view(-1, D)[rows] = _rotate(st, st["idx_k_new"], st["pos"]).view(-1, D)
        out.update(idx_k=st["idx_k_cache"], idx_q=_rotate(st, st["idx_q"], st["pos"]))
    return out


def _fp8_append_one(st, name, x):
    """Append rows x [n][G][128] (float32) to the 8-bit cache `name`."""
    G = st["case"]["groups"]
    first = _row_ids(st, st["blocks"][:, 0], st["blocks"][:, 1] * D) // D          # [blocks][G]: rows of the scales
    cache8, scale = st[name + "_cache"].view(-1, D, D), st[name + "_scale"].view(-1)
    top = torch.zeros(first.shape, device=DEV).scatter_reduce(
        0, st["token_block"][:, None].expand(-1, G), x.abs().amax(2), "amax")
    before = torch.where(st["fresh"][:, None], 0.0, scale[first])
    after = torch.maximum(before, _scale_of(top))
    ratio = torch.where(before > 0, before / after, 1.0)
    cache = cache8.view(torch.uint8)
    held = cache[first].view(torch.float8_e4m3fn).float() * ratio[..., None, None]
    cache[first] = held.to(torch.float8_e4m3fn).view(torch.uint8)
    scale[first] = after
    rows = _row_ids(st, st["stream"], st["pos"])
    y = (x / after[st["token_block"]][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    cache.view(-1, D)[rows] = y.view(torch.uint8)


def _fp8_append_plain(st):
    _fp8_append_one(st, "k", _rotate(st, st["k_new"], st["pos"]))
    _fp8_append_one(st, "v", st["v_new"].float())
    return {n: st[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _rows_as_float(st, name, rows):
    """Rows of the K or V cache, as the float32 values they stand for."""
    if not st["case"]["fp8"]:
        return st[name + "_cache"].view(-1, D)[rows].float()
    x = st[name + "_cache"].view(torch.uint8).view(-1, D)[rows].view(torch.float8_e4m3fn).float()
    return x * st[name + "_scale"].view(-1)[rows // D][..., None]


def _softmax_pv(s, seen, v):
    s = s / math.sqrt(D)
    s = torch.where(seen, s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return (p @ v) / p.sum(-1, keepdim=True)


def _gathered_plain(st, slot, seen):
    """Attention of query i over its own slots slot[i] ([n][G or 1][rows]), where seen."""
    c = st["case"]
    n, G = c["streams"] * c["new"], c["groups"]
    slot = slot.expand(n, G, -1)
    ids = _row_ids(st, st["stream"][:, None, None].expand_as(slot), slot)             # [n][G][rows][G]
    rows = ids.diagonal(dim1=1, dim2=3).transpose(1, 2)                                # group g's rows
    q = st["q"].view(n, G, HPG, D).float()
    s = q @ _rows_as_float(st, "k", rows).transpose(2, 3)
    out = _softmax_pv(s, seen.expand(n, G, -1)[:, :, None], _rows_as_float(st, "v", rows))
    return out.to(torch.bfloat16).view(n, G * HPG, D)


def _sparse_plain(st):
    sel = st["sel"].long()
    slot = (sel.clamp_min(0)[..., None] * D + torch.arange(D, device=DEV)).flatten(2)
    seen = (sel >= 0).repeat_interleave(D, 2) & (slot <= st["pos"][:, None, None])
    return _gathered_plain(st, slot.clamp_max(st["capacity"] - 1), seen)


def _window_plain(st):
    c = st["case"]
    S, G, new, W, sink = c["streams"], c["groups"], c["new"], c["window"], c["sink"]
    if new == 1:
        p = st["pos"].long()[:, None, None]
        slot = torch.cat((torch.arange(sink, device=DEV).expand(S, 1, -1),
                          p - torch.arange(min(W, c["ctx"]), device=DEV)), 2)
        first = torch.arange(slot.shape[2], device=DEV) < sink
        seen = torch.where(first, slot <= p - W, slot >= 0)
        return _gathered_plain(st, slot.clamp(0, st["capacity"] - 1), seen)
    # a chunk of new tokens for each stream, at the same places: all of its queries against all keys that one of them sees
    lo = max(0, c["ctx"] - new - W + 1)
    slot = torch.cat((torch.arange(min(sink, lo), device=DEV), torch.arange(lo, c["ctx"], device=DEV)))
    ids = _row_ids(st, torch.arange(S, device=DEV)[:, None].expand(S, slot.numel()), slot.expand(S, -1)).transpose(1, 2)
    q = st["q"].view(S, new, G, HPG, D).permute(0, 2, 3, 1, 4).float()                # [S][G][16][new][128]
    s = q @ _rows_as_float(st, "k", ids)[:, :, None].transpose(3, 4)
    p = st["pos"].long()[:new, None]
    seen = (slot <= p) & ((slot > p - W) | (slot < sink))
    out = _softmax_pv(s, seen, _rows_as_float(st, "v", ids)[:, :, None])
    return out.permute(0, 3, 1, 2, 4).reshape(S * new, G * HPG, D).to(torch.bfloat16)


# ---- one pass ----------------------------------------------------------------------------------------------------
def _run_own(st):
    import block_sparse_attention_maxpool_b200 as msa
    c = st["case"]
    shape = msa.Shape(c["streams"], st["capacity"], c["groups"] * HPG, c["groups"])
    pages = None if st["table"] is None else msa.Pages(st["table"], st["n_pages"])
    if c["op"] == "rope_append":
        rope = msa.Rope(st["inv_freq"], c["interleaved"])
        q, idx_q = msa.msa_rope_append(shape, rope, st["k_cache"], st["v_cache"], st["k_new"], st["v_new"],
                                       st["stream"], st["pos"], q=st["q"], q_pos=st["pos"],
                                       idx_k_cache=st.get("idx_k_cache"), idx_k_new=st.get("idx_k_new"),
                                       idx_q=st.get("idx_q"), pages=pages)
        out = dict(k=st["k_cache"], v=st["v_cache"], q=q)
        if c["indexer"]:
            out.update(idx_k=st["idx_k_cache"], idx_q=idx_q)
        return out
    if c["op"] == "fp8_append":
        msa.msa_kv_append_fp8(shape, st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["k_new"],
                              st["v_new"], st["stream"], st["pos"], rope=msa.Rope(st["inv_freq"], c["interleaved"]),
                              pages=pages)
        return {n: st[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    if c["op"] == "sparse_fp8":
        attend = msa.msa_sparse_attn_prefill_fp8 if c["new"] > 1 else msa.msa_sparse_attn_decode_fp8
        return attend(shape, st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["sel"],
                      st["stream"], st["pos"], pages=pages)
    attend = msa.msa_window_attn_prefill if c["new"] > 1 else msa.msa_window_attn_decode
    return attend(shape, st["q"], st["k_cache"], st["v_cache"], st["stream"], st["pos"], c["window"], c["sink"],
                  pages=pages, k_scale=st.get("k_scale"), v_scale=st.get("v_scale"))


def run(st):
    if own:
        return _run_own(st)
    return {"rope_append": _rope_append_plain, "fp8_append": _fp8_append_plain, "sparse_fp8": _sparse_plain,
            "window": _window_plain}[st["case"]["op"]](st)


# ---- what a pass cannot do without ---------------------------------------------------------------------------------
def _visible(case, p):
    if case["op"] == "sparse_fp8":
        b = p // D
        return p + 1 if b < TOP_K else (TOP_K - 1) * D + p % D + 1
    near = min(case["window"], p + 1)
    return near + min(case["sink"], p + 1 - near)


def work(case):
    S, G, new, ctx = case["streams"], case["groups"], case["new"], case["ctx"]
    n, Hq = S * new, G * HPG
    if case["op"] == "rope_append":
        rows = n * (2 * G + Hq) * D
        return {"bytes": 4 * rows + (16 * n * G * D if case["indexer"] else 0) + 8 * n, "flops": 3 * rows}
    if case["op"] == "fp8_append":
        return {"bytes": n * G * D * 6 + 16 * n, "flops": 5 * n * G * D}
    row = 2 * D * (1 if case["fp8"] else 2)                                          # bytes of a K and a V row
    # ragged lengths lie evenly between a quarter of the context and all of it: the mean is taken at five places
    at = [int(ctx * (1 + 3 * i / 4) / 4) - 1 for i in range(5)] if case["ragged"] else [ctx - 1]
    at = [max(p, new - 1) for p in at]
    seen = sum(_visible(case, p - i) for p in at for i in range(new)) * S / len(at)  # (query, row) pairs of a group
    if case["op"] == "sparse_fp8":
        # queries of a stream share rows: at most every row of the context is read
        read = min(seen, sum(p + 1 for p in at) * S / len(at))
    else:
        read = sum(min(p + 1, case["window"] + new - 1 + case["sink"]) for p in at) * S / len(at)
    return {"bytes": read * G * row + 4 * n * Hq * D, "flops": 4 * D * HPG * G * seen}


# ---- the definition in 64 bits -------------------------------------------------------------------------------------
def _turn64(x, pos, freq, interleaved):
    """Rotation as a product of complex numbers."""
    r = 2 * freq.numel()
    z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None] * freq)[:, None]
    y = x.double().clone()
    i = torch.arange(r // 2, device=DEV)
    re, im = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    w = torch.complex(y[..., re], y[..., im]) * z
    y[..., re], y[..., im] = w.real, w.imag
    return y


def _e4m3_64(x):
    """x (float64) rounded to the nearest e4m3 value, ties to even, beyond 448 to 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))).clamp_min(-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _block_row64(st, s, g, b):
    if st["table"] is None:
        return (s * st["case"]["groups"] + g) * (st["capacity"] // D) + b
    return int(st["table_host"][s][b]) * st["case"]["groups"] + g


def _fp8_append_exact(st):
    c = st["case"]
    out = {}
    x = {"k": _turn64(st["k_new"], st["pos"], st["inv_freq"], c["interleaved"]), "v": st["v_new"].double()}
    slots = st["pos"].tolist()
    for name in ("k", "v"):
        held = st[name + "_cache"].view(-1, D, D).double()
        scale = st[name + "_scale"].double().view(-1).clone()
        for s in range(c["streams"]):
            mine = slots[s * c["new"]:(s + 1) * c["new"]]
            for b in range(mine[0] // D, mine[-1] // D + 1):
                first, end = max(mine[0], b * D), min(mine[-1] + 1, b * D + D)
                for g in range(c["groups"]):
                    row = _block_row64(st, s, g, b)
                    rows = x[name][s * c["new"] + first - mine[0]:s * c["new"] + end - mine[0], g]
                    top = float(rows.abs().max())
                    need = 2.0 ** max(E_MIN, math.ceil(math.log2(top / 448))) if top > 0 else 2.0 ** E_MIN
                    old = float(scale[row])
                    if first > b * D and old >= need:
                        need = old
                    elif first > b * D and old > 0:
                        held[row] = _e4m3_64(held[row] * (old / need))
                    scale[row] = need
                    held[row, first - b * D:end - b * D] = _e4m3_64(rows / need)
        out[name + "_cache"] = held.view(st[name + "_cache"].shape)
        out[name + "_scale"] = scale.view(st[name + "_scale"].shape)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    S, G, new = c["streams"], c["groups"], c["new"]
    if st["table"] is not None:
        st["table_host"] = st["table"].tolist()
    if c["op"] == "fp8_append":
        return None if S * new * G > 40000 else _fp8_append_exact(st)
    if c["op"] == "rope_append":
        turn = lambda x: _turn64(x, st["pos"], st["inv_freq"], c["interleaved"])  # noqa: E731
        out = {"k": st["k_cache"].double(), "v": st["v_cache"].double(), "q": turn(st["q"])}
        rows = {"k": turn(st["k_new"]), "v": st["v_new"].double()}
        if c["indexer"]:
            out.update(idx_k=st["idx_k_cache"].double(), idx_q=turn(st["idx_q"]))
            rows["idx_k"] = turn(st["idx_k_new"])
        s, p = st["stream"].long(), st["pos"].long()
        for name, x in rows.items():
            if st["table"] is None:
                out[name][s, :, p] = x
            else:
                out[name][st["table"][s, p // D].long(), :, p % D] = x
        return out
    # attention: one stream and group at a time
    if 16 * G * S * new * min(c["ctx"], 1 << 30) > 2 ** 38:
        return None
    out = torch.empty((S * new, G, HPG, D), dtype=torch.float64, device=DEV)
    qs = st["q"].view(S, new, G, HPG, D).double()
    slots = torch.arange(st["capacity"], device=DEV)
    for s in range(S):
        p = st["pos"][s * new:(s + 1) * new].long()[:, None]
        for g in range(G):
            kv = []
            for name in ("k", "v"):
                rows = st[name + "_cache"]
                rows = rows[s, g] if st["table"] is None else rows.view(torch.uint8 if c["fp8"] else rows.dtype)[
                    st["table"][s].long(), g].view(rows.dtype).reshape(-1, D)
                rows = rows.double()
                if c["fp8"]:
                    sc = st[name + "_scale"][s, g] if st["table"] is None else st[name + "_scale"][st["table"][s].long(), g]
                    rows = rows * sc.double().repeat_interleave(D)[:, None]
                kv.append(rows)
            if c["op"] == "window":
                seen = (slots <= p) & ((p - slots < c["window"]) | (slots < c["sink"]))
            else:
                chosen = torch.zeros((new, st["capacity"] // D + 1), dtype=torch.bool, device=DEV)
                chosen.scatter_(1, st["sel"][s * new:(s + 1) * new, g].long() % (st["capacity"] // D + 1), True)
                seen = chosen[:, :-1].repeat_interleave(D, 1) & (slots <= p)
            for h in range(HPG):
                z = qs[s, :, g, h] @ kv[0].T * D ** -0.5
                w = torch.softmax(z.masked_fill(~seen, -math.inf), 1)
                out[s * new:(s + 1) * new, g, h] = w @ kv[1]
    return out.view(S * new, G * HPG, D)
