"""The operators around the rotated and the 8-bit paged cache: cases, plain forms and calls.

Four operators of a serving step, over a paged cache whose block tables and lengths the
program holds on the GPU:

  rope_append      each new token's query and key heads are (optionally) RMS-normed and
                   rotated by position; keys and values go to their cache slots (16 bits)
  rope_append_q8   the same into a cache of e4m3 codes [blocks, heads, block, dim] with one
                   power-of-two scale for each block and head; a block that older tokens
                   share keeps the larger scale and its older rows are brought to it
  decode_q8        attention of one query token per sequence over that cache
  expand_q8        blocks of that cache back to a 16-bit pool, so that prefill can run over
                   an 8-bit prefix

Lengths come from the case alone (evenly or geometrically spaced and then shuffled by the
seed), so that work() knows them; everything else comes from the seed.
"""
import math

import torch

own = False

EPS = 1e-6
MIN_EXP = -64                   # the smallest scale is 2^-64 (an all-zero block has it)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn


def _case(name, op, seqs, lo, hi, q_heads, kv_heads, head_dim, block, dtype, spread="even", new=1,
          rotary=0, interleaved=False, norm=False, packed=False):
    """new: new tokens of a sequence (its last ones), 0 for all of them."""
    c = dict(op=op, seqs=seqs, lo=lo, hi=hi, spread=spread, q_heads=q_heads, kv_heads=kv_heads,
             head_dim=head_dim, block=block, dtype=dtype)
    if op.startswith("rope"):
        c |= dict(new=new, rotary=rotary or head_dim, interleaved=interleaved, norm=norm,
                  packed=packed)
    return c | dict(name=name) if name else c


def listed():
    return [
        # a step of four short requests on a small model: latency alone
        _case("rope_step_small", "rope_append", 4, 5, 64, 4, 4, 64, 16, "fp16", interleaved=True),
        # a step of 64 requests, normed heads, q/k/v as slices of one projection's output
        _case("rope_step_norm", "rope_append", 64, 128, 4096, 32, 8, 128, 16, "bf16", norm=True,
              packed=True),
        # eight whole prompts: the write of a prefill, bound by memory
        _case("rope_prompts", "rope_append", 8, 512, 4096, 32, 8, 128, 16, "bf16", new=0),
        # a step of 256 requests of very different age into the 8-bit cache
        _case("rope_q8_step", "rope_append_q8", 256, 1, 8192, 32, 8, 128, 16, "bf16",
              spread="geometric", norm=True),
        # chunks of prompts that begin and end inside a block, half of each head rotated
        _case("rope_q8_chunks", "rope_append_q8", 16, 1024, 8192, 40, 8, 128, 32, "fp16", new=500,
              rotary=64, packed=True),
        # a step of four short requests on a small model
        _case("decode_q8_small", "decode_q8", 4, 5, 64, 4, 4, 64, 16, "fp16"),
        # the ordinary step: 64 requests, 135,000 tokens
        _case("decode_q8_batch", "decode_q8", 64, 128, 4096, 32, 8, 128, 16, "bf16"),
        # long documents, eight query heads to a key head
        _case("decode_q8_long", "decode_q8", 8, 32768, 131072, 64, 8, 128, 32, "bf16"),
        # very many short requests
        _case("decode_q8_many", "decode_q8", 2048, 16, 1024, 32, 8, 128, 16, "bf16"),
        # one request alone with a long odd context: only the split over its length fills the GPU
        _case("decode_q8_one", "decode_q8", 1, 50001, 50001, 40, 8, 128, 64, "fp16"),
        # a few blocks of a small model
        _case("expand_q8_small", "expand_q8", 3, 7, 50, 4, 4, 64, 8, "fp16"),
        # the cached prefixes of a chunked prefill
        _case("expand_q8_prefixes", "expand_q8", 16, 512, 7680, 32, 8, 128, 16, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope_append", "rope_append_q8", "decode_q8", "decode_q8", "expand_q8"])
    head_dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32])
    group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 16])
    if kv_heads * group > 128:
        group = 128 // kv_heads
    seqs = _log_int(rng, 1, 2048)
    # no more of K than the long documents of listed() have
    most = max(2, min(131072, (5 << 27) // (seqs * kv_heads * head_dim)))
    new = 1
    if op.startswith("rope"):
        new = rng.choice([1, 1, 0, _log_int(rng, 2, 2000)])
        if new != 1:              # at most 2^15 new tokens, 2^27 elements of q
            seqs = _log_int(rng, 1, 64)
            tokens = min(1 << 15, (1 << 27) // (kv_heads * group * head_dim))
            most = max(2, min(most, 32768, tokens // seqs))
    hi = _log_int(rng, 2, most)
    lo = _log_int(rng, 1, hi)
    rotary = rng.choice([head_dim, head_dim, head_dim // 2, 16 * rng.randint(1, head_dim // 16)])
    return _case(None, op, seqs, lo, hi, kv_heads * group, kv_heads, head_dim,
                 rng.choice([8, 16, 16, 32, 64]), rng.choice(["bf16", "fp16"]),
                 rng.choice(["even", "geometric"]), new, rotary, rng.random() < 0.3,
                 rng.random() < 0.5, rng.random() < 0.5)


def _lengths(case):
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    at = [(i + 0.5) / n for i in range(n)]
    if case["spread"] == "geometric":
        return [round(lo * (hi / lo) ** x) for x in at]
    return [round(lo + (hi - lo) * x) for x in at]


def _new_counts(case, lens):
    return [n if case["new"] == 0 else min(n, case["new"]) for n in lens]


def work(case):
    lens = _lengths(case)
    Hq, H, D, bs = case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    blocks = sum(-(-n // bs) for n in lens)
    if case["op"] == "decode_q8":
        tokens = sum(lens)
        return {"bytes": 2 * tokens * H * D + blocks * (8 * H + 4) + 4 * case["seqs"] * Hq * D,
                "flops": 4 * tokens * Hq * D}
    if case["op"] == "expand_q8":
        return {"bytes": blocks * (H * (6 * bs * D + 8) + 8), "flops": 2 * blocks * H * bs * D}
    counts = _new_counts(case, lens)
    T = sum(counts)
    flops = T * (Hq + H) * (3 * case["rotary"] + (4 * D if case["norm"] else 0))
    table = len(set(p for n, c in zip(lens, counts) for p in (range(n - c, n)))) * case["rotary"] * 4
    index = 4 * T + 8 * case["seqs"]
    if case["op"] == "rope_append":
        return {"bytes": T * (Hq + 2 * H) * D * 4 + table + index, "flops": flops}
    touched = sum((n - 1) // bs - (n - c) // bs + 1 for n, c in zip(lens, counts))
    return {"bytes": T * (4 * Hq + 6 * H) * D + touched * 8 * H + table + index,
            "flops": flops + 4 * T * H * D}


# ------------------------------------------------------------------------------ inputs

def _scale_of(amax):
    """The smallest power of two s >= 2^MIN_EXP with amax <= 448 s: amax = m 2^x with
    m in [1/2, 1), 448 = 7/8 2^9."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(min=MIN_EXP)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP))
    return torch.ldexp(torch.ones_like(amax), e)


def _cache8(blocks, H, bs, D, g):
    """Codes and scales of normal values whose size differs from head to head and block to
    block; a head has a channel that is eight times the others."""
    codes = torch.empty(blocks, H, bs, D, dtype=E4M3, device="cuda")
    scales = torch.empty(blocks, H, dtype=torch.float32, device="cuda")
    head = torch.exp2(3 * torch.rand(1, H, 1, 1, generator=g, device="cuda") - 1.5)
    channel = torch.ones(1, H, 1, D, device="cuda")
    at = torch.randint(0, D, (1, H, 1, 1), generator=g, device="cuda")
    channel.scatter_(3, at, 8.0)
    step = max(1, (1 << 27) // (H * bs * D))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn(n, H, bs, D, generator=g, device="cuda")
        x *= head * channel * (0.75 + torch.rand(n, 1, 1, 1, generator=g, device="cuda"))
        s = _scale_of(x.abs().amax((2, 3)))
        codes[i:i + n] = (x / s[:, :, None, None]).to(E4M3)
        scales[i:i + n] = s
    return codes, scales


def prepare(case, seed):
    """What the serving program holds before the call: the cache with the sequences' older
    tokens, block tables, lengths, the rotation's table, the new tokens' q, k, v."""
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    op = case["op"]
    Hq, H, D, bs = case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    dt = DTYPES[case["dtype"]]
    lens = torch.tensor(_lengths(case))[torch.randperm(case["seqs"], generator=host)]
    used = -(-lens // bs)
    total = int(used.sum())
    blocks = total + total // 10 + 1
    order = torch.randperm(blocks, generator=host)[:total].to(torch.int32)
    tables = torch.full((case["seqs"], int(used.max())), -1, dtype=torch.int32)
    tables[torch.arange(tables.shape[1])[None] < used[:, None]] = order
    st = {"case": case, "tables": tables.cuda(), "lens": lens.to(torch.int32).cuda(),
          "max_len": int(lens.max())}
    if op == "rope_append":
        for n in ("k", "v"):
            st[n + "_pool"] = torch.randn(blocks, bs, H, D, generator=g, device="cuda", dtype=dt)
    else:
        for n in ("k", "v"):
            st[n + "_pool"], st[n + "_scale"] = _cache8(blocks, H, bs, D, g)
    if op == "expand_q8":
        # the blocks in table order, to a staging pool filled from its first block on
        st["pairs"] = torch.stack([order, torch.arange(total, dtype=torch.int32)], 1).cuda()
        for n in ("k", "v"):
            st[n + "_out"] = torch.zeros(total, bs, H, D, dtype=dt, device="cuda")
        return st
    if op == "decode_q8":
        st["q"] = torch.randn(case["seqs"], Hq, D, generator=g, device="cuda").to(dt)
        st["out"] = torch.empty_like(st["q"])
        return st
    counts = torch.tensor(_new_counts(case, lens.tolist()))
    st["q_start"] = None if case["new"] == 1 else torch.cat(
        [torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
    T = int(counts.sum())
    qkv = torch.randn(T, Hq + 2 * H, D, generator=g, device="cuda")
    qkv *= torch.exp2(2 * torch.rand(1, Hq + 2 * H, 1, generator=g, device="cuda") - 1)
    qkv = qkv.to(dt)
    st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    if not case["packed"]:
        for n in "qkv":
            st[n] = st[n].contiguous()
    st["q_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
    for n in ("q_weight", "k_weight"):
        st[n] = (0.5 + torch.rand(D, generator=g, device="cuda")).to(dt) if case["norm"] else None
    R = case["rotary"]
    angle = torch.arange(st["max_len"], dtype=torch.float64, device="cuda")[:, None] * torch.exp(
        torch.arange(0, R, 2, dtype=torch.float64, device="cuda") * (-math.log(500000.0) / R))
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return st


# ------------------------------------------------------------------------- plain forms

def _place(st):
    """Sequence, position, block and row of every new token."""
    lens = st["lens"].long()
    if st["q_start"] is None:
        b = torch.arange(lens.numel(), device="cuda")
        pos = lens - 1
    else:
        start = st["q_start"].long()
        tok = torch.arange(st["q"].shape[0], device="cuda")
        b = torch.searchsorted(start[1:].contiguous(), tok, right=True)
        pos = lens[b] - (start[b + 1] - tok)
    bs = st["case"]["block"]
    return pos, st["tables"].long()[b, pos // bs], pos % bs


def _turned(x, w, cs, case):
    """[T, heads, D] normed (where there is a weight) and rotated by cs [T, R], in 32 bits."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    R = case["rotary"]
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    if case["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_append(st):
    case = st["case"]
    pos, block, row = _place(st)
    cs = st["cos_sin"][pos]
    st["q_out"].copy_(_turned(st["q"], st["q_weight"], cs, case))
    st["k_pool"][block, row] = _turned(st["k"], st["k_weight"], cs, case).to(st["k"].dtype)
    st["v_pool"][block, row] = st["v"]


def _values(pool, blocks):
    """Blocks of codes, in 32 bits."""
    return pool.view(torch.uint8)[blocks].view(E4M3).float()


def _plain_store8(pool, scales, x, block, row, lens, counts, tables):
    """x [T, H, D] (32 bits) to rows of the 8-bit pool, with the blocks' new scales."""
    bs = pool.shape[2]
    # the first block that each sequence writes, and how many older rows it keeps
    first = lens - counts
    older = torch.where(counts > 0, first % bs, torch.zeros_like(first))
    at = torch.where(counts > 0, first, torch.zeros_like(first)) // bs
    seq = torch.arange(lens.numel(), device="cuda")
    held = tables[seq, at.clamp(max=tables.shape[1] - 1)].clamp(min=0)
    H = pool.shape[1]
    need = torch.zeros(pool.shape[0], H, device="cuda")
    need.scatter_reduce_(0, block[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    need = _scale_of(need)
    keeps = older > 0
    before = torch.where(keeps[:, None], scales[held], torch.zeros(1, device="cuda"))
    need.scatter_reduce_(0, held[:, None].expand(-1, H), before, "amax")
    # rows of older tokens, brought to the new scale
    old = _values(pool, held) * (scales[held] / need[held])[:, :, None, None]
    stays = (torch.arange(bs, device="cuda")[None] < older[:, None])[:, None, :, None]
    codes = pool.view(torch.uint8)
    kept = torch.where(stays, old.to(E4M3).view(torch.uint8), codes[held])
    codes[held] = kept
    codes[block, :, row] = (x / need[block][:, :, None]).to(E4M3).view(torch.uint8)
    scales[block] = need[block]


def _plain_append8(st):
    case = st["case"]
    pos, block, row = _place(st)
    cs = st["cos_sin"][pos]
    st["q_out"].copy_(_turned(st["q"], st["q_weight"], cs, case))
    lens = st["lens"].long()
    counts = st["q_start"].long().diff() if st["q_start"] is not None else torch.ones_like(lens)
    where = (block, row, lens, counts, st["tables"].long())
    _plain_store8(st["k_pool"], st["k_scale"], _turned(st["k"], st["k_weight"], cs, case), *where)
    _plain_store8(st["v_pool"], st["v_scale"], st["v"].float(), *where)


def _plain_decode8(st):
    B, Hq, D = st["q"].shape
    bs = st["case"]["block"]
    table = st["tables"].long().clamp(min=0)
    H = st["k_pool"].shape[1]

    def rows(pool, scales):        # [B, H, longest, D] in 32 bits, padded rows zero
        x = _values(pool, table).mul_(scales[table][..., None, None])
        x = x.transpose(1, 2).reshape(B, H, -1, D)
        live = torch.arange(x.shape[2], device="cuda")[None] < st["lens"][:, None]
        return x.masked_fill_(~live[:, None, :, None], 0.0), live

    k, live = rows(st["k_pool"], st["k_scale"])
    s = st["q"].float().view(B, H, Hq // H, D) @ k.transpose(2, 3)
    del k
    s = (s * D ** -0.5).masked_fill_(~live[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    v, _ = rows(st["v_pool"], st["v_scale"])
    out = (p @ v) / p.sum(-1, keepdim=True)
    st["out"].copy_(out.view(B, Hq, D))


def _plain_expand8(st):
    src, dst = st["pairs"][:, 0].long(), st["pairs"][:, 1].long()
    for n in ("k", "v"):
        x = _values(st[n + "_pool"], src) * st[n + "_scale"][src][:, :, None, None]
        most = torch.finfo(st[n + "_out"].dtype).max
        st[n + "_out"][dst] = x.clamp(-most, most).transpose(1, 2).to(st[n + "_out"].dtype)


# ------------------------------------------------------------------------------ passes

def _outputs(st):
    op = st["case"]["op"]
    if op == "decode_q8":
        return {"out": st["out"]}
    if op == "expand_q8":
        return {"k": st["k_out"], "v": st["v_out"]}
    got = {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    if op == "rope_append_q8":
        got |= {"k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    return got


def _own(st):
    import paged_kv_cache_301_gb300 as pa
    case, op = st["case"], st["case"]["op"]
    if op == "decode_q8":
        if "workspace" not in st:      # once for a shape, as a serving program keeps it
            st["workspace"] = pa.workspace_for_q8(st["q"], st["k_pool"], st["max_len"])
        pa.pa_decode_q8(st["out"], st["q"], st["k_pool"], st["v_pool"], st["k_scale"],
                        st["v_scale"], st["tables"], st["lens"], case["head_dim"] ** -0.5,
                        max_seq_len=st["max_len"], workspace=st["workspace"])
    elif op == "expand_q8":
        pa.pa_expand_blocks_q8(st["k_out"], st["v_out"], st["k_pool"], st["v_pool"],
                               st["k_scale"], st["v_scale"], st["pairs"])
    elif op == "rope_append":
        pa.pa_rope_append(st["q_out"], st["k_pool"], st["v_pool"], st["q"], st["k"], st["v"],
                          st["cos_sin"], st["tables"], st["lens"], q_start=st["q_start"],
                          q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                          interleaved=case["interleaved"])
    else:
        pa.pa_rope_append_q8(st["q_out"], st["k_pool"], st["v_pool"], st["k_scale"],
                             st["v_scale"], st["q"], st["k"], st["v"], st["cos_sin"],
                             st["tables"], st["lens"], q_start=st["q_start"],
                             q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                             interleaved=case["interleaved"])


def run(state):
    if own:
        _own(state)
    else:
        {"rope_append": _plain_append, "rope_append_q8": _plain_append8,
         "decode_q8": _plain_decode8, "expand_q8": _plain_expand8}[state["case"]["op"]](state)
    return _outputs(state)


# ------------------------------------------------------------------------------- exact

def _exact_scale(amax):
    """Of a number: 2^e by trying exponents from the logarithm on."""
    if amax <= 0:
        return 2.0 ** MIN_EXP
    e = math.floor(math.log2(amax / 448.0)) - 1
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, MIN_EXP)


def _exact_head(x, w, pos, case):
    """Complex numbers times e^(i angle), the angles as the 32-bit table has them."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    R = case["rotary"]
    f = torch.arange(R // 2, dtype=torch.float64, device=x.device)
    angle = pos.double()[:, None] * torch.exp(f * 2 * (-math.log(500000.0) / R))
    z = torch.complex(angle.cos().float().double(), angle.sin().float().double())[:, None]
    y = x.clone()
    one, two = (slice(0, R, 2), slice(1, R, 2)) if case["interleaved"] else \
        (slice(0, R // 2), slice(R // 2, R))
    t = torch.complex(x[..., one], x[..., two]) * z
    y[..., one], y[..., two] = t.real, t.imag
    return y


def _exact_rope(case, st):
    lens = st["lens"].tolist()
    counts = _new_counts(case, lens)
    tables = st["tables"].tolist()
    eight = case["op"] == "rope_append_q8"
    bs = case["block"]
    got = {"q": torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")}
    for n in ("k", "v"):
        got[n + "_pool"] = st[n + "_pool"].double()
        if eight:
            got[n + "_scale"] = st[n + "_scale"].double()
    at = 0
    for b, (L, c) in enumerate(zip(lens, counts)):
        pos = torch.arange(L - c, L, device="cuda")
        mine = slice(at, at + c)
        at += c
        got["q"][mine] = _exact_head(st["q"][mine], st["q_weight"], pos, case)
        new = {"k": _exact_head(st["k"][mine], st["k_weight"], pos, case),
               "v": st["v"][mine].double()}
        for j in range((L - c) // bs, (L - 1) // bs + 1):
            lo, hi = max(L - c, j * bs), min(L, (j + 1) * bs)
            block, rows = tables[b][j], slice(lo - j * bs, hi - j * bs)
            for n, x in new.items():
                part = x[lo - (L - c):hi - (L - c)]
                pool = got[n + "_pool"]
                if not eight:
                    pool[block, rows] = part
                    continue
                scale = got[n + "_scale"]
                was = scale[block].tolist()
                need = [_exact_scale(a) for a in part.abs().amax((0, 2)).tolist()]
                if rows.start > 0:
                    need = [max(a, b) for a, b in zip(need, was)]
                    ratio = torch.tensor([a / b for a, b in zip(was, need)], device="cuda")
                    old = (pool[block, :, :rows.start] * ratio[:, None, None]).float()
                    pool[block, :, :rows.start] = old.to(E4M3).double()
                s = torch.tensor(need, dtype=torch.float64, device="cuda")
                pool[block, :, rows] = (part / s[:, None]).transpose(0, 1)
                scale[block] = s
    return got


def exact(case, seed):
    """Sequence by sequence and block by block from the definition, in 64 bits.  New codes
    come back before their rounding, in units of the block's scale."""
    if case["op"].startswith("rope"):
        lens = _lengths(case)
        if sum(c // case["block"] + 2 for c in _new_counts(case, lens)) > 6000:
            return None
    elif case["op"] == "decode_q8" and case["seqs"] * case["kv_heads"] > 40000:
        return None
    st = prepare(case, seed)
    if case["op"].startswith("rope"):
        return _exact_rope(case, st)
    if case["op"] == "expand_q8":
        got = {}
        for n in ("k", "v"):
            out = torch.zeros(st[n + "_out"].shape, dtype=torch.float64, device="cuda")
            for i in range(0, st["pairs"].shape[0], 512):
                src, dst = st["pairs"][i:i + 512].long().unbind(1)
                x = torch.einsum("bhtd,bh->bthd", _values(st[n + "_pool"], src).double(),
                                 st[n + "_scale"][src].double())
                out[dst] = x
            got[n] = out
        return got
    q = st["q"].double()
    B, Hq, D = q.shape
    H, bs = case["kv_heads"], case["block"]
    out = torch.zeros_like(q)
    for b, L in enumerate(st["lens"].tolist()):
        block = st["tables"][b, :-(-L // bs)].long()
        for h in range(H):
            k, v = ((st[n + "_pool"].view(torch.uint8)[block, h].view(E4M3).double() *
                     st[n + "_scale"][block, h].double()[:, None, None]).reshape(-1, D)[:L]
                    for n in ("k", "v"))
            mine = slice(h * (Hq // H), (h + 1) * (Hq // H))
            p = torch.softmax(torch.einsum("gd,td->gt", q[b, mine], k) / math.sqrt(D), -1)
            out[b, mine] = torch.einsum("gt,td->gd", p, v)
    return {"out": out}
