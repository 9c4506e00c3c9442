"""Latent attention over a paged cache, and attention of drafted trees: cases, plain forms, calls.

Five operators of a serving step.  A latent cache holds one row [c | r] a token, shared by all
query heads: c a vector of `latent` elements that keys and values are expanded from, r a rotated
key part of 64.

  latent_append    new tokens: c is RMS-normed, r rotated, both go to their cache slots; the
                   rotated part of the query heads is rotated into its place in the queries
  latent_gather    the rows of sequences, in order, as one matrix (what is expanded for prompts)
  latent_decode    absorbed form: queries [c part | r part] against the rows themselves, values
                   are the rows' c; one new token of a sequence, or a tree of drafted ones
  latent_prefill   expanded form: causal attention of prompt tokens, keys [own 128 | shared 64],
                   values of 128
  decode_tree      a tree of drafted tokens of each sequence over a paged cache of K and V

Drafted tokens are the last ones of their sequence; each sees all older tokens and, of the
drafted ones, itself and its ancestors.  Lengths come from the case alone (evenly or
geometrically spaced and then shuffled by the seed), so that work() knows them.
"""
import math

import torch

own = False

EPS = 1e-6
P = 64                          # the rotated part
DN, DV = 128, 128               # expanded form: a head's own key part, its value
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, seqs, lo, hi, q_heads, dtype, block=16, spread="even", latent=512,
          kv_heads=0, head_dim=0, new=1, interleaved=False, norm=True, packed=True):
    """new: new tokens of a sequence (its last ones), 0 for all of them; of latent_decode and
    decode_tree the drafted ones."""
    c = dict(op=op, seqs=seqs, lo=lo, hi=hi, spread=spread, q_heads=q_heads, dtype=dtype)
    if op != "latent_prefill":
        c |= dict(block=block)
    if op == "decode_tree":
        c |= dict(kv_heads=kv_heads, head_dim=head_dim)
    elif op != "latent_prefill":
        c |= dict(latent=latent)
    if op != "latent_gather":
        c |= dict(new=new)
    if op == "latent_append":
        c |= dict(interleaved=interleaved, norm=norm, packed=packed)
    return c | dict(name=name) if name else c


def listed():
    return [
        # a step of 64 requests: a token each
        _case("latent_append_step", "latent_append", 64, 128, 4096, 16, "bf16"),
        # eight whole prompts: the write of a prefill, bound by memory
        _case("latent_append_prompts", "latent_append", 8, 512, 4096, 32, "bf16", new=0,
              interleaved=True),
        # a few short prefixes of a small model
        _case("latent_gather_small", "latent_gather", 3, 7, 50, 4, "fp16", block=8, latent=256),
        # the cached prefixes of a chunked prefill
        _case("latent_gather_prefixes", "latent_gather", 16, 512, 7680, 32, "bf16"),
        # a step of four short requests on a small model: latency alone
        _case("latent_decode_small", "latent_decode", 4, 5, 64, 16, "fp16", latent=256),
        # the ordinary step of a large model: 64 requests, 128 heads
        _case("latent_decode_batch", "latent_decode", 64, 128, 4096, 128, "bf16"),
        # long documents, three drafted tokens a step
        _case("latent_decode_long", "latent_decode", 8, 32768, 131072, 16, "bf16", block=64,
              new=3),
        # whole prompts
        _case("latent_prefill_prompts", "latent_prefill", 4, 512, 4096, 32, "bf16", new=0),
        # chunks of odd length over prefixes of very different length
        _case("latent_prefill_chunks", "latent_prefill", 6, 500, 8191, 16, "fp16", new=500,
              spread="geometric"),
        # a small tree of four short requests on a small model
        _case("tree_small", "decode_tree", 4, 20, 80, 4, "fp16", kv_heads=4, head_dim=64, new=5),
        # verifying trees of 16 drafted tokens for 64 requests
        _case("tree_batch", "decode_tree", 64, 128, 4096, 32, "bf16", kv_heads=8, head_dim=128,
              new=16),
        # one request alone with a long odd context and a large tree
        _case("tree_one", "decode_tree", 1, 50001, 50001, 40, "bf16", block=32, kv_heads=8,
              head_dim=128, new=60),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["latent_append", "latent_gather", "latent_decode", "latent_decode",
                     "latent_prefill", "decode_tree", "decode_tree"])
    dtype, spread = rng.choice(["bf16", "fp16"]), rng.choice(["even", "geometric"])
    block = rng.choice([8, 16, 16, 32, 64])
    latent = rng.choice([256, 512, 512])
    heads = rng.choice([1, 3, 4, 8, 16, 20, 32, 40, 64, 96, 128])
    if op == "latent_prefill":
        heads = rng.choice([1, 2, 4, 8, 16, 32])
        seqs = _log_int(rng, 1, 16)
        hi = _log_int(rng, 2, 8192)
        new = rng.choice([0, 0, _log_int(rng, 1, 1000)])
        # no more scores of a padded batch than the listed prompts have
        while seqs * heads * hi * (new or hi) > 1 << 31:
            seqs, hi = max(1, seqs // 2), max(2, hi * 3 // 4)
        return _case(None, op, seqs, _log_int(rng, 1, hi), hi, heads, dtype, spread=spread,
                     new=new)
    if op == "latent_gather":
        seqs = _log_int(rng, 1, 256)
        hi = _log_int(rng, 2, max(2, min(32768, 65536 // seqs)))
        return _case(None, op, seqs, _log_int(rng, 1, hi), hi, heads, dtype, block, spread, latent)
    if op == "latent_append":
        new = rng.choice([1, 1, 0, _log_int(rng, 2, 2000)])
        seqs = _log_int(rng, 1, 1024) if new == 1 else _log_int(rng, 1, 64)
        most = 32768 if new == 1 else min(32768, max(2, 589824 // (seqs * heads)))
        hi = _log_int(rng, 2, max(2, min(most, (1 << 19) // seqs)))
        return _case(None, op, seqs, _log_int(rng, 1, hi), hi, heads, dtype, block, spread, latent,
                     new=new, interleaved=rng.random() < 0.3, norm=rng.random() < 0.7,
                     packed=rng.random() < 0.7)
    seqs = _log_int(rng, 1, 1024)
    if op == "latent_decode":
        new = rng.choice([1, 1, rng.randint(2, 8), rng.randint(9, 33)])
        row, tokens = latent + P, 131072 * 4 // (latent // 128)
        columns = heads * new
    else:
        head_dim = rng.choice([64, 128, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 16])
        new = rng.choice([rng.randint(1, 8), rng.randint(9, 33), 64])
        row, tokens = 2 * kv_heads * head_dim, (1 << 27) // (kv_heads * head_dim)
        columns, heads = kv_heads * group * new, kv_heads * group
    # no more scores of a padded batch than the listed trees have, and no more of the cache
    hi = _log_int(rng, 2, max(2, min(131072, tokens // seqs, (1 << 27) // (seqs * columns))))
    lo = _log_int(rng, 1, hi)
    if op == "latent_decode":
        return _case(None, op, seqs, lo, hi, heads, dtype, block, spread, latent, new=new)
    return _case(None, op, seqs, lo, hi, heads, dtype, block, spread, kv_heads=kv_heads,
                 head_dim=head_dim, new=new)


def _lengths(case):
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    at = [(i + 0.5) / n for i in range(n)]
    if case["spread"] == "geometric":
        return [round(lo * (hi / lo) ** x) for x in at]
    return [round(lo + (hi - lo) * x) for x in at]


def _new_counts(case, lens):
    return [n if case["new"] == 0 else min(n, case["new"]) for n in lens]


def work(case):
    lens, H = _lengths(case), case["q_heads"]
    S = sum(lens)
    if case["op"] == "latent_gather":
        blocks = sum(-(-n // case["block"]) for n in lens)
        return {"bytes": 4 * S * (case["latent"] + P) + 4 * blocks + 8 * case["seqs"], "flops": 0}
    counts = _new_counts(case, lens)
    T = sum(counts)
    if case["op"] == "latent_append":
        R = case["latent"]
        turns = len(set(p for n, c in zip(lens, counts) for p in range(n - c, n)))
        return {"bytes": 4 * T * (R + P + H * P) + 4 * P * turns + 4 * T + 8 * case["seqs"],
                "flops": T * (3 * P * (H + 1) + (4 * R if case["norm"] else 0))}
    # an older token of each row's, and itself: a tree adds its ancestors to that
    pairs = sum(c * (n - c + 1) for n, c in zip(lens, counts))
    if case["op"] == "latent_prefill":
        pairs += sum(c * (c - 1) // 2 for c in counts)
        return {"bytes": 2 * T * H * (DN + P + DV) + 2 * S * (H * (DN + DV) + P),
                "flops": 2 * (DN + P + DV) * H * pairs}
    blocks = sum(-(-n // case["block"]) for n in lens)
    index = 4 * blocks + 12 * case["seqs"] + 4 * T * -(-case["new"] // 32)
    if case["op"] == "latent_decode":
        R = case["latent"]
        return {"bytes": 2 * S * (R + P) + 2 * T * H * (2 * R + P) + index,
                "flops": 2 * (2 * R + P) * H * pairs}
    D = case["head_dim"]
    return {"bytes": 4 * S * case["kv_heads"] * D + 4 * T * H * D + index,
            "flops": 4 * D * H * pairs}


# ------------------------------------------------------------------------------ inputs

def _pages(case, lens, host):
    """Block tables of the sequences over a pool a tenth larger than they need, as a pool is
    that has served others: the blocks in no order.  And the pool's blocks."""
    bs = case["block"]
    used = -(-lens // bs)
    total = int(used.sum())
    blocks = total + total // 10 + 1
    order = torch.randperm(blocks, generator=host)[:total].to(torch.int32)
    tables = torch.full((lens.numel(), int(used.max())), -1, dtype=torch.int32)
    tables[torch.arange(tables.shape[1])[None] < used[:, None]] = order
    return tables.cuda(), blocks


def _starts(counts):
    return torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()


def _tree(counts, most, host):
    """For each drafted token the set of drafted tokens that it sees, as words of 32 bits: node i
    hangs on a random earlier node, or on the context itself.  [T, words] int32."""
    words = -(-most // 32)
    sets = []
    for n in counts.tolist():
        pick = torch.rand(n, generator=host).tolist()
        seen = []
        for i in range(n):
            parent = int(pick[i] * (i + 1)) - 1
            seen.append((1 << i) | (seen[parent] if parent >= 0 else 0))
        sets += seen
    rows = [[(s >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for s in sets]
    mask = torch.tensor(rows, dtype=torch.int64)
    return torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32).cuda()


def prepare(case, seed):
    """What the serving program holds before the call: the cache with the sequences' tokens,
    block tables, lengths, the rotation's table, the new tokens' projections."""
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    op, H, dt = case["op"], case["q_heads"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    lens = torch.tensor(_lengths(case))[torch.randperm(case["seqs"], generator=host)]
    st = {"case": case, "lens": lens.to(torch.int32).cuda(), "max_len": int(lens.max())}
    if op != "latent_gather":
        counts = torch.tensor(_new_counts(case, lens.tolist()))
        T = int(counts.sum())
        st["max_q"] = int(counts.max())
        st["q_start"] = _starts(counts)
    if op in ("latent_gather", "latent_prefill"):
        st["kv_start"] = _starts(lens)
    if op == "latent_prefill":
        S = int(lens.sum())
        st["q"] = normal(T, H, DN + P)
        st["kv"] = normal(S, H, DN + DV)
        st["key_rope"] = normal(S, P)
        st["out"] = torch.empty(T, H, DV, dtype=dt, device="cuda")
        return st
    st["tables"], blocks = _pages(case, lens, host)
    if op == "decode_tree":
        shape = (blocks, case["block"], case["kv_heads"], case["head_dim"])
        st["k_pool"], st["v_pool"] = normal(*shape), normal(*shape)
        st["q"] = normal(T, H, case["head_dim"])
        st["out"] = torch.empty_like(st["q"])
        st["mask"] = _tree(counts, case["new"], host)
        return st
    R = case["latent"]
    st["pool"] = normal(blocks, case["block"], R + P)
    if op == "latent_gather":
        st["out"] = torch.zeros(int(lens.sum()), R + P, dtype=dt, device="cuda")
        return st
    if op == "latent_decode":
        st["q"] = normal(T, H, R + P)
        st["out"] = torch.empty(T, H, R, dtype=dt, device="cuda")
        st["mask"] = _tree(counts, case["new"], host) if case["new"] > 1 else None
        if case["new"] == 1:
            st["q_start"] = None
        return st
    if case["new"] == 1:
        st["q_start"] = None
    # latent and key part come out of one projection, the queries out of another
    both = normal(T, R + P) * 2.0
    st["latent"], st["key_rope"] = both[:, :R], both[:, R:]
    if not case["packed"]:
        st["latent"], st["key_rope"] = st["latent"].contiguous(), st["key_rope"].contiguous()
    st["weight"] = (0.5 + torch.rand(R, generator=g, device="cuda")).to(dt) if case["norm"] else None
    st["q_rope"] = normal(T, H, DN + P)[..., DN:]
    st["q_out"] = torch.zeros(T, H, R + P, dtype=dt, device="cuda")[..., R:]
    angle = torch.arange(st["max_len"], dtype=torch.float64, device="cuda")[:, None] * torch.exp(
        torch.arange(0, P, 2, dtype=torch.float64, device="cuda") * (-math.log(10000.0) / P))
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return st


# ------------------------------------------------------------------------- plain forms

def _rows_of(starts):
    """Sequence of every row, and its number in it."""
    at = torch.arange(int(starts[-1]), device="cuda")
    b = torch.searchsorted(starts[1:].contiguous(), at, right=True)
    return b, at - starts[b]


def _new_tokens(st):
    """Sequence and position of every new token."""
    lens = st["lens"].long()
    if st["q_start"] is None:
        return torch.arange(lens.numel(), device="cuda"), lens - 1
    b, i = _rows_of(st["q_start"].long())
    return b, lens[b] - st["q_start"].long().diff()[b] + i


def _turn(x, cs, interleaved):
    """x [T, heads, P] rotated by cs [T, P], in 32 bits."""
    x, c, s = x.float(), cs[:, None, :P // 2], cs[:, None, P // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x[..., :P // 2], x[..., P // 2:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _plain_append(st):
    case, dt = st["case"], st["pool"].dtype
    b, pos = _new_tokens(st)
    bs = case["block"]
    block, row = st["tables"].long()[b, pos // bs], pos % bs
    cs = st["cos_sin"][pos]
    c = st["latent"].float()
    if st["weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * st["weight"].float()
    r = _turn(st["key_rope"][:, None], cs, case["interleaved"])[:, 0]
    st["pool"][block, row] = torch.cat([c, r], 1).to(dt)
    st["q_out"].copy_(_turn(st["q_rope"], cs, case["interleaved"]))


def _plain_gather(st):
    b, t = _rows_of(st["kv_start"].long())
    bs = st["case"]["block"]
    st["out"].copy_(st["pool"][st["tables"].long()[b, t // bs], t % bs])


def _padded(x, st):
    """Rows of queries [T, ...] as [B, most, ...] in 32 bits, and where each row is."""
    B = st["lens"].numel()
    if st["q_start"] is None:
        return x.float()[:, None], (torch.arange(B, device="cuda"), 0)
    at = _rows_of(st["q_start"].long())
    p = torch.zeros(B, st["max_q"], *x.shape[1:], device="cuda")
    p[at] = x.float()
    return p, at


def _visible(st, keys):
    """[B, most new, keys]: what each new token sees."""
    lens = st["lens"].long()
    if st["q_start"] is None:
        return (torch.arange(keys, device="cuda")[None] < lens[:, None])[:, None]
    n = st["q_start"].long().diff()
    t = torch.arange(keys, device="cuda")[None, None]
    i = torch.arange(st["max_q"], device="cuda")[None, :, None]
    old = (lens - n)[:, None, None]
    if st.get("mask") is None:
        return (t <= old + i) & (t < lens[:, None, None])
    words, at = _padded_words(st)
    j = (t - old).clamp(min=0, max=32 * words.shape[2] - 1)
    word = torch.gather(words, 2, (j >> 5).expand(-1, st["max_q"], -1))
    bit = (word >> (j & 31)) & 1
    return (t < old) | ((bit != 0) & (t < lens[:, None, None]))


def _padded_words(st):
    at = _rows_of(st["q_start"].long())
    w = torch.zeros(st["lens"].numel(), st["max_q"], st["mask"].shape[1], dtype=torch.int64,
                    device="cuda")
    w[at] = st["mask"].long()
    return w, at


def _attend(q, k, v, visible, scale):
    """softmax(scale q k^T) v in 32 bits: q [B, heads, n, *], k and v [B, heads or 1, keys, *],
    visible [B, 1, n, keys]."""
    s = (q @ k.transpose(2, 3)).mul_(scale).masked_fill_(~visible, -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    total = s.sum(-1, keepdim=True)
    return (s @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_latent_decode(st):
    R = st["case"]["latent"]
    B = st["lens"].numel()
    rows = st["pool"][st["tables"].long().clamp(min=0)].float().flatten(1, 2)     # [B, keys, R+P]
    live = torch.arange(rows.shape[1], device="cuda")[None] < st["lens"][:, None]
    rows = rows.masked_fill_(~live[..., None], 0.0)[:, None]
    q, at = _padded(st["q"], st)                                                  # [B, n, H, R+P]
    n, H = q.shape[1:3]
    seen = _visible(st, rows.shape[2]).repeat_interleave(H, 1)[:, None]
    out = _attend(q.reshape(B, 1, n * H, -1), rows, rows[..., :R], seen, (DN + P) ** -0.5)
    st["out"].copy_(out.view(B, n, H, R)[at])


def _plain_tree(st):
    H, D = st["case"]["kv_heads"], st["case"]["head_dim"]
    B = st["lens"].numel()
    live = None
    kv = []
    for pool in (st["k_pool"], st["v_pool"]):
        x = pool[st["tables"].long().clamp(min=0)].float().flatten(1, 2).transpose(1, 2)
        live = torch.arange(x.shape[2], device="cuda")[None] < st["lens"][:, None]
        kv.append(x.masked_fill(~live[:, None, :, None], 0.0))                    # [B, H, keys, D]
    q, at = _padded(st["q"], st)                                                  # [B, n, Hq, D]
    n, G = q.shape[1], q.shape[2] // H
    q = q.view(B, n, H, G, D).transpose(1, 2).reshape(B, H, n * G, D)
    seen = _visible(st, kv[0].shape[2]).repeat_interleave(G, 1)[:, None]
    out = _attend(q, *kv, seen, D ** -0.5)
    out = out.view(B, H, n, G, D).transpose(1, 2).reshape(B, n, H * G, D)
    st["out"].copy_(out[at])


def _plain_prefill(st):
    B, H = st["lens"].numel(), st["case"]["q_heads"]
    at = _rows_of(st["kv_start"].long())
    k = torch.zeros(B, st["max_len"], H, DN + P, device="cuda")
    v = torch.zeros(B, st["max_len"], H, DV, device="cuda")
    k[at] = torch.cat([st["kv"][..., :DN], st["key_rope"][:, None].expand(-1, H, -1)], 2).float()
    v[at] = st["kv"][..., DN:].float()
    q, rows = _padded(st["q"], st)
    out = _attend(q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2),
                  _visible(st, st["max_len"])[:, None], (DN + P) ** -0.5)
    st["out"].copy_(out.transpose(1, 2)[rows])


# ------------------------------------------------------------------------------ passes

def _own(st):
    import paged_kv_cache_301_gb300 as pa
    case, op = st["case"], st["case"]["op"]
    if op == "latent_append":
        pa.pa_latent_append(st["pool"], st["latent"], st["key_rope"], st["cos_sin"], st["tables"],
                            st["lens"], q_start=st["q_start"], weight=st["weight"], eps=EPS,
                            interleaved=case["interleaved"], q_rope=st["q_rope"],
                            q_out=st["q_out"])
    elif op == "latent_gather":
        pa.pa_latent_gather(st["out"], st["pool"], st["tables"], st["lens"], st["kv_start"])
    elif op == "latent_decode":
        if "workspace" not in st:      # once for a shape, as a serving program keeps it
            st["workspace"] = pa.workspace_for_latent(st["out"], st["pool"], st["max_q"])
        pa.pa_latent_decode(st["out"], st["q"], st["pool"], st["tables"], st["lens"],
                            (DN + P) ** -0.5, q_start=st["q_start"], tree_mask=st["mask"],
                            max_q_len=st["max_q"], max_seq_len=st["max_len"],
                            workspace=st["workspace"])
    elif op == "latent_prefill":
        pa.pa_latent_prefill(st["out"], st["q"], st["kv"], st["key_rope"], st["q_start"],
                             st["kv_start"], (DN + P) ** -0.5, max_q_len=st["max_q"])
    else:
        if "workspace" not in st:
            st["workspace"] = pa.workspace_for_tree(st["q"], st["k_pool"], st["max_q"])
        pa.pa_decode_tree(st["out"], st["q"], st["k_pool"], st["v_pool"], st["tables"], st["lens"],
                          st["q_start"], case["head_dim"] ** -0.5, tree_mask=st["mask"],
                          max_q_len=st["max_q"], max_seq_len=st["max_len"],
                          workspace=st["workspace"])


def run(state):
    op = state["case"]["op"]
    if own:
        _own(state)
    else:
        {"latent_append": _plain_append, "latent_gather": _plain_gather,
         "latent_decode": _plain_latent_decode, "latent_prefill": _plain_prefill,
         "decode_tree": _plain_tree}[op](state)
    if op == "latent_append":
        return {"pool": state["pool"], "q": state["q_out"]}
    return {"out": state["out"]}


# ------------------------------------------------------------------------------- exact

def _exact_turn(x, pos, interleaved):
    """Complex numbers times e^(i angle), the angles' cosines and sines as the 32-bit table has
    them.  x [T, heads, P]."""
    f = torch.arange(P // 2, dtype=torch.float64, device=x.device)
    angle = pos.double()[:, None] * torch.exp(f * 2 * (-math.log(10000.0) / P))
    z = torch.complex(angle.cos().float().double(), angle.sin().float().double())[:, None]
    one, two = (slice(0, P, 2), slice(1, P, 2)) if interleaved else \
        (slice(0, P // 2), slice(P // 2, P))
    x = x.double()
    t = torch.complex(x[..., one], x[..., two]) * z
    y = torch.empty_like(x)
    y[..., one], y[..., two] = t.real, t.imag
    return y


def _exact_rows(pool, table, n, bs):
    """The first n rows of a sequence, block after block."""
    return torch.cat([pool[i] for i in table[:-(-n // bs)]])[:n]


def exact(case, seed):
    """Sequence by sequence from the definition, in 64 bits."""
    op = case["op"]
    lens = _lengths(case)
    blocks = sum(n // case.get("block", 1 << 30) + 1 for n in lens)
    if blocks > 50000:
        return None
    st = prepare(case, seed)
    lens = st["lens"].tolist()
    if op == "latent_append":
        bs, R = case["block"], case["latent"]
        pool = st["pool"].double()
        q = torch.empty(st["q_rope"].shape, dtype=torch.float64, device="cuda")
        tables = st["tables"].tolist()
        at = 0
        for b, (L, c) in enumerate(zip(lens, _new_counts(case, lens))):
            pos = torch.arange(L - c, L, device="cuda")
            mine = slice(at, at + c)
            at += c
            x = st["latent"][mine].double()
            if st["weight"] is not None:
                x = x / torch.sqrt((x * x).sum(1, keepdim=True) / R + EPS) * st["weight"].double()
            y = _exact_turn(st["key_rope"][mine, None], pos, case["interleaved"])[:, 0]
            q[mine] = _exact_turn(st["q_rope"][mine], pos, case["interleaved"])
            for j in range((L - c) // bs, (L - 1) // bs + 1):
                lo, hi = max(L - c, j * bs), min(L, (j + 1) * bs)
                new = slice(lo - (L - c), hi - (L - c))
                pool[tables[b][j], lo - j * bs:hi - j * bs, :R] = x[new]
                pool[tables[b][j], lo - j * bs:hi - j * bs, R:] = y[new]
        return {"pool": pool, "q": q}
    if op == "latent_gather":
        rows = [_exact_rows(st["pool"], st["tables"][b].tolist(), L, case["block"])
                for b, L in enumerate(lens)]
        return {"out": torch.cat(rows).double()}
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    at = kv_at = 0
    for b, (L, c) in enumerate(zip(lens, _new_counts(case, lens))):
        # [c, L]: a row's own set of drafted tokens behind the older ones
        seen = torch.ones(c, L, dtype=torch.bool, device="cuda")
        new = torch.tril(torch.ones(c, c, dtype=torch.bool, device="cuda"))
        if st.get("mask") is not None:
            sets = [sum((w & 0xFFFFFFFF) << (32 * k) for k, w in enumerate(row))
                    for row in st["mask"][at:at + c].tolist()]
            new = torch.tensor([[s >> j & 1 for j in range(c)] for s in sets],
                               dtype=torch.bool, device="cuda")
        seen[:, L - c:] = new
        mine = slice(at, at + c)
        at += c
        q = st["q"][mine].double()
        if op == "latent_prefill":
            kv, r = st["kv"][kv_at:kv_at + L].double(), st["key_rope"][kv_at:kv_at + L].double()
            kv_at += L
            for h in range(case["q_heads"]):
                s = q[:, h, :DN] @ kv[:, h, :DN].T + q[:, h, DN:] @ r.T
                w = torch.softmax((s / math.sqrt(DN + P)).masked_fill(~seen, -math.inf), 1)
                out[mine, h] = w @ kv[:, h, DN:]
            continue
        table = st["tables"][b].tolist()
        if op == "latent_decode":
            x = _exact_rows(st["pool"], table, L, case["block"]).double()
            s = torch.einsum("nhd,td->nht", q, x) / math.sqrt(DN + P)
            w = torch.softmax(s.masked_fill(~seen[:, None], -math.inf), 2)
            out[mine] = torch.einsum("nht,td->nhd", w, x[:, :case["latent"]])
            continue
        k = _exact_rows(st["k_pool"], table, L, case["block"]).double()
        v = _exact_rows(st["v_pool"], table, L, case["block"]).double()
        G = case["q_heads"] // case["kv_heads"]
        for h in range(case["kv_heads"]):
            heads = slice(h * G, (h + 1) * G)
            s = torch.einsum("ngd,td->ngt", q[:, heads], k[:, h]) / math.sqrt(case["head_dim"])
            w = torch.softmax(s.masked_fill(~seen[:, None], -math.inf), 2)
            out[mine, heads] = torch.einsum("ngt,td->ngd", w, v[:, h])
    return {"out": out}
