"""What is measured of the 8-bit paged cache: appending with the position rotation, attention over the cache for one or
many query tokens per sequence, and the merge of partial attentions by their log-sum-exp.

``run`` computes each operator in its plain form (elementary torch operations in fp32) where ``own`` is false, and
makes the calls of ``residual_kv_cache_delta_b200.deltakv`` where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
FLOOR = 2.0 ** -64  # a block's largest magnitude counts as at least this
QMAX = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _append(name, seqs, new, start, code, hq=32, hkv=8, d=128, block=16, rot=128, pairs=False, dtype="bf16"):
    return dict(name=name, op="append", dtype=dtype, code=code, seqs=seqs, new=new, start=start, hq=hq, hkv=hkv, d=d,
                block=block, rot=rot, pairs=pairs)


def _attend(name, seqs, queries, ctx, code, ragged=True, hq=32, hkv=8, d=128, block=16, softcap=0.0, alibi=False,
            window=0, prefix=0, docs=0, dtype="bf16"):
    return dict(name=name, op="attention", dtype=dtype, code=code, seqs=seqs, queries=queries, ctx=ctx, ragged=ragged,
                hq=hq, hkv=hkv, d=d, block=block, softcap=softcap, alibi=alibi, window=window, prefix=prefix, docs=docs)


def _merge(name, parts, rows, heads, d=128, dtype="bf16"):
    return dict(name=name, op="merge", dtype=dtype, parts=parts, rows=rows, heads=heads, d=d)


def listed():
    return [
        # one decode step of a 64-sequence batch: each sequence's new token goes into its last block
        _append("append-64x1", 64, 1, 8000, "int8"),
        # chunked prefill of four prompts, 2048 tokens a step, chunks that begin inside a block
        _append("append-4x2048", 4, 2048, 5000, "e4m3", block=32),
        # two whole prompts of the bench's length, appended at once
        _append("append-2x32768", 2, 32768, 0, "int8", rot=64, pairs=True),
        # a single short conversation: latency
        _attend("decode-1x1000", 1, 1, 1000, "int8"),
        # the bench's batch: 8 sequences of 32768 tokens
        _attend("decode-8x32768", 8, 1, 32768, "int8", ragged=False),
        # ragged serving mix with capped scores, a sliding window and always-visible first tokens
        _attend("decode-24-window", 24, 1, 16384, "e4m3", block=32, softcap=30.0, window=4096, prefix=64),
        # one very long context, 8 query heads to a kv head
        _attend("decode-1x131072", 1, 1, 131072, "e4m3", hq=64, block=64),
        # verification of 5 drafted tokens per sequence, distance bias, 64-wide heads
        _attend("verify-8x5", 8, 5, 5000, "int8", hq=24, d=64, alibi=True),
        # one 2048-token prefill chunk at the end of a 32768-token context
        _attend("chunk-2048-32768", 1, 2048, 32768, "int8", ragged=False),
        # packed documents prefilled at once, capped scores
        _attend("docs-8192", 1, 8192, 8192, "e4m3", ragged=False, hq=16, hkv=4, softcap=50.0, docs=5),
        # two partial attentions of a decode batch
        _merge("merge-2x64", 2, 64, 32),
        # three partial attentions of a large prefill step
        _merge("merge-3x16381", 3, 16381, 32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "attention", "merge"])
    d, block, code = rng.choice([64, 128]), rng.choice([16, 32, 64]), rng.choice(["int8", "e4m3"])
    hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        seqs = _log(rng, 1, 64)
        new = rng.choice([1, 1, _log(rng, 2, 65536 // seqs)])
        c = _append("", seqs, new, _log(rng, 1, 20000), code, hkv * min(group, 4), hkv, d, block,
                    rng.choice([d, d // 2]), rng.choice([True, False]), rng.choice(["bf16", "bf16", "bf16", "f32"]))
    elif op == "merge":
        c = _merge("", rng.choice([2, 3, 4]), _log(rng, 1, 12000), hkv * min(group, 4), d,
                   rng.choice(["bf16", "bf16", "bf16", "f32"]))
    else:
        mask = dict(softcap=rng.choice([0.0, 0.0, 30.0]), alibi=rng.choice([False, False, True]),
                    window=rng.choice([0, 0, 100, 1000, 5000]), prefix=rng.choice([0, 0, 5, 700]))
        kind = rng.choice(["decode", "verify", "chunk"])
        if kind == "chunk":
            queries = _log(rng, 17, 3000)
            ctx = queries + _log(rng, 1, 16000)
            c = _attend("", 1 if queries > 500 else rng.choice([1, 2, 3]), queries, ctx, code,
                        hq=hkv * min(group, 4), hkv=hkv, d=d, block=block, docs=rng.choice([0, 0, 3]), **mask)
        else:
            seqs = _log(rng, 1, 48)
            ctx = _log(rng, 20, min(131072, 262144 // seqs))
            queries = 1 if kind == "decode" else rng.choice([2, 3, 4, 6, 8])
            c = _attend("", seqs, queries, ctx, code, hq=hkv * group, hkv=hkv, d=d, block=block, **mask)
            if kind == "decode" and ctx * seqs < 50000 and rng.random() < 0.25:
                c["dtype"] = "f32"
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------------------
# Sizes that follow from a case alone
# ---------------------------------------------------------------------------------------------------------------
def _spread(n, lo, hi, step=0.6180339887498949):
    """n whole numbers in [lo, hi], spread over their logarithm; the first is hi."""
    lo, hi = max(lo, 1), max(hi, 1)
    return [int(round(hi * (lo / hi) ** ((i * step) % 1.0))) for i in range(n)]


def _append_sizes(c):
    """(new tokens, first position) of each sequence."""
    new = _spread(c["seqs"], (c["new"] + 1) // 2, c["new"])
    start = [0] * c["seqs"] if c["start"] == 0 else _spread(c["seqs"], c["start"] // 4, c["start"], 0.7548776662466927)
    return new, start


def _attend_sizes(c):
    """(query tokens, context length) of each sequence; the queries are the context's last tokens."""
    ctx = [c["ctx"]] * c["seqs"] if not c["ragged"] else _spread(c["seqs"], c["ctx"] // 8, c["ctx"])
    most = c["queries"]
    nq = [most] * c["seqs"] if not c["ragged"] or most == 1 else _spread(c["seqs"], (most + 1) // 2, most)
    return [min(q, t) for q, t in zip(nq, ctx)], ctx


def _first_keys(c, nq, ctx):
    """First visible position of each query row: the start of its document (documents cut the context evenly)."""
    if not c["docs"]:
        return None
    rows = []
    for q, t in zip(nq, ctx):
        size = -(-t // c["docs"])
        rows += [p // size * size for p in range(t - q, t)]
    return rows


def work(c):
    es = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] == "merge":
        return {"bytes": c["rows"] * c["heads"] * (c["parts"] + 1) * (c["d"] * es + 4), "flops": 0}
    if c["op"] == "append":
        n = sum(_append_sizes(c)[0])
        blocks = sum((s + k - 1) // c["block"] - s // c["block"] + 1 for k, s in zip(*_append_sizes(c)))
        kv = n * c["hkv"] * 2 * c["d"] * (es + 1) + blocks * c["hkv"] * 8
        return {"bytes": kv + n * c["hq"] * c["d"] * 2 * es + n * c["rot"] * 4, "flops": 0}
    nq, ctx = _attend_sizes(c)
    first = _first_keys(c, nq, ctx)
    pairs = keys = row = 0
    for q, t in zip(nq, ctx):
        low = None
        for p in range(t - q, t):
            f = first[row] if first else 0
            lo = max(f, p - c["window"] + 1 if c["window"] else 0)
            seen = p + 1 - lo
            pre = min(c["prefix"], t)
            seen += max(0, min(pre, lo) - f) + max(0, pre - max(p + 1, f))
            pairs += seen
            low = lo if low is None else min(low, lo)
            row += 1
        keys += t - low + max(0, min(c["prefix"], low))
    n = sum(nq)
    return {"bytes": keys * c["hkv"] * (2 * c["d"] + 8 / c["block"]) + n * c["hq"] * (2 * c["d"] * es + 4),
            "flops": 4.0 * c["d"] * c["hq"] * pairs}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _pool(c, blocks, gen):
    """A paged cache of `blocks` blocks as earlier appends left it: codes of normal data, scales that differ by block and
    head, and stale bytes (not-a-number codes among the e4m3 ones) wherever a sequence's last block is not full."""
    shape = (blocks, c["hkv"], 2, c["block"], c["d"])
    scales = torch.exp(0.5 * torch.randn(shape[:3], device=DEV, generator=gen))
    if c["code"] == "int8":
        codes = torch.empty(shape, dtype=torch.int8, device=DEV)
        for i in range(0, blocks, 4096):  # a normal value's block has its largest magnitude near 3.5 deviations
            x = torch.randn((min(4096, blocks - i),) + shape[1:], device=DEV, generator=gen)
            codes[i:i + 4096] = (x * (127 / 3.5)).round().clamp(-127, 127).to(torch.int8)
        return codes, scales * (3.5 / 127)
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    for i in range(0, blocks, 4096):
        x = torch.randn((min(4096, blocks - i),) + shape[1:], device=DEV, generator=gen)
        codes[i:i + 4096] = (x * (448 / 3.5)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, scales * (3.5 / 448)


def _tables(c, first, last, gen):
    """Block tables of sequences whose blocks first..last-1 lie at random places of a pool; -1 elsewhere."""
    total = sum(b - a for a, b in zip(first, last))
    ids = torch.randperm(total, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((len(last), max(last)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, (a, b) in enumerate(zip(first, last)):
        table[s, a:b] = ids[at:at + b - a]
        at += b - a
    return table, total


def _cu(sizes):
    return torch.tensor([0] + sizes, device=DEV).cumsum(0).to(torch.int32)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) % (1 << 62))
    dt = TYPE[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, device=DEV, generator=gen, dtype=dt)

    if c["op"] == "merge":
        outs = [normal(c["rows"], c["heads"], c["d"]) for _ in range(c["parts"])]
        lses = [5 + 2 * torch.randn(c["rows"], c["heads"], device=DEV, generator=gen) for _ in range(c["parts"])]
        lses[-1][::7] = -math.inf  # rows whose last part saw no key
        return dict(c=c, outs=outs, lses=lses, out=torch.empty_like(outs[0]), lse=torch.empty_like(lses[0]))

    B = c["block"]
    if c["op"] == "append":
        new, start = _append_sizes(c)
        # only the blocks that the new tokens go into are mapped
        table, blocks = _tables(c, [s // B for s in start], [(s + n - 1) // B + 1 for s, n in zip(start, new)], gen)
        codes, scales = _pool(c, blocks, gen)
        n = sum(new)
        qkv = normal(n, c["hq"] + 2 * c["hkv"], c["d"])  # the fused projection's result: q, k and v are views of it
        q, k, v = qkv.split([c["hq"], c["hkv"], c["hkv"]], 1)
        top = max(s + m for s, m in zip(start, new))
        freq = 500000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        angle = torch.arange(top, device=DEV, dtype=torch.float64)[:, None] * freq
        rope = torch.cat([angle.cos(), angle.sin()], 1).float()
        return dict(c=c, codes=codes, scales=scales, table=table, cu=_cu(new), q=q, k=k, v=v, rope=rope, max_new=max(new),
                    start=torch.tensor(start, dtype=torch.int32, device=DEV),
                    q_out=torch.empty(n, c["hq"], c["d"], dtype=dt, device=DEV))

    nq, ctx = _attend_sizes(c)
    table, blocks = _tables(c, [0] * len(ctx), [-(-t // B) for t in ctx], gen)
    codes, scales = _pool(c, blocks, gen)
    for s, t in enumerate(ctx):
        if t % B:
            codes[table[s, t // B].long(), :, :, t % B:] = torch.tensor(127, dtype=torch.uint8, device=DEV).view(CODE[c["code"]])
    n = sum(nq)
    st = dict(c=c, codes=codes, scales=scales, table=table, cu=_cu(nq), q=normal(n, c["hq"], c["d"]), max_q=max(nq),
              max_ctx=max(ctx), ctx=torch.tensor(ctx, dtype=torch.int32, device=DEV),
              out=torch.empty(n, c["hq"], c["d"], dtype=dt, device=DEV),
              lse=torch.empty(n, c["hq"], dtype=torch.float32, device=DEV), slopes=None, prefix=None, first=None)
    if c["alibi"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["hq"] + 1, device=DEV) / c["hq"]).float()
    if c["prefix"]:
        st["prefix"] = torch.full((len(ctx),), c["prefix"], dtype=torch.int32, device=DEV)
    if c["docs"]:
        st["first"] = torch.tensor(_first_keys(c, nq, ctx), dtype=torch.int32, device=DEV)
    if own:  # the workspace that a program allocates once for its largest step
        from residual_kv_cache_delta_b200 import deltakv as D
        st["ws"] = D.alloc_workspace(D.kv8_attention_workspace(_shape(c), len(ctx), n, max(nq), max(ctx)), DEV)
    return st


# ---------------------------------------------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------------------------------------------
def _shape(c):
    from residual_kv_cache_delta_b200 import deltakv as D
    return D.KV8Shape(c["hq"], c["hkv"], c["d"], c["block"], TYPE[c["dtype"]], c["code"])


def run(state):
    return {"append": _run_append, "attention": _run_attention, "merge": _run_merge}[state["c"]["op"]](state)


def _run_merge(st):
    if own:
        from residual_kv_cache_delta_b200 import deltakv as D
        D.deltakv_merge_attention(st["outs"], st["lses"], st["out"], st["lse"])
        return st["out"], st["lse"]
    lses = torch.stack(st["lses"])
    m = lses.amax(0)
    w = torch.exp(lses - torch.where(m == -math.inf, 0.0, m))
    total = w.sum(0)
    out = (w[..., None] * torch.stack(st["outs"]).float()).sum(0) / torch.where(total > 0, total, 1.0)[..., None]
    return out.to(st["out"].dtype), torch.log(total) + m


def _rotate(x, cs, pairs):
    """Rotation of the first rot dimensions of x [n, heads, d] by cs [n, rot] (cosines, then sines)."""
    rot = cs.shape[1]
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if pairs else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _quantise(x, code):
    x = x.clamp(-QMAX[code], QMAX[code])
    return x.round().to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _run_append(st):
    c = st["c"]
    if own:
        from residual_kv_cache_delta_b200 import deltakv as D
        D.deltakv_kv8_append(_shape(c), D.KV8Cache(st["codes"], st["scales"]), st["k"], st["v"], st["cu"], st["start"],
                             st["table"], st["max_new"], rope=st["rope"], rope_pairs=c["pairs"], q=st["q"],
                             q_out=st["q_out"])
        return st["codes"], st["scales"], st["q_out"]
    B, codes, scales, start = c["block"], st["codes"], st["scales"], st["start"].long()
    cu = st["cu"].long()
    n = st["k"].shape[0]
    row = torch.arange(n, device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    pos = start[seq] + row - cu[seq]
    block, offset = st["table"][seq, pos // B].long(), pos % B
    cs = st["rope"][pos]
    kv = torch.stack([_rotate(st["k"].float(), cs, c["pairs"]), st["v"].float()], 2)  # [n, head, half, d]
    q_out = _rotate(st["q"].float(), cs, c["pairs"]).to(st["q"].dtype)
    # the largest magnitude of each block's new rows, then the scale: it never shrinks while a block holds earlier rows
    top = torch.zeros_like(scales).index_reduce_(0, block, kv.abs().amax(-1), "amax")
    touched = torch.zeros(len(scales), dtype=torch.bool, device=DEV)
    touched[block] = True
    held = torch.zeros(len(scales), dtype=torch.long, device=DEV)  # rows that the block holds already
    held[st["table"][torch.arange(len(start), device=DEV), start // B].long()] = start % B
    old = torch.where(held[:, None, None] > 0, scales, 0.0)
    grown = torch.maximum(top.clamp(min=FLOOR) * (1.0 / QMAX[c["code"]]), old)
    inv = torch.ones_like(grown) / grown
    # earlier rows follow the scale
    some = held.nonzero()[:, 0]
    ratio = (old * inv)[some][..., None, None]
    rows = torch.arange(B, device=DEV)[:, None] < held[some][:, None, None, None, None]
    codes_b = codes.view(torch.uint8)
    codes_b[some] = torch.where(rows, _quantise(codes[some].float() * ratio, c["code"]).view(torch.uint8), codes_b[some])
    # the new rows
    codes_b[block, :, :, offset] = _quantise(kv * inv[block][..., None], c["code"]).view(torch.uint8)
    scales.copy_(torch.where(touched[:, None, None], grown, scales))
    return codes, scales, q_out


def _run_attention(st):
    c = st["c"]
    if own:
        from residual_kv_cache_delta_b200 import deltakv as D
        D.deltakv_kv8_attention(_shape(c), D.KV8Cache(st["codes"], st["scales"]), st["q"], st["cu"], st["ctx"],
                                st["table"], st["max_q"], st["max_ctx"], st["out"], st["lse"], st["ws"],
                                softcap=c["softcap"], window=c["window"], alibi_slopes=st["slopes"],
                                prefix_lens=st["prefix"], first_key=st["first"])
        return st["out"], st["lse"]
    S, H, G, d, Q, T = c["seqs"], c["hkv"], c["hq"] // c["hkv"], c["d"], st["max_q"], st["max_ctx"]
    ctx, cu = st["ctx"].long(), st["cu"].long()
    table = st["table"].long().clamp(min=0)
    t = torch.arange(table.shape[1] * c["block"], device=DEV)
    kv = st["codes"][table].float() * st["scales"][table][..., None, None]  # [S, blocks, H, 2, B, d]
    kv = kv.permute(3, 0, 2, 1, 4, 5).flatten(3, 4)                          # [2, S, H, T, d]
    kv = torch.where((t < ctx[:, None])[:, None, :, None], kv, 0.0)
    # rows of the queries, padded to Q per sequence
    i = torch.arange(Q, device=DEV)
    nq = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp(max=len(st["q"]) - 1)                    # [S, Q]
    pos = (ctx - nq)[:, None] + i
    q = st["q"].float().view(-1, H, G, d)[row].permute(0, 2, 3, 1, 4)         # [S, H, G, Q, d]
    x = (q.flatten(2, 3) @ kv[0].transpose(-1, -2)).unflatten(2, (G, Q)) * (1.0 / math.sqrt(d))
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    gap = pos[:, :, None] - t                                                 # [S, Q, T]
    if c["alibi"]:
        x = x - st["slopes"].view(H, G, 1, 1) * gap.abs()[:, None, None]
    see = gap >= 0
    if c["window"]:
        see = see & (gap < c["window"])
    if c["prefix"]:
        see = see | (t < st["prefix"][:, None])[:, None]
    if c["docs"]:
        see = see & (t >= st["first"][row][:, :, None])
    see = see & (t < ctx[:, None])[:, None]
    x = torch.where(see[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    out = (x.flatten(2, 3) @ kv[1]).unflatten(2, (G, Q)) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + m)[..., 0]
    seq = torch.repeat_interleave(torch.arange(S, device=DEV), nq, output_size=len(st["q"]))
    at = torch.arange(len(st["q"]), device=DEV) - cu[seq]
    out, lse = out.permute(0, 3, 1, 2, 4)[seq, at], lse.permute(0, 3, 1, 2)[seq, at]
    return out.flatten(1, 2).to(st["q"].dtype), lse.flatten(1, 2)


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "merge":
        weight, out = 0.0, 0.0
        top = torch.stack(st["lses"]).double().max(0).values
        for o, l in zip(st["outs"], st["lses"]):
            w = (l.double() - top).exp()
            weight, out = weight + w, out + w[..., None] * o.double()
        return out / weight[..., None], top + weight.log()
    if c["op"] == "append":
        return _exact_append(c, st)
    return _exact_attention(c, st)


def _exact_append(c, st):
    B, rot, half = c["block"], c["rot"], c["rot"] // 2
    new, start = _append_sizes(c)
    first = torch.arange(0, rot, 2, device=DEV) if c["pairs"] else torch.arange(half, device=DEV)
    second = first + (1 if c["pairs"] else half)
    q_out = torch.empty(st["q_out"].shape, dtype=torch.float64, device=DEV)
    codes, scales = st["codes"].double() if c["code"] == "e4m3" else None, st["scales"].double()
    at = 0
    for s, (n, p0) in enumerate(zip(new, start)):
        rows = slice(at, at + n)
        at += n
        cs = st["rope"][p0:p0 + n].double()
        cos, sin = cs[:, None, :half], cs[:, None, half:]
        turned = []
        for x in (st["q"][rows].double(), st["k"][rows].double()):
            y = x.clone()
            y[..., first] = x[..., first] * cos - x[..., second] * sin
            y[..., second] = x[..., second] * cos + x[..., first] * sin
            turned.append(y)
        q_out[rows] = turned[0]
        kv = torch.stack([turned[1], st["v"][rows].double()], 2)
        # rows of whole blocks, the held rows of the first block as nothing
        b0, b1 = p0 // B, (p0 + n - 1) // B + 1
        ids = st["table"][s, b0:b1].long()
        x = torch.zeros(((b1 - b0) * B,) + kv.shape[1:], dtype=torch.float64, device=DEV)
        x[p0 - b0 * B:p0 - b0 * B + n] = kv
        x = x.unflatten(0, (b1 - b0, B)).permute(0, 2, 3, 1, 4)                # [blocks, H, 2, B, d]
        step = x.abs().amax((-1, -2)).clamp(min=FLOOR) / QMAX[c["code"]]
        if p0 % B:
            step[0] = torch.maximum(step[0], scales[ids[0]])
        if codes is not None:
            y = codes[ids]
            if p0 % B:
                y[0, :, :, :p0 % B] *= (scales[ids[0]] / step[0])[..., None, None]
            r = torch.arange((b1 - b0) * B, device=DEV).view(b1 - b0, 1, 1, B, 1) - (p0 - b0 * B)
            codes[ids] = torch.where((r >= 0) & (r < n), x / step[..., None, None], y)
        scales[ids] = step
    return codes, scales, q_out


def _exact_attention(c, st):
    nq, ctx = _attend_sizes(c)
    G, B, d = c["hq"] // c["hkv"], c["block"], c["d"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for s, (n, T) in enumerate(zip(nq, ctx)):
        ids = st["table"][s, :-(-T // B)].long()
        key = torch.arange(T, device=DEV)
        for r0 in range(0, n, 512):
            rows = slice(at + r0, at + min(n, r0 + 512))
            p = T - n + torch.arange(r0, min(n, r0 + 512), device=DEV)[:, None]
            hide = key > p
            if c["window"]:
                hide |= key <= p - c["window"]
            if c["prefix"]:
                hide &= key >= c["prefix"]
            if c["docs"]:
                hide |= key < st["first"][rows].long()[:, None]
            for h in range(c["hkv"]):
                k, v = ((st["codes"][ids, h, j].double() * st["scales"][ids, h, j].double()[:, None, None])
                        .flatten(0, 1)[:T] for j in (0, 1))
                for g in range(h * G, h * G + G):
                    x = st["q"][rows, g].double() @ k.T / math.sqrt(d)
                    if c["softcap"]:
                        x = c["softcap"] * torch.tanh(x / c["softcap"])
                    if c["alibi"]:
                        x = x - st["slopes"][g].double() * (p - key).abs()
                    x.masked_fill_(hide, -math.inf)
                    lse[rows, g] = torch.logsumexp(x, -1)
                    out[rows, g] = torch.softmax(x, -1).nan_to_num(0.0) @ v
        at += n
    return out, lse
