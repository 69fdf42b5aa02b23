"""Plain implementations of the 8-bit cache's operators for the tests (CPU): the append's fp32 definition step by step,
attention and merge in fp64, and the error bounds that the kernels are held to."""
import math

import torch

from residual_kv_cache_delta_b200 import deltakv as D

FLOOR = 2.0 ** -64
TOP = {"int8": 127.0, "e4m3": 448.0}


def f32(x):
    return torch.tensor(x, dtype=torch.float32)


def quantise(y, code):
    y = y.clamp(-TOP[code], TOP[code])
    return y.round().to(torch.int8) if code == "int8" else y.to(torch.float8_e4m3fn)


def rotate(x, cs, pairs, dtype=torch.float32):
    """Rotates x [n, heads, d] by rows cs [n, rot] (cosines, then sines); every step in `dtype`."""
    x, cs = x.to(dtype), cs.to(dtype)
    rot = cs.shape[1]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    first = torch.arange(0, rot, 2) if pairs else torch.arange(rot // 2)
    second = first + (1 if pairs else rot // 2)
    y = x.clone()
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def append(shape, codes, scales, k, v, cu, start, table, rope=None, pairs=False, positions=None):
    """The append in fp32, block by block; codes [nb, H, 2, B, d] and scales are changed in place."""
    B, top = shape.block_tokens, f32(TOP[shape.code])
    for s in range(len(start)):
        n, p0 = cu[s + 1] - cu[s], start[s]
        if n == 0:
            continue
        rows = slice(cu[s], cu[s + 1])
        pos = torch.arange(p0, p0 + n) if positions is None else positions[rows].long()
        kk = k[rows].float()
        if rope is not None:
            ok = (pos >= 0) & (pos < len(rope))
            turned = rotate(kk, rope[pos.clamp(0, len(rope) - 1)], pairs)
            kk = torch.where(ok[:, None, None], turned, kk)
        x = torch.stack([kk, v[rows].float()], 2)  # [n, H, 2, d]
        for b in range(p0 // B, (p0 + n - 1) // B + 1):
            r0, r1 = max(b * B, p0) - p0, min((b + 1) * B, p0 + n) - p0
            off = r0 + p0 - b * B
            blk = int(table[s, b])
            for h in range(x.shape[1]):
                for j in range(2):
                    y = x[r0:r1, h, j]
                    old = scales[blk, h, j].clone() if off > 0 else f32(0.0)
                    if not torch.isfinite(y).all() or not torch.isfinite(old):
                        scales[blk, h, j] = math.nan
                        codes[blk, h, j, off:off + r1 - r0] = quantise(torch.zeros_like(y), shape.code)
                        continue
                    now = torch.maximum(y.abs().max(), f32(FLOOR)) * (f32(1.0) / top)
                    now = torch.maximum(now, old)
                    inv = f32(1.0) / now
                    if off > 0 and now > old:
                        codes[blk, h, j, :off] = quantise(codes[blk, h, j, :off].float() * (old * inv), shape.code)
                    codes[blk, h, j, off:off + r1 - r0] = quantise(y * inv, shape.code)
                    scales[blk, h, j] = now


def random_codes(shape, dims, gen):
    raw = torch.randint(0, 256, dims, generator=gen, dtype=torch.int64).to(torch.uint8)
    if shape.code == "int8":
        raw[raw == 128] = 0
        return raw.view(torch.int8)
    # values of a filled block: magnitudes up to 448, no NaN codes
    x = torch.randn(dims, generator=gen) * 120
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def cache_for(shape, ctx, gen, spare=3, scale=0.02):
    """A CPU cache whose sequences hold `ctx` tokens at shuffled blocks: (codes, scales, table).  Rows behind a sequence's
    last token hold the byte 0x7f (an e4m3 NaN), blocks of no sequence too, with NaN scales; table entries that no
    sequence needs are -1."""
    B, H, d = shape.block_tokens, shape.num_kv_heads, shape.head_dim
    need = [-(-t // B) for t in ctx]
    nb = sum(need) + spare
    codes = random_codes(shape, (nb, H, 2, B, d), gen)
    scales = scale * torch.exp(0.7 * torch.randn(nb, H, 2, generator=gen))
    ids = torch.randperm(nb, generator=gen)
    table = torch.full((len(ctx), max(need + [1]) + 1), -1, dtype=torch.int32)
    raw = codes.view(torch.uint8)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n].int()
        if ctx[s] % B:
            raw[ids[at + n - 1], :, :, ctx[s] % B:] = 0x7f
        at += n
    raw[ids[at:]] = 0x7f
    scales[ids[at:]] = math.nan
    return codes, scales, table


def visible(nq, T, window, prefix, first):
    p = (T - nq + torch.arange(nq))[:, None]
    t = torch.arange(T)[None]
    see = t <= p
    if window:
        see &= p - t < window
    see |= t < prefix
    if first is not None:
        see &= t >= first[:, None]
    return see


def attention(shape, codes, scales, table, q, cu, ctx, scale=0.0, softcap=0.0, window=0, slopes=None, prefix=None,
              first=None):
    """(out, lse, bound on |out - kernel's|, bound on |lse - kernel's|) in fp64, rows of no sequence left NaN.

    The kernels' error: a score is a sum of d products in fp32 (d 2^-24 of the sum of magnitudes), then a handful of
    fp32 roundings of the score and its bias (and 2^-20 of the cap); the weights' hardware exponential is off by
    2^-21, their fp16 rounding (bf16 storage) by 2^-11 of the weight; what is rounded there is weight times V scale
    relative to the row's largest such product, so below the smallest normal fp16 by 2^-25 of that, times the code; sums over T keys by T 2^-24; the result by half a step of its type."""
    n, Hq, d = q.shape
    G, B = Hq // shape.num_kv_heads, shape.block_tokens
    sc = scale if scale > 0 else 1.0 / math.sqrt(d)
    out = torch.full((n, Hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((n, Hq), math.nan, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    bf = shape.dtype == torch.bfloat16
    for s, T in enumerate(ctx):
        r0, nq = cu[s], cu[s + 1] - cu[s]
        if nq == 0:
            continue
        rows = slice(r0, r0 + nq)
        ids = table[s, :-(-T // B)].long()
        kv = (codes[ids].double() * scales[ids].double()[..., None, None]).permute(2, 1, 0, 3, 4).flatten(2, 3)
        k, v = kv[0][:, :T], kv[1][:, :T]  # [H, T, d]
        see = visible(nq, T, window, int(prefix[s]) if prefix is not None else 0,
                      first[rows].long() if first is not None else None)
        gap = ((T - nq + torch.arange(nq))[:, None] - torch.arange(T)[None]).abs().double()
        for h in range(Hq):
            qq, kk, vv = q[rows, h].double(), k[h // G], v[h // G]
            x = qq @ kk.T * sc
            err = 2.0 ** -24 * d * (qq.abs() @ kk.abs().T * sc)
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                err = err + 2.0 ** -20 * softcap
            if slopes is not None:
                bias = slopes[h].double() * gap
                err = err + 2.0 ** -22 * bias
                x = x - bias
            err = err + 2.0 ** -22 * x.abs()
            x = x.masked_fill(~see, -math.inf)
            lse[rows, h] = torch.logsumexp(x, -1) if T else -math.inf
            any_ = see.any(-1)
            w = torch.softmax(x, -1).masked_fill(~any_[:, None], 0.0) if T else x
            out[rows, h] = w @ vv.masked_fill(~see.any(0)[:, None], 0.0) if T else 0.0
            if T == 0 or not any_.any():
                continue
            e = err.masked_fill(~see, 0.0).nan_to_num(0.0).amax(-1) + 2.0 ** -21 + T * 2.0 ** -24
            vv = vv.nan_to_num(0.0).abs()
            wsum = w.nan_to_num(0.0) @ vv
            half = 2.0 ** -8 if bf else 2.0 ** -24
            t = (2 * e[:, None] + (2.0 ** -11 if bf else 0.0)) * wsum * 1.01 + half * 1.01 * out[rows, h].abs()
            if bf:
                vs = scales[ids, h // G, 1].double().repeat_interleave(B)[:T].nan_to_num(0.0)
                code = codes[ids, h // G, 1].double().flatten(0, 1)[:T].abs().masked_fill(~see.any(0)[:, None], 0.0)
                t = t + 2.0 ** -25 * (w.nan_to_num(0.0) * vs).amax(-1, keepdim=True) * code.sum(0)
            tol[rows, h] = t + 1e-30
            tol_l[rows, h] = e + 2.0 ** -22 * lse[rows, h].abs().nan_to_num(0.0, posinf=0.0)
    return out, lse, tol, tol_l


def check(got, ref, tol, what):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    fin = torch.isfinite(ref)
    over = ((got - ref).abs() - tol)[fin]
    worst = ((got - ref).abs() / tol.clamp(min=1e-300))[fin]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: error is {worst.max():.3g} of its bound"


def run_attention(shape, codes, scales, table, q, cu, ctx, dev, max_q=None, max_ctx=None, slopes=None, prefix=None,
                  first=None, cu_none=False, stream=None, fill=math.nan, **kw):
    nq = [b - a for a, b in zip(cu[:-1], cu[1:])]
    max_q, max_ctx = max_q or max(nq), max_ctx if max_ctx is not None else max(ctx)

    def to(t):
        return None if t is None else t.to(dev)

    n = q.shape[0]
    cache = D.KV8Cache(codes.view(torch.uint8).to(dev).view(shape.code_dtype), scales.to(dev))
    out = torch.full((n, shape.num_q_heads, shape.head_dim), fill, dtype=shape.dtype, device=dev)
    lse = torch.full((n, shape.num_q_heads), fill, dtype=torch.float32, device=dev)
    ws = D.alloc_workspace(D.kv8_attention_workspace(shape, len(ctx), n, max_q, max_ctx), dev).fill_(0xff)
    D.deltakv_kv8_attention(shape, cache, q.to(dev), None if cu_none else torch.tensor(cu, dtype=torch.int32, device=dev),
                            torch.tensor(ctx, dtype=torch.int32, device=dev), table.to(dev), max_q, max_ctx, out, lse,
                            ws, alibi_slopes=to(slopes), prefix_lens=to(prefix), first_key=to(first), stream=stream, **kw)
    torch.cuda.synchronize()
    return out, lse
