"""The 8-bit paged cache on the GPU (deltakv_kv8_append, deltakv_kv8_attention, deltakv_merge_attention) against plain
implementations: the append bit by bit against its fp32 definition, attention and merge against fp64 within bounds that
follow from the arithmetic (tests/_kv8.py)."""
import math

import numpy as np
import pytest
import torch

from residual_kv_cache_delta_b200 import deltakv as D
from residual_kv_cache_delta_b200 import synth

import _cases as C  # noqa: E402
import _kv8 as K  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from residual_kv_cache_delta_b200 import build
    build.build()
    D.load_library()
    yield
    assert D.deltakv_get_device_error() == 0


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _cu(sizes):
    return [0] + list(np.cumsum(sizes))


def _i32(x, dev="cuda"):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device=dev)


def _rope(n, rot, gen):
    ang = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


# ------------------------------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------------------------------
def _append_case(shape, new, start, rot, pairs, seed, strided=False, positions=None, edit=None, max_new=None):
    """Runs an append on a cache that already holds `start` tokens and compares every byte of it."""
    g = _gen(seed)
    H, Hq, d = shape.num_kv_heads, shape.num_q_heads, shape.head_dim
    codes, scales, table = K.cache_for(shape, [s + n for s, n in zip(start, new)], g)
    n, cu = sum(new), _cu(new)
    qkv = (torch.randn(n, Hq + 2 * H, d, generator=g) * torch.exp(torch.randn(n, 1, 1, generator=g))).to(shape.dtype)
    if edit is not None:
        edit(qkv, Hq, H)
    rope = _rope(max([s + m for s, m in zip(start, new)] + [1]), rot, g) if rot else None
    dev = "cuda"
    dq = qkv.to(dev)
    q, k, v = dq.split([Hq, H, H], 1)
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cache = D.KV8Cache(codes.view(torch.uint8).to(dev).view(shape.code_dtype), scales.to(dev))
    q_out = torch.full((n, Hq, d), 7.0, dtype=shape.dtype, device=dev) if rot else None
    pos = None if positions is None else positions.to(dev)
    D.deltakv_kv8_append(shape, cache, k, v, _i32(cu), _i32(start), table.to(dev), max_new or max(new),
                         rope=None if rope is None else rope.to(dev), rope_pairs=pairs, positions=pos,
                         q=q if rot else None, q_out=q_out)
    torch.cuda.synchronize()
    cq, ck, cv = qkv.split([Hq, H, H], 1)
    K.append(shape, codes, scales, ck, cv, cu, start, table, rope, pairs, positions)
    got, want = cache.codes.view(torch.uint8).cpu(), codes.view(torch.uint8)
    assert torch.equal(got, want), f"{(got != want).sum()} of {want.numel()} codes differ"
    assert torch.equal(cache.scales.cpu().view(torch.int32), scales.view(torch.int32)) or \
        torch.equal(cache.scales.cpu().nan_to_num(-1.0), scales.nan_to_num(-1.0))
    if rot:
        p = torch.cat([torch.arange(s, s + m) for s, m in zip(start, new)]) if positions is None else positions.long()
        assert torch.equal(q_out.cpu(), K.rotate(cq, rope[p], pairs).to(shape.dtype))
    return codes, scales, table, ck, cv, cu, rope


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,B,rot,pairs,hq,hkv", [(128, 16, 128, False, 8, 2), (128, 32, 64, True, 3, 3),
                                                  (64, 64, 64, False, 6, 2), (64, 16, 32, True, 16, 1),
                                                  (128, 64, 96, False, 5, 5), (64, 32, 0, False, 4, 4)])
def test_append_matches_its_definition_bit_by_bit(code, dtype, d, B, rot, pairs, hq, hkv):
    shape = D.KV8Shape(hq, hkv, d, B, dtype, code)
    _append_case(shape, [1, 37, 0, B, 2 * B + 1, 1], [0, 5, 3, B - 1, 2 * B, B], rot, pairs, 1)
    _append_case(shape, [1, 1, 1], [B - 1, B, 7], rot, pairs, 2, strided=True)
    _append_case(shape, [300], [0], rot, pairs, 3, strided=True, max_new=1000)


def test_append_value_error_is_half_a_step():
    """Against fp64: a code is within half a step (e4m3: half a step of its binade) of the rotated value, plus the
    roundings of the fp32 rotation and of the two products in front of the code (2^-22 of the largest value)."""
    for code in ("int8", "e4m3"):
        shape = D.KV8Shape(4, 2, 128, 32, BF, code)
        codes, scales, table, k, v, cu, rope = _append_case(shape, [95], [0], 128, False, 5)
        ids = table[0, :3].long()
        val = (codes[ids].double() * scales[ids].double()[..., None, None]).permute(0, 3, 1, 2, 4).flatten(0, 1)[:95]
        true = torch.stack([K.rotate(k, rope[:95], False, torch.float64), v.double()], 2)
        step = scales[ids].double().repeat_interleave(32, 0)[:95][..., None]
        if code == "int8":
            bound = 0.5 * step + 2.0 ** -22 * 127 * step
        else:  # half a step: 2^-4 of the value, at least half the smallest subnormal (2^-10)
            bound = torch.maximum(2.0 ** -4 * true.abs(), 2.0 ** -10 * step) * (1 + 2.0 ** -20) + 2.0 ** -22 * 448 * step
        assert ((val - true).abs() <= bound).all()


def test_append_token_by_token_recodes_a_growing_block():
    """One token at a time, magnitudes rising and falling: each step equals the definition, scales never shrink."""
    for code in ("int8", "e4m3"):
        shape = D.KV8Shape(2, 2, 64, 16, BF, code)
        g = _gen(3)
        n = 40
        x = torch.randn(n, 4, 64, generator=g) * torch.tensor([1.0, 3.0, 0.1, 9.0] * 10)[:, None, None]
        x = x.to(BF)
        codes, scales, table = K.cache_for(shape, [n], g)
        cache = D.KV8Cache(codes.view(torch.uint8).cuda().view(shape.code_dtype), scales.cuda())
        for i in range(n):
            k, v = x[i:i + 1, :2].contiguous(), x[i:i + 1, 2:].contiguous()
            D.deltakv_kv8_append(shape, cache, k.cuda(), v.cuda(), _i32([0, 1]), _i32([i]), table.cuda(), 1)
            before = scales[table[0, i // 16].long()].clone()
            K.append(shape, codes, scales, k, v, [0, 1], [i], table)
            assert i % 16 == 0 or (scales[table[0, i // 16].long()] >= before).all()
        torch.cuda.synchronize()
        assert torch.equal(cache.codes.view(torch.uint8).cpu(), codes.view(torch.uint8))
        assert torch.equal(cache.scales.cpu().nan_to_num(-1.0), scales.nan_to_num(-1.0))


def test_append_positions_of_their_own_and_outside_the_table():
    shape = D.KV8Shape(4, 2, 64, 16, BF, "int8")
    pos = torch.tensor([5, 5, 0, 29, 1] + list(range(25)), dtype=torch.int32)
    _append_case(shape, [5, 25], [4, 5], 64, False, 9, positions=pos)
    g = _gen(10)
    codes, scales, table = K.cache_for(shape, [3], g)
    k = torch.randn(3, 2, 64, generator=g).to(BF)
    cache = D.KV8Cache(codes.cuda(), scales.cuda())
    rope = _rope(2, 64, g)
    D.deltakv_kv8_append(shape, cache, k.cuda(), k.cuda(), _i32([0, 3]), _i32([0]), table.cuda(), 3, rope=rope.cuda())
    assert D.deltakv_get_device_error() == 3  # position 2 lies outside the table's two rows: not rotated, recorded
    K.append(shape, codes, scales, k, k, [0, 3], [0], table, rope)
    assert torch.equal(cache.codes.cpu(), codes)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_of_values_that_are_not_finite(bad, code):
    shape = D.KV8Shape(2, 2, 128, 16, BF, code)

    def edit(x, hq, h):
        x[3, hq, 70] = bad          # K of token 3, head 0
        x[30, hq + h + 1, 5] = bad  # V of token 30, head 1

    _append_case(shape, [40], [0], 0, False, 4, edit=edit)
    _append_case(shape, [40], [6], 128, False, 4, edit=edit)


def test_append_of_zeros_tiny_and_huge_values():
    shape = D.KV8Shape(2, 1, 64, 16, F32, "int8")
    for code in ("int8", "e4m3"):
        shape = D.KV8Shape(2, 1, 64, 16, F32, code)
        for f in (0.0, 1e-30, 1e-41, 3e37):
            _append_case(shape, [20], [0], 64, False, 6, edit=lambda x, hq, h: x.mul_(f))


def test_append_writes_nothing_for_lengths_that_break_their_bounds():
    shape = D.KV8Shape(2, 1, 64, 16, BF, "int8")
    g = _gen(8)
    codes, scales, table = K.cache_for(shape, [40, 40], g)
    k = torch.randn(20, 1, 64, generator=g).to(BF).cuda()
    for cu, start, tab, code in (([0, 10, 20], [0, -1], table, 3), ([0, 12, 20], [0, 0], table, 3),
                                 ([0, 10, 25], [0, 0], table, 3), ([0, 10, 20], [0, 100000], table, 1),
                                 ([0, 10, 20], [0, 0], table.clone().fill_(codes.shape[0]), 1)):
        cache = D.KV8Cache(codes.cuda(), scales.cuda())
        D.deltakv_kv8_append(shape, cache, k, k, _i32(cu), _i32(start), tab.cuda(), 10)
        assert D.deltakv_get_device_error() == code
        bad = {tuple([0, 12, 20]): 0}.get(tuple(cu), 1)
        keep = table[bad].long()
        keep = keep[keep >= 0]
        assert torch.equal(cache.codes.cpu()[keep], codes[keep])
        assert torch.equal(cache.scales.cpu()[keep], scales[keep])


# ------------------------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------------------------
def _attention_case(shape, nq, ctx, seed, mods=(), cu_none=False, max_q=None, scale=0.0):
    g = _gen(seed)
    n, cu = sum(nq), _cu(nq)
    codes, scales, table = K.cache_for(shape, ctx, g)
    q = (torch.randn(n, shape.num_q_heads, shape.head_dim, generator=g) *
         torch.exp2(torch.randint(-3, 2, (n, shape.num_q_heads, 1), generator=g).float())).to(shape.dtype)
    kw, ref = dict(softmax_scale=scale), dict(scale=scale)
    for m in mods:
        if m == "softcap":
            kw["softcap"] = ref["softcap"] = 5.0
        elif m == "alibi":
            kw["slopes"] = ref["slopes"] = torch.exp2(-torch.arange(shape.num_q_heads).float() / 2)
        elif m.startswith("window"):
            kw["window"] = ref["window"] = int(m[6:])
        elif m.startswith("prefix"):
            p = torch.tensor([int(m[6:]) + 3 * s for s in range(len(ctx))], dtype=torch.int32)
            kw["prefix"] = p
            ref["prefix"] = p
        elif m == "docs":  # documents of uneven length; some rows' documents begin behind them: nothing is seen
            first = []
            for a, t in zip(nq, ctx):
                for p in range(t - a, t):
                    first.append(p // 37 * 37 if p % 11 else p + 1)
            kw["first"] = ref["first"] = torch.tensor(first, dtype=torch.int32)
    out, lse = K.run_attention(shape, codes, scales, table, q, cu, ctx, "cuda", cu_none=cu_none, max_q=max_q, **kw)
    ro, rl, to, tl = K.attention(shape, codes, scales, table, q, cu, ctx, **ref)
    K.check(lse, rl, tl, "lse")
    K.check(out, ro, to, "out")


DECODE_CTX = [1, 15, 16, 17, 0, 64, 65, 255, 1000]
MODS = [(), ("softcap",), ("alibi",), ("window7",), ("window100", "prefix20"), ("docs",),
        ("softcap", "alibi", "window300", "prefix5"), ("docs", "prefix50", "window64")]


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,hq,hkv,d,B", [(BF, 8, 2, 128, 16), (BF, 5, 1, 64, 32), (F32, 6, 2, 128, 64),
                                              (BF, 16, 1, 128, 64), (BF, 2, 2, 64, 16), (F32, 4, 4, 64, 16)])
def test_single_token_attention(dtype, hq, hkv, d, B, code, mods):
    shape = D.KV8Shape(hq, hkv, d, B, dtype, code)
    _attention_case(shape, [1] * len(DECODE_CTX), DECODE_CTX, 1, mods, cu_none=True)


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,hq,hkv,d,B", [(BF, 8, 2, 128, 16), (BF, 7, 1, 64, 32), (F32, 6, 2, 128, 64),
                                              (BF, 2, 2, 64, 64)])
def test_few_token_attention(dtype, hq, hkv, d, B, code, mods):
    shape = D.KV8Shape(hq, hkv, d, B, dtype, code)
    _attention_case(shape, [2, 5, 0, 1, 4, 3], [2, 5, 40, 129, 300, 1], 2, mods)
    _attention_case(shape, [8, 8], [900, 8], 3, mods)


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,hq,hkv,d,B", [(BF, 8, 2, 128, 16), (BF, 6, 2, 64, 32), (F32, 2, 1, 64, 16),
                                              (BF, 3, 3, 128, 64)])
def test_many_token_attention(dtype, hq, hkv, d, B, code, mods):
    shape = D.KV8Shape(hq, hkv, d, B, dtype, code)
    _attention_case(shape, [70, 0, 130, 33, 1], [70, 10, 301, 20, 129], 4, mods)
    _attention_case(shape, [257], [400], 5, mods, max_q=300)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("nq", [1, 6, 200])
def test_attention_long_context_and_scale(code, nq):
    _attention_case(D.KV8Shape(4, 1, 128, 16, BF, code), [nq, 1], [9001, 5000], 6, scale=0.3)
    _attention_case(D.KV8Shape(4, 2, 64, 64, BF, code), [nq], [12345], 7, ("window4000", "prefix64"))


def test_attention_of_every_group_size():
    for G in range(1, 17):
        for nq in (1, 3, 20):
            _attention_case(D.KV8Shape(2 * G, 2, 64 if G % 2 else 128, 16, BF, "int8"), [nq, 1], [333, 47], G)


def test_attention_rows_of_strided_queries_and_rows_behind_the_last_sequence():
    shape = D.KV8Shape(8, 2, 128, 16, BF, "int8")
    for nq in ([1, 1], [3, 2], [40, 30]):
        g = _gen(11)
        ctx = [200, 90]
        codes, scales, table = K.cache_for(shape, ctx, g)
        n, cu = sum(nq), _cu(nq)
        qkv = torch.randn(n + 4, 12, 128, generator=g).to(BF)
        q = qkv[:, :8]
        cache = D.KV8Cache(codes.cuda(), scales.cuda())
        out = torch.full((n + 4, 8, 128), 3.0, dtype=BF, device="cuda")
        lse = torch.full((n + 4, 8), 3.0, device="cuda")
        ws = D.alloc_workspace(D.kv8_attention_workspace(shape, 2, n + 4, max(nq) + 4, 300))
        D.deltakv_kv8_attention(shape, cache, qkv.cuda()[:, :8], _i32(cu), _i32(ctx), table.cuda(), max(nq) + 4, 300 if
                                table.shape[1] * 16 >= 300 else table.shape[1] * 16, out, lse, ws)
        ro, rl, to, tl = K.attention(shape, codes, scales, table, q[:n], cu, ctx)
        K.check(out[:n], ro, to, "out")
        K.check(lse[:n], rl, tl, "lse")
        assert (out[n:] == 3.0).all() and (lse[n:] == 3.0).all()


@pytest.mark.parametrize("nq", [1, 4, 60])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_attention_of_poisoned_blocks_queries_and_masked_places(nq, code):
    """A block whose scale is NaN makes NaN of the rows that see it and of no other; a query that holds NaN or an
    infinity makes NaN of its own row and head alone."""
    shape = D.KV8Shape(4, 2, 128, 16, BF, code)
    g = _gen(13)
    ctx, cu = [400, 400], _cu([nq, nq])
    codes, scales, table = K.cache_for(shape, ctx, g)
    scales[table[0, 3].long(), 1, 0] = math.nan  # K of tokens 48..63, kv head 1
    scales[table[1, 9].long(), 0, 1] = math.nan  # V of tokens 144..159, kv head 0
    q = torch.randn(2 * nq, 4, 128, generator=g).to(BF)
    q[0, 0, 5] = math.nan
    q[nq, 3, 7] = math.inf
    out, lse = K.run_attention(shape, codes, scales, table, q, cu, ctx, "cuda")
    assert out[:nq, 2:].isnan().all() and lse[:nq, 2:].isnan().all() and out[nq:, :2].isnan().all()
    assert out[0, 0].isnan().all() and out[nq, 3].isnan().all() and lse[0, 0].isnan() and lse[nq, 3].isnan()
    clean = torch.ones(2 * nq, 4, dtype=torch.bool)
    clean[:nq, 2:] = clean[nq:, :2] = False
    clean[0, 0] = clean[nq, 3] = False
    qc = q.clone()
    qc[0, 0], qc[nq, 3] = 0, 0
    ro, rl, to, tl = K.attention(shape, codes, scales, table, qc, cu, ctx)
    assert torch.isfinite(ro[clean]).all()
    K.check(out.cpu()[clean], ro[clean], to[clean], "out")
    K.check(lse.cpu()[clean], rl[clean], tl[clean], "lse")
    # the same blocks out of every row's sight
    q = qc
    out, lse = K.run_attention(shape, codes, scales, table, q, cu, ctx, "cuda", window=100)
    ro, rl, to, tl = K.attention(shape, codes, scales, table, q, cu, ctx, window=100)
    assert torch.isfinite(ro).all()
    K.check(out, ro, to, "out")
    K.check(lse, rl, tl, "lse")


@pytest.mark.parametrize("nq", [1, 4, 60])
def test_attention_of_scales_and_scores_far_apart(nq):
    """Blocks whose scales differ by 2^30, blocks of zeros with the smallest scale, and queries large enough that one key
    takes all the weight."""
    shape = D.KV8Shape(4, 1, 64, 16, BF, "int8")
    g = _gen(17)
    ctx = [300]
    codes, scales, table = K.cache_for(shape, ctx, g)
    ids = table[0, :19].long()
    scales[ids, 0, 1] = 0.01 * torch.exp2(torch.randint(-15, 15, (19,), generator=g).float())
    codes[ids[4:7]] = 0
    scales[ids[4:7]] = 2.0 ** -64 / 127
    for size in (1.0, 1e3, 1e-20, 1e25):
        q = (size * torch.randn(nq, 4, 64, generator=g)).to(BF)
        out, lse = K.run_attention(shape, codes, scales, table, q, [0, nq], ctx, "cuda")
        ro, rl, to, tl = K.attention(shape, codes, scales, table, q, [0, nq], ctx)
        K.check(lse, rl, tl, "lse")
        if size <= 1.0:  # beyond, the scores' own error decides which of near keys takes the weight
            K.check(out, ro, to, "out")
        assert torch.isfinite(out).all()


def test_attention_records_bad_blocks_and_lengths():
    shape = D.KV8Shape(8, 2, 128, 16, BF, "int8")
    g = _gen(19)
    for nq in (1, 3, 50):
        ctx, cu = [200, 200, 200], _cu([nq] * 3)
        codes, scales, table = K.cache_for(shape, ctx, g)
        q = torch.randn(3 * nq, 8, 128, generator=g).to(BF)
        ro, rl, to, tl = K.attention(shape, codes, scales, table, q, cu, ctx)
        good = slice(2 * nq, 3 * nq)
        for bad_id in (-1, codes.shape[0], 1 << 30):
            t2 = table.clone()
            t2[1, 4] = bad_id
            out, lse = K.run_attention(shape, codes, scales, t2, q, cu, ctx, "cuda")
            assert D.deltakv_get_device_error() == 1
            K.check(out[good], ro[good], to[good], "out")
            assert torch.isfinite(out).all()
        out, lse = K.run_attention(shape, codes, scales, table, q, cu, [200, 201, 200], "cuda", max_ctx=200, fill=3.0)
        assert D.deltakv_get_device_error() == 3
        K.check(out[good], ro[good], to[good], "out")
        assert (out[nq:2 * nq] == 3.0).all() and (lse[nq:2 * nq] == 3.0).all()
        if nq > 1:
            out, lse = K.run_attention(shape, codes, scales, table, q, [0, nq, 2 * nq + 1, 3 * nq], ctx, "cuda", max_q=nq,
                                       fill=3.0)
            assert D.deltakv_get_device_error() == 3
            assert (out[nq:2 * nq] == 3.0).all()


def test_attention_offsets_past_32_bits():
    """A pool of more than 2^32 bytes, the sequence's blocks at its far end."""
    shape = D.KV8Shape(4, 2, 128, 64, BF, "e4m3")
    per = 2 * 2 * 64 * 128
    nb = (1 << 32) // per + 40
    g = _gen(23)
    ctx = [600]
    codes, scales, table = K.cache_for(shape, ctx, g, spare=0)
    cache = D.KV8Cache(torch.empty((nb, 2, 2, 64, 128), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                       torch.empty((nb, 2, 2), device="cuda"))
    far = nb - codes.shape[0]
    cache.codes.view(torch.uint8)[far:] = codes.view(torch.uint8).cuda()
    cache.scales[far:] = scales.cuda()
    t2 = torch.where(table >= 0, table + far, table).cuda()
    for nq in (1, 5, 100):
        q = torch.randn(nq, 4, 128, generator=g).to(BF)
        out = torch.empty(nq, 4, 128, dtype=BF, device="cuda")
        lse = torch.empty(nq, 4, device="cuda")
        ws = D.alloc_workspace(D.kv8_attention_workspace(shape, 1, nq, nq, 600))
        D.deltakv_kv8_attention(shape, cache, q.cuda(), _i32([0, nq]), _i32(ctx), t2, nq, 600, out, lse, ws)
        ro, rl, to, tl = K.attention(shape, codes, scales, table, q, [0, nq], ctx)
        K.check(out, ro, to, "out")
        K.check(lse, rl, tl, "lse")
    k = torch.randn(1, 2, 128, generator=g).to(BF)
    D.deltakv_kv8_append(shape, cache, k.cuda(), k.cuda(), _i32([0, 1]), _i32([599]), t2, 1)
    K.append(shape, codes, scales, k, k, [0, 1], [599], table)
    assert torch.equal(cache.codes.view(torch.uint8)[far:].cpu(), codes.view(torch.uint8))


def test_attention_twice_is_bit_identical_and_no_sequences_is_a_no_op():
    shape = D.KV8Shape(8, 2, 128, 16, BF, "int8")
    g = _gen(29)
    for nq in (1, 4, 70):
        ctx, cu = [3000, 800], _cu([nq, nq])
        codes, scales, table = K.cache_for(shape, ctx, g)
        q = torch.randn(2 * nq, 8, 128, generator=g).to(BF)
        a = K.run_attention(shape, codes, scales, table, q, cu, ctx, "cuda")
        b = K.run_attention(shape, codes, scales, table, q, cu, ctx, "cuda", stream=torch.cuda.Stream())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cache = D.KV8Cache(codes.cuda(), scales.cuda())
    empty = torch.empty(0, 8, 128, dtype=BF, device="cuda")
    D.deltakv_kv8_attention(shape, cache, empty, _i32([0]), _i32([]), table[:0].cuda(), 1, 16, empty, None, None)
    D.deltakv_kv8_append(shape, cache, empty[:, :2], empty[:, :2], _i32([0]), _i32([]), table[:0].cuda(), 1)


@pytest.mark.parametrize("hq,hkv,d,B,code,softcap", [(16, 4, 128, 16, "e4m3", 0.0), (16, 4, 128, 16, "e4m3", 50.0),
                                                     (8, 2, 64, 64, "int8", 0.0)])
def test_long_prompts_over_and_over(hq, hkv, d, B, code, softcap):
    """Many waves of CTAs of the tcgen05 kernel, twenty times: every wait is met (the device error word stays 0) and every
    run gives the same bits; rows far apart are checked against fp64."""
    shape, T = D.KV8Shape(hq, hkv, d, B, BF, code), 6000
    g = _gen(41)
    codes, scales, table = K.cache_for(shape, [T], g)
    q = torch.randn(T, hq, d, generator=g).to(BF)
    cache = D.KV8Cache(codes.view(torch.uint8).cuda().view(shape.code_dtype), scales.cuda())
    ws = D.alloc_workspace(D.kv8_attention_workspace(shape, 1, T, T, T))
    dq, cu, ctx, tab = q.cuda(), _i32([0, T]), _i32([T]), table.cuda()
    first = None
    for _ in range(20):
        out, lse = torch.empty_like(dq), torch.empty(T, hq, device="cuda")
        D.deltakv_kv8_attention(shape, cache, dq, cu, ctx, tab, T, T, out, lse, ws, softcap=softcap)
        assert D.deltakv_get_device_error() == 0
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    for p in (0, 1, 129, 2047, 4444, T - 1):  # a row is the last token of a shorter sequence in the same blocks
        ro, rl, to, tl = K.attention(shape, codes, scales, table, q[p:p + 1], [0, 1], [p + 1], softcap=softcap)
        K.check(first[0][p:p + 1], ro, to, "out")
        K.check(first[1][p:p + 1], rl, tl, "lse")


def test_two_graphs_share_a_workspace_and_two_streams_do_not():
    """Graphs of different shapes that use one workspace, replayed in turn, and calls on two streams with a workspace each."""
    g = _gen(43)
    shape = D.KV8Shape(8, 2, 128, 16, BF, "int8")
    ctx = [5000, 3000]
    codes, scales, table = K.cache_for(shape, ctx, g)
    cache = D.KV8Cache(codes.cuda(), scales.cuda())
    dctx, tab = _i32(ctx), table.cuda()
    sizes = (1, 2, 40)
    q = {n: torch.randn(2 * n, 8, 128, generator=g).to(BF) for n in sizes}
    ws = D.alloc_workspace(max(D.kv8_attention_workspace(shape, 2, 2 * n, n, 5000) for n in sizes)).fill_(0xff)
    ref = {n: K.attention(shape, codes, scales, table, q[n], [0, n, 2 * n], ctx) for n in sizes}

    def call(n, out, lse, work, stream=None):
        D.deltakv_kv8_attention(shape, cache, dq[n], cus[n], dctx, tab, n, 5000, out, lse,
                                work, stream=stream)

    dq, cus = {n: q[n].cuda() for n in sizes}, {n: _i32([0, n, 2 * n]) for n in sizes}
    outs = {n: (torch.empty_like(dq[n]), torch.empty(2 * n, 8, device="cuda")) for n in sizes}
    graphs = {}
    for n in sizes:
        graphs[n] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[n]):
            call(n, *outs[n], ws)
    for _ in range(3):
        for n in sizes:
            graphs[n].replay()
    torch.cuda.synchronize()
    for n in sizes:
        K.check(outs[n][0], ref[n][0], ref[n][2], "out")
        K.check(outs[n][1], ref[n][1], ref[n][3], "lse")
    streams = [torch.cuda.Stream() for _ in sizes]
    own = [D.alloc_workspace(D.kv8_attention_workspace(shape, 2, 2 * n, n, 5000)) for n in sizes]
    two = {n: (torch.empty_like(dq[n]), torch.empty(2 * n, 8, device="cuda")) for n in sizes}
    torch.cuda.synchronize()
    for _ in range(5):
        for n, st, w in zip(sizes, streams, own):
            call(n, *two[n], w, st)
    torch.cuda.synchronize()
    for n in sizes:
        assert torch.equal(two[n][0], outs[n][0]) and torch.equal(two[n][1], outs[n][1])


# ------------------------------------------------------------------------------------------------------------------
# merge
# ------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("parts", range(1, 9))
def test_merge(dtype, d, parts):
    g = _gen(parts)
    for rows in (1, 7, 333):
        outs = [torch.randn(rows, 3, d, generator=g).to(dtype) for _ in range(parts)]
        lses = [4 * torch.randn(rows, 3, generator=g) for _ in range(parts)]
        lses[0][::2] = -math.inf
        outs[0][::2] = math.nan  # what a part that saw nothing holds does not matter
        if rows > 4:
            for x in lses:
                x[3] = -math.inf
        out = torch.empty(rows, 3, d, dtype=dtype, device="cuda")
        lse = torch.empty(rows, 3, device="cuda")
        D.deltakv_merge_attention([o.cuda() for o in outs], [x.cuda() for x in lses], out, lse)
        x = torch.stack(lses).double()
        rl = torch.logsumexp(x, 0)
        w = torch.where(x == -math.inf, 0.0, torch.exp(x - torch.where(rl == -math.inf, 0.0, rl)))[..., None]
        o = torch.stack(outs).double()
        o = torch.where(w == 0, 0.0, o)
        # fp32: the exponent's argument (of size |lse_i - max| < 64) rounds twice, 2^x to 2^-22, then parts sums
        rel = 64 * 2.0 ** -23 + (parts + 4) * 2.0 ** -23
        K.check(out, (w * o).sum(0), (w * o.abs()).sum(0) * rel + (w * o).sum(0).abs() *
                (2.0 ** -8 if dtype == BF else 2.0 ** -24) * 1.01 + 1e-37, "out")
        K.check(lse, rl, 2.0 ** -22 * (rl.abs().nan_to_num(0.0, posinf=0.0) + 64) + 0 * rl.nan_to_num(0.0, neginf=0.0), "lse")


def test_merge_in_place_without_lse_and_with_nan_and_infinite_lse():
    g = _gen(3)
    a, b = (torch.randn(50, 4, 128, generator=g).to(BF).cuda() for _ in range(2))
    la, lb = (torch.randn(50, 4, generator=g).cuda() for _ in range(2))
    out, lse = torch.empty_like(a), torch.empty_like(la)
    D.deltakv_merge_attention([a, b], [la, lb], out, lse)
    a2, la2 = a.clone(), la.clone()
    D.deltakv_merge_attention([a2, b], [la2, lb], a2, la2)
    assert torch.equal(a2, out) and torch.equal(la2, lse)
    b2, lb2 = b.clone(), lb.clone()
    D.deltakv_merge_attention([a, b2], [la, lb2], b2, None)
    assert torch.equal(b2, out) and torch.equal(lb2, lb)
    la[0, 0] = math.nan
    lb[1, 1] = math.inf
    D.deltakv_merge_attention([a, b], [la, lb], out, lse)
    assert out[0, 0].isnan().all() and lse[0, 0].isnan()
    assert torch.equal(out[1, 1], b[1, 1]) and lse[1, 1] == math.inf  # infinite weight: that part alone


# ------------------------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------------------------
def _serve(shape, dev, graph):
    """A prompt, then decode steps: append with rotation, attend, each step checked against fp64 over the cache's values."""
    g = _gen(31)
    H, Hq, d, B = shape.num_kv_heads, shape.num_q_heads, shape.head_dim, shape.block_tokens
    prompt, steps = [75, 20, 33], 6
    S, most = len(prompt), max(prompt) + steps
    nblk = -(-most // B)
    table = torch.randperm(S * nblk, generator=g).int().view(S, nblk)
    codes = torch.full((S * nblk, H, 2, B, d), 0x7f, dtype=torch.uint8).view(shape.code_dtype)
    scales = torch.full((S * nblk, H, 2), math.nan)
    cache = D.KV8Cache(codes.view(torch.uint8).to(dev).view(shape.code_dtype), scales.to(dev))
    rope = _rope(most, d, g)
    dtab, drope = table.to(dev), rope.to(dev)

    def step(x, cu, start, q_rot, out, lse, ws, ctx, max_new):
        q, k, v = x.split([Hq, H, H], 1)
        D.deltakv_kv8_append(shape, cache, k, v, cu, start, dtab, max_new, rope=drope, q=q, q_out=q_rot)
        D.deltakv_kv8_attention(shape, cache, q_rot, cu, ctx, dtab, max_new, most, out, lse, ws)

    def verify(x, cu, start, out, lse):
        n = x.shape[0]
        q, k, v = x.split([Hq, H, H], 1)
        K.append(shape, codes, scales, k, v, cu, start, table, rope)
        assert torch.equal(cache.codes.view(torch.uint8).cpu(), codes.view(torch.uint8))
        ctx = [s + b - a for s, a, b in zip(start, cu[:-1], cu[1:])]
        pos = torch.cat([torch.arange(s, t) for s, t in zip(start, ctx)])
        qr = K.rotate(q, rope[pos], False).to(shape.dtype)
        ro, rl, to, tl = K.attention(shape, codes, scales, table, qr, cu, ctx)
        K.check(out[:n], ro, to, "out")
        K.check(lse[:n], rl, tl, "lse")

    def buffers(n, max_new):
        return (torch.empty(n, Hq, d, dtype=shape.dtype, device=dev), torch.empty(n, Hq, d, dtype=shape.dtype, device=dev),
                torch.empty(n, Hq, device=dev),
                D.alloc_workspace(D.kv8_attention_workspace(shape, S, n, max_new, most), dev))

    n, cu, start = sum(prompt), _cu(prompt), [0] * S
    x = torch.randn(n, Hq + 2 * H, d, generator=g).to(shape.dtype)
    q_rot, out, lse, ws = buffers(n, max(prompt))
    step(x.to(dev), _i32(cu, dev), _i32(start, dev), q_rot, out, lse, ws, _i32(prompt, dev), max(prompt))
    torch.cuda.synchronize(dev)
    verify(x, cu, start, out, lse)
    cu = list(range(S + 1))
    q_rot, out, lse, ws = buffers(S, 1)
    dx = torch.empty(S, Hq + 2 * H, d, dtype=shape.dtype, device=dev)
    dcu, dstart, dctx = _i32(cu, dev), _i32(prompt, dev), _i32([p + 1 for p in prompt], dev)
    G = None
    for i in range(steps):
        x = torch.randn(S, Hq + 2 * H, d, generator=g).to(shape.dtype)
        start = [p + i for p in prompt]
        dx.copy_(x)
        dstart.copy_(_i32(start, dev))
        dctx.copy_(_i32([s + 1 for s in start], dev))
        if graph:
            if G is None:
                G = torch.cuda.CUDAGraph()
                with torch.cuda.graph(G):
                    step(dx, dcu, dstart, q_rot, out, lse, ws, dctx, 1)
            G.replay()
        else:
            step(dx, dcu, dstart, q_rot, out, lse, ws, dctx, 1)
        torch.cuda.synchronize(dev)
        verify(x, cu, start, out, lse)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype,code,hq,hkv,d,B", [(BF, "int8", 8, 2, 128, 16), (BF, "e4m3", 6, 2, 64, 32),
                                                   (F32, "int8", 4, 2, 64, 16)])
def test_prompt_then_decode_steps(dtype, code, hq, hkv, d, B, graph):
    _serve(D.KV8Shape(hq, hkv, d, B, dtype, code), torch.device("cuda"), graph)


def test_compressed_past_and_8_bit_recent_tokens_merge_into_one_attention():
    """A sequence whose old tokens lie in the compressed cache and whose recent ones in the 8-bit cache: decode over each,
    merged by log-sum-exp, equals softmax attention over all the tokens' cached values in fp64."""
    w = synth.workload(1, seq_len=2000, num_kv_heads=2, num_q_heads=8)
    lens, recent = [2000, 700, 48], [100, 17, 1]
    L = C.make_layer(w, lens)
    old = C.gpu_compress(L)
    shape = D.KV8Shape(8, 2, w.head_dim, w.ref_stride, BF, "int8")
    g = _gen(37)
    codes, scales, table = K.cache_for(shape, recent, g, scale=0.03)
    q = torch.randn(3, 8, w.head_dim, generator=g).to(BF)
    qn = q.double().numpy()
    cache = D.KV8Cache(codes.cuda(), scales.cuda())
    o1, o2, o = (torch.empty(3, 8, w.head_dim, dtype=BF, device="cuda") for _ in range(3))
    l1, l2, l = (torch.empty(3, 8, device="cuda") for _ in range(3))
    ds = C.shape_of(w)
    bt = torch.from_numpy(L.bt).cuda()
    ws1 = D.alloc_workspace(D.decode_workspace(ds, 3, 2000))
    ws2 = D.alloc_workspace(D.kv8_attention_workspace(shape, 3, 3, 1, 100))
    D.deltakv_decode_attention(ds, L.mu.cuda(), L.basis.cuda(), old, q.cuda(), _i32(lens), bt, 2000, o1, l1, ws1)
    D.deltakv_kv8_attention(shape, cache, q.cuda(), None, _i32(recent), table.cuda(), 1, 100, o2, l2, ws2)
    D.deltakv_merge_attention([o1, o2], [l1, l2], o, l)
    torch.cuda.synchronize()
    ro, rl, to, tl = K.attention(shape, codes, scales, table, q, [0, 1, 2, 3], recent)
    for s in range(3):
        a, la = C.oracle_decode_sparse_from_cache(L, old, s, qn[s], np.arange(lens[s]))
        la = torch.as_tensor(np.asarray(la)).double()
        want_l = torch.logaddexp(la, rl[s])
        want = torch.exp(la - want_l)[:, None] * torch.as_tensor(np.asarray(a)).double() + \
            torch.exp(rl[s] - want_l)[:, None] * ro[s]
        # The merge is a mean of the two parts with weights that add to 1, so it is off by at most the larger of their
        # errors (the compressed decode's tolerance of 2e-2, which holds its bf16 rounding; the 8-bit part's bound), and
        # by one bf16 rounding more of its own, 2^-8 of the value.
        want_err = torch.clamp(to[s], min=2e-2) + 2.0 ** -8 * want.abs()
        got = o[s].double().cpu()
        assert ((got - want).abs() <= want_err).all()
        assert (got - want).norm() <= (1e-2 + 2.0 ** -8) * want.norm()
        assert (l[s].double().cpu() - want_l).abs().max() <= 1e-3


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_poisoned_v_blocks_reach_only_the_rows_that_see_them(dtype, code, d):
    """A block whose V scale is NaN, in front of some rows of a CTA and behind or outside the others' sight: causal rows of one
    sequence, windows, packed documents, a prefix."""
    shape = D.KV8Shape(2, 1, d, 16, dtype, code)
    g = _gen(47)
    for nq, T, block in ((4, 66, 4), (40, 90, 4), (60, 200, 8)):
        codes, scales, table = K.cache_for(shape, [T], g)
        q = torch.randn(nq, 2, d, generator=g).to(dtype)
        p = T - nq + torch.arange(nq)
        bad = scales.clone()
        bad[table[0, block].long(), 0, 1] = math.nan
        first = torch.where(p % 2 == 0, 0, 16 * block + 16).to(torch.int32)
        for kw in (dict(), dict(window=20), dict(first=first), dict(window=5, prefix=torch.tensor([40], dtype=torch.int32))):
            out, lse = K.run_attention(shape, codes, bad, table, q, [0, nq], [T], "cuda", **kw)
            ro, rl, to, tl = K.attention(shape, codes, scales, table, q, [0, nq], [T], **kw)
            see = K.visible(nq, T, kw.get("window", 0), int(kw["prefix"][0]) if "prefix" in kw else 0,
                            first.long() if "first" in kw else None)
            hit = see[:, 16 * block:16 * block + 16].any(1)
            assert hit.any() and not hit.all() or nq == 60 and not kw
            assert out[hit].isnan().all()
            K.check(out[~hit], ro[~hit], to[~hit], "out")
            K.check(lse[~hit], rl[~hit], tl[~hit], "lse")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_leaves_the_queries_of_refused_sequences(dtype):
    """A sequence whose lengths break a bound is recorded and nothing of it is written: not its queries either, in place or
    not; the other sequence's are rotated."""
    shape = D.KV8Shape(4, 1, 64, 16, dtype, "int8")
    g = _gen(53)
    codes, scales, table = K.cache_for(shape, [40, 40], g)
    k = torch.randn(20, 1, 64, generator=g).to(dtype)
    q = torch.randn(20, 4, 64, generator=g).to(dtype)
    rope = _rope(64, 64, g)
    for cu, start, bad in (([0, 10, 20], [3, -1], 1), ([0, 12, 20], [0, 5], 0), ([0, 10, 25], [7, 0], 1),
                           ([0, 10, 20], [0, (1 << 31) - 20], 1)):
        for inplace in (False, True):
            cache = D.KV8Cache(codes.cuda(), scales.cuda())
            dq = q.cuda()
            q_out = dq if inplace else torch.full_like(dq, 7.0)
            D.deltakv_kv8_append(shape, cache, k.cuda(), k.cuda(), _i32(cu), _i32(start), table.cuda(), 10,
                                 rope=rope.cuda(), q=dq, q_out=q_out)
            assert D.deltakv_get_device_error() == 3
            got = q_out.cpu()
            for s in (0, 1):
                rows = slice(cu[s], min(cu[s + 1], 20))
                if s == bad:
                    want = q[rows] if inplace else torch.full_like(q[rows], 7.0)
                else:
                    want = K.rotate(q[rows], rope[start[s]:start[s] + cu[s + 1] - cu[s]], False).to(dtype)
                assert torch.equal(got[rows], want), (cu, start, inplace, s)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_one_workspace_serves_every_step_of_a_program(dtype, d):
    """A workspace sized once, for the largest batch, step and context: decode steps of batches that come and go, verification
    and prefill chunks all run in it, and nothing behind its end is written."""
    shape, T, most = D.KV8Shape(4, 2, d, 16, dtype, "int8"), 4000, 40
    g = _gen(59)
    ctx = [T - 61 * i for i in range(most)]
    codes, scales, table = K.cache_for(shape, ctx, g)
    cache, tab = D.KV8Cache(codes.cuda(), scales.cuda()), table.cuda()
    need = D.kv8_attention_workspace(shape, most, 300, 200, T)
    ws = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    for sizes in ([1], [1] * 2, [1] * 9, [1] * 18, [1] * 19, [1] * 37, [1] * 40, [5] * 3, [9, 1, 9], [20], [40, 3], [200, 100], [200]):
        S, n, cu = len(sizes), sum(sizes), _cu(sizes)
        q = torch.randn(n, 4, d, generator=g).to(dtype)
        out = torch.full((n, 4, d), math.nan, dtype=dtype, device="cuda")
        lse = torch.full((n, 4), math.nan, device="cuda")
        D.deltakv_kv8_attention(shape, cache, q.cuda(), _i32(cu), _i32(ctx[:S]), tab[:S], max(sizes), T, out, lse, ws[:need])
        rows = [i for i in range(S) if i in (0, S // 2, S - 1)]
        for s in rows:  # a sequence at a time in fp64
            part = slice(cu[s], cu[s + 1])
            ro, rl, to, tl = K.attention(shape, codes, scales, table[s:s + 1], q[part], [0, sizes[s]], ctx[s:s + 1])
            K.check(out[part], ro, to, "out")
            K.check(lse[part], rl, tl, "lse")
    assert (ws[need:] == 0xa5).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mods", [(), ("softcap", "alibi", "window300", "prefix5")])
def test_row_counts_on_either_side_of_a_kernel_s_limit(d, mods):
    """Rows per kv head around 8, 16, 64, 80 and 96, where one kernel or row tile gives way to the next."""
    shape = D.KV8Shape(2, 1, d, 16, BF, "e4m3")
    for nq in (3, 4, 5, 8, 9, 31, 32, 33, 39, 40, 41, 47, 48, 49):
        _attention_case(shape, [nq, 1], [700, 90], nq, mods)


def test_prefills_and_compress_on_streams_of_their_own():
    """Kernels that take a whole SM's tensor memory, launched side by side: many-row attention with both head sizes on two
    streams, the compressed cache's search on a third.  Each ends, and with the bits of a run by itself."""
    g = _gen(61)
    w = synth.workload(1, seq_len=1500, num_kv_heads=2, num_q_heads=8)
    L = C.make_layer(w, [1500, 900])
    alone = C.gpu_compress(L)
    runs = []
    for d, code, cap in ((64, "int8", 0.0), (64, "e4m3", 30.0), (128, "int8", 0.0)):
        shape, T = D.KV8Shape(8, 2, d, 16, BF, code), 1800
        codes, scales, table = K.cache_for(shape, [T], g)
        cache = D.KV8Cache(codes.view(torch.uint8).cuda().view(shape.code_dtype), scales.cuda())
        q = torch.randn(T, 8, d, generator=g).to(BF).cuda()
        args = (shape, cache, q, _i32([0, T]), _i32([T]), table.cuda(), T, T)
        bufs = [(torch.empty_like(q), torch.empty(T, 8, device="cuda"),
                 D.alloc_workspace(D.kv8_attention_workspace(shape, 1, T, T, T))) for _ in range(2)]
        D.deltakv_kv8_attention(*args, *bufs[0], softcap=cap)
        runs.append((args, cap, bufs, torch.cuda.Stream()))
    side = torch.cuda.Stream()
    cache2 = D.alloc_cache(C.shape_of(w), L.num_blocks, "cuda")
    torch.cuda.synchronize()
    for _ in range(6):
        for args, cap, bufs, st in runs:
            for _ in range(3):
                D.deltakv_kv8_attention(*args, *bufs[1], softcap=cap, stream=st)
        with torch.cuda.stream(side):
            C.gpu_compress(L, cache=cache2)
    torch.cuda.synchronize()
    assert D.deltakv_get_device_error() == 0
    for args, cap, bufs, st in runs:
        assert torch.equal(bufs[0][0], bufs[1][0]) and torch.equal(bufs[0][1], bufs[1][1])
    assert torch.equal(alone.codes, cache2.codes) and torch.equal(alone.ref_idx, cache2.ref_idx)


@pytest.mark.parametrize("nq", [1, 4, 100])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequences_that_share_blocks(dtype, nq):
    """Sequences with one prefix in the same physical blocks, one of them there twice."""
    shape = D.KV8Shape(6, 2, 64, 16, dtype, "e4m3")
    g = _gen(67)
    ctx = [300, 208 + nq, 300, 300]
    codes, scales, table = K.cache_for(shape, ctx, g)
    table[1, :13] = table[0, :13]
    table[2] = table[0]
    q = torch.randn(4 * nq, 6, 64, generator=g).to(dtype)
    cu = _cu([nq] * 4)
    out, lse = K.run_attention(shape, codes, scales, table, q, cu, ctx, "cuda")
    ro, rl, to, tl = K.attention(shape, codes, scales, table, q, cu, ctx)
    K.check(lse, rl, tl, "lse")
    K.check(out, ro, to, "out")
