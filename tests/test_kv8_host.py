"""The 8-bit cache's entry points on a host without a GPU: sizes, and refusals before any launch."""
import ctypes
import math

import pytest
import torch

from residual_kv_cache_delta_b200 import build as B
from residual_kv_cache_delta_b200 import deltakv as D

BF = torch.bfloat16
OK, ARG, UNS, WS = D.DKV_OK, D.DKV_ERR_INVALID_ARG, D.DKV_ERR_UNSUPPORTED, D.DKV_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    B.build()
    return D.load_library()


def _shape(**kw):
    a = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, block_tokens=16, dtype=D.DKV_BF16, code=0)
    a.update(kw)
    return D.DkvKv8Shape(**a)


BAD_SHAPES = [(dict(num_q_heads=0), ARG), (dict(num_kv_heads=-1), ARG), (dict(num_q_heads=7), ARG), (dict(code=2), ARG),
              (dict(dtype=D.DKV_BF16_Q4), ARG), (dict(dtype=9), ARG), (dict(head_dim=96), UNS), (dict(head_dim=256), UNS),
              (dict(block_tokens=8), UNS), (dict(block_tokens=48), UNS), (dict(block_tokens=128), UNS),
              (dict(num_q_heads=34), UNS), (dict(head_dim=0), ARG), (dict(block_tokens=0), ARG)]


def append(lib, shape=None, rope=None, k=256, ks=256, v=256, vs=256, cu=256, start=256, table=256, max_blocks=4, seqs=1,
           total=8, max_new=8, q=0, qs=0, q_out=0, cache=(256, 256, 4), shape_null=False, cache_null=False):
    sh = shape or _shape()
    cc = D.DkvKv8Cache(*cache)
    return lib.deltakv_kv8_append(None if shape_null else ctypes.byref(sh), None if cache_null else ctypes.byref(cc),
                                  ctypes.byref(rope) if rope else None, k, ks, v, vs, cu, start, table, max_blocks, seqs,
                                  total, max_new, q, qs, q_out, None)


def attend(lib, shape=None, score=None, q=256, qs=1024, cu=256, ctx=256, table=256, max_blocks=4, seqs=1, total=4, max_q=4,
           max_ctx=64, scale=0.0, out=256, lse=0, ws=256, ws_bytes=1 << 40, cache=(256, 256, 4), cache_null=False):
    sh = shape or _shape()
    cc = D.DkvKv8Cache(*cache)
    return lib.deltakv_kv8_attention(ctypes.byref(sh), None if cache_null else ctypes.byref(cc),
                                     ctypes.byref(score) if score else None, q, qs, cu, ctx, table, max_blocks, seqs, total,
                                     max_q, max_ctx, scale, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", BAD_SHAPES)
def test_shapes_refused_by_every_entry_point(lib, over, status):
    sh = _shape(**over)
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.deltakv_kv8_cache_bytes(ctypes.byref(sh), 4, ctypes.byref(a), ctypes.byref(b)) == status
    assert lib.deltakv_kv8_attention_workspace(ctypes.byref(sh), 1, 1, 1, 64, ctypes.byref(a)) == status
    assert append(lib, sh) == status
    assert attend(lib, sh) == status


def test_cache_bytes_match_the_tensors(lib):
    for code in ("int8", "e4m3"):
        sh = D.KV8Shape(32, 8, 128, 32, BF, code)
        c = D.alloc_kv8_cache(sh, 5, "cpu")
        assert D.kv8_cache_bytes(sh, 5) == (c.codes.numel(), c.scales.numel() * 4)
        assert c.nbytes() == 5 * 8 * 2 * (32 * 128 + 4)
    with pytest.raises(D.DeltaKVError):
        D.kv8_cache_bytes(sh, -1)
    with pytest.raises(ValueError):
        D.kv8_cache_bytes(D.KV8Shape(32, 8, 128, 32, torch.float16, "int8"), 1)
    with pytest.raises(ValueError):
        D.kv8_cache_bytes(D.KV8Shape(32, 8, 128, 32, BF, "int4"), 1)


def test_append_refusals(lib):
    assert append(lib, shape_null=True) == ARG and append(lib, cache_null=True) == ARG
    for bad in (dict(k=0), dict(v=0), dict(cu=0), dict(start=0), dict(table=0), dict(k=260), dict(v=264), dict(ks=255),
                dict(ks=260), dict(vs=0), dict(vs=-256), dict(ks=1 << 60), dict(max_blocks=-1), dict(seqs=-1),
                dict(total=-1), dict(max_new=-1), dict(total=9), dict(cache=(0, 256, 4)), dict(cache=(256, 0, 4)),
                dict(cache=(256, 256, 0)), dict(cache=(264, 256, 4)), dict(cache=(256, 260, 4)), dict(q=256, qs=1024),
                dict(q_out=256)):
        assert append(lib, **bad) == ARG, bad
    rope = lambda **kw: D.DkvKv8Rope(**{**dict(table=256, positions=0, max_pos=64, rot_dim=128, pairs=0), **kw})  # noqa: E731
    for bad in (dict(table=0), dict(table=260), dict(max_pos=0), dict(rot_dim=0), dict(rot_dim=-16), dict(rot_dim=24),
                dict(rot_dim=144)):
        assert append(lib, rope=rope(**bad)) == ARG, bad
    for bad in (dict(q=256, qs=1000, q_out=256), dict(q=256, qs=1024, q_out=260), dict(q=264, qs=1024, q_out=256),
                dict(q=256, qs=2048, q_out=256)):
        assert append(lib, rope=rope(), **bad) == ARG, bad
    assert append(lib, q=256, qs=1024, q_out=512) == ARG  # queries without a rotation
    assert append(lib, cache=(256, 256, 1 << 30)) == UNS
    assert append(lib, seqs=1 << 20, total=1 << 31, max_new=1 << 20) == UNS
    for nothing in (dict(seqs=0, total=0), dict(total=0), dict(max_new=0, total=0)):
        assert append(lib, **nothing) == OK


def test_attention_refusals(lib):
    assert attend(lib, cache_null=True) == ARG
    for bad in (dict(q=0), dict(q=260), dict(qs=1023), dict(qs=1028), dict(ctx=0), dict(table=0), dict(out=0), dict(out=264),
                dict(max_blocks=3), dict(max_blocks=-1), dict(seqs=-1), dict(total=-1), dict(total=5), dict(max_q=-1),
                dict(max_ctx=-1), dict(cu=0), dict(scale=math.nan), dict(cache=(0, 256, 4)), dict(cache=(256, 256, -4)),
                dict(cu=0, total=1, max_q=0)):
        assert attend(lib, **bad) == ARG, bad
    score = lambda **kw: D.DkvKv8Score(**{**dict(softcap=0.0, window=0), **kw})  # noqa: E731
    for bad in (dict(softcap=-1.0), dict(softcap=math.nan), dict(softcap=math.inf), dict(softcap=1e-7),
                dict(softcap=1e31), dict(window=-1)):
        assert attend(lib, score=score(**bad)) == ARG, bad
    assert attend(lib, cache=(256, 256, 1 << 30)) == UNS
    assert attend(lib, seqs=1 << 20, total=1 << 29, max_q=1 << 10) == UNS
    # a split call needs its workspace
    long = dict(max_ctx=32768, max_blocks=2048, total=1, max_q=1)
    need = D.kv8_attention_workspace(D.KV8Shape(8, 2, 128, 16, BF, "int8"), 1, 1, 1, 32768)
    assert need > 0
    assert attend(lib, ws_bytes=need - 1, **long) == WS
    assert attend(lib, ws=0, **long) == ARG
    assert attend(lib, ws=264, **long) == ARG
    for nothing in (dict(seqs=0, total=0, max_blocks=0, q=0), dict(total=0, q=0, out=0)):
        assert attend(lib, **nothing) == OK


def test_merge_refusals(lib):
    P2 = ctypes.c_void_p * 2

    def merge(dtype=D.DKV_BF16, d=128, rows=4, parts=2, outs=(256, 512), lses=(256, 512), out=256, lse=0):
        return lib.deltakv_merge_attention(dtype, d, rows, parts, P2(*outs) if outs else None, P2(*lses) if lses else None,
                                           out, lse, None)

    for bad in (dict(dtype=2), dict(d=0), dict(rows=-1), dict(parts=0), dict(parts=9), dict(outs=None), dict(lses=None),
                dict(out=0), dict(out=264), dict(outs=(256, 0)), dict(outs=(256, 264)), dict(lses=(0, 256))):
        assert merge(**bad) == ARG, bad
    assert merge(d=96) == UNS and merge(rows=1 << 60) == UNS
    assert merge(rows=0, outs=None, lses=None, out=0) == OK


def test_workspace_grows_with_its_bounds(lib):
    sh = D.KV8Shape(32, 8, 128, 16, BF, "int8")
    assert D.kv8_attention_workspace(sh, 1, 1, 1, 16) == 0  # nothing to split
    a = [D.kv8_attention_workspace(sh, 1, 1, 1, t) for t in (4096, 32768, 131072)]
    assert a == sorted(a)
    with pytest.raises(D.DeltaKVError):
        D.kv8_attention_workspace(sh, 1, 2, 1, 64)


def test_binding_refuses_tensors_that_do_not_fit(lib):
    """Shapes, types and devices are checked before the library is called (CPU tensors never reach it)."""
    sh = D.KV8Shape(8, 2, 128, 16, BF, "int8")
    cache = D.alloc_kv8_cache(sh, 4, "cpu")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    k, table = torch.zeros(3, 2, 128, dtype=BF), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        D.deltakv_kv8_append(sh, cache, k, k, i32(0, 3), i32(0), table, 3)  # not on a GPU
    with pytest.raises(ValueError):
        D.deltakv_kv8_append(sh, D.KV8Cache(cache.codes, cache.scales[:, :1]), k, k, i32(0, 3), i32(0), table, 3)
    q = torch.zeros(3, 8, 128, dtype=BF)
    with pytest.raises(ValueError):
        D.deltakv_kv8_attention(sh, cache, q, i32(0, 3), i32(3), table, 3, 64, q, None, None)
    with pytest.raises(ValueError):
        D.deltakv_merge_attention([q], [], q, None)
    with pytest.raises(ValueError):
        D.deltakv_merge_attention([q] * 9, [q[..., 0].float()] * 9, q, None)
    with pytest.raises(ValueError):
        D.deltakv_merge_attention([q.half()], [q[..., 0].float()], q.half(), None)


def test_append_refuses_tokens_without_room_for_them(lib):
    """New tokens, but no sequence or a bound of 0 per sequence: refused as attention refuses it, not passed over."""
    for bad in (dict(max_new=0), dict(seqs=0), dict(seqs=0, max_new=0), dict(total=1, max_new=0)):
        assert append(lib, **bad) == ARG, bad
    for bad in (dict(max_q=0), dict(seqs=0)):
        assert attend(lib, **bad) == ARG, bad
    for nothing in (dict(total=0, max_new=0, seqs=0), dict(total=0), dict(total=0, k=0, v=0, cu=0)):
        assert append(lib, **nothing) == OK, nothing


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64), (64, 8, 128), (16, 1, 64)])
def test_a_workspace_for_the_largest_step_serves_every_smaller_one(lib, dtype, hq, hkv, d):
    """The size never falls as a bound grows, whatever the split plan makes of the batch."""
    sh = D.KV8Shape(hq, hkv, d, 16, dtype, "int8")
    seqs, most_q, ctxs = (1, 2, 5, 37, 48, 74, 80, 128), (1, 2, 5, 16, 17, 64, 300, 2048), (16, 300, 4096, 32768, 131072)
    need = {(s, q, t): D.kv8_attention_workspace(sh, s, s * q, q, t) for s in seqs for q in most_q for t in ctxs}
    for axis, steps in enumerate((seqs, most_q, ctxs)):
        for key, n in need.items():
            i = steps.index(key[axis])
            if i:
                below = list(key)
                below[axis] = steps[i - 1]
                assert need[tuple(below)] <= n, (key, axis)
    # fewer query rows than the bounds allow, and a bound that no longer grows with the batch
    assert D.kv8_attention_workspace(sh, 8, 8, 300, 4096) <= need[37, 300, 4096]
    assert max(need.values()) <= 512 << 20
