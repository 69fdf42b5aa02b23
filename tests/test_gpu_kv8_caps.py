"""Score caps of the 8-bit cache's attention: softcap tanh(x / softcap) has to hold for every cap that is accepted, in every
kernel (CUDA cores, mma.sync, tcgen05), with an error that follows the score and not the cap."""
import math

import pytest
import torch

from residual_kv_cache_delta_b200 import deltakv as D

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


def _reference(shape, codes, scales, table, q, cu, ctx, cap, slopes=None):
    """(out, lse, bound on out, bound on lse) in fp64, causal.

    A score x = scale q.k is off by d 2^-24 of the sum of its products' magnitudes.  Its capped value c = cap tanh(x / cap)
    is off by that (the slope of tanh is at most 1) and by a share of its own size: x / cap and the product with cap round
    by 2^-22 in all; tanh by a polynomial of relative error 2^-23 and five roundings below 2^-22 for |x / cap| <= 0.6, where
    |tanh| is within 0.54 above; beyond, cap - 2 cap / (1 + e^(2 x / cap)) with an exponential off by 2^-22 and a
    reciprocal off by 2^-23 is off by less than 4.2e-7 cap, 2^-20.3 of the least value there.  So 2^-20 |c|, whatever the cap.
    Then as for scores without a cap: 2^-22 of the score and of its bias, the exponential 2^-21, the sum of T weights T 2^-24;
    bf16 storage rounds weights to fp16 (2^-11) and the result by half a step."""
    n, Hq, d = q.shape
    G, B = Hq // shape.num_kv_heads, shape.block_tokens
    bf = shape.dtype == BF
    out = torch.full((n, Hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((n, Hq), math.nan, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for s, T in enumerate(ctx):
        rows, nq = slice(cu[s], cu[s + 1]), cu[s + 1] - cu[s]
        ids = table[s, :-(-T // B)].long()
        kv = (codes[ids].double() * scales[ids].double()[..., None, None]).permute(2, 1, 0, 3, 4).flatten(2, 3)[:, :, :T]
        gap = (T - nq + torch.arange(nq))[:, None] - torch.arange(T)[None]
        for h in range(Hq):
            k, v = kv[0, h // G], kv[1, h // G]
            qq = q[rows, h].double()
            x = qq @ k.T / math.sqrt(d)
            err = 2.0 ** -24 * d * (qq.abs() @ k.abs().T / math.sqrt(d))
            x = cap * torch.tanh(x / cap)
            err = err + 2.0 ** -20 * x.abs()
            if slopes is not None:
                bias = slopes[h].double() * gap.abs()
                err = err + 2.0 ** -22 * bias
                x = x - bias
            err = err + 2.0 ** -22 * x.abs()
            x = x.masked_fill(gap < 0, -math.inf)
            lse[rows, h] = torch.logsumexp(x, -1)
            w = torch.softmax(x, -1)
            out[rows, h] = w @ v
            e = err.masked_fill(gap < 0, 0.0).amax(-1) + 2.0 ** -21 + T * 2.0 ** -24
            t = (2 * e[:, None] + (2.0 ** -11 if bf else 0.0)) * (w @ v.abs()) * 1.01
            t = t + (2.0 ** -8 if bf else 2.0 ** -24) * 1.01 * out[rows, h].abs()
            if bf:  # weights below fp16's smallest normal, relative to the row's largest weight times V scale
                vs = scales[ids, h // G, 1].double().repeat_interleave(B)[:T]
                code = codes[ids, h // G, 1].double().flatten(0, 1)[:T].abs()
                t = t + 2.0 ** -25 * (w * vs).amax(-1, keepdim=True) * code.sum(0)
            tol[rows, h] = t + 1e-30
            tol_l[rows, h] = e + 2.0 ** -22 * lse[rows, h].abs()
    return out, lse, tol, tol_l


def _case(shape, nq, ctx, cap, seed, grow=None, slopes=None):
    g = torch.Generator()
    g.manual_seed(seed)
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    codes, scales, table = K.cache_for(shape, ctx, g)
    q = torch.randn(cu[-1], shape.num_q_heads, shape.head_dim, generator=g)
    if grow is not None:  # rows of very different size beside one another
        q *= grow ** torch.randint(0, 3, (cu[-1], shape.num_q_heads, 1), generator=g).float()
    q = q.to(shape.dtype)
    out, lse = K.run_attention(shape, codes, scales, table, q, cu, ctx, "cuda", softcap=cap, slopes=slopes)
    ro, rl, to, tl = _reference(shape, codes, scales, table, q, cu, ctx, cap, slopes)
    K.check(lse, rl, tl, "lse")
    K.check(out, ro, to, "out")


# one token; a few tokens; enough rows for the tcgen05 kernel
ROWS = {"one": ([1, 1, 1], [700, 33, 1]), "few": ([5, 3], [400, 20]), "many": ([70, 130], [301, 150])}


@pytest.mark.parametrize("cap", [1e-6, 1.0, 30.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e30])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype,code,d", [(BF, "int8", 128), (BF, "e4m3", 64), (F32, "int8", 64), (F32, "e4m3", 128)])
def test_caps_of_every_size(dtype, code, d, rows, cap):
    _case(D.KV8Shape(8, 2, d, 16, dtype, code), *ROWS[rows], cap, 1)


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype,code,d", [(BF, "int8", 128), (BF, "e4m3", 64), (F32, "int8", 64)])
def test_caps_of_scores_far_apart(dtype, code, d, rows):
    """Rows far below their cap beside rows that reach it: neither form of the cap may be taken for both."""
    shape = D.KV8Shape(8, 2, d, 16, dtype, code)
    _case(shape, *ROWS[rows], 1e3, 2, grow=40.0)
    _case(shape, *ROWS[rows], 3.0, 3, grow=3.0)
    _case(shape, *ROWS[rows], 1e5, 4, grow=100.0, slopes=torch.exp2(-torch.arange(8).float()))
