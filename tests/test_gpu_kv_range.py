"""The key/value cache calls where the magnitudes lie far apart or at the ends of their types, for both attention kernels:
scales from the subnormals to the top of bf16, zero scales, long tails of the softmax.  The 64-bit result and the bound
are computed here, per token, so that one page's size does not loosen the bound of another's."""
import math

import numpy as np
import pytest
import torch

from tests import gpu_helpers as H
from tests import kv_reference as R
from tests import test_gpu_kv as T

pytestmark = pytest.mark.gpu

WIDE = 128      # query rows of a key/value head that go to the tcgen05 kernel whatever the number of jobs


def exact(c, requests):
    """(y, bound) [tokens][heads][dim] in 64 bits, NaN in rows of no request.  How far a kernel may be off:
    - logits: fp32 sums of products of up to 255 (INT8's offset codes, its 128 taken off: 383) or 448 times the scale, 16
      roundings of 2^-24, and 4 of the logit itself: a weight's relative error 2 dx;
    - weights: half a step of fp16 (2^-11 of the weight) or, where they are subnormal, 2^-25 of what holds them: 2^-7 of
      the reference's, in numerator and sum, for the mma.sync kernel; for the tcgen05 kernel, in the numerator, 2^-6 of the
      reference's and twice the largest V scale of the same 128 tokens (here: within 128 on either side), or of 2^-100 if
      that is more, and the values of pages whose V scale is 2^-40 of that or less count as 0;
    - sums: a rounding of what is summed up per 16 tokens, which is the weighted |values| and, for INT8 in the mma.sync
      kernel, 128 scales a weight more that are taken off again;
    - the type's half step (of its subnormals: eps / 2 of the smallest normal number);
    - half a subnormal step of fp32 of each of these sums: 2^-149 a step."""
    fmt, page, D = c["fmt"], c["page"], c["dim"]
    top = 383.0 if fmt == R.INT8 else 448.0
    table = torch.from_numpy(R.value(np.arange(256), fmt)).cuda()
    codes = [torch.from_numpy(k).cuda() for k in c["codes"]]
    scales = torch.from_numpy(c["scales"]).cuda().double()
    kv, group = c["kv_heads"], c["heads"] // c["kv_heads"]
    q = c["q"].cuda().double()
    y = torch.full(q.shape, math.nan, dtype=torch.float64, device="cuda")
    bound = y.clone()
    eps, least = torch.finfo(T.TYPES[c["xdt"]]).eps, torch.finfo(T.TYPES[c["xdt"]]).smallest_normal
    for b in requests:
        L, n, first = int(c["lens"][b]), int(c["cu"][b + 1] - c["cu"][b]), int(c["cu"][b])
        ids = torch.from_numpy(np.asarray(c["table"][b, :-(-L // page)])).cuda().long()
        for h in range(kv):
            k, v = [(table[x[ids, h].long()] * scales[i, ids, h][:, None, None]).reshape(-1, D)[:L] for i, x in enumerate(codes)]
            ks, vs = [scales[i, ids, h].repeat_interleave(page)[:L] for i in (0, 1)]
            near = torch.nn.functional.max_pool1d(vs[None, None], 257, 1, 128)[0, 0].clamp(min=2.0 ** -100)
            for t in range(n):
                p = L - n + t
                lo = max(0, p - c["window"] + 1) if c["window"] else 0
                rows = q[first + t, h * group:(h + 1) * group]
                x = rows @ k[lo:p + 1].T * c["scale"]
                w = torch.exp(x - x.amax(1, keepdim=True))
                w = w / w.sum(1, keepdim=True)
                peak = w.amax(1, keepdim=True)                     # 1 / the sum of weights relative to the largest
                r = w @ v[lo:p + 1]
                vv, sv, nv = v[lo:p + 1].abs(), vs[lo:p + 1], near[lo:p + 1]
                size = w @ vv
                dx = 2.0 ** -20 * top * abs(c["scale"]) * rows.abs().sum(1, keepdim=True) * ks[lo:p + 1].max() + 2.0 ** -22 * x.abs().amax(1, keepdim=True)
                steps = (p + 1 - lo) / 16 + 16
                summed = size if fmt == R.E4M3 or n * group >= WIDE else size + 256 * (w @ sv)[:, None]
                if n * group >= WIDE:
                    cut = 2.0 ** -30 * R.TOP[fmt] * nv.sum() * peak + 2.0 ** -39 * R.TOP[fmt] * (w @ nv)[:, None]
                else:
                    cut = 2.0 ** -32 * peak * (vv.sum(0) + (p + 1 - lo) * r.abs())
                bound[first + t, h * group:(h + 1) * group] = ((2.0 ** -11 + 2 * dx) * (size + r.abs()) + cut + steps * 2.0 ** -23 * summed
                                                               + eps / 2 * (r.abs() * 1.01 + least) + 2.0 ** -149 * steps)
                y[first + t, h * group:(h + 1) * group] = r
    return y, bound


def copies(c, times):
    """The same requests `times` over, on the same pages: jobs enough that a CTA goes through several tiles of one."""
    n = int(c["cu"][-1])
    return dict(c, lens=np.tile(c["lens"], times), table=np.tile(c["table"], (times, 1)), q=c["q"][:n].repeat(times, 1, 1), tokens=n * times,
                cu=np.concatenate([c["cu"][:-1] + n * t for t in range(times)] + [[n * times]]), times=times)


def check(c):
    y = T.call_attn(c)
    assert c["status"] == 0
    times = c.get("times", 1)
    want, bound = exact(c, range(len(c["lens"]) // times))
    part = len(want) // times
    want, bound = (x[:part].repeat(times, 1, 1) if times > 1 else x for x in (want, bound))
    live = ~want.isnan()
    err = (y.double() - want).abs()
    bad = ~(err <= bound) & live
    assert not bad.any(), (int(bad.sum()), float((err / bound)[live].max()), y[bad][:3], want[bad][:3], bad.nonzero()[:3])
    return y


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("top", [2e9, 1e20, 3e38])
def test_append_quotients_that_underflow(fmt, top):
    """x / s below the smallest subnormal is a zero with x's sign, whatever its sign, and no NaN."""
    page, dim, heads = 16, 64, 1
    x = torch.zeros(2, 5, dim)
    x[:, :, 0] = top
    tiny = torch.tensor([1e-40, 9.2e-41, 1.2e-38, 1e-36, 1e-30, 1e-20, 1e-10])
    for t in range(5):
        x[0, t, 1 + t:8 + t], x[1, t, 1 + t:8 + t] = tiny, -tiny
        x[0, t, 20 + t:27 + t], x[1, t, 20 + t:27 + t] = -tiny, tiny
    codes, scales = T.make_cache(9, fmt, 2, heads, page, dim)
    T.check_append(fmt, 1, page, dim, heads, codes, scales, x.bfloat16(), np.arange(5))


# ------------------------------------------------------------------ V scales
def far_apart(kind, fmt, xdt, dim, page, group, new, lens=(700, 333)):
    c = T.make_attn(dim + page + group, fmt, xdt, page, 1, group, dim, list(lens), [new] * len(lens), nan_behind=False)
    r = np.random.default_rng(len(kind))
    tb, s = c["table"], c["scales"]
    tiles = max(1, 128 // page)                                    # pages of 128 tokens
    if kind == "decades":
        s[1] *= (10.0 ** r.integers(-8, 4, s[1].shape)).astype(np.float32)
        s[:, tb[0, 1]] = 0
    elif kind == "one page":
        for b in range(len(lens)):
            s[1, tb[b, 1]] = [1e-40, 1e-43, 1e-38, 0.0][b % 4]
    elif kind == "subnormal tile":
        s[1, tb[0, tiles:2 * tiles]] = 1e-40
        s[1, tb[1, :tiles]] = 1e-44
    elif kind == "zero tiles":
        s[1, tb[0, :tiles]] = 0
        s[1, tb[0, 2 * tiles:3 * tiles]] = 0
        s[1, tb[1, tiles:2 * tiles]] = 0
    elif kind == "up and down":
        f = (10.0 ** np.array([0, 12, -12, 25, -25, 3, -30, 30, -3, 0, 1, -1])).astype(np.float32)
        for b in range(len(lens)):
            for j in range(-(-lens[b] // page)):
                s[1, tb[b, j]] = 1e-2 * f[(j // tiles) % len(f)]
    elif kind == "all tiny":
        s[1] *= np.float32(1e-36)
    elif kind == "bits":
        s[1] = (2.0 ** r.uniform(-150, 3, s[1].shape)).astype(np.float32)
    return c


@pytest.mark.parametrize("kind", ["decades", "one page", "subnormal tile", "zero tiles", "up and down", "all tiny", "bits"])
@pytest.mark.parametrize("fmt,xdt,dim,page", [(R.INT8, 1, 128, 64), (R.E4M3, 0, 64, 16), (R.E4M3, 1, 256, 32), (R.INT8, 0, 64, 128)])
@pytest.mark.parametrize("group,new", [(4, 40), (2, 1)])
def test_attn_v_scales_far_apart(kind, fmt, xdt, dim, page, group, new):
    c = far_apart(kind, fmt, 1 if kind in ("all tiny", "up and down") else xdt, dim, page, group, new)
    check(c)
    check(copies(c, 150))


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
def test_attn_long_tail_behind_a_page_of_large_values(fmt):
    """Tokens of 2^-20 of the largest weight each, 65536 of them: a sixteenth of the largest weight together.  The first page's V scale is
    60 times the others'.  148 requests over the same pages keep a job whole."""
    L, page, dim, group = 65536, 64, 64, WIDE
    pages = L // page
    codes = np.full((2, pages, 1, page, dim), 128 if fmt == R.INT8 else 0, np.uint8)
    r = np.random.default_rng(5)
    codes[0, 0, 0, 3, 0] = 255 if fmt == R.INT8 else 0x7E          # the token that takes most
    big = r.integers(60, 100, (pages, page, dim))
    codes[1, :, 0] = R.nearest(big.astype(np.float64) * (1 if fmt == R.INT8 else 3), fmt)
    codes[1, 0, 0] = R.nearest(r.integers(-2, 3, (page, dim)).astype(np.float64), fmt)
    scales = np.full((2, pages, 1), 1 / R.TOP[fmt], np.float32)
    scales[1, 0] *= 60
    q = torch.zeros(1, group, dim)
    q[:, :, 0] = 20 * math.log(2) * 8
    c = dict(fmt=fmt, xdt=0, page=page, pages=pages, width=pages, kv_heads=1, heads=group, dim=dim, lens=np.array([L]), cu=np.array([0, 1]),
             table=np.arange(pages)[None], codes=codes, scales=scales, q=q.half(), tokens=1, window=0, scale=0.125, max_new=1)
    check(copies(c, 148))


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
def test_attn_long_tail_of_single_tokens(fmt):
    """Tokens of 2^-25.5 of the largest weight each, 262144 of them: half a percent of the sum.  600 requests over the same
    pages keep a job whole."""
    L, page, dim, group = 262144, 128, 64, 8
    pages = L // page
    codes = np.full((2, pages, 1, page, dim), 128 if fmt == R.INT8 else 0, np.uint8)
    codes[0, 0, 0, 3, 0] = 255 if fmt == R.INT8 else 0x7E
    codes[1] = 228 if fmt == R.INT8 else R.nearest(np.array([300.0]), fmt)[0]
    codes[1, 0] = codes[0, 1, 0, 0, 1]                             # zero
    scales = np.full((2, pages, 1), 1 / R.TOP[fmt], np.float32)
    q = torch.zeros(1, group, dim)
    q[:, :, 0] = 25.5 * math.log(2) * 8
    q[:, 1:, 1:] = 1e-3 * torch.randn(group - 1, dim - 1, generator=torch.Generator().manual_seed(1))
    c = dict(fmt=fmt, xdt=0, page=page, pages=pages, width=pages, kv_heads=1, heads=group, dim=dim, lens=np.array([L]), cu=np.array([0, 1]),
             table=np.arange(pages)[None], codes=codes, scales=scales, q=q.half(), tokens=1, window=0, scale=0.125, max_new=1)
    check(copies(c, 600))


# ------------------------------------------------------------------ the ends of bf16
@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("group,new", [(4, 40), (8, 1)])
@pytest.mark.parametrize("lens", [(300, 200), (20011, 50)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [1e6, 1e8, 1e9, 1e12, 1e25, 1e32, 1e36])
def test_attn_logits_of_any_size(fmt, group, new, lens, sign, size):
    """Every logit is `size` or so, of one sign, a token's twice or half that: it takes all."""
    page, dim = 64, 64
    c = T.make_attn(8, fmt, 1, page, 1, group, dim, lens, [new, new], nan_behind=False)
    code = {k: R.nearest(np.full((1,), k * R.TOP[fmt]), fmt)[0] for k in (-1.0, -0.5, 0.5, 1.0)}
    most, rest = (1.0, 0.5) if sign > 0 else (-0.5, -1.0)
    c["codes"][0] = code[rest]
    c["codes"][0, c["table"][0, 2], 0, 5] = c["codes"][0, c["table"][1, 0], 0, 1] = code[most]
    c["scales"][0] = np.float32(1e-3 / R.TOP[fmt])
    c["q"][:] = size / 64 * 1e3 / c["scale"]
    y = T.call_attn(c)
    assert c["status"] == 0
    for b, (pg, tok) in enumerate(((2, 5), (0, 1))):
        at = c["table"][b, pg]
        want = torch.from_numpy(R.value(c["codes"][1, at, 0, tok], fmt) * float(c["scales"][1, at, 0])).cuda()
        got = y[int(c["cu"][b]):int(c["cu"][b + 1])].double()
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 1e-30).all(), (got.flatten()[:4], want[:4])


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("group,new", [(4, 40), (8, 1)])
def test_attn_queries_of_zero_meet_keys_of_any_size(fmt, group, new):
    """Their logits are 0: an even mean."""
    c = T.make_attn(7, fmt, 1, 32, 1, group, 128, [300, 200], [new, new], nan_behind=False)
    c["scales"][0] = np.float32(1e36)
    c["q"][:] = 0
    check(c)


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("dim,page,lens", [(64, 16, (20011, 200)), (128, 64, (9001, 40)), (256, 32, (333, 70))])
@pytest.mark.parametrize("group,new", [(4, 40), (8, 1)])
@pytest.mark.parametrize("size", [7.9e28, 1e20, 1e-31, 1e-36])
def test_attn_values_of_any_size(fmt, dim, page, lens, group, new, size):
    """Values up to 2^96, the most that the calls take, and down to the subnormals, split jobs among them."""
    c = T.make_attn(dim + page, fmt, 1, page, 1, group, dim, lens, [new] * len(lens), spread=0.0, nan_behind=False)
    c["scales"][1] = np.float32(size / R.TOP[fmt])
    check(c)


# ------------------------------------------------------------------ slots
@pytest.mark.parametrize("width,length", [(4, 64), (1 << 14, 1 << 18)])
def test_slots_more_pages_released_than_there_are(width, length):
    """Every request claims the same pages: the stack ends full, nothing is written behind it, and the call is not held up."""
    Q = H.q()
    page, pages, rows = 16, 5, 64
    d = Q.kv_desc(R.INT8, page, pages, 1, 64)
    table = torch.arange(width, dtype=torch.int32, device="cuda").remainder(pages).repeat(rows, 1)
    free = T.dev(np.full(pages + 3, 77))
    ln, cu, sl, left, st = T.dev(np.zeros(rows)), T.dev(np.zeros(rows + 1)), T.dev([7]), T.dev([0]), T.dev([0])
    Q.qnt_kv_slots(d, T.dev(np.full(rows, length)), T.dev(np.full(rows, -1)), table, free, T.dev([0]), ln, cu, sl, left, rows, width, 1, st)
    torch.cuda.synchronize()
    assert int(st) == Q.QNT_ERR_ARG and int(left) == pages and ln.tolist() == [0] * rows and sl.tolist() == [-1]
    assert free.tolist() == [j % width % pages for j in range(pages)] + [77] * 3
