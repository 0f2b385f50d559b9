"""The key/value cache calls on the GPU against the 64-bit reference: qnt_kv_slots and qnt_kv_append bit for bit,
qnt_kv_attn within a bound derived from its roundings (kv_reference.attn)."""
import math

import numpy as np
import pytest
import torch

from tests import gpu_helpers as H
from tests import kv_reference as R

pytestmark = pytest.mark.gpu
TYPES = {0: torch.float16, 1: torch.bfloat16}


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to("cuda", dtype)


# ------------------------------------------------------------------ slots
def run_slots(page, pages, length, add, table, free, count, tokens):
    Q = H.q()
    rows, width = table.shape
    d = Q.kv_desc(Q.QNT_KV_INT8, page, pages, 1, 64)
    t, f = dev(table), dev(free)
    ln, cu, sl = dev(np.full(rows, 77)), dev(np.full(rows + 1, 77)), dev(np.full(tokens + 5, 77))
    left, st = dev([77]), dev([0])
    for _ in range(2):      # a repeated call gives the same outputs
        Q.qnt_kv_slots(d, dev(length), dev(add), t, f, dev([count]), ln, cu, sl, left, rows, width, tokens, st)
    torch.cuda.synchronize()
    assert sl[tokens:].eq(77).all()
    return t.cpu().numpy(), f.cpu().numpy(), ln.cpu().numpy(), cu.cpu().numpy(), sl[:tokens].cpu().numpy(), int(left), int(st)


def check_slots(*args):
    got, want = run_slots(*args), R.slots(*args)
    for g, w, name in zip(got, want, ["table", "free", "len_out", "cu", "slots", "free count", "status"]):
        assert np.array_equal(g, w), (name, g, w)


def random_slots(seed, rows, page, most, spare, releases=10, prompts=10, prompt=100):
    r = np.random.default_rng(seed)
    length = r.integers(0, most + 1, rows)
    add = np.where(r.integers(0, 100, rows) < prompts, r.integers(0, prompt + 1, rows), r.integers(0, 2, rows))
    add = np.where(r.integers(0, 100, rows) < releases, -1, add)
    up = lambda v: -(-v // page)  # noqa: E731
    n = np.maximum(add, 0)
    used, need = up(length), up(length + n) - up(length)
    width = up(most + prompt)
    held, pool = int(used.sum()), int(need.sum()) * spare // 100
    pages = held + pool + 3
    order = r.permutation(pages)
    table = np.full((rows, width), -1)
    table[np.arange(width)[None] < used[:, None]] = order[:held]
    free = np.full(pages, -1)
    free[:pool] = order[held:held + pool]
    return page, pages, length, add, table, free, pool, int(n.sum()) + 4


@pytest.mark.parametrize("seed,rows,page,most,spare", [(1, 1, 16, 40, 100), (2, 3, 16, 0, 100), (3, 33, 32, 100, 100), (4, 255, 64, 300, 100),
                                                       (5, 256, 16, 200, 70), (6, 257, 16, 200, 100), (7, 1025, 128, 900, 40), (8, 4096, 16, 60, 90),
                                                       (9, 37, 16, 50, 0)])
def test_slots_random(seed, rows, page, most, spare):
    check_slots(*random_slots(seed, rows, page, most, spare))


def test_slots_all_released_then_reused():
    r = np.random.default_rng(11)
    table = r.permutation(12).reshape(3, 4)
    check_slots(16, 12, np.array([64, 33, 64]), np.array([-1, -1, -1]), table, np.full(12, -1), 0, 4)
    # pages pushed in the call are popped in the call
    check_slots(16, 12, np.array([64, 33, 0]), np.array([-1, 15, 60]), np.where(np.arange(4)[None] < np.array([[4], [3], [0]]), table, -1),
                np.array([table[2, 0]] + [-1] * 11), 1, 75)


def test_slots_no_room():
    table = np.array([[0, 1], [2, -1], [3, -1], [-1, -1]])
    free = np.array([4, 5, 6, 7, -1, -1, -1, -1])
    check_slots(16, 8, np.array([32, 16, 5, 0]), np.array([1, 1, 11, 8]), table, free, 4, 21)      # row 0's table is full
    check_slots(16, 8, np.array([32, 16, 5, 0]), np.array([0, 1, 11, 8]), table, free, 4, 15)      # row 3 passes the token rows
    check_slots(16, 8, np.array([33, -1, 5, 0]), np.array([0, 1, 1, 1]), table, free, 4, 9)        # lengths outside the table
    check_slots(16, 8, np.array([33, -1, 5, 0]), np.array([-1, -1, 1, 1]), table, free, 4, 9)
    check_slots(16, 8, np.array([16, 16, 5, 0]), np.array([1, 1, 1, 1]), np.array([[0, -1], [2, -1], [3, -1], [-1, -1]]), free, 4, 0)
    check_slots(16, 8, np.array([0] * 4), np.array([2 ** 30, 2 ** 30, 2 ** 31 - 1, 1]), np.full((4, 2), -1), free, 4, 9)


# ------------------------------------------------------------------ append
def make_cache(seed, fmt, pages, heads, page, dim, nan=False):
    r = np.random.default_rng(seed)
    codes = r.integers(0, 256, (2, pages, heads, page, dim)).astype(np.uint8)
    if fmt == R.INT8:
        codes = np.maximum(codes, 1)
    elif not nan:
        codes[(codes & 127) == 127] = 9
    scales = (np.exp(r.normal(0, 0.5, (2, pages, heads))) * 3 / R.TOP[fmt]).astype(np.float32)
    return codes, scales


def check_append(fmt, xdt, page, dim, heads, codes, scales, x, slot, want_status=0, times=1):
    """x: tensor [2][tokens][heads * dim] on the CPU, in its type."""
    Q = H.q()
    pages = codes.shape[1]
    d = Q.kv_desc(fmt, page, pages, heads, dim)
    tokens = len(slot)
    buf = torch.zeros(tokens, 3 * heads * dim + 24, dtype=TYPES[xdt], device="cuda")     # rows of a larger matrix
    k, v = buf[:, 8:8 + heads * dim], buf[:, 16 + heads * dim:16 + 2 * heads * dim]
    k.copy_(x[0])
    v.copy_(x[1])
    gc, gs, st = dev(codes, torch.uint8), dev(scales, torch.float32), dev([0])
    for _ in range(times):
        Q.qnt_kv_append(d, gc[0], gc[1], gs[0], gs[1], k, v, buf.stride(0), dev(slot), tokens, xdt, st)
    torch.cuda.synchronize()
    status = 0
    for i in range(2):
        c, s, e = R.append(fmt, page, codes[i], scales[i], x[i].double().numpy().reshape(tokens, heads, dim), slot)
        status = max(status, e)
        assert np.array_equal(gs[i].cpu().numpy(), s), ("scales", i)
        got = gc[i].cpu().numpy()
        if not np.array_equal(got, c):
            at = np.argwhere(got != c)
            raise AssertionError(("codes", i, len(at), at[:4], got[tuple(at[0])], c[tuple(at[0])]))
    assert int(st) == status == want_status


def random_slots_of(r, page, pages, runs):
    """Slots of requests: (begin, count) pairs laid out over random pages."""
    order, at, out = r.permutation(pages), 0, []
    for begin, count in runs:
        for t in range(count):
            p = begin % page + t
            out.append(order[at + p // page] * page + p % page)
        at += -(-(begin % page + count) // page)
    return out


def values(seed, tokens, width, xdt, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, tokens, width, generator=g) * torch.exp(0.7 * torch.randn(2, tokens, 1, generator=g)) * scale
    return x.to(TYPES[xdt])


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("xdt", [0, 1])
@pytest.mark.parametrize("page,dim,heads", [(16, 64, 3), (32, 128, 2), (64, 128, 1), (128, 256, 1), (16, 256, 2), (128, 64, 2)])
def test_append_runs(fmt, xdt, page, dim, heads):
    r = np.random.default_rng(page + dim + fmt)
    runs = [(0, 1), (5, 1), (page - 1, 1), (page - 1, 2), (0, page), (3, 8), (3, 9), (0, 2 * page + 3), (page // 2, page), (1, 7)]
    pages = sum(-(-(b % page + n) // page) for b, n in runs) + 2
    slot = random_slots_of(r, page, pages, runs)
    for at in (0, 3, len(slot)):     # the last one falls into the last run, whose second part is refused
        slot.insert(at, -1)
    codes, scales = make_cache(3, fmt, pages, heads, page, dim)
    check_append(fmt, xdt, page, dim, heads, codes, scales, values(7, len(slot), heads * dim, xdt), np.array(slot), want_status=R.ARG)
    check_append(fmt, xdt, page, dim, heads, codes, scales, values(8, len(slot), heads * dim, xdt), np.array(slot), want_status=R.ARG, times=2)
    check_append(fmt, xdt, page, dim, heads, codes, scales, values(8, len(slot) - 3, heads * dim, xdt), np.array(slot[:-3]), times=2)


@pytest.mark.parametrize("fmt,xdt", [(R.INT8, 0), (R.E4M3, 1)])
def test_append_token_by_token_with_growing_scale(fmt, xdt):
    """A page filled one token a call: the scale grows now and then, the codes before are rounded again."""
    Q = H.q()
    page, dim, heads, pages = 32, 128, 2, 3
    d = Q.kv_desc(fmt, page, pages, heads, dim)
    x = values(21, page, heads * dim, xdt)
    x[:, :4] = 0                                            # the first tokens are zero: scale 0
    codes, scales = make_cache(5, fmt, pages, heads, page, dim)
    gc, gs, st = dev(codes, torch.uint8), dev(scales, torch.float32), dev([0])
    grew = 0
    for t in range(page):
        k, v = x[0, t:t + 1].cuda(), x[1, t:t + 1].cuda()
        Q.qnt_kv_append(d, gc[0], gc[1], gs[0], gs[1], k, v, heads * dim, dev([page + t]), 1, xdt, st)
        for i in range(2):
            before = scales[i].copy()
            codes[i], scales[i], _ = R.append(fmt, page, codes[i], scales[i], x[i, t:t + 1].double().numpy().reshape(1, heads, dim), np.array([page + t]))
            grew += int((scales[i] > before).sum()) if t else 0
            assert np.array_equal(gs[i].cpu().numpy(), scales[i]) and np.array_equal(gc[i].cpu().numpy(), codes[i]), t
    assert grew > 4 and int(st) == 0


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
def test_append_ties_and_near_ties(fmt):
    """Quotients at ties and next to them: x = k a / m for scales a / top with short and long mantissas."""
    page, dim, heads = 16, 256, 1
    rows = []
    for a in (127.0, 448.0, 1.0, 224.0, 2.0 ** -10 * 127, 1.9375, 255.0, 65504.0, 97.0):
        base = np.concatenate([np.arange(1, 128) * a / 254, (np.arange(0, 64) + 0.5) * a / 127, (np.arange(1, 65) * 2 - 1) * a / 64])
        rows.append(np.concatenate([[a], base])[:dim])
    x = torch.tensor(np.array(rows)).to(torch.float16)
    x = torch.where(x.abs() > x[:, :1], x[:, :1], x)
    x = torch.stack([x, -x])
    slot = np.arange(len(rows)) * page
    codes, scales = make_cache(6, fmt, len(rows), heads, page, dim)
    check_append(fmt, 0, page, dim, heads, codes, scales, x, slot)


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e30, 0.0])
def test_append_extreme_magnitudes(fmt, scale):
    page, dim, heads = 16, 64, 2
    codes, scales = make_cache(9, fmt, 4, heads, page, dim)
    scales[:] = np.float32(scale)
    x = values(31, 20, heads * dim, 1, scale)
    slot = np.concatenate([np.arange(5, 16), np.arange(32, 41)])
    check_append(fmt, 1, page, dim, heads, codes, scales, x, slot)


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
def test_append_non_finite_and_bad_slots(fmt):
    Q = H.q()
    page, dim, heads, pages = 16, 64, 2, 4
    codes, scales = make_cache(9, fmt, pages, heads, page, dim)
    x = values(32, 6, heads * dim, 0)
    # slots beyond the cache, and a second run of a page next to the first, are not written
    check_append(fmt, 0, page, dim, heads, codes, scales, x, np.array([3, 4, pages * page, 2 ** 31 - 1, 20, 21]), want_status=R.ARG)
    check_append(fmt, 0, page, dim, heads, codes, scales, x, np.array([3, 4, 6, 7, 20, 21]), want_status=R.ARG)
    check_append(fmt, 0, page, dim, heads, codes, scales, x, np.array([3, 4, 4, 0, 20, 21]), want_status=R.ARG)
    y = x.clone()
    y[0, 1, 5], y[0, 2, 9], y[1, 3, 70] = math.inf, math.nan, -math.inf
    d = Q.kv_desc(fmt, page, pages, heads, dim)
    gc, gs, st = dev(codes, torch.uint8), dev(scales, torch.float32), dev([0])
    Q.qnt_kv_append(d, gc[0], gc[1], gs[0], gs[1], y[0].cuda(), y[1].cuda(), heads * dim, dev(np.arange(6)), 6, 0, st)
    assert int(st) == Q.QNT_ERR_NONFINITE
    fin = torch.where(torch.isfinite(y), y, torch.zeros_like(y)).double().numpy().reshape(2, 6, heads, dim)
    for i in range(2):
        c, s, _ = R.append(fmt, page, codes[i], scales[i], fin[i], np.arange(6))
        assert np.array_equal(gs[i].cpu().numpy(), s)
        ok = torch.isfinite(y[i]).numpy().reshape(6, heads, dim).transpose(1, 0, 2)
        got = gc[i].cpu().numpy()
        assert np.array_equal(got[0, :, :6][ok], c[0, :, :6][ok])
        assert np.isfinite(R.value(got[0, :, :6], fmt)).all()


# ------------------------------------------------------------------ attention
def make_attn(seed, fmt, xdt, page, kv_heads, group, dim, lens, news, window=0, spread=1.0, nan_behind=True, pad=2):
    """A cache of random pages, its bytes behind the last token of a request anything at all, and queries."""
    r = np.random.default_rng(seed)
    lens, news = np.array(lens), np.array(news)
    used = -(-lens // page)
    width, pages = max(1, int(used.max())) + 1, int(used.sum()) + 2
    order = r.permutation(pages)
    table = np.full((len(lens), width), -1)
    table[np.arange(width)[None] < used[:, None]] = order[:used.sum()]
    codes = np.empty((2, pages, kv_heads, page, dim), np.uint8)
    scales = np.empty((2, pages, kv_heads), np.float32)
    for i in range(2):
        x = r.normal(size=(pages, kv_heads, page, dim)) * np.exp(spread * r.normal(size=(pages, kv_heads, 1, 1)))
        scales[i] = (np.abs(x).max((2, 3)) / R.TOP[fmt]).astype(np.float32)
        codes[i] = R.nearest(x / scales[i][..., None, None].astype(np.float64), fmt)
    if nan_behind:
        for b in range(len(lens)):
            if lens[b] % page:
                codes[:, table[b, lens[b] // page], :, lens[b] % page:] = 0x7F
        codes[:, order[used.sum():]] = 0xFF
        scales[:, order[used.sum():]] = np.nan
    cu = np.concatenate([[0], np.cumsum(news)])
    tokens = int(cu[-1]) + pad
    q = torch.tensor(r.normal(size=(tokens, kv_heads * group, dim)) * 1.5).to(TYPES[xdt])
    return dict(fmt=fmt, xdt=xdt, page=page, pages=pages, width=width, kv_heads=kv_heads, heads=kv_heads * group, dim=dim, lens=lens, cu=cu, table=table,
                codes=codes, scales=scales, q=q, tokens=tokens, window=window, scale=1 / math.sqrt(dim), max_new=int(max(1, news.max())))


def call_attn(c, work=None, gpu=None, max_new=None):
    """The GPU's y [tokens][heads][dim]: q and y are slices of wider rows, y is filled with 3 before."""
    Q = H.q()
    d = Q.kv_desc(c["fmt"], c["page"], c["pages"], c["kv_heads"], c["dim"])
    max_new = max_new or c["max_new"]
    if work is None:
        work = H.dev_bytes(Q.qnt_kv_attn_work_bytes(d, c["heads"], max_new))
    row = c["heads"] * c["dim"]
    qb = torch.zeros(c["tokens"], row + 24, dtype=TYPES[c["xdt"]], device="cuda")
    yb = torch.full((c["tokens"], row + 8), 3.0, dtype=TYPES[c["xdt"]], device="cuda")
    qb[:, 16:16 + row] = c["q"].reshape(c["tokens"], row)
    gc, gs = dev(c["codes"], torch.uint8), dev(c["scales"], torch.float32)
    st = dev([0])
    Q.qnt_kv_attn(d, gc[0], gc[1], gs[0], gs[1], qb[:, 16:], qb.stride(0), yb, yb.stride(0), c["heads"], dev(c["cu"]), dev(c["lens"]),
                  dev(c["table"]), len(c["lens"]), c["width"], c["tokens"], max_new, c["scale"], c["window"], work, c["xdt"], st)
    torch.cuda.synchronize()
    assert yb[:, row:].eq(3).all()
    c["status"] = int(st)
    return yb[:, :row].reshape(c["tokens"], c["heads"], c["dim"])


def check_attn(c, y=None, status=0, **kw):
    y = call_attn(c, **kw) if y is None else y
    assert c["status"] == status
    want, bound = R.attn(c["fmt"], c["page"], c["codes"][0], c["codes"][1], c["scales"][0], c["scales"][1], c["q"].double().numpy(), c["cu"], c["lens"],
                         c["table"], c["scale"], c["window"], torch.finfo(TYPES[c["xdt"]]).eps)
    got = y.double().cpu().numpy()
    live = ~np.isnan(want)
    assert (got[~live] == 3).all()                          # rows of no request are left as they were
    err = np.abs(got - want)[live]
    bad = ~(err <= bound[live])
    assert not bad.any(), (int(bad.sum()), float((err / bound[live]).max()), np.argwhere(~(np.abs(got - want) <= bound) & live)[:3])
    return y


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("xdt", [0, 1])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page,kv_heads,group", [(16, 2, 4), (32, 1, 1), (64, 3, 8), (128, 2, 7), (16, 1, 16)])
def test_attn_single_tokens(fmt, xdt, dim, page, kv_heads, group):
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 300, 511]
    check_attn(make_attn(dim + page, fmt, xdt, page, kv_heads, group, dim, lens, [1] * len(lens)))


@pytest.mark.parametrize("fmt,xdt,dim,page", [(R.INT8, 1, 128, 16), (R.E4M3, 0, 64, 32), (R.INT8, 0, 256, 64), (R.E4M3, 1, 128, 128)])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_attn_several_tokens(fmt, xdt, dim, page, group):
    """New tokens see those before them: drafts, and prompts that begin at nothing."""
    lens = [5, 40, 2, 100, 37, 64, 0, 3]
    news = [5, 3, 2, 1, 37, 20, 0, 1]
    check_attn(make_attn(2 * dim + page, fmt, xdt, page, 2, group, dim, lens, news))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 33, 100, 10 ** 6])
@pytest.mark.parametrize("fmt,xdt,dim,page", [(R.INT8, 1, 256, 32), (R.E4M3, 0, 128, 16)])
def test_attn_window(window, fmt, xdt, dim, page):
    lens = [1, 16, 17, 50, 260, 33, 40]
    news = [1, 1, 2, 1, 1, 33, 20]
    check_attn(make_attn(window, fmt, xdt, page, 1, 4, dim, lens, news, window=window))


@pytest.mark.parametrize("fmt,xdt", [(R.INT8, 0), (R.E4M3, 1)])
@pytest.mark.parametrize("new", [1, 4])
def test_attn_long_rows_are_split(fmt, xdt, new):
    """A long request is shared by many CTAs, beside short ones; twice with one workspace, bit for bit alike."""
    Q = H.q()
    c = make_attn(77, fmt, xdt, 64, 2, 4, 128, [20011, 3, 700, new], [new] * 3 + [new] if new < 4 else [4, 3, 2, 4])
    work = H.dev_bytes(Q.qnt_kv_attn_work_bytes(Q.kv_desc(fmt, 64, c["pages"], 2, 128), c["heads"], new))
    y = check_attn(c, work=work)
    again = call_attn(c, work=work)
    assert torch.equal(y, again)
    assert torch.equal(y, call_attn(c, max_new=1)) or new > 1      # max_new chooses the kernel only


def test_attn_max_new_is_a_hint():
    c = make_attn(78, R.INT8, 0, 16, 2, 4, 128, [50, 90, 17], [1, 6, 9])
    check_attn(c, max_new=1)
    check_attn(c, max_new=1000)


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
def test_attn_scales_far_apart(fmt):
    """Pages whose scales differ by many orders of magnitude, zero among them: no page's values are lost beside another's."""
    c = make_attn(79, fmt, 0, 16, 2, 2, 128, [200, 333], [1, 2])
    r = np.random.default_rng(1)
    c["scales"][1] *= (10.0 ** r.integers(-8, 4, c["scales"][1].shape)).astype(np.float32)
    c["scales"][0] *= (10.0 ** r.integers(-3, 1, c["scales"][0].shape)).astype(np.float32)
    c["scales"][:, c["table"][0, 1]] = 0
    c["scales"][1, c["table"][1, :5]] = 0
    check_attn(c)


@pytest.mark.parametrize("fmt,xdt", [(R.INT8, 0), (R.E4M3, 1)])
def test_attn_peaked_and_flat(fmt, xdt):
    """Logits of hundreds (one token takes it all, the reference moves again and again) and queries of zero."""
    c = make_attn(80, fmt, xdt, 32, 1, 8, 128, [400, 400], [1, 1])
    c["q"][0, ::2] *= 60
    c["q"][0, 1] = 0
    c["q"][1] *= 1e-3
    check_attn(c)


def test_attn_bf16_queries_of_any_size():
    c = make_attn(81, R.INT8, 1, 32, 1, 8, 128, [60], [1])
    for h, s in enumerate([1e-38, 1e-30, 1e-10, 1e-2, 10.0, 1e5, 0.0, 1.0]):
        c["q"][0, h] *= s
    c["scales"][0] *= np.float32(1e-4)
    check_attn(c)


def test_attn_non_finite_queries_stay_in_their_row():
    c = make_attn(82, R.INT8, 0, 16, 1, 8, 128, [70, 50], [1, 1])
    y0 = call_attn(c)
    c["q"][0, 2, 5], c["q"][1, 7, 0] = math.nan, math.inf
    y1 = call_attn(c)
    same = torch.ones(c["tokens"], 8, dtype=torch.bool)
    same[0, 2] = same[1, 7] = False
    assert torch.equal(y0[same], y1[same]) and y1[0, 2].isnan().all()


def test_attn_rows_that_see_nothing():
    """len < n (a request that got no room) and len = 0: those queries see nothing and get 0."""
    c = make_attn(83, R.E4M3, 0, 16, 2, 2, 64, [0, 20, 5], [3, 1, 2])
    c["lens"] = np.array([0, 20, 1])
    check_attn(c)


def test_attn_bad_pages_and_lengths_are_reported():
    """A page number outside the cache is read as page 0, a length beyond the table is cut: both set the status."""
    Q = H.q()
    c = make_attn(84, R.INT8, 0, 16, 2, 2, 64, [40, 50], [1, 1], nan_behind=False)
    for bad in (-5, c["pages"], 2 ** 31 - 1):
        d = dict(c, table=c["table"].copy())
        d["table"][1, 1] = bad
        y = call_attn(d)
        assert d["status"] == Q.QNT_ERR_ARG
        d["table"][1, 1] = 0
        check_attn(d, y=y, status=Q.QNT_ERR_ARG)
    # cut at width * page, whose last page does not exist here: page 0
    d = dict(c, table=np.where(c["table"] < 0, 0, c["table"]), lens=np.array([40, 10 ** 9]))
    y = call_attn(d)
    assert d["status"] == Q.QNT_ERR_ARG
    d["lens"] = np.array([40, c["width"] * 16])
    check_attn(d, y=y, status=Q.QNT_ERR_ARG)


def test_attn_many_rows():
    r = np.random.default_rng(5)
    lens = r.integers(1, 40, 1500)
    check_attn(make_attn(85, R.INT8, 0, 16, 1, 1, 64, lens, [1] * 1500))


# ------------------------------------------------------------------ together
def test_streams_and_two_calls_at_once():
    """Two calls on two streams with a workspace each, beside work on the default stream."""
    Q = H.q()
    cases = [make_attn(90 + i, R.INT8, 0, 64, 2, 4, 128, [9000, 50], [1, 1]) for i in range(2)]
    want = [call_attn(c).clone() for c in cases]
    args, outs = [], []
    for c in cases:
        d = Q.kv_desc(c["fmt"], c["page"], c["pages"], c["kv_heads"], c["dim"])
        row = c["heads"] * c["dim"]
        q, gc, gs = c["q"].reshape(c["tokens"], row).cuda(), dev(c["codes"], torch.uint8), dev(c["scales"], torch.float32)
        y = torch.full((c["tokens"], row), 3.0, dtype=torch.float16, device="cuda")
        work = H.dev_bytes(Q.qnt_kv_attn_work_bytes(d, c["heads"], 1))
        args.append((d, gc[0], gc[1], gs[0], gs[1], q, row, y, row, c["heads"], dev(c["cu"]), dev(c["lens"]), dev(c["table"]), 2, c["width"], c["tokens"],
                     1, c["scale"], 0, work))
        outs.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for a, s in zip(args, streams):
            Q.qnt_kv_attn(*a, stream=s)
    torch.cuda.synchronize()
    for y, w in zip(outs, want):
        assert torch.equal(y.view(w.shape), w)


@pytest.mark.parametrize("fmt,xdt", [(R.INT8, 0), (R.E4M3, 1)])
def test_decode_steps_together(fmt, xdt):
    """Steps as a server runs them, the steps' launches captured into one CUDA graph: places for the new tokens, the qkv
    product (qnt_gemm), the append, the attention and the o product.  One request draws on pages that another released."""
    Q = H.q()
    from dequant_gemv_rtn_b200 import synth
    from oracle import oracle as orc
    B, heads, kv, dim, page, width, pages = 4, 4, 2, 64, 16, 4, 12
    K, row = 256, heads * dim
    N = row + 2 * kv * dim
    mats = []
    for n, k, seed in ((N, K, 1), (K, row, 2)):
        ref = orc.quantize(orc.INT4, synth.llama_like(n, k, seed=seed), 64)
        pc, pm = orc.pack(ref)
        mats.append((Q.desc(Q.QNT_INT4_ASYM, n, k, 64), torch.from_numpy(pc).cuda(), torch.from_numpy(pm).cuda()))
    d = Q.kv_desc(fmt, page, pages, kv, dim)
    T, dt = 24, TYPES[xdt]
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    length, add, len_out, cu, sl, table = i32(B), i32(B), i32(B), i32(B + 1), i32(T), i32(B, width) - 1
    free, count, left, st = torch.arange(pages, dtype=torch.int32, device="cuda"), i32(1) + pages, i32(1), i32(1)
    codes = torch.randint(0, 256, (2, pages, kv, page, dim), dtype=torch.uint8, device="cuda")
    scales = torch.rand(2, pages, kv, device="cuda")
    x, y = torch.zeros(T, K, dtype=dt, device="cuda"), torch.zeros(T, row, dtype=dt, device="cuda")
    qkv, out = torch.zeros(T, N, dtype=dt, device="cuda"), torch.zeros(T, K, dtype=dt, device="cuda")
    work = H.dev_bytes(Q.qnt_kv_attn_work_bytes(d, heads, T))

    def step():
        Q.qnt_kv_slots(d, length, add, table, free, count, len_out, cu, sl, left, B, width, T, st)
        Q.qnt_gemm(*mats[0], x, qkv, T, xdt, st)
        Q.qnt_kv_append(d, codes[0], codes[1], scales[0], scales[1], qkv[:, row:], qkv[:, row + kv * dim:], N, sl, T, xdt, st)
        Q.qnt_kv_attn(d, codes[0], codes[1], scales[0], scales[1], qkv, N, y, row, heads, cu, len_out, table, B, width, T, T, 0.125, 0, work, xdt, st)
        Q.qnt_gemm(*mats[1], y, out, T, xdt, st)
        length.copy_(len_out)
        count.copy_(left)

    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        step()                                              # adds nothing
    warm.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    cpu = lambda t: t.cpu().numpy()  # noqa: E731
    g = torch.Generator().manual_seed(5)
    for news in ([10, 3, 0, 5], [1, 1, 7, 1], [1, -1, 1, 12], [5, 0, 1, 1], [1, 9, 1, 1], [1, 1, -1, 1], [20, 1, 0, 1], [1, 1, 2, 1]):
        add.copy_(torch.tensor(news, dtype=torch.int32))
        x.copy_(torch.randn(T, K, generator=g).to(dt))
        before = [cpu(t).copy() for t in (length, table, free, count, codes, scales)]
        graph.replay()
        torch.cuda.synchronize()
        want = R.slots(page, pages, before[0], np.array(news), before[1], before[2], int(before[3][0]), T)
        for got, w in zip((table, free, len_out, cu, sl, left), want):
            assert np.array_equal(cpu(got).reshape(np.shape(w)), w)
        flat = qkv.double().cpu().numpy()
        for i in range(2):
            part = flat[:, row + i * kv * dim:row + (i + 1) * kv * dim].reshape(T, kv, dim)
            c, s, _ = R.append(fmt, page, before[4][i], before[5][i], part, cpu(sl))
            assert np.array_equal(cpu(codes[i]), c) and np.array_equal(cpu(scales[i]), s)
        ref, bound = R.attn(fmt, page, cpu(codes[0]), cpu(codes[1]), cpu(scales[0]), cpu(scales[1]), flat[:, :row].reshape(T, heads, dim), cpu(cu), cpu(len_out),
                            cpu(table), 0.125, 0, torch.finfo(dt).eps)
        live = ~np.isnan(ref)
        err = np.abs(y.double().cpu().numpy().reshape(T, heads, dim) - ref)
        assert (err[live] <= bound[live]).all(), float((err / bound)[live].max())
    assert int(st) == 0


# ------------------------------------------------------------------ many query rows (tensor-memory kernel)
@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("xdt", [0, 1])
@pytest.mark.parametrize("dim,page,kv_heads,group,lens,news,window", [
    (128, 64, 1, 4, [5], [5], 0), (128, 16, 1, 4, [40], [33], 0), (64, 32, 2, 8, [300, 17], [40, 17], 0), (256, 128, 1, 4, [200, 64, 1], [64, 40, 1], 0),
    (128, 16, 2, 7, [129, 30, 260], [5, 3, 41], 0), (64, 16, 1, 16, [90, 400], [16, 33], 50), (256, 16, 1, 1, [700], [150], 100), (128, 32, 1, 3, [700, 9], [300, 0], 130)])
def test_attn_many_query_rows(fmt, xdt, dim, page, kv_heads, group, lens, news, window):
    check_attn(make_attn(3 * dim + page + group, fmt, xdt, page, kv_heads, group, dim, lens, news, window=window))


@pytest.mark.parametrize("fmt,xdt,dim,group,len_,new", [(R.E4M3, 0, 64, 8, 20011, 9), (R.INT8, 1, 128, 4, 9001, 130), (R.INT8, 0, 256, 4, 7003, 33), (R.E4M3, 1, 128, 65, 20011, 1)])
def test_attn_many_query_rows_split(fmt, xdt, dim, group, len_, new):
    """One request on one key/value head is shared by every CTA; twice with one workspace, bit for bit alike."""
    Q = H.q()
    c = make_attn(len_ + dim, fmt, xdt, 64, 1, group, dim, [len_, 70], [new, 1])
    work = H.dev_bytes(Q.qnt_kv_attn_work_bytes(Q.kv_desc(fmt, 64, c["pages"], 1, dim), c["heads"], new))
    y = check_attn(c, work=work)
    assert torch.equal(y, call_attn(c, work=work))
    assert int(work[:16384].max()) == 0                    # ready for the next call


def test_attn_wait_expires_and_next_call_is_correct():
    """The tcgen05 kernel of the test build: in CTA 0 a decode warp never reports the first tile, so the waits behind it
    expire (50 ms).  The call returns QNT_ERR_TIMEOUT in the status, has freed its tensor memory and leaves the
    workspace ready: the next calls with it, the product library's and the test build's, are correct."""
    import ctypes
    import time
    Q = H.q()
    from dequant_gemv_rtn_b200 import build
    f = ctypes.CDLL(build.build(test=True)).qnt_test_kv_attn_fault
    P, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    f.restype, f.argtypes = I, [P, P, P, P, P, P, L, P, L, I, P, P, P, I, I, I, I, ctypes.c_float, I, P, I, P, P, I, ctypes.c_ulonglong]
    c = make_attn(95, R.INT8, 0, 16, 2, 4, 128, [300, 5000], [40, 33])
    d = Q.kv_desc(c["fmt"], c["page"], c["pages"], c["kv_heads"], c["dim"])
    work = H.dev_bytes(Q.qnt_kv_attn_work_bytes(d, c["heads"], c["max_new"]))
    row = c["heads"] * c["dim"]
    q, gc, gs = c["q"].reshape(c["tokens"], row).cuda(), dev(c["codes"], torch.uint8), dev(c["scales"], torch.float32)
    y, cu, ln, tb, st = torch.full_like(q, 3.0), dev(c["cu"]), dev(c["lens"]), dev(c["table"]), dev([0])

    def call(fault, timeout_ns):
        return f(ctypes.addressof(d), gc[0].data_ptr(), gc[1].data_ptr(), gs[0].data_ptr(), gs[1].data_ptr(), q.data_ptr(), row, y.data_ptr(), row, c["heads"],
                 cu.data_ptr(), ln.data_ptr(), tb.data_ptr(), 2, c["width"], c["tokens"], c["max_new"], c["scale"], 0, work.data_ptr(), 0, st.data_ptr(),
                 torch.cuda.current_stream().cuda_stream, fault, timeout_ns)

    torch.cuda.synchronize()
    t0 = time.time()
    assert call(1, 50_000_000) == Q.QNT_OK
    torch.cuda.synchronize()
    assert int(st) == Q.QNT_ERR_TIMEOUT and 0.05 <= time.time() - t0 < 10.0
    check_attn(c, work=work)
    st.zero_()
    y.fill_(3)
    assert call(0, 2_000_000_000) == Q.QNT_OK
    torch.cuda.synchronize()
    c["status"] = int(st)
    check_attn(c, y=y.reshape(c["tokens"], c["heads"], c["dim"]))


@pytest.mark.parametrize("scale", [-0.2, 0.0])
@pytest.mark.parametrize("new", [2, 50])
def test_attn_scale_of_any_sign(scale, new):
    c = make_attn(96, R.INT8, 1, 32, 1, 4, 64, [90, 200], [1, new])
    c["scale"] = scale
    check_attn(c)


@pytest.mark.parametrize("dim,page,tokens", [(64, 32, 1300), (128, 16, 700), (256, 128, 330)])
@pytest.mark.parametrize("fmt,xdt", [(R.INT8, 1), (R.E4M3, 0)])
def test_append_prompts(dim, page, tokens, fmt, xdt):
    """Enough rows for the wide windows: prompts of several pages, decode rows between them."""
    r = np.random.default_rng(dim)
    heads, runs, left = 16, [], tokens
    while left > 0:
        n = min(left, int(r.choice([1, 1, 3, page, 2 * page + 5, 7 * page + 1])))
        runs.append((int(r.integers(0, page)), n))
        left -= n
    pages = sum(-(-(b % page + n) // page) for b, n in runs) + 2
    slot = random_slots_of(r, page, pages, runs) + [-1] * 5
    codes, scales = make_cache(4, fmt, pages, heads, page, dim)
    check_append(fmt, xdt, page, dim, heads, codes, scales, values(9, len(slot), heads * dim, xdt), np.array(slot))


def test_attn_window_needs_no_page_before_it():
    """Pages that lie wholly before every new token's window may be gone (their table entries -1)."""
    for new, group in ((1, 4), (3, 4), (60, 4)):
        c = make_attn(97, R.INT8, 0, 16, 1, group, 128, [700, 350], [new, 1], window=100)
        for b in range(2):
            first = max(0, int(c["lens"][b]) - int(c["cu"][b + 1] - c["cu"][b]) + 1 - 100) // 16
            c["table"][b, :first] = -1
        y = call_attn(c)
        assert c["status"] == 0
        full = dict(c, table=np.where(c["table"] < 0, 0, c["table"]))
        check_attn(full, y=y)


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("new", [1, 40])
def test_cache_beyond_32_bit_offsets(fmt, new):
    """Codes of 5.2 GB: pages at both ends, written by an append and read by attention."""
    Q = H.q()
    page, heads, dim, pages = 128, 8, 128, 40000
    d = Q.kv_desc(fmt, page, pages, heads, dim)
    assert Q.qnt_kv_codes_bytes(d) > 2 ** 32
    codes = [torch.empty(Q.qnt_kv_codes_bytes(d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = torch.zeros(2, pages, heads, device="cuda")
    ids, L, tokens = [39998, 5, 39999], 300, 300
    slot = np.array([ids[t // page] * page + t % page for t in range(L)])
    x = values(3, tokens, heads * dim, 0)
    st = dev([0])
    Q.qnt_kv_append(d, codes[0], codes[1], scales[0], scales[1], x[0].cuda(), x[1].cuda(), heads * dim, dev(slot), tokens, 0, st)
    q = torch.randn(new, 2 * heads * dim, generator=torch.Generator().manual_seed(1)).half()
    y = torch.zeros(new, 2 * heads * dim, dtype=torch.float16, device="cuda")
    work = H.dev_bytes(Q.qnt_kv_attn_work_bytes(d, 2 * heads, new))
    Q.qnt_kv_attn(d, codes[0], codes[1], scales[0], scales[1], q.cuda(), 2 * heads * dim, y, 2 * heads * dim, 2 * heads, dev([0, new]), dev([L]), dev([ids]),
                  1, 3, new, new, 0.09, 0, work, 0, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    c = [k.view(pages, heads, page, dim)[ids].cpu().numpy() for k in codes]
    s = [k[ids].cpu().numpy() for k in scales]
    small = np.array([t for t in range(L)])
    for i in range(2):
        want_c, want_s, _ = R.append(fmt, page, c[i], np.zeros((3, heads), np.float32), x[i].double().numpy().reshape(tokens, heads, dim), small)
        assert np.array_equal(s[i], want_s) and np.array_equal(c[i][:2], want_c[:2]) and np.array_equal(c[i][2, :, :L - 256], want_c[2, :, :L - 256])
    want, bound = R.attn(fmt, page, c[0], c[1], s[0], s[1], q.double().numpy().reshape(new, 2 * heads, dim), np.array([0, new]), np.array([L]),
                         np.array([[0, 1, 2]]), 0.09, 0, torch.finfo(torch.float16).eps)
    assert (np.abs(y.double().cpu().numpy().reshape(want.shape) - want) <= bound).all()


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 128)])
@pytest.mark.parametrize("new", [1, 2, 70])
def test_attn_bytes_before_the_window_may_be_nan(dim, page, new):
    """The window begins inside a page: what is before it there, seen by no query, does not reach the result."""
    c = make_attn(dim + new, R.E4M3, 0, page, 1, 4, dim, [700, 357], [new, 1], window=99)
    for b in range(2):
        first = max(0, int(c["lens"][b]) - int(c["cu"][b + 1] - c["cu"][b]) + 1 - 99)
        c["codes"][:, c["table"][b, first // page], :, :first % page] = 0x7F
    check_attn(c)


def test_append_second_run_behind_a_bad_slot_is_refused():
    """A slot beyond the cache is a skipped row, also between two runs of a page."""
    Q = H.q()
    page, heads, dim, pages = 16, 2, 64, 3
    d = Q.kv_desc(R.INT8, page, pages, heads, dim)
    slot = np.array([16, 17, pages * page + 4, -1, 20, 21, 32, 33])
    x = values(11, len(slot), heads * dim, 0)
    codes = [dev(np.full((pages, heads, page, dim), 200), torch.uint8) for _ in range(2)]
    scales = torch.zeros(2, pages, heads, device="cuda")
    st = dev([0])
    Q.qnt_kv_append(d, codes[0], codes[1], scales[0], scales[1], x[0].cuda(), x[1].cuda(), heads * dim, dev(slot), len(slot), 0, st)
    torch.cuda.synchronize()
    assert int(st) == R.ARG
    for i in range(2):
        want_c, want_s, status = R.append(R.INT8, page, np.full((pages, heads, page, dim), 200, np.uint8), np.zeros((pages, heads), np.float32),
                                          x[i].double().numpy().reshape(-1, heads, dim), slot)
        assert status == R.ARG
        assert np.array_equal(codes[i].cpu().numpy(), want_c) and np.array_equal(scales[i].cpu().numpy(), want_s)


def test_slots_of_pages_outside_the_cache():
    """Their tokens get a slot that qnt_kv_append refuses, whatever the product with the page size would wrap to."""
    Q = H.q()
    page, pages, rows, width, tokens = 16, 40, 4, 5, 12
    length, add = np.array([18, 3, 16, 16]), np.array([2, 1, 2, 3])
    table = np.zeros((rows, width), np.int64)
    table[0, :2], table[1, 0], table[2, 0], table[3, 0] = [4, 1 << 28], -1, 5, 6
    free = np.zeros(pages, np.int64)
    free[:3] = [7, (1 << 28) + 1, 9]
    d = Q.kv_desc(R.INT8, page, pages, 1, 64)
    t, f, out, cu, slot, count, st = dev(table), dev(free), dev(np.zeros(rows)), dev(np.zeros(rows + 1)), dev(np.zeros(tokens)), dev([0]), dev([0])
    Q.qnt_kv_slots(d, dev(length), dev(add), t, f, dev([3]), out, cu, slot, count, rows, width, tokens, st)
    torch.cuda.synchronize()
    none = 2 ** 31 - 1
    assert slot.tolist() == [none, none, none, 9 * page, 9 * page + 1, none, none, none] + [-1] * 4
    assert [int(x) for x in R.slots(page, pages, length, add, table, free, 3, tokens)[4]] == slot.tolist()
    assert t[2, 1] == 9 and t[3, 1] == (1 << 28) + 1 and int(count) == 1
