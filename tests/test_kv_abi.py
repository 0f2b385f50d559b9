"""The key/value cache calls without a GPU: descriptor and buffer sizes, refusals (nothing is launched), and the 64-bit
reference of the GPU tests pinned by hand."""
import numpy as np
import pytest

from tests import kv_reference as R

A = 1 << 20   # a fake, 16-byte aligned address: validation fails before any CUDA call


@pytest.fixture(scope="module")
def q():
    from dequant_gemv_rtn_b200 import build
    build.build()
    from dequant_gemv_rtn_b200 import qnt
    return qnt


def test_descriptor(q):
    good = q.kv_desc(q.QNT_KV_INT8, 16, 3, 2, 64)
    assert q.qnt_check_kv_desc(good) == q.QNT_OK
    assert q.qnt_kv_codes_bytes(good) == 3 * 2 * 16 * 64 and q.qnt_kv_scales_bytes(good) == 3 * 2 * 4
    big = q.kv_desc(q.QNT_KV_E4M3, 128, (1 << 24) - 1, 8, 256)
    assert q.qnt_kv_codes_bytes(big) == ((1 << 24) - 1) * 8 * 128 * 256
    for bad, code in [((0, 16, 3, 2, 64), q.QNT_ERR_ARG), ((3, 16, 3, 2, 64), q.QNT_ERR_ARG), ((1, 8, 3, 2, 64), q.QNT_ERR_SHAPE),
                      ((1, 48, 3, 2, 64), q.QNT_ERR_SHAPE), ((1, 256, 3, 2, 64), q.QNT_ERR_SHAPE), ((1, 16, 0, 2, 64), q.QNT_ERR_SHAPE),
                      ((1, 128, 1 << 24, 2, 64), q.QNT_ERR_SHAPE), ((1, 16, 3, 0, 64), q.QNT_ERR_SHAPE), ((1, 16, 3, 1025, 64), q.QNT_ERR_SHAPE),
                      ((1, 16, 3, 2, 80), q.QNT_ERR_SHAPE)]:
        d = q.kv_desc(*bad)
        assert q.qnt_check_kv_desc(d) == code, bad
        assert q.qnt_kv_codes_bytes(d) == 0 and q.qnt_kv_scales_bytes(d) == 0 and q.qnt_kv_attn_work_bytes(d, 4, 1) == 0
    assert q.qnt_strerror(q.QNT_ERR_PAGES) and "unknown" not in q.qnt_strerror(q.QNT_ERR_PAGES)


def test_work_bytes(q):
    d = q.kv_desc(q.QNT_KV_INT8, 16, 3, 2, 64)
    assert q.qnt_kv_attn_work_bytes(d, 4, 1) > 0
    assert q.qnt_kv_attn_work_bytes(d, 5, 1) == 0 and q.qnt_kv_attn_work_bytes(d, 0, 1) == 0 and q.qnt_kv_attn_work_bytes(d, 4, 0) == 0


def test_work_bytes_refuses_the_heads_that_the_call_refuses(q):
    d = q.kv_desc(q.QNT_KV_INT8, 16, 3, 2, 64)
    assert q.qnt_kv_attn_work_bytes(d, 65536, 1) > 0 and q.qnt_kv_attn_work_bytes(d, 65538, 1) == 0


def test_slots_refusals(q):
    d = q.kv_desc(q.QNT_KV_INT8, 16, 3, 2, 64)
    names = ["length", "add", "table", "free", "free_count", "len_out", "cu", "slots", "free_count_out"]
    good = {n: A + 64 * i for i, n in enumerate(names)}

    def call(desc=d, rows=4, width=2, tokens=4, **change):
        return q.qnt_kv_slots(desc, *{**good, **change}.values(), rows, width, tokens, check=False, stream=0)

    for n in names:
        assert call(**{n: None}) == q.QNT_ERR_ARG, n
        assert call(**{n: good[n] + 2}) == q.QNT_ERR_ALIGN, n
    assert call(len_out=good["length"]) == q.QNT_ERR_ARG and call(len_out=good["add"]) == q.QNT_ERR_ARG
    assert call(free_count_out=good["free_count"]) == q.QNT_ERR_ARG
    for kw in ({"rows": 0}, {"rows": q.QNT_KV_MAX_ROWS + 1}, {"width": 0}, {"width": (1 << 26) + 1}, {"tokens": -1},
               {"tokens": q.QNT_KV_MAX_TOKENS + 1}, {"desc": q.kv_desc(1, 17, 3, 2, 64)}):
        assert call(**kw) == q.QNT_ERR_SHAPE, kw
    with pytest.raises(q.QntError):
        q.qnt_kv_slots(d, *good.values(), 0, 2, 4, stream=0)


def test_append_refusals(q):
    d = q.kv_desc(q.QNT_KV_E4M3, 16, 3, 2, 64)
    names = ["k_codes", "v_codes", "k_scales", "v_scales", "k", "v"]
    good = {n: A for n in names}

    def call(desc=d, stride=128, slots=A, tokens=4, xdtype=0, **change):
        return q.qnt_kv_append(desc, *{**good, **change}.values(), stride, slots, tokens, xdtype, check=False, stream=0)

    for n in names:
        assert call(**{n: None}) == q.QNT_ERR_ARG, n
        assert call(**{n: A + (2 if n.endswith("scales") else 8)}) == q.QNT_ERR_ALIGN, n
    assert call(slots=None) == q.QNT_ERR_ARG and call(slots=A + 1) == q.QNT_ERR_ALIGN and call(xdtype=2) == q.QNT_ERR_ARG
    assert call(stride=120) == q.QNT_ERR_SHAPE and call(stride=132) == q.QNT_ERR_SHAPE and call(tokens=-1) == q.QNT_ERR_SHAPE
    assert call(tokens=q.QNT_KV_MAX_TOKENS + 1) == q.QNT_ERR_SHAPE and call(desc=q.kv_desc(9, 16, 3, 2, 64)) == q.QNT_ERR_ARG
    assert call(tokens=0) == q.QNT_OK                       # nothing to do, nothing launched


def test_attn_refusals(q):
    d = q.kv_desc(q.QNT_KV_INT8, 16, 3, 2, 64)
    names = ["k_codes", "v_codes", "k_scales", "v_scales", "q", "y", "cu", "length", "table", "work"]
    good = {n: A for n in names}

    def call(desc=d, q_stride=256, y_stride=256, heads=4, rows=2, width=2, tokens=4, max_new=1, scale=0.1, window=0, xdtype=0, **change):
        p = {**good, **change}
        return q.qnt_kv_attn(desc, p["k_codes"], p["v_codes"], p["k_scales"], p["v_scales"], p["q"], q_stride, p["y"], y_stride, heads, p["cu"],
                             p["length"], p["table"], rows, width, tokens, max_new, scale, window, p["work"], xdtype, check=False, stream=0)

    four = {"k_scales", "v_scales", "cu", "length", "table"}
    for n in names:
        assert call(**{n: None}) == q.QNT_ERR_ARG, n
        assert call(**{n: A + (2 if n in four else 8)}) == q.QNT_ERR_ALIGN, n
    for kw in ({"heads": 0}, {"heads": 5}, {"tokens": q.QNT_KV_MAX_TOKENS}, {"heads": 65538}, {"q_stride": 248}, {"q_stride": 260}, {"y_stride": 248}, {"y_stride": 260}, {"rows": 0},
               {"rows": q.QNT_KV_MAX_ROWS + 1}, {"width": 0}, {"width": (1 << 26) + 1}, {"tokens": -1}, {"tokens": q.QNT_KV_MAX_TOKENS + 1}):
        assert call(**kw) == q.QNT_ERR_SHAPE, kw
    for kw in ({"max_new": 0}, {"window": -1}, {"scale": float("nan")}, {"scale": float("inf")}, {"xdtype": 7}):
        assert call(**kw) == q.QNT_ERR_ARG, kw
    assert call(tokens=0) == q.QNT_OK


def test_attn_refuses_scales_that_overflow_the_logits_factor(q):
    d = q.kv_desc(q.QNT_KV_INT8, 16, 3, 2, 64)

    def call(scale):
        return q.qnt_kv_attn(d, A, A, A, A, A, 256, A, 256, 4, A, A, A, 2, 2, 0, 1, scale, 0, A, check=False, stream=0)

    for scale in (3e38, -3e38, 2.0 ** 65, float("-inf")):
        assert call(scale) == q.QNT_ERR_ARG, scale
    assert call(2.0 ** 64) == q.QNT_OK and call(-(2.0 ** 64)) == q.QNT_OK     # no tokens: nothing launched


def test_current_stream_without_the_raw_number(q, monkeypatch):
    """A torch that does not offer the stream's number: the Stream object is asked."""
    import types

    import torch
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    assert q._current_stream() == 1003
    monkeypatch.delattr(torch._C, "_cuda_getDevice")
    assert q._current_stream() == 77


# ------------------------------------------------------------------ the reference itself
def test_reference_e4m3_rounding_against_torch():
    import torch
    vals = R.e4m3_table()
    got = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(vals), np.isnan(got)) and np.array_equal(vals[~np.isnan(vals)], got[~np.isnan(got)])
    x = np.concatenate([np.linspace(-448, 448, 40001), (R.e4m3_table()[:126] + R.e4m3_table()[1:127]) / 2, [2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11]])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()      # x here is exact in fp32 or far from a tie
    near = np.abs(x - x.astype(np.float32)) == 0
    assert np.array_equal(R.nearest(x, R.E4M3)[near], want[near])


def test_reference_slots_by_hand():
    # page 16, 2 columns: row 0 goes on in its page, row 1 leaves (pages 7, 3), row 2 is new with 20 tokens
    table = np.array([[5, -1], [7, 3], [-1, -1]])
    t, f, ln, cu, sl, left, st = R.slots(16, 8, np.array([14, 17, 0]), np.array([2, -1, 20]), table, np.array([1, 0, 0, 0, 0, 0, 0, 0]), 1, 24)
    assert t.tolist() == [[5, -1], [7, 3], [3, 7]] and ln.tolist() == [16, 0, 20] and cu.tolist() == [0, 2, 2, 22] and left == 1 and st == 0
    assert sl.tolist() == [94, 95] + list(range(48, 64)) + [112, 113, 114, 115] + [-1, -1]
    # a stack of one page: row 0 takes it, row 1 gets none, row 2 needs none
    t, f, ln, cu, sl, left, st = R.slots(16, 8, np.array([16, 16, 3]), np.array([1, 1, 1]), np.array([[0, -1], [1, -1], [2, -1]]), np.array([4] + [0] * 7), 1, 3)
    assert t.tolist() == [[0, 4], [1, -1], [2, -1]] and ln.tolist() == [17, 16, 4] and sl.tolist() == [64, -1, 35] and left == 0 and st == R.PAGES


def test_reference_append_by_hand():
    # INT8: 2.0 / s = 127, then 0.5 / s = 31.75 -> 32; the page grows to 4 / 127: 127 -> 63.5 -> 64 (even), 32 -> 16
    codes, scales = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.float32)
    x = np.zeros((2, 1, 64))
    x[0, 0, 0], x[1, 0, 0] = 2.0, -0.5
    c, s, st = R.append(R.INT8, 16, codes, scales, x, np.array([0, 1]))
    assert st == 0 and s[0, 0] == np.float32(2 / 127) and c[0, 0, 0, 0] == 255 and c[0, 0, 1, 0] == 128 - 32 and c[0, 0, 0, 1] == 128
    y = np.zeros((1, 1, 64))
    y[0, 0, 3] = 4.0
    c, s, st = R.append(R.INT8, 16, c, s, y, np.array([2]))
    assert s[0, 0] == np.float32(4 / 127) and c[0, 0, 0, 0] == 128 + 64 and c[0, 0, 1, 0] == 128 - 16 and c[0, 0, 2, 3] == 255
