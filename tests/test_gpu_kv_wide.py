"""qnt_kv_attn's tcgen05 kernel: its own tests of masks, magnitudes, splits and refused pages, and of which requests it
takes.  (The cases of test_gpu_kv.py with few query rows run the mma.sync kernel.)"""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import gpu_helpers as H
from tests import kv_reference as R
from tests import test_gpu_kv as T
from tests import test_gpu_kv_range as G

pytestmark = pytest.mark.gpu


def goes_wide(c):
    """Whether the tcgen05 kernel has rows of this call: in the test build a decode warp of its CTA 0 never reports a tile, so
    the call ends with QNT_ERR_TIMEOUT after the wait's limit (30 ms) if it has, and without if not."""
    Q = H.q()
    from dequant_gemv_rtn_b200 import build
    f = ctypes.CDLL(build.build(test=True)).qnt_test_kv_attn_fault
    P, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    f.restype, f.argtypes = I, [P, P, P, P, P, P, L, P, L, I, P, P, P, I, I, I, I, ctypes.c_float, I, P, I, P, P, I, ctypes.c_ulonglong]
    d = Q.kv_desc(c["fmt"], c["page"], c["pages"], c["kv_heads"], c["dim"])
    work = H.dev_bytes(Q.qnt_kv_attn_work_bytes(d, c["heads"], c["max_new"]))
    row = c["heads"] * c["dim"]
    q, gc, gs = c["q"].reshape(c["tokens"], row).cuda(), T.dev(c["codes"], torch.uint8), T.dev(c["scales"], torch.float32)
    y, cu, ln, tb, st = torch.zeros_like(q), T.dev(c["cu"]), T.dev(c["lens"]), T.dev(c["table"]), T.dev([0])
    assert f(ctypes.addressof(d), gc[0].data_ptr(), gc[1].data_ptr(), gs[0].data_ptr(), gs[1].data_ptr(), q.data_ptr(), row, y.data_ptr(), row, c["heads"],
             cu.data_ptr(), ln.data_ptr(), tb.data_ptr(), len(c["lens"]), c["width"], c["tokens"], c["max_new"], c["scale"], c["window"], work.data_ptr(),
             c["xdt"], st.data_ptr(), torch.cuda.current_stream().cuda_stream, 1, 30_000_000) == Q.QNT_OK
    torch.cuda.synchronize()
    assert int(st) in (Q.QNT_OK, Q.QNT_ERR_TIMEOUT)
    return int(st) == Q.QNT_ERR_TIMEOUT


@pytest.mark.parametrize("dim,heads,group,rows,new,wide", [
    (128, 1, 4, 2, 32, True), (64, 1, 8, 1, 13, True), (128, 1, 97, 2, 1, True), (256, 1, 4, 2, 32, True), (128, 8, 2, 1, 60, True),
    (128, 8, 8, 16, 1, False), (128, 8, 8, 4, 1, False), (64, 2, 4, 3, 4, False), (256, 1, 4, 24, 1, False), (128, 8, 8, 64, 5, True)])
def test_which_kernel(dim, heads, group, rows, new, wide):
    """A hundred query rows of a key/value head and more go to the tcgen05 kernel, 32 of many jobs too; those of single tokens do not."""
    assert goes_wide(T.make_attn(1, R.INT8, 0, 16, heads, group, dim, [max(40, new)] * rows, [new] * rows)) is wide


@pytest.mark.parametrize("fmt,xdt,dim,group,len_,new", [(R.E4M3, 0, 64, 8, 20011, 13), (R.INT8, 1, 64, 97, 9001, 1), (R.INT8, 0, 128, 97, 20011, 1),
                                                        (R.E4M3, 1, 128, 4, 20011, 70), (R.E4M3, 1, 256, 7, 20011, 18), (R.INT8, 0, 256, 130, 9001, 2)])
def test_split_in_many_parts(fmt, xdt, dim, group, len_, new):
    """More parts than the merge takes in one round; twice with one workspace, bit for bit alike."""
    Q = H.q()
    c = T.make_attn(len_ + dim, fmt, xdt, 64, 1, group, dim, [len_, 70], [new, 1])
    work = H.dev_bytes(Q.qnt_kv_attn_work_bytes(Q.kv_desc(fmt, 64, c["pages"], 1, dim), c["heads"], new))
    y = T.check_attn(c, work=work)
    for _ in range(3):
        assert torch.equal(y, T.call_attn(c, work=work))
    assert int(work[:16384].max()) == 0


@pytest.mark.parametrize("fmt,xdt,dim", [(R.INT8, 0, 128), (R.E4M3, 1, 64), (R.INT8, 1, 256), (R.E4M3, 0, 128)])
def test_mixed_batches(fmt, xdt, dim):
    """Requests on both sides of the border in one call, of few and of many jobs, full, partial and empty warps of rows."""
    T.check_attn(T.make_attn(dim, fmt, xdt, 16, 1, 1, dim, [400, 50, 300, 0, 97, 1, 260], [97, 1, 200, 0, 97, 1, 129]))
    c = T.make_attn(dim + 1, fmt, xdt, 32, 8, 1, dim, [40] * 13 + [130, 97, 33], [1] * 8 + [32, 33, 31, 34, 40, 97, 96, 33])
    T.check_attn(c)
    T.check_attn(c, max_new=1)


def test_max_new_selects_the_kernel():
    for hint in (1, 30, 1000):
        T.check_attn(T.make_attn(78, R.INT8, 0, 16, 1, 4, 128, [50, 190, 217], [1, 30, 40]), max_new=hint)


@pytest.mark.parametrize("fmt,xdt", [(R.INT8, 0), (R.E4M3, 1), (R.INT8, 1), (R.E4M3, 0)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_peaked_and_flat(fmt, xdt, dim):
    c = T.make_attn(80, fmt, xdt, 32, 1, 8, dim, [400, 400], [40, 40])
    c["q"][:40, ::2] *= 60
    c["q"][:40, 1] = 0
    c["q"][40:] *= 1e-3
    T.check_attn(c)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_bf16_queries_of_any_size(dim):
    c = T.make_attn(81, R.INT8, 1, 32, 1, 8, dim, [260], [50])
    for h, s in enumerate([1e-38, 1e-30, 1e-10, 1e-2, 10.0, 1e5, 0.0, 1.0]):
        c["q"][:, h] *= s
    c["scales"][0] *= np.float32(1e-4)
    T.check_attn(c)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_non_finite_queries_stay_in_their_row(dim):
    c = T.make_attn(82, R.INT8, 0, 16, 1, 8, dim, [270, 150], [40, 30])
    y0 = T.call_attn(c)
    c["q"][20, 2, 5], c["q"][60, 7, 0] = math.nan, math.inf
    y1 = T.call_attn(c)
    same = torch.ones(c["tokens"], 8, dtype=torch.bool)
    same[20, 2] = same[60, 7] = False
    assert torch.equal(y0[same], y1[same]) and y1[20, 2].isnan().all()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_see_nothing(dim):
    c = T.make_attn(83, R.E4M3, 0, 16, 1, 2, dim, [0, 150, 75], [90, 70, 64])
    c["lens"] = np.array([0, 150, 20])
    T.check_attn(c)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_bad_pages_and_lengths_are_reported(dim):
    Q = H.q()
    c = T.make_attn(84, R.INT8, 0, 16, 1, 4, dim, [140, 150], [40, 40], nan_behind=False)
    for bad in (-5, c["pages"], 2 ** 31 - 1):
        d = dict(c, table=c["table"].copy())
        d["table"][1, 1] = bad
        y = T.call_attn(d)
        assert d["status"] == Q.QNT_ERR_ARG
        d["table"][1, 1] = 0
        T.check_attn(d, y=y, status=Q.QNT_ERR_ARG)
    d = dict(c, table=np.where(c["table"] < 0, 0, c["table"]), lens=np.array([140, 10 ** 9]))
    y = T.call_attn(d)
    assert d["status"] == Q.QNT_ERR_ARG
    d["lens"] = np.array([140, c["width"] * 16])
    T.check_attn(d, y=y, status=Q.QNT_ERR_ARG)


@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
def test_cache_beyond_32_bit_offsets(fmt):
    """Codes of 5.2 GB, read by 120 query rows of a head."""
    Q = H.q()
    page, heads, dim, pages, new, L = 128, 8, 128, 40000, 60, 300
    d = Q.kv_desc(fmt, page, pages, heads, dim)
    assert Q.qnt_kv_codes_bytes(d) > 2 ** 32
    ids = [39998, 5, 39999]
    small = T.make_attn(3, fmt, 0, page, heads, 2, dim, [L], [new], pad=0, nan_behind=False)
    codes = [torch.empty(Q.qnt_kv_codes_bytes(d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = torch.zeros(2, pages, heads, device="cuda")
    for i in range(2):
        codes[i].view(pages, heads, page, dim)[ids] = T.dev(small["codes"][i][small["table"][0, :3]], torch.uint8)
        scales[i, ids] = T.dev(small["scales"][i][small["table"][0, :3]], torch.float32)
    y = torch.zeros(new, 2 * heads * dim, dtype=torch.float16, device="cuda")
    work, st = H.dev_bytes(Q.qnt_kv_attn_work_bytes(d, 2 * heads, new)), T.dev([0])
    Q.qnt_kv_attn(d, codes[0], codes[1], scales[0], scales[1], small["q"].reshape(new, -1).cuda(), 2 * heads * dim, y, 2 * heads * dim, 2 * heads, T.dev([0, new]),
                  T.dev([L]), T.dev([ids]), 1, 3, new, new, small["scale"], 0, work, 0, st)
    torch.cuda.synchronize()
    small["status"] = int(st)
    T.check_attn(small, y=y.view(new, 2 * heads, dim))


def test_calls_repeat_bit_for_bit():
    """Both kernels' results do not depend on timing: beside other work, on another stream, after other sizes with the same workspace."""
    Q = H.q()
    cases = [T.make_attn(90, R.INT8, 0, 64, 2, 4, 128, [9000, 50, 3000], [1, 1, 1]), T.make_attn(91, R.E4M3, 1, 16, 2, 4, 128, [5000, 300], [40, 70]),
             T.make_attn(92, R.E4M3, 0, 32, 1, 7, 64, [2500, 700], [20, 5])]
    work = [H.dev_bytes(max(Q.qnt_kv_attn_work_bytes(Q.kv_desc(c["fmt"], c["page"], c["pages"], c["kv_heads"], c["dim"]), c["heads"], c["max_new"]) for c in cases))
            for _ in range(2)]
    first = [T.call_attn(c, work=work[0]).clone() for c in cases]
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.float16)
    side = torch.cuda.Stream()
    for k in range(12):
        with torch.cuda.stream(side):
            for _ in range(k % 4):
                a @ a
        for i, c in enumerate(cases):
            assert torch.equal(T.call_attn(c, work=work[k % 2]), first[i])


@pytest.mark.parametrize("fmt,xdt,dim,page,kv_heads,group,new,lens,window", [
    (R.INT8, 1, 64, 32, 2, 64, 22, [169], 0), (R.E4M3, 1, 64, 64, 1, 64, 26, [276, 271], 129), (R.E4M3, 0, 128, 16, 1, 7, 44, [271, 273], 0),
    (R.INT8, 0, 128, 64, 1, 7, 42, [166, 177], 0), (R.INT8, 1, 64, 16, 1, 7, 40, [70, 157], 500), (R.INT8, 0, 64, 64, 1, 130, 10, [15, 744, 2102, 612], 500),
    (R.E4M3, 1, 128, 128, 1, 1, 300, [900, 1300], 0)])
def test_jobs_of_one_tile_of_rows_beside_jobs_of_two(fmt, xdt, dim, page, kv_heads, group, new, lens, window):
    """A CTA's next job has rows for both streams after one that had rows for the first only (up to 128 rows over a multiple of 256)."""
    assert 0 < new * group % 256 <= 128
    G.check(G.copies(T.make_attn(dim + group, fmt, xdt, page, kv_heads, group, dim, lens, [new] * len(lens), window=window), 150))
