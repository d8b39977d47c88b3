"""Refusals of the rotated appends and the 16-bit attention, on the host: every
argument error is found before any CUDA call, so a context's memory with
made-up contents stands in for one (nothing on a device is reached: a call
whose arguments are all good ends with the CUDA error of a machine without
one)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA, ALIGNMENT = 0, -1, -2, -4, -5, -6


@pytest.fixture(scope="module")
def native():
    import compressed_space_decode_b200 as csd
    from compressed_space_decode_b200 import build
    build.build()
    return csd


@pytest.fixture(scope="module")
def ctx():
    """The memory of a context of 2 KV heads: {device, num_kv_heads, num_sms, ..}."""
    if torch.cuda.is_available():
        pytest.skip("a call with good arguments would launch on this machine's device")
    buf = (ctypes.c_int32 * 4096)()
    buf[0], buf[1], buf[2] = 0, 2, 148
    return buf


P = 1 << 20  # any aligned address: it is never followed


def test_structures_match_the_header(native):
    text = open(os.path.join(ROOT, "include", "isoquant.h")).read()
    for name, struct in (("isoquant_rope", native._Rope), ("isoquant_dense_cache", native._DenseCache)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
        fields = re.findall(r"(\w+);", body)
        assert fields == [f for f, _ in struct._fields_]
    assert ctypes.sizeof(native._Rope) == 24 and ctypes.sizeof(native._DenseCache) == 24
    for name, value in (("POS_RANGE", native.DEVERR_POS_RANGE), ("SEQ_RANGE", native.DEVERR_SEQ_RANGE)):
        assert int(re.search(r"ISOQUANT_DEVERR_" + name + r" (\d+)u", text).group(1)) == value


def test_null_contexts(native):
    L, sz = native.lib(), ctypes.c_size_t()
    assert L.isoquant_decode_prep_rope(None, None, P, P, 1, P, P, P, 1, 1, 8, P, None, P, None) == INVALID
    assert L.isoquant_dense_prep(None, None, P, P, 1, P, P, P, 1, 1, 8, P, None, P, P, None) == INVALID
    assert L.isoquant_dense_workspace_size(None, 1, 1, 8, ctypes.byref(sz)) == INVALID
    assert L.isoquant_dense_attend(None, None, P, 1, 1, 8, P, 1, P, 0, 0.0, P, 1 << 30, P, None) == INVALID
    assert L.isoquant_prompt_attend(None, P, P, P, 1, 1, 8, 1024, 256, 256, P, 1, 1, 0.0, P, None) == INVALID


def test_append_refusals(native, ctx):
    L = native.lib()
    packed, dense = native._Cache(P, P, 4, 64), native._DenseCache(P, 1, 4, 64)

    def rope(table=P, n=10, rot=128):
        return native._Rope(table, n, rot, 0)

    def prep(cache=packed, k=P, v=P, n=3, sl=P, kp=P, q=P, dt=1, rows=3, heads=8, qp=P, r=rope(), out=P):
        return L.isoquant_decode_prep_rope(ctx, cache, k, v, n, sl, kp, q, dt, rows, heads, qp, r, out, None)

    def dprep(cache=dense, k=P, v=P, n=3, sl=P, kp=P, q=P, dt=1, rows=3, heads=8, qp=P, r=rope(), out=P, ko=None):
        return L.isoquant_dense_prep(ctx, cache, k, v, n, sl, kp, q, dt, rows, heads, qp, r, ko, out, None)

    for call in (prep, dprep):
        assert call() == CUDA
        assert call(n=0, rows=0) == OK
        for bad in (dict(n=-1), dict(rows=-1), dict(heads=0), dict(heads=7), dict(k=None), dict(v=None), dict(sl=None),
                    dict(kp=None), dict(q=None), dict(qp=None), dict(out=None), dict(r=rope(table=None)),
                    dict(r=rope(n=0)), dict(rows=1 << 30)):
            assert call(**bad) == INVALID, bad
        for bad in (dict(dt=9), dict(r=rope(rot=0)), dict(r=rope(rot=40)), dict(r=rope(rot=160))):
            assert call(**bad) == UNSUPPORTED, bad
        for bad in (dict(sl=P + 4), dict(kp=P + 4), dict(qp=P + 4), dict(out=P + 8), dict(r=rope(table=P + 8)),
                    dict(k=P + 2), dict(v=P + 2), dict(q=P + 2)):
            assert call(**bad) == ALIGNMENT, bad
    assert prep(r=None) == INVALID and dprep(r=None) == CUDA
    assert prep(cache=None) == INVALID
    assert dprep(cache=None) == INVALID and dprep(cache=None, ko=P) == CUDA
    assert dprep(cache=None, ko=P, v=None, sl=None) == CUDA
    assert dprep(dt=0) == UNSUPPORTED and dprep(dt=2) == UNSUPPORTED
    assert dprep(n=1 << 30, rows=0) == INVALID
    assert dprep(ko=P + 8) == ALIGNMENT
    for bad, status in ((native._DenseCache(None, 1, 4, 64), INVALID), (native._DenseCache(P, 1, 0, 64), INVALID),
                        (native._DenseCache(P, 0, 4, 64), UNSUPPORTED), (native._DenseCache(P, 1, 4, 48), UNSUPPORTED),
                        (native._DenseCache(P + 8, 1, 4, 64), ALIGNMENT)):
        assert dprep(cache=bad) == status


def test_cache_attention_refusals(native, ctx):
    L, sz = native.lib(), ctypes.c_size_t()
    dense = native._DenseCache(P, 1, 4, 64)
    assert L.isoquant_dense_workspace_size(ctx, 3, 2, 8, ctypes.byref(sz)) == OK
    need = sz.value
    assert need >= 256 and need % 16 == 0

    def call(cache=dense, q=P, B=3, nq=2, heads=8, pt=P, mp=2, sl=P, scale=0.0, ws=P, wb=need, o=P):
        return L.isoquant_dense_attend(ctx, cache, q, B, nq, heads, pt, mp, sl, 0, scale, ws, wb, o, None)

    assert call() == CUDA and call(B=0) == OK
    for bad in (dict(q=None), dict(pt=None), dict(sl=None), dict(ws=None), dict(o=None), dict(B=-1), dict(nq=0),
                dict(heads=5), dict(mp=0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(nq=1 << 30), dict(cache=None), dict(cache=native._DenseCache(P, 1, 1 << 24, 64))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(q=P + 8), dict(o=P + 2), dict(ws=P + 8), dict(pt=P + 2), dict(sl=P + 2)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(wb=need - 1) == WORKSPACE
    # a workspace grows with the rows of a row tile, not with the batch
    sizes = []
    for B, nq, heads in ((1, 1, 2), (700, 1, 2), (1, 1, 16), (1, 16, 16), (1, 8192, 16)):
        assert L.isoquant_dense_workspace_size(ctx, B, nq, heads, ctypes.byref(sz)) == OK
        sizes.append(sz.value)
    assert sizes[0] == sizes[1] < sizes[2] < sizes[3] == sizes[4] < 1 << 26


def test_prompt_refusals(native, ctx):
    L = native.lib()

    def call(q=P, k=P, v=P, dt=1, T=50, heads=8, qs=1024, ks=256, vs=256, cu=P, B=2, scale=0.0, o=P):
        return L.isoquant_prompt_attend(ctx, q, k, v, dt, T, heads, qs, ks, vs, cu, B, 1, scale, o, None)

    assert call() == CUDA and call(T=0) == OK and call(B=0) == OK
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(o=None), dict(T=-1), dict(B=-1),
                dict(heads=0), dict(heads=9), dict(qs=1016), dict(ks=248), dict(vs=-256), dict(ks=1 << 40),
                dict(scale=-1.0), dict(scale=float("nan")), dict(T=1 << 30), dict(B=1 << 29)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=0), dict(dt=5), dict(heads=258, qs=258 * 128)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=P + 8), dict(k=P + 8), dict(v=P + 2), dict(o=P + 8), dict(cu=P + 2), dict(qs=1028),
                dict(ks=260), dict(vs=257)):
        assert call(**bad) == ALIGNMENT, bad


def test_python_calls_check_shapes_and_types(native):
    class Ctx:
        handle, num_kv_heads, device = None, 2, 0

    ctx = Ctx()
    bf = torch.bfloat16
    k, q = torch.zeros(5, 2, 128, dtype=bf), torch.zeros(5, 8, 128, dtype=bf)
    pos, table = torch.zeros(5, dtype=torch.int64), torch.zeros(9, 128)
    rope = native.Rope(table)
    packed = native.PagedCache(torch.zeros((2, 2, 2, 13, 64), dtype=torch.int32),
                               torch.zeros((2, 2, 2, 64), dtype=torch.float16), 64)
    dense = native.DenseCache(torch.zeros((2, 2, 2, 64, 128), dtype=bf), 64)
    q_rot = torch.zeros(5, 8, 128)

    def refused(fn, *a, **kw):
        with pytest.raises(AssertionError):
            fn(*a, **kw)

    good = [ctx, packed, k, k, pos, pos, q, pos, rope, q_rot]
    for i, bad in ((2, k[:4]), (2, k.float()), (3, k.transpose(0, 1)), (4, pos[:4]), (4, pos.int()), (5, pos[:0]),
                   (6, q.half()), (7, pos[:2]), (9, q_rot.to(bf)), (9, q_rot[:4]), (2, torch.zeros(5, 3, 128, dtype=bf))):
        args = list(good)
        args[i] = bad
        refused(native.isoquant_decode_prep_rope, *args)
    good = [ctx, dense, k, k, pos, pos, q, pos, rope, q]
    for i, bad in ((2, k[:4]), (3, k[:3]), (4, pos[::2]), (5, None), (6, q.half()), (9, q[:4]), (9, q.float())):
        args = list(good)
        args[i] = bad
        refused(lambda *a: native.isoquant_dense_prep(*a), *args) if bad is not None else None
    refused(native.isoquant_dense_prep, *good, k_out=k[:2])
    q4, pt, sl = q.view(5, 1, 8, 128), torch.zeros(5, 3, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.int32)
    good = [ctx, dense, q4, pt, sl, ws, q4]
    for i, bad in ((2, q4.half()), (3, pt[:4]), (3, pt.long()), (4, sl[:2]), (4, sl.long()), (6, q4[:3]),
                   (6, q4.float())):
        args = list(good)
        args[i] = bad
        refused(native.isoquant_dense_attend, *args)
    cu = torch.zeros(3, dtype=torch.int32)
    good = [ctx, q, k, k, cu, q]
    for i, bad in ((1, q.half()), (2, k[:4]), (3, k.transpose(1, 2)), (4, cu.long()), (4, cu[::2]), (5, q[:, :4]),
                   (5, q.transpose(0, 1)), (2, torch.zeros(5, 3, 128, dtype=bf))):
        args = list(good)
        args[i] = bad
        refused(native.isoquant_prompt_attend, *args)
    refused(native.Rope, table.double())
    refused(native.Rope, table, 64)
    refused(native.DenseCache, torch.zeros((2, 2, 2, 64, 128)), 64)
    refused(native.DenseCache, torch.zeros((2, 2, 2, 64, 128), dtype=bf), 32)


@pytest.mark.parametrize("rot", [32, 64, 96, 128])
def test_rope_tables(native, rot):
    """Angles in 64 bits before one rounding: half a step of fp32 at far positions."""
    import math
    t = native.Rope.table(70000, rot, base=500000.0, device="cpu")
    assert t.shape == (70000, rot) and t.dtype == torch.float32
    for p in (0, 1, 12345, 69999):
        for i in (0, 1, rot // 2 - 1):
            a = p * 500000.0 ** (-2 * i / rot)
            assert abs(float(t[p, i]) - math.cos(a)) <= 2.0 ** -24
            assert abs(float(t[p, rot // 2 + i]) - math.sin(a)) <= 2.0 ** -24
