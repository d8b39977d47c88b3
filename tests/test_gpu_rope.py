"""Appends with the position rotation: isoquant_decode_prep_rope (packed
cache) and isoquant_dense_prep (16-bit cache).

Packed codes and norms are those of the key rotated in exact arithmetic on
the fp32 table, bit for bit (compare_compressed of the other parity tests);
16-bit results within half a step plus the fp32 rotation's error."""
import numpy as np
import pytest
import torch

import oracle
from tests.dense_ref import U, check_rotated, rope64, rope_table
from tests.parity import compare_compressed

pytestmark = pytest.mark.gpu
D = 128


def draw(seed, n, heads, dtype, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, D), generator=g)
    if spread:
        x = x * torch.exp(torch.rand((heads, D), generator=g) * 4 - 2)
    return x.to(dtype)


def make_slots(seed, n, pages, ps, skip):
    g = torch.Generator().manual_seed(seed)
    slots = torch.randperm(pages * ps, generator=g)[:n]
    if skip:
        slots[torch.randperm(n, generator=g)[:skip]] = -1
    return slots


CASES = [  # bits, dtype, n_tok, H, G, page size, rot, interleaved, skipped
    (3, torch.bfloat16, 1, 1, 1, 32, 128, False, 0),
    (3, torch.bfloat16, 37, 4, 8, 256, 128, False, 5),
    (3, torch.float16, 301, 2, 3, 64, 96, True, 0),
    (3, torch.float32, 70, 8, 4, 128, 64, False, 9),
    (2, torch.bfloat16, 65, 3, 2, 32, 32, False, 1),
    (2, torch.float32, 19, 1, 6, 64, 128, True, 0),
    (4, torch.float16, 130, 2, 1, 128, 96, False, 30),
    (4, torch.bfloat16, 33, 5, 2, 256, 64, True, 33),
    (3, torch.bfloat16, 2000, 8, 4, 256, 128, True, 100),
]


@pytest.mark.parametrize("bits,dtype,n,H,G,ps,rot,inter,skip", CASES)
def test_packed_append_is_bit_exact(cuda_lib, bits, dtype, n, H, G, ps, rot, inter, skip):
    csd = cuda_lib
    signs, quats = csd.synthetic.rotation_params(n + bits, H)
    ctx = csd.isoquant_init(signs, quats, bits=bits)
    pages = (n + ps - 1) // ps + 1
    table = rope_table(5000, rot)
    k, v, q = draw(1, n, H, dtype), draw(2, n, H, dtype), draw(3, n, H * G, dtype)
    g = torch.Generator().manual_seed(n)
    kp, qp = (torch.randint(0, 5000, (n,), generator=g) for _ in range(2))
    slots = make_slots(n, n, pages, ps, skip)
    cache = csd.PagedCache.allocate(H, pages, ps, bits=bits)
    cache.codes.fill_(0x12345678)
    cache.norms.fill_(3.0)
    q_rot = torch.full((n, H * G, D), float("nan"), device="cuda")
    rope = csd.Rope(table.cuda(), rot, inter)
    csd.isoquant_decode_prep_rope(ctx, cache, k.cuda(), v.cuda(), slots.cuda(), kp.cuda(), q.cuda(), qp.cuda(), rope,
                                  q_rot)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0
    assert csd.isoquant_last_launch_count(ctx) == 1
    codes, norms = cache.codes.cpu(), cache.norms.cpu()
    live = slots >= 0
    page, off = slots[live] // ps, slots[live] % ps
    k64 = rope64(k, kp, table, rot, inter)[0]
    for side, x in ((0, k64), (1, v.double())):
        for h in range(H):
            got = codes[page, side, h][torch.arange(len(page)), :, off].to(torch.int64) & 0xFFFFFFFF
            nb = norms[page, side, h, off].view(torch.int16).to(torch.int64) & 0xFFFF
            if len(page):
                stats, _, _ = compare_compressed(x[live][:, h].numpy(), signs[h].numpy(), quats[h].numpy(),
                                                 got.numpy(), nb.numpy(), bits=bits)
                assert stats["code_mismatch"] == 0 and stats["norm_mismatch"] == 0
    # slots that no token took are as they were
    rest = torch.ones(pages * ps, dtype=torch.bool)
    rest[slots[live]] = False
    r = rest.nonzero()[:, 0]
    assert (codes[r // ps, :, :, :, r % ps] == 0x12345678).all() and (norms[r // ps, :, :, r % ps] == 3.0).all()
    # queries: 7 butterfly levels, a 4-term product and the rotation by
    # position, each within u of the vector's length per stage
    q64, _ = rope64(q, qp, table, rot, inter)
    for hq in range(0, H * G, max(1, H * G // 4)):
        want = oracle.rotate(signs[hq // G].numpy(), quats[hq // G].numpy(), q64[:, hq].numpy())
        err = np.abs(q_rot[:, hq].double().cpu().numpy() - want).max(1)
        assert (err <= 32 * U * np.linalg.norm(want, axis=1) + 1e-30).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,H,G,ps,rot,inter,skip,k_out", [
    (1, 1, 1, 32, 128, False, 0, False),
    (16, 4, 8, 256, 128, False, 0, True),
    (333, 3, 5, 64, 96, False, 40, True),
    (129, 2, 1, 128, 64, True, 0, False),
    (77, 7, 3, 32, 32, True, 76, True),
    (50, 5, 2, 64, 32, False, 50, False),
    (4100, 6, 5, 256, 128, False, 100, True),   # large enough for four heads per item, and odd head counts
    (4099, 9, 3, 64, 96, True, 0, False),
])
def test_dense_append(cuda_lib, dtype, n, H, G, ps, rot, inter, skip, k_out):
    csd = cuda_lib
    signs, quats = csd.synthetic.rotation_params(1, H)
    ctx = csd.isoquant_init(signs, quats)
    pages = (n + ps - 1) // ps + 1
    table = rope_table(5000, rot)
    k, v, q = draw(1, n, H, dtype), draw(2, n, H, dtype), draw(3, n, H * G, dtype)
    v[0, 0, :3] = torch.tensor([float("inf"), float("nan"), -0.0])
    g = torch.Generator().manual_seed(n)
    kp, qp = (torch.randint(0, 5000, (n,), generator=g) for _ in range(2))
    slots = make_slots(n, n, pages, ps, skip)
    cache = csd.DenseCache.allocate(H, pages, ps, dtype)
    cache.data.fill_(7.0)
    q_out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    ko = torch.full(k.shape, float("nan"), dtype=dtype, device="cuda") if k_out else None
    rope = csd.Rope(table.cuda(), rot, inter)
    csd.isoquant_dense_prep(ctx, cache, k.cuda(), v.cuda(), slots.cuda(), kp.cuda(), q.cuda(), qp.cuda(), rope,
                            q_out, k_out=ko)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0
    k64, kr = rope64(k, kp, table, rot, inter)
    q64, qr = rope64(q, qp, table, rot, inter)
    check_rotated(q_out.cpu(), q64, qr)
    data = cache.data.cpu()
    live = slots >= 0
    page, off = slots[live] // ps, slots[live] % ps
    got_k = data[page, 0, :, off]
    check_rotated(got_k, k64[live], kr[live])
    assert torch.equal(data[page, 1, :, off].view(torch.int16), v[live].view(torch.int16))
    if k_out:
        check_rotated(ko.cpu(), k64, kr)
        assert torch.equal(ko.cpu()[live], got_k)
    rest = torch.ones(pages * ps, dtype=torch.bool)
    rest[slots[live]] = False
    r = rest.nonzero()[:, 0]
    assert (data[r // ps, :, :, r % ps] == 7.0).all()


def test_dense_prep_in_place_without_cache_and_without_rotation(cuda_lib):
    csd = cuda_lib
    H, G, n, dtype = 2, 3, 41, torch.bfloat16
    signs, quats = csd.synthetic.rotation_params(1, H)
    ctx = csd.isoquant_init(signs, quats)
    table = rope_table(100, 128)
    rope = csd.Rope(table.cuda())
    assert torch.equal(csd.Rope.table(100).cpu(), table) or (csd.Rope.table(100).cpu() - table).abs().max() <= 2 * U
    k, v, q = (draw(i, n, h, dtype).cuda() for i, h in ((1, H), (2, H), (3, H * G)))
    pos = torch.arange(n, device="cuda") + 50
    ko, qo = torch.empty_like(k), torch.empty_like(q)
    csd.isoquant_dense_prep(ctx, None, k, None, None, pos, q, pos, rope, qo, k_out=ko)
    k2, q2 = k.clone(), q.clone()
    csd.isoquant_dense_prep(ctx, None, k2, None, None, pos, q2, pos, rope, q2, k_out=k2)
    assert torch.equal(k2, ko) and torch.equal(q2, qo)
    check_rotated(ko.cpu(), *rope64(k.cpu(), pos.cpu(), table, 128, False))
    # rope None: a plain append and copy
    cache = csd.DenseCache.allocate(H, 2, 32, dtype)
    slots = torch.arange(n, device="cuda")
    csd.isoquant_dense_prep(ctx, cache, k, v, slots, None, q, None, None, qo, k_out=ko)
    assert torch.equal(ko, k) and torch.equal(qo, q)
    assert torch.equal(cache.data[:, 0].transpose(1, 2).reshape(-1, H, D)[:n], k)
    assert torch.equal(cache.data[:, 1].transpose(1, 2).reshape(-1, H, D)[:n], v)
    # either half empty
    none_k, none_q = k[:0], q[:0]
    qo.zero_()
    csd.isoquant_dense_prep(ctx, cache, none_k, none_k, slots[:0], pos[:0], q, pos, rope, qo)
    check_rotated(qo.cpu(), *rope64(q.cpu(), pos.cpu(), table, 128, False))
    csd.isoquant_dense_prep(ctx, cache, k, v, slots, pos, none_q, pos[:0], rope, qo[:0], k_out=ko)
    check_rotated(ko.cpu(), *rope64(k.cpu(), pos.cpu(), table, 128, False))
    csd.isoquant_dense_prep(ctx, cache, none_k, none_k, slots[:0], pos[:0], none_q, pos[:0], rope, qo[:0])
    assert csd.isoquant_last_launch_count(ctx) == 0
    assert csd.isoquant_get_status(ctx) == 0


def test_bad_positions_and_slots_are_flagged(cuda_lib):
    """A position outside the table or a slot outside the cache skips its
    token, zeroes its rows and sets its status bit; the others are as if it
    were not there.  Positions of padding tokens are not looked at."""
    csd = cuda_lib
    H, G, n, ps = 2, 2, 9, 32
    signs, quats = csd.synthetic.rotation_params(4, H)
    ctx = csd.isoquant_init(signs, quats)
    table = rope_table(64, 128).cuda()
    rope = csd.Rope(table)
    dtype = torch.bfloat16
    k, v, q = (draw(i, n, h, dtype).cuda() for i, h in ((1, H), (2, H), (3, H * G)))
    slots = torch.arange(n, device="cuda") * 3
    good = torch.arange(n, device="cuda")

    def packed(sl, kp, qp):
        cache = csd.PagedCache.allocate(H, 1, ps)
        q_rot = torch.full(q.shape, float("nan"), device="cuda")
        csd.isoquant_decode_prep_rope(ctx, cache, k, v, sl, kp, q, qp, rope, q_rot)
        return cache.codes, cache.norms, q_rot, csd.isoquant_get_status(ctx)

    def dense(sl, kp, qp):
        cache = csd.DenseCache.allocate(H, 1, ps, dtype)
        qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
        csd.isoquant_dense_prep(ctx, cache, k, v, sl, kp, q, qp, rope, qo, k_out=ko)
        return cache.data, ko, qo, csd.isoquant_get_status(ctx)

    bad_k, bad_q, bad_s, pad = good.clone(), good.clone(), slots.clone(), slots.clone()
    bad_k[2], bad_k[7], bad_q[4], bad_q[0] = -1, 64, 2 ** 40, -5
    bad_s[5] = ps
    pad[2] = pad[7] = -1
    codes, norms, q_rot, status = packed(slots, good, good)
    assert status == 0
    c, m, r, status = packed(slots, bad_k, bad_q)
    assert status == csd.DEVERR_POS_RANGE
    keep = torch.tensor([i for i in range(n) if i not in (2, 7)], device="cuda") * 3
    assert torch.equal(c[..., keep], codes[..., keep]) and torch.equal(m[..., keep], norms[..., keep])
    assert (c[..., [6, 21]] == 0).all()
    assert (r[[0, 4]] == 0).all() and torch.equal(r[[1, 2, 3, 5, 6, 7, 8]], q_rot[[1, 2, 3, 5, 6, 7, 8]])
    c, m, r, status = packed(pad, bad_k, good)
    assert status == 0 and torch.equal(c[..., keep], codes[..., keep])
    c, m, r, status = packed(bad_s, good, good)
    assert status == csd.DEVERR_SLOT_RANGE and (c[..., 15] == 0).all() and torch.equal(c[..., 18], codes[..., 18])

    data, ko, qo, status = dense(slots, good, good)
    assert status == 0
    x, y, z, status = dense(slots, bad_k, bad_q)
    assert status == csd.DEVERR_POS_RANGE
    assert torch.equal(x[..., keep, :], data[..., keep, :]) and (x[..., [6, 21], :] == 0).all()
    assert (y[[2, 7]] == 0).all() and torch.equal(y[[0, 1, 3, 4, 5, 6, 8]], ko[[0, 1, 3, 4, 5, 6, 8]])
    assert (z[[0, 4]] == 0).all() and torch.equal(z[[1, 2, 3, 5, 6, 7, 8]], qo[[1, 2, 3, 5, 6, 7, 8]])
    x, y, z, status = dense(bad_s, good, good)
    assert status == csd.DEVERR_SLOT_RANGE and (x[..., 15, :] == 0).all() and torch.equal(y, ko)


def test_rope_argument_errors(cuda_lib):
    import ctypes
    csd = cuda_lib
    L, p = csd.lib(), csd._ptr
    signs, quats = csd.synthetic.rotation_params(4, 2)
    ctx = csd.isoquant_init(signs, quats)
    n, dtype = 4, torch.bfloat16
    k, v, q = (draw(i, n, h, dtype).cuda() for i, h in ((1, 2), (2, 2), (3, 4)))
    table = rope_table(64, 128).cuda()
    pos = torch.arange(n, device="cuda")
    q_rot = torch.empty(q.shape, device="cuda")
    packed, dense = csd.PagedCache.allocate(2, 1, 32), csd.DenseCache.allocate(2, 1, 32, dtype)
    s0 = csd._stream(None)
    null = ctypes.c_void_p(0)

    def off(t, by=4):
        return ctypes.c_void_p(t.data_ptr() + by)

    def rope(table_ptr=None, n_pos=64, rot=128):
        return csd._Rope(table.data_ptr() if table_ptr is None else table_ptr, n_pos, rot, 0)

    def prep(r=None, kp=None, qp=None, dt=1, heads=4, rows=n, out=None):
        return L.isoquant_decode_prep_rope(ctx.handle, packed.c_struct(), p(k), p(v), n, p(pos), kp or p(pos), p(q),
                                           dt, rows, heads, qp or p(pos), r, out or p(q_rot), s0)

    def dprep(r=None, cache=dense._c, dt=1, heads=4, kk=None, ko=None, qo=None, kp=None):
        return L.isoquant_dense_prep(ctx.handle, cache, kk or p(k), p(v), n, p(pos), kp or p(pos), p(q), dt, n,
                                     heads, p(pos), r, ko, qo or p(q_rot), s0)

    for call in (prep, dprep):
        assert call(rope(table_ptr=0)) == -1
        assert call(rope(n_pos=0)) == -1
        assert call(rope(rot=0)) == -2 and call(rope(rot=48)) == -2 and call(rope(rot=160)) == -2
        assert call(rope(table_ptr=table.data_ptr() + 4)) == -6
        assert call(rope(), heads=3) == -1
        assert call(rope(), dt=7) == -2
        assert call(rope(), kp=off(pos)) == -6
    assert prep(None) == -1
    assert prep(rope(), rows=-1) == -1
    assert prep(rope(), out=off(q_rot)) == -6
    assert dprep(rope(), dt=0) == -2                                   # fp32 has no 16-bit cache
    assert dprep(rope(), dt=2) == -2                                   # the cache is bf16
    assert dprep(rope(), cache=csd._DenseCache(dense.data.data_ptr(), 1, 1, 48)) == -2
    assert dprep(rope(), cache=csd._DenseCache(dense.data.data_ptr(), 0, 1, 32)) == -2
    assert dprep(rope(), cache=csd._DenseCache(0, 1, 1, 32)) == -1
    assert dprep(rope(), cache=csd._DenseCache(dense.data.data_ptr() + 8, 1, 1, 32)) == -6
    assert dprep(rope(), cache=None) == -1                             # nothing to write keys to
    assert dprep(rope(), ko=off(k, 8)) == -6
    assert dprep(rope(), kk=off(k, 8)) == -6
    assert L.isoquant_last_launch_count(ctx.handle) == 0
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0
    assert prep(rope()) == 0 and dprep(rope(), cache=None, ko=p(k)) == 0
    assert null is not None
