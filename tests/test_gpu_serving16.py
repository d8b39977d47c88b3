"""The 16-bit operators and the rotated appends together, as a serving step
uses them, and the places where they can go wrong apart from plain values:
non-finite values that only later tokens see, caches beyond 32-bit offsets,
many sequences, long chunks."""
import numpy as np
import pytest
import torch

import oracle
from tests.dense_ref import attend64, check_attention, half_step, rope64, rope_table
from tests.parity import ATTN_TOL, rowwise_rel_err
from tests.test_gpu_dense_attend import WEIGHT_BITS, Case
from tests.test_gpu_prompt import check as check_prompts
from tests.test_gpu_prompt import context, draw

pytestmark = pytest.mark.gpu
D = 128


def test_prompts_then_decode_steps(cuda_lib):
    """Prompts enter a 16-bit cache rotated, attend to themselves, and three
    decode steps follow: every output is that of attention over the cache's
    own keys and values, and those are the rotated inputs."""
    csd = cuda_lib
    H, G, ps, dtype = 2, 4, 32, torch.bfloat16
    lens, steps = [45, 130, 7], 3
    ctx = context(csd, H)
    table = rope_table(400, 96)
    rope = csd.Rope(table.cuda(), 96)
    T, B = sum(lens), len(lens)
    per = [-(-(L + steps) // ps) for L in lens]
    pages = torch.randperm(sum(per), generator=torch.Generator().manual_seed(3))
    pt = torch.zeros((B, max(per)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        pt[b, :n] = pages[at:at + n]
        at += n
    cache = csd.DenseCache.allocate(H, sum(per), ps, dtype)
    cache.data.fill_(float("nan"))

    def slots(b, t):
        return pt[b, t // ps].long() * ps + t % ps

    q, k, v, cu = draw(31, lens, H, G, dtype)
    pos = torch.cat([torch.arange(L) for L in lens])
    sl = torch.cat([slots(b, torch.arange(L)) for b, L in enumerate(lens)])
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    csd.isoquant_dense_prep(ctx, cache, k, v, sl.cuda(), pos.cuda(), q, pos.cuda(), rope, qr, k_out=kr)
    out = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, qr, kr, v, cu, out)
    torch.cuda.synchronize()
    check_prompts(out, qr, kr, v, lens, H, G, True)
    want, r = rope64(k.cpu(), pos, table, 96, False)
    assert ((kr.cpu().double() - want).abs() <= half_step(dtype) * want.abs() * 1.001 + 1e-6 * r).all()
    # decode: one token per sequence a step
    ws = csd.alloc_dense_workspace(ctx, B, 1, H * G)
    held_k, held_v = list(kr.split(lens)), list(v.split(lens))
    for s in range(steps):
        qn, kn, vn, _ = draw(40 + s, [1] * B, H, G, dtype)
        p = torch.tensor([L + s for L in lens])
        sn = torch.stack([slots(b, p[b]) for b in range(B)])
        qo, ko = torch.empty_like(qn), torch.empty_like(kn)
        csd.isoquant_dense_prep(ctx, cache, kn, vn, sn.cuda(), p.cuda(), qn, p.cuda(), rope, qo, k_out=ko)
        o = torch.empty((B, 1, H * G, D), dtype=dtype, device="cuda")
        sq = (p + 1).to(torch.int32).cuda()
        csd.isoquant_dense_attend(ctx, cache, qo.view(B, 1, H * G, D), pt.cuda(), sq, ws, o)
        torch.cuda.synchronize()
        for b in range(B):
            held_k[b], held_v[b] = torch.cat([held_k[b], ko[b:b + 1]]), torch.cat([held_v[b], vn[b:b + 1]])
            kk = held_k[b].transpose(0, 1).repeat_interleave(G, 0)
            vv = held_v[b].transpose(0, 1).repeat_interleave(G, 0)
            n = kk.shape[1]
            ref = attend64(qo[b].unsqueeze(1), kk, vv, torch.full((1,), n))
            check_attention(o[b, 0].unsqueeze(1), *ref, WEIGHT_BITS[dtype])
    assert csd.isoquant_get_status(ctx) == 0


def test_rotated_packed_step(cuda_lib):
    """decode_prep_rope and attend_decode: attention of rotated queries over a
    packed cache of rotated keys, against the oracle on its codes."""
    csd = cuda_lib
    H, G, ps, L = 2, 4, 64, 150
    signs, quats = csd.synthetic.rotation_params(8, H)
    ctx = csd.isoquant_init(signs, quats)
    table = rope_table(300, 128)
    rope = csd.Rope(table.cuda())
    q, k, v, _ = draw(50, [L], H, G, torch.bfloat16)
    cache = csd.PagedCache.allocate(H, 3, ps)
    pos = torch.arange(L) + 100
    q_rot = torch.empty(q.shape, device="cuda")
    csd.isoquant_decode_prep_rope(ctx, cache, k, v, torch.arange(L).cuda(), pos.cuda(), q, pos.cuda(), rope, q_rot)
    rows = q_rot[-1:].view(1, 1, H * G, D).contiguous()
    out = torch.empty_like(rows)
    ws = csd.alloc_workspace(ctx, 1, 1, H * G)
    csd.isoquant_attend_decode(ctx, cache, rows, torch.arange(3, dtype=torch.int32).cuda().view(1, 3),
                               torch.tensor([L], dtype=torch.int32).cuda(), ws, out)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0
    q64 = rope64(q.cpu(), pos, table, 128, False)[0]
    t = torch.arange(L)
    for h in range(H):
        part = []
        for side in range(2):
            codes = cache.codes.cpu()[t // ps, side, h][torch.arange(L), :, t % ps].to(torch.int64) & 0xFFFFFFFF
            norms = cache.norms.cpu()[t // ps, side, h, t % ps].view(torch.int16).to(torch.int64) & 0xFFFF
            part += [codes.numpy().astype(np.uint32), norms.numpy().astype(np.uint16)]
        rows64 = q64[-1, h * G:(h + 1) * G].numpy()
        ref = oracle.attend(signs[h].numpy(), quats[h].numpy(), rows64, part[0], part[1], part[2], part[3], [L] * G)
        got = out[0, 0, h * G:(h + 1) * G].double().cpu().numpy()
        assert rowwise_rel_err(got, ref).max() <= ATTN_TOL


def test_rotated_queries_into_a_16_byte_aligned_buffer(cuda_lib):
    """32-byte stores are taken only where the output allows them."""
    csd = cuda_lib
    H, G, n = 2, 3, 37
    signs, quats = csd.synthetic.rotation_params(9, H)
    ctx = csd.isoquant_init(signs, quats)
    rope = csd.Rope(rope_table(100, 64).cuda(), 64, True)
    q, k, v, _ = draw(51, [n], H, G, torch.float16)
    pos = torch.arange(n).cuda()
    cache = csd.PagedCache.allocate(H, 2, 32)
    buf = torch.full((n * H * G * D + 8,), 3.0, device="cuda")
    outs = []
    for off in (0, 4):
        o = buf[off:off + n * H * G * D].view(n, H * G, D)
        csd.isoquant_decode_prep_rope(ctx, cache, k[:0], v[:0], pos[:0], pos[:0], q, pos, rope, o)
        outs.append(o.clone())
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and (buf[-4:] == 3.0).all()


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_values_that_only_later_tokens_see(cuda_lib, dtype, G):
    """Infinite and NaN values reach exactly the rows that see them, in the
    dimension that holds them; every other output keeps its bits."""
    csd = cuda_lib
    ctx = context(csd, 1)
    lens = [50, 400, 30]
    q, k, v, cu = draw(60, lens, 1, G, dtype)
    clean = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, clean)
    bad = {50 + 3: (5, float("inf")), 50 + 130: (70, float("-inf")), 50 + 255: (127, float("nan")),
           50 + 399: (0, float("inf"))}
    for t, (d, x) in bad.items():
        v[t, 0, d] = x
    out = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out)
    torch.cuda.synchronize()
    want = clean.clone().float()
    for t, (d, x) in bad.items():
        want[t:450, :, d] = x
    same = torch.isfinite(want)
    assert torch.equal(out[same], clean[same])
    assert torch.equal(torch.nan_to_num(out.float()[~same], nan=7.0, posinf=8.0, neginf=9.0),
                       torch.nan_to_num(want[~same], nan=7.0, posinf=8.0, neginf=9.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,G,nq", [(2, 1, 5), (2, 4, 4), (1, 4, 16), (1, 8, 16)])
def test_chunk_values_that_only_later_tokens_see(cuda_lib, H, G, nq, dtype):
    """The same for chunks over the cache, in every kernel form and with
    several sequences (clean ones behind) in one block of work."""
    csd = cuda_lib
    lens = [140, 300, 129, 200, 64, 500, 33, 260] * 3
    c = Case(csd, lens, H, G, nq, 64, dtype, seed=70)
    clean = c.run(causal=True)
    bad = {}
    for b in (0, 3, 4, 10, 21):
        t = lens[b] - 2  # seen by the last two tokens
        page = int(c.table_cpu[b, t // 64])
        d = 11 * b % D
        x = float("inf") if b % 2 else float("nan")
        c.cache.data[page, 1, 0, t % 64, d] = x
        bad[b] = (d, x)
    out = c.run(causal=True)
    want = clean.clone().float()
    for b, (d, x) in bad.items():
        want[b, max(0, nq - 2):, :G, d] = x
    same = torch.isfinite(want)
    assert torch.equal(out[same], clean[same])
    assert torch.equal(torch.nan_to_num(out.float()[~same], nan=7.0, posinf=8.0),
                       torch.nan_to_num(want[~same], nan=7.0, posinf=8.0))


@pytest.mark.parametrize("lens,H,G,nq,ps", [([900, 750], 1, 4, 700, 128), ([400], 2, 1, 400, 32), ([130, 600], 1, 160, 3, 64)])
def test_long_chunks_and_large_groups(cuda_lib, lens, H, G, nq, ps):
    """A cache read by whole prompts, and groups of more than 128 heads."""
    c = Case(cuda_lib, lens, H, G, nq, ps, torch.bfloat16, seed=80)
    c.check(c.run(causal=True), causal=True)


def test_pages_beyond_32_bit_offsets(cuda_lib):
    """A cache of 5 GB: the sequence's pages lie behind 2^31 elements."""
    csd = cuda_lib
    H, ps = 2, 256
    pages = 20000  # 131072 elements each
    data = torch.zeros((pages, 2, H, ps, D), dtype=torch.bfloat16, device="cuda")
    cache = csd.DenseCache(data, ps)
    ctx = context(csd, H)
    order = torch.tensor([pages - 1, 17000, 19998], dtype=torch.int32)
    L = 600
    q, k, v, _ = draw(90, [L], H, 8, torch.bfloat16)
    slots = order[torch.arange(L) // ps].long() * ps + torch.arange(L) % ps
    csd.isoquant_dense_prep(ctx, cache, k, v, slots.cuda(), None, q[-1:], None, None, torch.empty_like(q[-1:]))
    out = torch.empty((1, 1, 16, D), dtype=torch.bfloat16, device="cuda")
    ws = csd.alloc_dense_workspace(ctx, 1, 1, 16)
    csd.isoquant_dense_attend(ctx, cache, q[-1:].view(1, 1, 16, D), order.cuda().view(1, 3),
                              torch.tensor([L], dtype=torch.int32).cuda(), ws, out)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0
    kk, vv = (x.transpose(0, 1).repeat_interleave(8, 0) for x in (k, v))
    ref = attend64(q[-1].unsqueeze(1), kk, vv, torch.full((1,), L))
    check_attention(out[0, 0].unsqueeze(1), *ref, 15)
    assert (data[:17000].view(torch.int16).abs().amax() == 0)


@pytest.mark.parametrize("causal", [True, False])
def test_thousands_of_prompts(cuda_lib, causal):
    """More pieces of work than the grid holds at once, most of them one row."""
    g = torch.Generator().manual_seed(5)
    lens = [int(x) for x in torch.randint(0, 4, (4000,), generator=g)]
    lens[1234], lens[3999] = 600, 257
    ctx = context(cuda_lib, 1)
    q, k, v, cu = draw(95, lens, 1, 2, torch.bfloat16)
    out = torch.zeros_like(q)
    cuda_lib.isoquant_prompt_attend(ctx, q, k, v, cu, out, causal=causal)
    torch.cuda.synchronize()
    assert cuda_lib.isoquant_get_status(ctx) == 0
    at = [0] + list(np.cumsum(lens))
    for b in [1234, 3999] + list(range(0, 4000, 401)):
        a, z = int(at[b]), int(at[b + 1])
        if z > a:
            check_prompts(out[a:z], q[a:z], k[a:z], v[a:z], [z - a], 1, 2, causal)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,H,G", [([255, 256, 257], 16, 2), ([1000], 16, 4), ([130, 61, 400], 16, 3),
                                      ([300, 17, 0, 5], 16, 8), ([90, 200], 16, 5), ([40, 70], 4, 71),
                                      ([30, 5], 8, 128), ([2500, 700], 4, 4), ([700], 48, 1)])
def test_prompts_of_many_heads(cuda_lib, lens, H, G, causal, dtype):
    """Enough work for jobs of two row tiles that share their key tiles (the
    cases of few heads take jobs of one row tile)."""
    ctx = context(cuda_lib, H)
    q, k, v, cu = draw(len(lens) + G, lens, H, G, dtype, 7)
    k[sum(lens):], v[sum(lens):], q[sum(lens):] = float("nan"), float("inf"), float("nan")
    out = torch.full_like(q, 5.0)
    before = out.clone()
    cuda_lib.isoquant_prompt_attend(ctx, q, k, v, cu, out, causal=causal)
    torch.cuda.synchronize()
    assert cuda_lib.isoquant_get_status(ctx) == 0
    check_prompts(out, q, k, v, lens, H, G, causal, before=before)


@pytest.mark.parametrize("rate", [0.002, 0.02, 0.2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_growing_maxima_of_many_heads(cuda_lib, dtype, rate):
    ctx = context(cuda_lib, 32)
    q, k, v, cu = draw(9, [1500], 32, 1, dtype)
    q[..., 0], k[..., 0] = 8.0, (torch.arange(1500, device="cuda") * rate)[:, None].to(k.dtype)
    out = torch.zeros_like(q)
    cuda_lib.isoquant_prompt_attend(ctx, q, k, v, cu, out)
    torch.cuda.synchronize()
    check_prompts(out, q, k, v, [1500], 32, 1, True)


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_values_of_many_heads_that_only_later_tokens_see(cuda_lib, dtype, G):
    """As above in jobs of two row tiles, one head's values alone bad."""
    csd = cuda_lib
    H = 64
    ctx = context(csd, H)
    lens = [50, 400, 30]
    q, k, v, cu = draw(61, lens, H, G, dtype)
    clean = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, clean)
    want = clean.clone().float()
    for t, h, d, x in ((53, 3, 5, float("inf")), (180, 3, 70, float("-inf")), (305, 40, 127, float("nan")),
                       (449, 63, 0, float("inf"))):
        v[t, h, d] = x
        want[t:450, h * G:(h + 1) * G, d] = x
    out = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out)
    torch.cuda.synchronize()
    same = torch.isfinite(want)
    assert torch.equal(out[same], clean[same])
    assert torch.equal(torch.nan_to_num(out.float()[~same], nan=7.0, posinf=8.0, neginf=9.0),
                       torch.nan_to_num(want[~same], nan=7.0, posinf=8.0, neginf=9.0))
