"""isoquant_prompt_attend: packed prompts attending to themselves, against
64-bit attention.  Weights are rounded to the inputs' type."""
import pytest
import torch

from tests.dense_ref import attend64, check_attention

pytestmark = pytest.mark.gpu
D = 128
WEIGHT_BITS = {torch.bfloat16: 8, torch.float16: 11}  # half a step relative: 2^-8, 2^-11


def context(csd, H, seed=0):
    signs, quats = csd.synthetic.rotation_params(seed, H)
    return csd.isoquant_init(signs, quats)


def draw(seed, lens, H, G, dtype, tail=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + tail
    q = torch.randn((T, H * G, D), generator=g)
    k = torch.randn((T, H, D), generator=g) * torch.exp(torch.rand((H, D), generator=g) - 0.5) * spread
    v = torch.randn((T, H, D), generator=g)
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    return q.to(dtype).cuda(), k.to(dtype).cuda(), v.to(dtype).cuda(), cu.cuda()


def check(out, q, k, v, lens, H, G, causal, scale=None, before=None, start=0):
    a = start
    for L in lens:
        rows = q[a:a + L].transpose(0, 1)
        kk = k[a:a + L].transpose(0, 1).repeat_interleave(G, 0)
        vv = v[a:a + L].transpose(0, 1).repeat_interleave(G, 0)
        limits = torch.arange(1, L + 1) if causal else torch.full((L,), L)
        if L:
            for i in range(0, L, 1024):
                j = min(L, i + 1024)
                end = j if causal else L
                o, A, d = attend64(rows[:, i:j], kk[:, :end], vv[:, :end], limits[i:j], scale)
                check_attention(out[a + i:a + j].transpose(0, 1), o, A, d, WEIGHT_BITS[q.dtype])
        a += L
    if before is not None:
        assert torch.equal(out[a:], before[a:]) and torch.equal(out[:start], before[:start])


CASES = [  # lens, H, G
    ([1], 1, 1),
    ([1, 2, 3, 0, 5], 2, 1),
    ([127, 128, 129], 1, 1),
    ([255, 256, 257], 2, 2),
    ([300, 17], 4, 8),
    ([1000], 1, 4),
    ([130, 61, 400], 2, 3),
    ([90, 200], 1, 5),
    ([64, 77], 3, 7),
    ([200, 33], 1, 16),
    ([40, 70], 1, 71),
    ([30, 5], 1, 128),
    ([2500, 3, 700], 2, 4),
    ([0, 0, 50, 0], 2, 6),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,H,G", CASES)
def test_prompts(cuda_lib, lens, H, G, causal, dtype):
    csd = cuda_lib
    ctx = context(csd, H)
    tail = 7
    q, k, v, cu = draw(len(lens) + G, lens, H, G, dtype, tail)
    # padding rows behind the last sequence hold what they like
    k[sum(lens):], v[sum(lens):], q[sum(lens):] = float("nan"), float("inf"), float("nan")
    out = torch.full_like(q, 5.0)
    before = out.clone()
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out, causal=causal)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0 and csd.isoquant_last_launch_count(ctx) == 1
    check(out, q, k, v, lens, H, G, causal, before=before)


@pytest.mark.parametrize("causal", [True, False])
def test_many_short_prompts(cuda_lib, causal):
    g = torch.Generator().manual_seed(2)
    lens = [int(x) for x in torch.randint(0, 40, (500,), generator=g)]
    ctx = context(cuda_lib, 2)
    q, k, v, cu = draw(6, lens, 2, 4, torch.bfloat16)
    out = torch.zeros_like(q)
    cuda_lib.isoquant_prompt_attend(ctx, q, k, v, cu, out, causal=causal)
    torch.cuda.synchronize()
    assert cuda_lib.isoquant_get_status(ctx) == 0
    check(out, q, k, v, lens, 2, 4, causal)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale,spread", [(0.7, 3.0), (1e-3, 1.0)])
def test_scales_and_peaked_softmax(cuda_lib, dtype, scale, spread):
    ctx = context(cuda_lib, 2)
    lens = [700, 300]
    q, k, v, cu = draw(8, lens, 2, 4, dtype, spread=spread)
    # a late key with far larger scores: the running maximum moves by hundreds
    k[650], k[900] = k[650] * 20, k[900] * 20
    out = torch.zeros_like(q)
    cuda_lib.isoquant_prompt_attend(ctx, q, k, v, cu, out, scale=scale)
    torch.cuda.synchronize()
    check(out, q, k, v, lens, 2, 4, True, scale)


def test_growing_maxima(cuda_lib):
    """Scores that rise along the prompt, by less and by more per tile than
    the running maximum lets pass."""
    ctx = context(cuda_lib, 1)
    for rate in (0.002, 0.02, 0.2):
        q, k, v, cu = draw(9, [1500], 1, 4, torch.bfloat16)
        q[..., 0], k[..., 0] = 8.0, (torch.arange(1500, device="cuda") * rate)[:, None].to(k.dtype)
        out = torch.zeros_like(q)
        cuda_lib.isoquant_prompt_attend(ctx, q, k, v, cu, out)
        torch.cuda.synchronize()
        check(out, q, k, v, [1500], 1, 4, True)


def test_fused_projection_slices(cuda_lib):
    """q, k and v as slices of one [T][(Hq + 2 H) 128] projection, and with
    tokens further apart still."""
    csd = cuda_lib
    H, G, lens = 2, 4, [333, 50]
    ctx = context(csd, H)
    q, k, v, cu = draw(10, lens, H, G, torch.bfloat16)
    want = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, want)
    for pad in (0, 24):
        fused = torch.full((383, (H * G + 2 * H) * D + pad), float("nan"), dtype=q.dtype, device="cuda")
        qs = fused[:, :H * G * D].view(383, H * G, D) if pad == 0 else fused[:, :H * G * D].unflatten(1, (H * G, D))
        ks = fused[:, H * G * D:(H * G + H) * D].unflatten(1, (H, D))
        vs = fused[:, (H * G + H) * D:(H * G + 2 * H) * D].unflatten(1, (H, D))
        qs.copy_(q), ks.copy_(k), vs.copy_(v)
        out = torch.zeros_like(q)
        csd.isoquant_prompt_attend(ctx, qs, ks, vs, cu, out)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_neighbours_do_not_leak(cuda_lib):
    """NaN and infinite rows of one prompt stay in it."""
    csd = cuda_lib
    ctx = context(csd, 2)
    lens = [100, 77, 300]
    q, k, v, cu = draw(11, lens, 2, 2, torch.bfloat16)
    clean = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, clean)
    k[100:177], v[100:177], q[100:177] = float("nan"), float("inf"), float("inf")
    out = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out)
    torch.cuda.synchronize()
    assert torch.equal(out[:100], clean[:100]) and torch.equal(out[177:], clean[177:])
    assert torch.isnan(out[100:177]).all()


def test_nan_key_reaches_only_rows_that_see_it(cuda_lib):
    csd = cuda_lib
    ctx = context(csd, 1)
    q, k, v, cu = draw(12, [400], 1, 4, torch.bfloat16)
    clean = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, clean)
    k[250, 0, 3] = float("nan")
    out = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out)
    torch.cuda.synchronize()
    assert torch.equal(out[:250], clean[:250]) and torch.isnan(out[250:]).all()


def test_bad_sequence_bounds_are_flagged(cuda_lib):
    csd = cuda_lib
    ctx = context(csd, 2)
    lens = [50, 60, 70]
    q, k, v, cu = draw(13, lens, 2, 2, torch.float16)
    clean = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, clean)
    for bad in ([0, 50, 110, 181], [-3, 50, 110, 180], [0, 50, 20, 180]):
        out = torch.full_like(q, 9.0)
        csd.isoquant_prompt_attend(ctx, q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out)
        torch.cuda.synchronize()
        assert csd.isoquant_get_status(ctx) == csd.DEVERR_SEQ_RANGE
        a = 50 if bad[0] < 0 else 0
        b = 50 if bad[2] == 20 else 110
        if bad[2] != 20:
            assert torch.equal(out[a:b], clean[a:b])
        if bad[3] == 181:
            assert (out[110:] == 9.0).all()
    # a first sequence that starts behind the first token
    out = torch.full_like(q, 9.0)
    csd.isoquant_prompt_attend(ctx, q, k, v, torch.tensor([50, 110], dtype=torch.int32, device="cuda"), out)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0
    assert torch.equal(out[50:110], clean[50:110]) and (out[:50] == 9.0).all() and (out[110:] == 9.0).all()


def test_streams_graphs_and_repeats(cuda_lib):
    csd = cuda_lib
    ctx = context(csd, 2)
    lens = [900, 100, 333]
    q, k, v, cu = draw(14, lens, 2, 4, torch.bfloat16)
    want = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, want)
    torch.cuda.synchronize()
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        csd.isoquant_prompt_attend(ctx, q, k, v, cu, out)
    other = torch.zeros_like(q)
    for _ in range(10):
        out.zero_()
        torch.cuda.synchronize()
        gr.replay()
        csd.isoquant_prompt_attend(ctx, q, k, v, cu, other, stream=side)  # two calls at once
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want)
    # other lengths through the same graph
    cu.copy_(torch.tensor([0, 5, 1000, 1333], dtype=torch.int32))
    gr.replay()
    torch.cuda.synchronize()
    check(out, q, k, v, [5, 995, 333], 2, 4, True)


def test_argument_errors(cuda_lib):
    import ctypes
    csd = cuda_lib
    L, p = csd.lib(), csd._ptr
    ctx = context(csd, 2)
    q, k, v, cu = draw(15, [20, 30], 2, 4, torch.bfloat16)
    out = torch.zeros_like(q)
    s0 = csd._stream(None)

    def call(qp=None, kp=None, vp=None, dt=1, T=50, Hq=8, qs=1024, ks=256, vs=256, cup=None, B=2, scale=0.0, o=None):
        return L.isoquant_prompt_attend(ctx.handle, qp or p(q), kp or p(k), vp or p(v), dt, T, Hq, qs, ks, vs,
                                        cup or p(cu), B, 1, scale, o or p(out), s0)

    def off(t, by=8):
        return ctypes.c_void_p(t.data_ptr() + by)

    assert call(dt=0) == -2 and call(dt=9) == -2
    assert call(T=-1) == -1 and call(B=-1) == -1 and call(Hq=0) == -1 and call(Hq=9) == -1
    assert call(Hq=2 * 129, qs=129 * 256) == -2
    assert call(scale=-0.5) == -1 and call(scale=float("nan")) == -1
    assert call(qs=1016) == -1 and call(ks=248) == -1 and call(vs=0) == -1 and call(ks=1 << 40) == -1
    assert call(qs=1028) == -6 and call(ks=260) == -6 and call(vs=257) == -6
    assert call(qp=off(q)) == -6 and call(kp=off(k)) == -6 and call(vp=off(v)) == -6 and call(o=off(out)) == -6
    assert call(cup=off(cu, 2)) == -6
    assert call(T=1 << 30) == -1
    assert L.isoquant_last_launch_count(ctx.handle) == 0
    assert call(T=0) == 0 and call(B=0) == 0 and L.isoquant_last_launch_count(ctx.handle) == 0
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0
    assert call() == 0
    torch.cuda.synchronize()
    check(out, q, k, v, [20, 30], 2, 4, True)
