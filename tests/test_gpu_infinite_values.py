"""Infinite and NaN values that every row of a tile sees, under the 16-bit
attention: an infinite value makes its element infinite for the rows that see
its token, however small the weight; both signs, or a NaN, make it NaN.  A row
whose every score is -inf stays zero."""
import pytest
import torch

from tests.test_gpu_attend16_values import same_values
from tests.test_gpu_dense_attend import Case
from tests.test_gpu_prompt import context, draw

pytestmark = pytest.mark.gpu
D = 128
INF, NAN = float("inf"), float("nan")
# (token, dim, value): dim 20 holds both signs
EARLY = [(5, 3, INF), (200, 9, -INF), (6, 20, INF), (130, 20, -INF), (7, 30, NAN), (131, 127, INF)]
FORMS = [(2, 1, 1), (4, 8, 1), (1, 24, 1), (1, 16, 4), (2, 8, 16)]  # rows of a product: 16, 16, 32, 64, 128


def put(c, b, side, t, d, x, heads=slice(None)):
    """A value (side 1) or key (side 0) element of sequence b's token t."""
    c.cache.data[int(c.table_cpu[b, t // c.ps]), side, heads, t % c.ps, d] = x


def place(want, b, t, d, x, lim):
    """x joins element d of the rows [nq][heads][128] whose limit is beyond t."""
    rows = torch.tensor([l > t for l in lim], device=want.device)
    old = want[b, rows, :, d]
    want[b, rows, :, d] = torch.where(torch.isfinite(old), torch.full_like(old, x), old + x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,G,nq", FORMS)
@pytest.mark.parametrize("lens", [[1000], [700, 300, 1500] * 30])
def test_cache(cuda_lib, lens, H, G, nq, dtype):
    c = Case(cuda_lib, lens, H, G, nq, 64, dtype, seed=3)
    want = c.run(causal=True)
    for b, L in enumerate(lens):
        if b % 4 == 2:
            continue  # a clean one between
        for t, d, x in EARLY:
            put(c, b, 1, t, d, x)
            place(want, b, t, d, x, [L - nq + i + 1 for i in range(nq)])
    same_values(c.run(causal=True), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,G,nq", FORMS)
@pytest.mark.parametrize("lens", [[1000], [700, 400] * 40])
@pytest.mark.parametrize("late", [20, 390])
def test_cache_weights_of_nothing(cuda_lib, late, lens, H, G, nq, dtype):
    """One key takes all: the others' weights are e^-280 and less."""
    c = Case(cuda_lib, lens, H, G, nq, 64, dtype, seed=4)
    c.q[..., 0] = 16.0
    c.cache.data[:, 0, :, :, 0] = 0.0
    for b in range(len(lens)):
        put(c, b, 0, late, 0, 200.0)
    want = c.run()
    for b, L in enumerate(lens):
        for t, d, x in EARLY:
            put(c, b, 1, t, d, x)
            place(want, b, t, d, x, [L] * nq)
    same_values(c.run(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,G,nq", FORMS)
@pytest.mark.parametrize("lens", [[1000], [700, 400] * 40])
@pytest.mark.parametrize("causal", [True, False])
def test_cache_rows_of_minus_infinity(cuda_lib, causal, lens, H, G, nq, dtype):
    """Every score of head 0's rows is -inf: zeros, whatever the values."""
    c = Case(cuda_lib, lens, H, G, nq, 64, dtype, seed=5)
    want = c.run(causal=causal)
    want[:, :, :G] = 0.0
    c.q[:, :, :G, 7] = 1.0
    c.cache.data[:, 0, 0, :, 7] = -INF
    for b, L in enumerate(lens):
        for t, d, x in EARLY + [(L - 1, 50, INF)]:
            put(c, b, 1, t, d, x, heads=0)
    same_values(c.run(causal=causal), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,G", [(1, 1), (1, 4), (2, 8), (64, 1), (16, 8)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("late", [20, 390])
def test_prompt_weights_of_nothing(cuda_lib, late, causal, H, G, dtype):
    csd = cuda_lib
    ctx = context(csd, H)
    lens = [700, 30, 500]
    q, k, v, cu = draw(9, lens, H, G, dtype)
    q[..., 0], k[..., 0] = 16.0, 0.0
    k[late, :, 0] = k[730 + late, :, 0] = 200.0
    clean = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, clean, causal=causal)
    want = clean.clone()
    for at, L in ((0, 700), (730, 500)):
        part = want[at:at + L][None]
        for t, d, x in EARLY:
            v[at + t, :, d] = x
            place(part, 0, t, d, x, [i + 1 if causal else L for i in range(L)])
    out = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out, causal=causal)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0
    same_values(out, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,G", [(2, 1), (2, 8), (64, 1), (16, 8)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_rows_of_minus_infinity(cuda_lib, causal, H, G, dtype):
    csd = cuda_lib
    ctx = context(csd, H)
    lens = [300, 30, 500]
    q, k, v, cu = draw(10, lens, H, G, dtype)
    want = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, want, causal=causal)
    want[:, :G] = 0.0
    q[:, :G, 7], k[:, 0, 7] = 1.0, -INF
    for t, d, x in ((5, 3, INF), (200, 9, -INF), (7, 30, NAN), (299, 50, INF), (329, 60, INF), (829, 0, NAN)):
        v[t, 0, d] = x
    out = torch.full_like(q, 5.0)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out, causal=causal)
    torch.cuda.synchronize()
    same_values(out, want)
