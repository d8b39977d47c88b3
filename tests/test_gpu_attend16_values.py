"""Non-finite values under the 16-bit attention: they reach the rows that see
their token, in the dimension that holds them, and no others."""
import pytest
import torch

from tests.test_gpu_prompt import context, draw

pytestmark = pytest.mark.gpu
D = 128
BAD = (float("inf"), float("-inf"), float("nan"))


def same_values(got, want):
    """NaN equal to NaN, everything else bit for bit."""
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,G,count,longest", [(64, 1, 300, 16), (16, 8, 300, 16), (64, 1, 120, 300), (1, 1, 70, 400),
                                               (1, 8, 90, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_prompt_holds_one(cuda_lib, dtype, H, G, count, longest, causal):
    """Each piece of work of a CTA has values of its own to keep apart."""
    csd = cuda_lib
    ctx = context(csd, H)
    g = torch.Generator().manual_seed(count + H)
    lens = [int(x) for x in torch.randint(1, longest + 1, (count,), generator=g)]
    q, k, v, cu = draw(7, lens, H, G, dtype)
    clean = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, clean, causal=causal)
    want, at = clean.clone(), 0
    for b, L in enumerate(lens):
        t, d, x = max(0, L - 2 - b % 3), (7 * b) % D, BAD[b % 3]
        v[at + t, :, d] = x
        want[at + (t if causal else 0):at + L, :, d] = x
        at += L
    out = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out, causal=causal)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(ctx) == 0
    same_values(out, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_one_prompt_of_more_pieces_than_sms(cuda_lib, dtype):
    """Few heads: both sides of a CTA on one row tile's keys."""
    csd = cuda_lib
    ctx = context(csd, 1)
    L = 26000  # 204 row tiles of 128
    q, k, v, cu = draw(8, [L], 1, 1, dtype)
    clean = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, clean)
    want = clean.clone()
    for i, t in enumerate(range(100, L, 256)):
        v[t, 0, i % D] = BAD[2]
        want[t:, 0, i % D] = BAD[2]
    out = torch.zeros_like(q)
    csd.isoquant_prompt_attend(ctx, q, k, v, cu, out)
    torch.cuda.synchronize()
    same_values(out, want)
