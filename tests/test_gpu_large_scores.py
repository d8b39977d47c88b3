"""Scores so large that fp32 holds them in steps of 2^5 to 2^12: a softmax
takes differences of scores, so equal scores weigh the same however large."""
import pytest
import torch

from tests.dense_ref import check_attention
from tests.test_gpu_dense_attend import WEIGHT_BITS, Case
from tests.test_gpu_prompt import WEIGHT_BITS as PROMPT_BITS
from tests.test_gpu_prompt import context, draw

pytestmark = pytest.mark.gpu
D = 128
# |q|: products with keys of 30000 (29952 in bf16) sum to 2^28 to 2^36 once scaled
SIZES = [1000.0, 3100.0, 9000.0, 17000.0, 27000.0, 31000.0, 60000.0]


def check(got, v, n, dtype, bits):
    """Means of the first n values: n equal weights 1 / n, whose sum and
    products stay within the bound with no score error (d = 0)."""
    o = v.double()[:n].mean(0)
    check_attention(got, o.expand_as(got), v.double()[:n].abs().mean(0).expand_as(got), torch.zeros(1).cuda(), bits)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,G,nq", [(2, 1, 1), (1, 24, 1), (1, 16, 4), (1, 8, 16)])
def test_cache(cuda_lib, H, G, nq, dtype):
    c = Case(cuda_lib, [700], H, G, nq, 64, dtype, seed=6)
    c.cache.data[:, 0] = 30000.0
    v = c.cache.data[c.table[0].long()].transpose(0, 2).reshape(H, 2, -1, D)[:, 1, :700]
    for size in SIZES:
        c.q[:] = size
        c.q[..., 1::2] *= 1 + 2.0 ** -6  # products that need more than a few bits
        out = c.run()
        for h in range(H):
            check(out[0, :, h * G:(h + 1) * G].reshape(-1, D), v[h], 700, dtype, WEIGHT_BITS[dtype])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,G", [(1, 2), (64, 1)])
def test_prompts(cuda_lib, H, G, dtype):
    csd = cuda_lib
    ctx = context(csd, H)
    L = 600
    q, k, v, cu = draw(11, [L], H, G, dtype)
    k[:] = 30000.0
    for size in SIZES:
        q[:] = size
        q[..., 1::2] *= 1 + 2.0 ** -6
        out = torch.zeros_like(q)
        csd.isoquant_prompt_attend(ctx, q, k, v, cu, out, causal=False)
        torch.cuda.synchronize()
        for h in (0, H - 1):
            check(out[:, h * G:(h + 1) * G].reshape(-1, D), v[:, h], L, dtype, PROMPT_BITS[dtype])
