"""The weights' own precision in the attention's second product: columns of V
in which four tokens cancel, so that the output is as small as the error of the
weights and no rounding of the output hides it."""
import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
from test_gpu_parity import DEV, _say

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def badly_split(dtype, top):
    """A number x of the type in (-top, -top / 2] whose weight e^x loses most
    when it is held as two 16-bit numbers of the type (at least a quarter of the
    square of their unit)."""
    x = -(top * torch.arange(256, 512).double() / 512).to(dtype)
    p = torch.exp(x.double())
    hi = p.to(dtype).double()
    loss = (p - hi - (p - hi).to(dtype).double()).abs() / p
    i = int(loss.argmax())
    return x[i], float(loss[i])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,heads,width", [(64, 1, None), (128, 1, None), (128, 20, None), (128, 40, 600), (72, 3, None),
                                             (192, 2, 600), (256, 2, None), (256, 20, 600)])
def test_weights_that_cancel(dtype, dim, heads, width):
    _say("weights that cancel dim=%d heads=%d wide=%s %s" % (dim, heads, width, dtype))
    m = R.make([4], 1, dim, 16, dtype, heads=heads, seed=dim, width=width)
    page = m.table[0, 0].long()
    x1, loss = badly_split(dtype, 2.0)
    assert dtype is not torch.bfloat16 or loss >= R.UNIT[dtype] ** 2 / 4
    x = torch.stack([torch.zeros((), dtype=dtype), x1, torch.tensor(-6.0, dtype=dtype), torch.tensor(-9.0, dtype=dtype)])
    m.q[:], m.k[page, 0, :4] = 0.0, 0.0
    m.q[:, :, 0], m.k[page, 0, :4, 0] = 1.0, x
    p = torch.exp(x.double())
    v = torch.zeros(4, dim, dtype=dtype)
    v[0] = torch.randn(dim, generator=torch.Generator().manual_seed(dim)).to(dtype)
    for t in (1, 2, 3):             # each takes away what the ones before leave, as far as its type can
        v[t] = (-(p[:t] @ v[:t].double()) / p[t]).to(dtype)
    m.v[page, 0, :4] = v
    R.to_gpu(m, S)
    out = m.cache.attend(m.gq, S.KVWorkspace(m.cache, heads), scale=1.0)[0].double().cpu()
    p = p / p.sum()
    want, mix = p @ v.double(), p @ v.double().abs()
    # In units of 2^-24 of what a token adds: its logit is exact, its base-2
    # form is rounded twice (the constant, the product) and the largest is 0, so
    # that 2 |x| of them; the exponential 2; the parts of its weight 1 (bf16) or 4
    # (fp16).  Four tokens and up to three parts are 12 sums, the division and
    # its product 3 more roundings of at most that.
    tol = R.UNIT[dtype] * want.abs() + R.F32 * (p * (2 * x.double().abs() + 2 + 4 + 12 + 3)) @ v.double().abs()
    tol += torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps      # results below the normal ones
    assert bool((tol < 2.0 ** -18 * mix + R.UNIT[dtype] * want.abs() + 1e-7).all())
    worst = ((out - want).abs() / tol).max()
    assert float(worst) <= 1, float(worst)
