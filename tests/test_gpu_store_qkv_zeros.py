"""Signs of zero in 4-bit codes: 0 where the block's scale is 0, otherwise the sign of the value."""
import numpy as np
import pytest
import torch

from oracle import fourbit
from test_gpu_store_qkv import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -6])
def test_signs_of_zero(scale):
    c = Case(6, 1, 1, "e2m1", seed=20, norm=False, rot=0, scale=scale)
    v = torch.zeros(6, 128)
    v[0] = -1e-4                          # blocks whose scale rounds to zero
    v[1] = torch.tensor([1e-4, -1e-4, -0.0, 0.0]).repeat(32)
    v[2] = torch.tensor([-0.0, 3.0, 0.0, -1.0]).repeat(32)
    v[3] = torch.tensor([-0.0, 0.0, -1e-5, 1e-5, 6.0, -0.01, 0.01, -6.0]).repeat(16)
    v[4, ::2] = -0.0
    v[4, 64] = 2.0 ** 20                  # beyond the largest scale, beside zeros of both signs
    v[5] = torch.tensor([-0.0, 448 * 6.0, -1e-30, 1e-30]).repeat(32)
    c.v.copy_((v * scale)[:, None].to(torch.bfloat16))
    c.run()
    torch.cuda.synchronize()
    codes, sb = fourbit.unpack(c.vp.cpu().numpy())
    x = c.v[:, 0].float().cpu().double().numpy() / scale
    for t, slot in enumerate(c.slots.tolist()):
        ref_c, ref_b = fourbit.encode(x[t])
        assert (fourbit.e4m3_value(sb[slot // 64, 0, slot % 64]) == ref_b).all()
        assert (codes[slot // 64, 0, slot % 64] == ref_c).all(), t
    zero = np.repeat(fourbit.e4m3_value(sb[c.slots[0] // 64, 0, c.slots[0] % 64]), 16) == 0
    assert zero.all() and (codes[c.slots[0] // 64, 0, c.slots[0] % 64] == 0).all()
