"""Norms of queries and keys on the GPU: a row whose sum of squares is not finite in fp32 is lost as
a whole, and alone, whichever kernel its dimensions choose."""
import pytest
import torch

import kda_prefill_gb300 as kda
from tests.test_gpu_qk_norm_rope import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot,dtype", [(128, 128, torch.bfloat16), (128, 64, torch.float32), (64, 32, torch.bfloat16),
                                         (256, 256, torch.bfloat16), (66, 66, torch.bfloat16), (512, 256, torch.float32),
                                         (7, 2, torch.float32)])
@pytest.mark.parametrize("value", [1e20, 3e38, float("inf"), float("nan")])
def test_rows_whose_squares_are_not_finite(D, rot, dtype, layout, value):
    q, k, qw, kw, pos, freq = make(40, 3, 2, D, rot, dtype, seed=12)
    clean = [x.clone() for x in kda.qk_norm_rope(q.clone(), k.clone(), qw, kw, pos, freq, layout=layout)]
    q[0, 11, 1, D - 1] = value
    k[0, 20, 0] = value
    out = kda.qk_norm_rope(q, k, qw, kw, pos, freq, layout=layout)
    for x, y, (t, h) in zip(out, clean, ((11, 1), (20, 0))):
        rows = torch.ones(x.shape[1:3], dtype=torch.bool, device="cuda")
        rows[t, h] = False
        assert torch.equal(x[0][rows], y[0][rows])
        assert torch.isnan(x[0, t, h]).all()
