"""GPU parity of tree_verify_attn8 at the edges of its inputs: bad rows of Q, rows of very uneven values, long sums.

Tolerances as in test_gpu_kv8, with what a test adds to them derived beside it.
"""
import numpy as np
import pytest
import torch

from gpu_util import host

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from test_gpu_kv8 import attn_call, attn_check, attn_inputs


@pytest.mark.parametrize("R,G,hd", [(5, 1, 128), (8, 4, 128), (33, 1, 128), (40, 1, 128), (40, 4, 128), (70, 2, 128), (200, 1, 128), (6, 2, 64), (90, 4, 64)])
def test_verify_attn8_bad_query_row_that_sees_nothing(R, G, hd):
    """NaN or Inf in a row of Q: 0 and -Inf where it sees no key, NaN where it sees one; other rows are not touched.  Both kernels, both
    widths of the larger one's tile, with a prefix and without."""
    d = attn_inputs(R + G + 4, 2, R, 2 * G, 2, hd, [0, 20], 16, 16)
    d["see"][0, 1:3] = False
    good = d["Q"].copy()
    bad = [(0, 1), (0, 2), (0, 3), (1, 4)]
    d["Q"][0, 1], d["Q"][0, 2, :, 7], d["Q"][0, 3, :, 5], d["Q"][1, 4, :, 3] = np.nan, np.inf, np.nan, np.nan
    O, lse, err = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    O, lse = host(O).copy(), host(lse).copy()
    assert np.all(O[0, 1:3] == 0) and np.all(np.isneginf(lse[0, 1:3]))
    for b, i in bad[2:]:
        assert np.all(np.isnan(O[b, i])) and np.all(np.isnan(lse[b, i]))
    d["Q"] = good
    O2, lse2, _ = attn_call(d)
    torch.cuda.synchronize()
    for b, i in bad[2:]:
        O[b, i], lse[b, i] = host(O2)[b, i], host(lse2)[b, i]
    attn_check(d, torch.from_numpy(O), torch.from_numpy(lse))
