"""A prefill with more (request, head) pairs than its kernel's grid holds is refused before anything is enqueued, on CPU:
addresses are never followed."""
import ctypes

import numpy as np
import pytest

import mla_latent_kv_24_b200 as mla

P, UNSUPPORTED = 256, 2


@pytest.mark.parametrize("heads,batch,n_q", [(128, 512, 1), (16, 4096, 2), (1, 65536, 16)])
def test_more_requests_and_heads_than_a_grid_holds(heads, batch, n_q):
    d = mla.make_dims(n_heads=heads)
    lens = np.full(batch, 64, np.int32)
    with pytest.raises(mla.MlaError) as e:
        mla.mla_prefill_workspace_size(d, batch, n_q, lens)
    assert e.value.status == UNSUPPORTED
    assert mla.load().mla_prefill_expanded(ctypes.byref(d), P, P, P, P, P, lens.ctypes.data_as(ctypes.c_void_p), batch, n_q, 1, 1,
                                           P, P, 1 << 60, None) == UNSUPPORTED


def test_the_largest_grid_is_taken():
    assert mla.mla_prefill_workspace_size(mla.make_dims(), 511, 1, [64] * 511) > 0
