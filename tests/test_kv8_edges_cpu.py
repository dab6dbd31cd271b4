"""8-bit caches without a GPU: refusals of overlapping arrays and sizes at their limits."""
import pytest

import token_level_sparse_fwht_b200 as ad
from test_kv8_cpu import A, _evict, cache
from token_level_sparse_fwht_b200 import ERR_INVALID_ARG


@pytest.mark.parametrize("off", [-4, 4])
def test_new_lengths_beside_the_old_ones_are_refused(off):
    """In place they are the same array; one element off, a sequence would read another's new length."""
    far = dict(k=A + (1 << 24), v=A + (1 << 25), k_scale=A + (1 << 26), v_scale=A + (1 << 27))
    assert _evict(cache(), lens=A + 64, lens_out=A + 64 + off) == ERR_INVALID_ARG
    assert _evict(cache(), dst=cache(**far), w_out=A + (1 << 28), lens=A + 64,
                  lens_out=A + 64 + off) == ERR_INVALID_ARG
