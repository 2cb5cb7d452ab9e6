"""More host-side checks of the attention calls that need no GPU."""
import pytest

import hybrid_linear_attention_causal_b200 as gdn
from tests import test_attn_host as H


def test_numbers_of_requests():
    """The kernels count requests in steps in 32 bits."""
    for n in ((1 << 28) + 1, 2 ** 31 - 1):
        assert H.extend(N=n) == gdn.GDN_ERR_UNSUPPORTED
        assert H.append(N=n, T=n) == gdn.GDN_ERR_UNSUPPORTED


def test_a_cache_changed_in_place():
    """Pools that grow or shrink where they lie count anew, and are checked anew."""
    cfg = H.cfg()
    cache = gdn.alloc_attn_cache(cfg, 8, "cpu")
    assert cache.c().num_pages == 8 and cache.c() is cache.c()
    pools = (cache.k, cache.v, cache.k_exp, cache.v_exp)
    at = cache.k.data_ptr()
    for pages in (3, 6):
        for t in pools:
            t.resize_(pages, *t.shape[1:])
        assert cache.k.data_ptr() == at and cache.c().num_pages == cache.num_pages == pages
    cache.k.resize_(7, *cache.k.shape[1:])
    with pytest.raises(ValueError):
        cache.c()
