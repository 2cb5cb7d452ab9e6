"""More host-side checks of the attention calls that need no GPU."""

import hybrid_linear_attention_causal_b200 as gdn
from tests import test_attn_host as H


def test_numbers_of_requests():
    """The kernels count requests in steps in 32 bits."""
    for n in ((1 << 28) + 1, 2 ** 31 - 1):
        assert H.extend(N=n) == gdn.GDN_ERR_UNSUPPORTED
        assert H.append(N=n, T=n) == gdn.GDN_ERR_UNSUPPORTED
