"""Pool sizes that the page operators refuse before any launch (no GPU: the
addresses are stand-ins)."""
import ctypes as C

import pytest

from tests.gpu_helpers import built_lib

AT = [C.c_void_p(i << 20) for i in range(1, 13)]


@pytest.fixture(scope="module")
def B():
    built_lib()
    from q8_quantized_llama_gb300 import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("pool", [dict(n_pages=(1 << 31) - 1), dict(n_pages=(1 << 30) + 1), dict(n_layer=1 << 20, n_head_kv=17),
                                  dict(n_layer=1, n_head_kv=(1 << 19) + 1, page=256, head_dim=128)])
def test_page_operators_refuse_pools_past_their_limits(B, pool):
    """Among them counts whose passes, in 32 bits, would step over the last page and start again."""
    f = dict(k=AT[0], v=AT[1], type=B.GGUF_F16, n_layer=1, n_pages=100, page=8, n_head_kv=1, head_dim=64)
    f.update(pool)
    p = B.llama_q8_pages(*(f[n] for n, _ in B.llama_q8_pages._fields_))
    st = B.lib().llama_q8_pages_compact(C.addressof(p), 1, AT[2], 4, AT[3], AT[4], AT[5], AT[6], AT[7], 1 << 40, AT[8], None)
    assert st == B.LQ8_ERR_UNSUPPORTED
    st = B.lib().llama_q8_pages_fork(C.addressof(p), 1, AT[2], AT[3], 4, AT[4], 1, AT[5], 1, AT[6], AT[7], AT[8], AT[9],
                                     1 << 40, AT[10], None)
    assert st == B.LQ8_ERR_UNSUPPORTED
