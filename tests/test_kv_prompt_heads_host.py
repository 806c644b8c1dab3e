"""Host-only: an append's rows (heads by tokens of a block) are counted in 32 bits, so more than 2^24 key heads are refused,
as kv_norm_rotate refuses them."""
import pytest

from hybrid_ssm_gated_gb300 import build, gdn, kv
from tests.test_kv_host import FAKE, NULL, SHAPE, _cache, _rows


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kv.lib()


@pytest.mark.parametrize("Hkv", [(1 << 24) + 1, 1 << 27, (1 << 31) - 1])
@pytest.mark.parametrize("total", [0, 9])
def test_key_heads_of_an_append(lib, Hkv, total):
    call = lambda heads: lib.kv_append(_cache(Hkv=heads, counts=None), 2, total, 4, FAKE, FAKE, _rows(), _rows(), None, None, None,
                                       None, FAKE, None)
    assert call(Hkv) == SHAPE and "Hkv" in gdn.gdn_last_error_string()
    assert call(1 << 24) == NULL  # (its missing counts are what is refused)
