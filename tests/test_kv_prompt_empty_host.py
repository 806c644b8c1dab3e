"""Host-only checks of calls of the prompt operators that bring no row (total = 0: every sequence empty, or padding):
rows need no address then. No kernel is launched: each call ends at a later refusal."""
import pytest

from hybrid_ssm_gated_gb300 import build, gdn, kv
from tests.test_kv_host import FAKE, NULL, SHAPE, _cache, _rows

LAUNCH = -6


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kv.lib()


@pytest.mark.parametrize("rows", [None, _rows(p=None)], ids=["no rows", "rows without an address"])
def test_append_without_a_row(lib, rows):
    """What refuses the call is the check behind those of the rows: a cache with stamps needs counts."""
    r = kv.kv_rotary(None, None, 0, 0, 1e-6, 0.0, FAKE, FAKE, 32, 1, 0)
    append = lambda total, q, rotary: lib.kv_append(_cache(counts=None), 2, total, 4, FAKE, FAKE, rows, rows, rotary, None, q,
                                                    q, FAKE, None)
    for q, rotary in ((None, None), (None, r), (rows, r)):
        assert append(0, q, rotary) == NULL and "stamps needs counts" in gdn.gdn_last_error_string()
        assert append(1, q, rotary) == NULL and "k is NULL" in gdn.gdn_last_error_string()


@pytest.mark.parametrize("rows", [None, _rows(p=None)], ids=["no rows", "rows without an address"])
def test_prompt_attention_without_a_row(lib, rows):
    """What refuses the call is its workspace of no bytes (or the machine, where that has no device to size one for)."""
    call = lambda total, out: lib.kv_prompt_attention(_cache(), 2, total, 4, FAKE, FAKE, rows, 1.0, out, None, FAKE, 0, FAKE, None)
    assert call(0, None) in (SHAPE, LAUNCH)
    assert call(1, None) == NULL and call(1, FAKE) == NULL


def test_other_refusals_stand(lib):
    null = _rows(p=None)
    assert lib.kv_append(_cache(), 2, 0, 4, None, FAKE, null, null, None, None, None, None, FAKE, None) == NULL
    assert lib.kv_append(_cache(), 2, 0, 4, FAKE, None, null, null, None, None, None, None, FAKE, None) == NULL
    assert lib.kv_prompt_attention(_cache(), 2, 0, 4, FAKE, FAKE, null, 1.0, None, None, None, 1 << 30, FAKE, None) == NULL
    assert lib.kv_prompt_attention(_cache(), 2, 0, 4, FAKE, None, null, 1.0, None, None, FAKE, 1 << 30, FAKE, None) == NULL
