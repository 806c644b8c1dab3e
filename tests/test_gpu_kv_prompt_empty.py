"""Calls of the prompt operators that bring no row at all (total = 0), whose empty tensors have no address: nothing is
written, and slots, lengths and offsets are checked as in any other call."""
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, gdn, kv
from tests.kv_ref import TORCH

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Empty:
    """A cache of three slots (5, 0 and 40 entries) and a call of three sequences without a row."""

    def __init__(self, dtype, slots=(0, -1, 2), cu=(0, 0, 0, 0), lengths=(5, 0, 40), num_pages=12, d=64):
        dt = TORCH[dtype]
        self.cache = kv.KVCache.allocate(num_pages, 2, 16, d, 3, 4, dt)
        self.cache.page_table.copy_(torch.arange(12, dtype=torch.int32).view(3, 4))
        self.cache.k.fill_(1.0), self.cache.v.fill_(2.0)
        self.cache.lengths.copy_(i32(*lengths)), self.cache.counts.copy_(i32(*lengths))
        self.slots, self.cu, self.err = i32(*slots), i32(*cu), i32(0)
        self.q, self.k, self.v = (torch.empty(0, h, d, dtype=dt, device="cuda") for h in (4, 2, 2))
        self.ws = kv.kv_prompt_workspace(self.cache, len(slots), self.q)
        self.before = [x.clone() for x in self.state()]

    def state(self):
        c = self.cache
        return c.k, c.v, c.page_table, c.lengths, c.counts, c.weights, c.stamps

    def append(self, rotary=None):
        q = self.q if rotary else None
        kv.kv_append(self.cache, self.slots, self.cu, self.k, self.v, self.err, rotary=rotary, q=q,
                     q_out=torch.empty_like(self.q) if rotary else None)

    def attend(self, lse=True):
        out = torch.empty_like(self.q)
        kv.kv_prompt_attention(self.cache, self.slots, self.cu, self.q, out, self.err, self.ws,
                               lse=torch.empty(0, 4, device="cuda") if lse else None)

    def assert_unchanged(self, bit=0):
        torch.cuda.synchronize()
        assert int(self.err.item()) == bit
        assert all(torch.equal(a, b) for a, b in zip(self.state(), self.before))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rotated", [False, True])
def test_append_without_a_row(dtype, rotated):
    e = Empty(dtype)
    e.append(kv.Rotary([1.0] * 16) if rotated else None)
    e.assert_unchanged()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("lse", [False, True])
def test_attention_without_a_row(dtype, d, lse):
    e = Empty(dtype, d=d)
    e.attend(lse)
    e.assert_unchanged()


@pytest.mark.parametrize("what,bit", [(dict(slots=(0, 3, 1)), gdn.DEVERR_SLOT), (dict(lengths=(5, 0, 65)), kv.DEVERR_LENGTH),
                                      (dict(lengths=(-1, 0, 40)), kv.DEVERR_LENGTH), (dict(cu=(0, 1, 1, 1)), gdn.DEVERR_SEQLEN),
                                      (dict(cu=(0, 0, -1, 0)), gdn.DEVERR_SEQLEN)], ids=str)
@pytest.mark.parametrize("op", ["append", "attend"])
def test_what_is_refused_without_a_row(op, what, bit):
    e = Empty("bf16", **what)
    getattr(e, op)()
    e.assert_unchanged(bit)


def test_a_captured_step_that_brings_no_row():
    """Both operators in a graph, replayed twice, between steps that bring rows."""
    e = Empty("bf16")
    rot = kv.Rotary([1.0] * 16)
    one = torch.randn(1, 4, 64, device="cuda").bfloat16()
    out, ws = torch.empty_like(one), kv.kv_prompt_workspace(e.cache, 1, one)

    def step():
        k, v = one[:, :2], one[:, 2:]
        kv.kv_append(e.cache, i32(0), i32(0, 1), k, v, e.err, rotary=rot, q=one, q_out=torch.empty_like(one))
        kv.kv_prompt_attention(e.cache, i32(0), i32(0, 1), one, out, e.err, ws)
        torch.cuda.synchronize()

    def empty():
        e.append(rot)
        e.attend()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        empty()
    torch.cuda.current_stream().wait_stream(s)
    e.assert_unchanged()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        empty()
    for i in range(2):
        step()
        want = [x.clone() for x in e.state()]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(e.state(), want))
        assert int(e.err.item()) == 0 and e.cache.lengths.tolist() == [6 + i, 0, 40] and out.isfinite().all()
