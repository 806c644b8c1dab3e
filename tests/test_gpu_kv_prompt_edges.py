"""Edges of the prompt operators: rows that share memory, outputs and weights off the 16-byte grid, gaps between
sequences of activations, many sequences with two tiles of rows a unit, and the same bits from the same call."""
import numpy as np
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, kv
from tests import prompt_ref as ref
from tests.kv_ref import TORCH, host
from tests.prompt_ref import Prompt
from tests.test_gpu_kv_prompt import check_sampled, frequencies

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", [(0,), (1,), (0, 1)], ids=str)
def test_queries_shared_by_strides_of_zero(dtype, dims):
    c = Prompt(80, dtype, [(100, 20), (33, 0)], Hq=4, Hkv=2, d=64, page=16)
    x = c.q
    for i in dims:
        x = x.narrow(i, 0, 1)
    c.q = x.expand_as(c.q)
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_pool_whose_heads_share_memory(dtype):
    c = Prompt(81, dtype, [(100, 20), (33, 0)], Hq=4, Hkv=2, d=64, page=16)
    c.k, c.v = c.k[:, :1].expand_as(c.k), c.v[:, :1].expand_as(c.v)
    c.sync()
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 256])
def test_outputs_off_the_grid(dtype, d):
    c = Prompt(82, dtype, [(100, 300), (33, 0)], Hq=4, Hkv=2, d=d, page=16)
    room = torch.full((c.q.numel() + 2,), 7.0, dtype=c.q.dtype, device="cuda")
    out, lse = room[1:-1].view(c.q.shape), torch.empty(c.total, 4, device="cuda")
    kv.kv_prompt_attention(c.cache, c.d_slots, c.d_cu, c.q, out, c.err, kv.kv_prompt_workspace(c.cache, 2, c.q), lse=lse,
                           scale=c.scale)
    r = ref.prompt_attention(host(c.k), host(c.v), c.table, c.lengths, c.slots, c.cu, host(c.q), c.scale)
    c.compare(out, lse, *r, c.owned())
    assert room[0] == 7.0 and room[-1] == 7.0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences_with_two_tiles_a_unit(dtype, d):
    r = np.random.default_rng(83)
    prompts = [(int(r.integers(1, 120)), int(r.integers(0, 200))) for _ in range(40)]
    check_sampled(Prompt(83, dtype, prompts, Hq=64, Hkv=8, d=d, page=16, pad=(3, 17)), 31)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("prompts,Hq,Hkv,d", [([(2500, 0)], 16, 2, 128), ([(700, 5000)], 96, 8, 64), ([(600, 100)], 16, 2, 256)])
def test_the_same_call_gives_the_same_bits(dtype, prompts, Hq, Hkv, d):
    """Twenty times, over other bytes in the workspace."""
    c = Prompt(84, dtype, prompts, Hq=Hq, Hkv=Hkv, d=d, page=64)
    out, lse = torch.empty_like(c.q), torch.empty(c.total, Hq, device="cuda")
    ws = kv.kv_prompt_workspace(c.cache, 1, c.q)
    want = None
    for i in range(20):
        ws.fill_(i * 13)
        out.fill_(5.0)
        kv.kv_prompt_attention(c.cache, c.d_slots, c.d_cu, c.q, out, c.err, ws, lse=lse, scale=c.scale)
        if want is None:
            want = out.clone(), lse.clone()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_past_the_turned_part_stay(dtype, interleaved):
    x = torch.randn(1, 3, 2, 64, device="cuda").to(TORCH[dtype])
    x[0, 1, 0, 40], x[0, 1, 0, 50] = float("inf"), float("-inf")
    out = torch.empty_like(x)
    pos = torch.tensor([[5, 6, 7]], dtype=torch.int32, device="cuda")
    kv.kv_norm_rotate(kv.Rotary(frequencies(32), interleaved=interleaved), pos, q=x, q_out=out)
    assert torch.equal(out[..., 32:], x[..., 32:]) and out[..., :32].isfinite().all()


def _against(x, out, weight, rot, pos, d, dtype):
    z, size = ref.turned(host(x).reshape(-1, x.shape[2], d), weight, 1e-6, 0.0, frequencies(rot), [0] * (rot // 2),
                         pos.reshape(1, -1), False)
    assert (np.abs(host(out).reshape(z.shape) - z) <= ref.turn_bound(z, size, d, dtype)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("per_head", [False, True])
def test_norm_weights_off_the_grid(dtype, per_head):
    r = np.random.default_rng(85)
    x = torch.from_numpy(r.normal(size=(2, 9, 3, 64))).to(TORCH[dtype]).cuda()
    w = r.normal(size=(3, 64) if per_head else 64).astype(np.float32)
    room = torch.zeros(w.size + 3 + 1, device="cuda")
    if per_head:  # rows of 65 floats
        dw = room[:3 * 65].view(3, 65)[:, 1:]
    else:
        dw = room[1:65]
    dw.copy_(torch.from_numpy(w))
    pos = r.integers(0, 99, size=(2, 9)).astype(np.int32)
    out = torch.empty_like(x)
    kv.kv_norm_rotate(kv.Rotary(frequencies(32), q_norm=dw), torch.from_numpy(pos).cuda(), q=x, q_out=out)
    _against(x, out, w, 32, pos, 64, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,T", [(3, 5), (700, 3), (2, 900)])
def test_sequences_with_gaps_between_them(dtype, B, T):
    """Activations of T + 2 tokens a sequence, of which the first T are taken, into an output with other gaps."""
    r = np.random.default_rng(86)
    x = torch.from_numpy(r.normal(size=(B, T + 2, 4, 64))).to(TORCH[dtype]).cuda()
    room = torch.full((B, T + 1, 4, 64), 7.0, dtype=x.dtype, device="cuda")
    pos = r.integers(0, 5000, size=(B, T)).astype(np.int32)
    kv.kv_norm_rotate(kv.Rotary(frequencies(64)), torch.from_numpy(pos).cuda(), q=x[:, :T], q_out=room[:, :T])
    _against(x[:, :T].contiguous(), room[:, :T].contiguous(), None, 64, pos, 64, dtype)
    assert (room[:, T] == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_queue_of_appends_and_attention(dtype):
    """Ten chunks of a prompt queued without a wait between them, against the whole prompt at once."""
    Hq, Hkv, d, n = 4, 2, 64, 500
    r = np.random.default_rng(87)
    rows = lambda H: torch.from_numpy(r.normal(size=(n, H, d))).to(TORCH[dtype]).cuda()
    q, k, v = rows(Hq), rows(Hkv), rows(Hkv)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rot, slot = kv.Rotary(frequencies(64)), i32(0)

    def start():
        c = kv.KVCache.allocate(40, Hkv, 16, d, 1, 34, TORCH[dtype])
        c.page_table[0] = torch.from_numpy(r.permutation(40)[:34].astype(np.int32))
        return c

    whole, parts = start(), start()
    qt, want, got = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    kv.kv_append(whole, slot, i32(0, n), k, v, err, rotary=rot, q=q, q_out=qt)
    kv.kv_prompt_attention(whole, slot, i32(0, n), qt, want, err, kv.kv_prompt_workspace(whole, 1, q))
    ws, cu = kv.kv_prompt_workspace(parts, 1, q), i32(0, 50)
    torch.cuda.synchronize()
    for a in range(0, n, 50):
        x = q[a:a + 50].clone()
        kv.kv_append(parts, slot, cu, k[a:a + 50], v[a:a + 50], err, rotary=rot, q=x, q_out=x)  # (in place)
        kv.kv_prompt_attention(parts, slot, cu, x, got[a:a + 50], err, ws)
    assert int(err.item()) == 0 and int(parts.lengths[0]) == n
    pages = [c.page_table[0, :32].long() for c in (whole, parts)]
    assert torch.equal(whole.k[pages[0]], parts.k[pages[1]]) and torch.equal(whole.stamps[pages[0]], parts.stamps[pages[1]])
    # each side is within the bound of the same definition
    table, cu_n = whole.page_table.cpu().numpy(), np.array([0, n])
    out, lse, mag, smag = ref.prompt_attention(host(whole.k), host(whole.v), table, np.array([n]), np.array([0]), cu_n,
                                               host(qt), 1.0 / 8)
    bound = ref.out_bound(mag, smag, d, dtype)
    assert (np.abs(host(want) - out) <= bound).all() and (np.abs(host(got) - out) <= bound).all()
