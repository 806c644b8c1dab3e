"""Calls of the cache's operators on which tests/test_gpu_kv_waits.py compares the normal library with the build
whose waits run out. Run as a program (python -m tests.kv_stalled CALL NAME FILE, the library named by
GDN_LIBRARY), it leaves a call's results in a file."""
import sys

import numpy as np
import torch

from hybrid_ssm_gated_gb300 import kv
from tests.gpu_util import canaries_intact, guarded
from tests.kv_ref import Case, host

LONG, SHORT = [5000, 20, 1700, 0, 2900, 300], [130 + 17 * i % 171 for i in range(40)]
# of attention: lengths, nodes, query heads (of 8 key heads), head size
ATTENTION = {"shared units, 16 rows": (LONG, 5, 16, 64), "whole units": (SHORT, 5, 16, 128),
             "shared units, 128 rows": (LONG, 20, 48, 64), "whole units, 64 rows, two halves": (SHORT, 5, 64, 256)}


def attention(name: str) -> dict:
    lens, T, Hq, d = ATTENTION[name]
    c = Case(70, "bf16", lens, T=T, Hq=Hq, Hkv=8, d=d, page=64)
    guards = []
    out = guarded(c.q.shape, c.q.dtype, guards).fill_(7.0)
    lse = guarded(c.q.shape[:3], torch.float32, guards).fill_(7.0)
    ws = guarded((kv.kv_tree_workspace(c.cache, c.q).numel(),), torch.uint8, guards).fill_(1)
    kv.kv_tree_attention(c.cache, c.d_slots, c.q, c.kn, c.vn, c.d_mask, out, c.err, ws, num_nodes=c.d_nodes, lse=lse)
    assert canaries_intact(guards)
    return {"out": host(out), "lse": host(lse), "err": int(c.err.item())}


# of accumulation: nodes of the paths, query heads (of 8 key heads), head size
ACCUMULATION = {"one block of rows": (3, 16, 128), "two blocks of rows": (40, 48, 64), "four boxes": (3, 32, 256)}


def accumulation(name: str) -> dict:
    P, Hq, d = ACCUMULATION[name]
    c = Case(71, "bf16", [5000, 60, 1700, 41, 2900, 300], T=P, Hq=Hq, Hkv=8, d=d, page=64)
    guards = []
    c.weights = guarded(c.weights.shape, torch.float32, guards).copy_(c.weights)
    c.sync()
    before = host(c.weights)
    path = torch.arange(P, dtype=torch.int32, device="cuda").repeat(6, 1)
    n = torch.tensor([P, P, P - 1, P, 1, P], dtype=torch.int32, device="cuda")
    kv.kv_accumulate(c.cache, c.d_slots, c.q, torch.full((6, P, Hq), 3.0, device="cuda"), path, n, c.err, decay=0.5)
    assert canaries_intact(guards)
    return {"before": before, "weights": host(c.weights), "err": int(c.err.item())}


CALLS = {"attention": attention, "accumulation": accumulation}

if __name__ == "__main__":
    np.savez(sys.argv[3], **CALLS[sys.argv[1]](sys.argv[2]))
