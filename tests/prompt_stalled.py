"""Calls of the prompt attention on which tests/test_gpu_kv_prompt_waits.py compares the normal library with the build
whose waits run out. Run as a program (python -m tests.prompt_stalled NAME FILE, the library named by GDN_LIBRARY), it
leaves a call's results in a file."""
import sys

import numpy as np

from tests.kv_ref import host
from tests.prompt_ref import Prompt

# prompts (rows, entries before them), query and key heads (in odd numbers where ranges are short: the middle one
# then begins inside a unit), head size
CALLS = {"one tile, long units": ([(60, 5000), (3, 9000)], 12, 3, 64),
         "one tile, short units, two halves": ([(300, 10), (200, 0)], 14, 7, 256),
         "two tiles, short units": ([(700, 0), (650, 20)], 64, 8, 128),
         "two tiles, long units": ([(1000, 3000)], 64, 8, 64)}


def call(name: str) -> dict:
    prompts, Hq, Hkv, d = CALLS[name]
    c = Prompt(70, "bf16", prompts, Hq=Hq, Hkv=Hkv, d=d, page=64)
    out, lse = c.attend(fill=1)
    return {"out": host(out), "lse": host(lse), "err": int(c.err.item())}


if __name__ == "__main__":
    np.savez(sys.argv[2], **call(sys.argv[1]))
