"""The plain-decoding and 8-bit-cache calls at the edges of what they allow:
counts past 32 bits, offsets that overlap, values that are not finite, more
units than thread blocks, and the measured cases' own plain forms."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import speculative_decoding_tree_build_gb300 as tv
import test_gpu_decode_ops as base

pytestmark = pytest.mark.gpu

ROOT = base.ROOT
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def in_a_process(code):
    """A refusal must not end the interpreter, so it is looked at from outside."""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT,
                         env={**os.environ, "PYTHONPATH": ROOT})
    assert out.returncode == 0, (out.returncode, out.stderr[-2000:])
    return out.stdout


@pytest.mark.parametrize("call", ["rope", "read"])
def test_more_rows_than_32_bits_are_refused(call):
    """2^31 rows (8.6 GB) or requests: ValueError, and the process lives on and calls again."""
    said = in_a_process("""
import torch
import speculative_decoding_tree_build_gb300 as tv
n = 2 ** 31
big = torch.empty(n, dtype=torch.int32, device="cuda")
try:
    if %r == "rope":
        q = big.view(torch.bfloat16).view(n, 1, 2)
        tv.rope_axes(tv.rope_axes_geom(1, 0, 2, [1]), q, None, big[None], torch.ones(1, device="cuda"), q, None)
    else:
        pool = torch.zeros(1, 1, 16, 64, dtype=torch.int8, device="cuda")
        scale, out = torch.zeros(1, 1, 16, device="cuda"), torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
        tv.kv_quant_read(tv.geom(1, 1, 64), None, big, big[:, None], big, pool, pool, scale, scale, big[:, None], big,
                         out, out, big)
    print("no error")
except ValueError as e:
    print("refused:", e)
q = torch.ones(1, 1, 2, device="cuda")
tv.rope_axes(tv.rope_axes_geom(1, 0, 2, [1]), q, None, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
             torch.ones(1, device="cuda"), q, None)
print("and again", q.flatten().tolist())
""" % call)
    assert "refused:" in said and "out of range" in said and "and again [1.0, 1.0]" in said
