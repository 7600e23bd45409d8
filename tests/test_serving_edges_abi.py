"""Host side of the serving entry points beside test_serving_abi.py: refusals with int64 block tables, the binding's import."""
import os
import subprocess
import sys

import pytest
import torch

from tests.test_serving_abi import ALIAS, ALIGN, BF16, CUDA, NULL, SHAPE, A, L, refused
from w3a3_quantization_online_b200 import rsq


def _plan(ctx=A[0], new=A[1], B=4, tab=A[2], mb=8, bs=64, free=A[3], nf=100, cur=A[4], curo=A[5], cu=A[6], seq=A[7],
          pos=A[8], slots=A[9], T=16):
    return L.kv8_plan_i64(ctx, new, B, tab, mb, bs, free, nf, cur, curo, cu, seq, pos, slots, T, None)


def _attend(q=A[0], ldq=4096, kc=A[1], ks=A[2], vc=A[3], vs=A[4], tab=A[5], mb=8, seq=A[6], cu=A[7], B=4, out=A[8], T=4,
            h=32, kv=8, dh=128, bs=64, nb=16, ws=A[9], wsb=1 << 34):
    return L.kv8_attention_i64(q, ldq, kc, ks, vc, vs, tab, mb, seq, cu, B, 0.1, out, T, h, kv, dh, bs, nb, BF16, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tab=None), NULL), (dict(B=0), SHAPE), (dict(bs=8), SHAPE), (dict(tab=A[2] + 4), ALIGN),
    (dict(seq=A[2] + 4 * 8 * 8 - 4), ALIAS),     # the last half of the last of B x max_blocks 8-byte ids
    (dict(free=A[2]), ALIAS),
])
def test_plan_refuses(kw, want):
    refused(_plan(**kw), want, rsq.launch_count())


@pytest.mark.parametrize("kw,want", [
    (dict(tab=None), NULL), (dict(mb=0), SHAPE), (dict(tab=A[5] + 4), ALIGN), (dict(ws=A[5] + 4 * 8 * 8 - 16), ALIAS),
    (dict(out=A[5]), ALIAS),
])
def test_attention_refuses(kw, want):
    refused(_attend(**kw), want, rsq.launch_count())


def test_valid_calls_reach_the_launch():
    """Without a GPU a call that passes the checks ends with RSQ_ERR_CUDA (never run on fake pointers on a GPU)."""
    if torch.cuda.is_available():
        pytest.skip("would launch on fake pointers")
    assert _plan() == CUDA and _plan(seq=A[2] + 4 * 8 * 8) == CUDA
    assert _attend() == CUDA and _attend(ws=A[5] + 4 * 8 * 8) == CUDA


def test_binding_imports_without_torchs_short_cuts():
    """Builds of torch without CUDA lack them; where only they are gone, the public calls answer instead."""
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from w3a3_quantization_online_b200 import rsq\n"
            "torch.cuda.current_stream = lambda d: type('S', (), {'cuda_stream': 40 + d})\n"
            "assert rsq._raw_stream(2) == 42 and rsq._current_device is torch.cuda.current_device\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
