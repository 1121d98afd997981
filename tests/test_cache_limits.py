"""Sizes at the limits of the paged-cache calls: refused on the host, before any
CUDA work, where the kernels' 32-bit counts would not hold them.  The calls run in a
process of their own, so that one which ends the process fails its test (and those
behind it) only."""

import subprocess
import sys

import pytest
import torch

HEAD = """
import ctypes
from token_indexed_sparse_b200 import qsa
lib, P = qsa.library(), ctypes.c_void_p

def rope(T, H, G):
    rows = [P(4096), 0, 256, P(1 << 50), 0, 256]
    out = [P(4096), H * 256, 256, P(1 << 50), G * 256, 256]
    return lib.qsa_rope(*rows, *out, P(256), P(256), T, H, G, 64, 0, 1.0, 0, None)

def append(T, G, B=1, q=None):
    rows = [P(4096), 0, 256, P(1 << 50), 0, 256, P(q), 0, 256, P(q), 0, 256]
    return lib.qsa_cache_append(*rows, P(256) if q else None, 64, 0, 1.0, P(1 << 31), P(1 << 32), P(256), P(256),
                                P(256), T, B, 4, 16, 3, 12 * G, G, None)
"""


CAUSAL = "lib.qsa_paged_causal(*[P(256)] * 6, 8, {B}, 4, 16, 3, 12, 1, 0, 0, 1.0, *[P(256)] * 3, 1 << 40, None)"
ROUTED = "lib.qsa_paged_forward(*[P(256)] * 7, 8, {B}, 4, 16, 3, 12, 1, 4, 1.0, *[P(256)] * 3, 1 << 40, None)"

# 16 units a head, and 1024 behind them, have to fit 31 bits
HEADS = ["rope(1, 2**28, 0)", "rope(1, 2**28 - 1, 1)", "rope(1, 2**27, 0)", "rope(1, 2**27 - 64, 0)",
         "rope(1, 2**26, 2**26)", "rope(1, 2**31 - 1, 0)", "append(1, 2**27)", "append(1, 2**31 // 14)",
         "append(1, 2**27 // 14)", "append(1, 2**27 // 14, q=1 << 40)"]
# the search for a row's sequence looks up to 31 offsets past B, the plan up to 383
SEQUENCES = [call.format(B=B) for call in ("append(8, 1, {B})", CAUSAL, ROUTED)
             for B in ("2**31 - 1", "2**31 - 384", "2**30 + 1")]


@pytest.fixture(scope="module")
def status():
    from token_indexed_sparse_b200 import build
    build.build()
    code = "".join(f"\nprint('status', {call}, flush=True)" for call in HEADS + SEQUENCES)
    r = subprocess.run([sys.executable, "-c", HEAD + code], capture_output=True, text=True)
    found = [int(line.split()[1]) for line in r.stdout.splitlines() if line.startswith("status")]
    return {call: found[i] if i < len(found) else f"the process ended with {r.returncode}: {r.stderr}"
            for i, call in enumerate(HEADS + SEQUENCES)}


@pytest.mark.parametrize("call", HEADS)
def test_heads_past_the_kernels_counts_are_refused(status, call):
    assert status[call] == 1


@pytest.mark.parametrize("call", SEQUENCES)
def test_more_sequences_than_the_searches_count_are_refused(status, call):
    assert status[call] == 1


@pytest.mark.parametrize("name", ["window", "sinks"])
@pytest.mark.parametrize("value", [2**31, 2**32, 2**32 + 5, -2**31 - 1])
def test_the_binding_refuses_what_32_bits_do_not_hold(status, name, value):
    from token_indexed_sparse_b200 import qsa
    x, i = torch.zeros(2, 12, 256, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(1, 16, 1, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=f"{name} must fit 32 bits"):
        qsa.paged_causal(x, pages, pages, i[None], i[:1], i, **{name: value})
    with pytest.raises(ValueError, match=f"{name} must fit 32 bits"):
        qsa.paged_causal_workspace_size(2, 12, 1, 16, 1, **{name: value})


def test_the_workspace_sizes_refuse_what_32_bits_do_not_hold(status):
    from token_indexed_sparse_b200 import qsa
    for bad in ((2**32 + 12, 1, 4, 16), (12, 2**32 + 1, 4, 16), (12, 1, 2**32 + 4, 16), (12, 1, 4, 2**32 + 16)):
        with pytest.raises(ValueError, match="32 bits"):
            qsa.paged_forward_workspace_size(2, *bad, 3)
    x = torch.zeros(1, 1, 256, dtype=torch.bfloat16).expand(1, 2**32 + 12, 256)
    with pytest.raises(ValueError, match="heads of q must fit 32 bits"):
        qsa.rope(x, None, torch.zeros(1, dtype=torch.int32), torch.ones(8, dtype=torch.float64))


def test_the_status_word_is_the_workspace_s_first_int():
    from token_indexed_sparse_b200 import qsa
    ws = torch.zeros(512, dtype=torch.uint8)
    w = qsa.status_word(ws)
    assert w.dtype == torch.int32 and w.shape == (1,) and w.data_ptr() == ws.data_ptr()
    ws[:4] = torch.tensor([2, 0, 0, 0], dtype=torch.uint8)
    assert w.item() == 2
    for bad in (ws.int(), ws[:2], ws[::2], ws.view(2, 256)):
        with pytest.raises(ValueError, match="workspace"):
            qsa.status_word(bad)
