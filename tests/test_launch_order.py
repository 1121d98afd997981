"""Kernels that start while the kernel before them still runs (``after_previous`` in
``qsa_launch.cuh``) must not read what that kernel writes through the read-only
path, which is for data that nothing writes while the kernel lives.  Read from the
sources."""

import os
import re

import pytest

from token_indexed_sparse_b200 import build

# the call's own inputs: whole before the first kernel of the chain starts
INPUTS = {"paged_kernel": {"q", "k", "v"}}


def _kernels():
    """(name, parameters, body) of every kernel that waits for the one before it."""
    for f in sorted(os.listdir(build.CSRC)):
        if not f.endswith((".cu", ".cuh")):
            continue
        text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, f)).read())
        for m in re.finditer(r"__global__", text):
            open_at = text.index("{", m.end())
            head, depth, i = text[m.end():open_at], 0, open_at
            while True:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                if depth == 0:
                    break
                i += 1
            body = text[open_at:i + 1]
            if "after_previous()" in body:
                name, params = re.search(r"(\w+)\(((?:[^()]|\([^()]*\))*)\)\s*$", head).groups()
                yield name, params, body


KERNELS = list(_kernels())


def test_the_chains_are_found():
    assert {k[0] for k in KERNELS} == {"paged_kernel", "paged_join_kernel", "causal_join_kernel"}


@pytest.mark.parametrize("name,params,body", KERNELS, ids=[k[0] for k in KERNELS])
def test_no_read_only_loads_of_what_the_chain_writes(name, params, body):
    assert "__ldg" not in body and "__ldcs" not in body and "global.nc" not in body
    read_only = {re.search(r"(\w+)\s*$", p).group(1) for p in params.split(",")
                 if "__restrict__" in p and re.search(r"\bconst\b[^*]*\*", p)}
    assert read_only <= INPUTS.get(name, set())


@pytest.mark.parametrize("name,params,body", KERNELS, ids=[k[0] for k in KERNELS])
def test_nothing_is_read_from_memory_before_the_wait(name, params, body):
    before = body[:body.index("after_previous()")]
    pointers = {re.search(r"(\w+)\s*$", p).group(1) for p in params.split(",") if "*" in p}
    for p in pointers:  # named at most to form an address
        assert not re.search(rf"\b{p}\s*\[|\*\s*{p}\b(?!\s*\))", before), p
