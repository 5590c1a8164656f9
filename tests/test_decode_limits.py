"""Limits of the decode-step calls that hold without a GPU: workspace sizes of shapes that the
calls refuse."""

import subprocess
import sys

import pytest

import fp8_grouped_expert_gb300 as fge
from conftest import ROOT

HEADER = 256


@pytest.fixture(scope="module", autouse=True)
def built():
    from fp8_grouped_expert_gb300 import build
    build.build()
    fge.lib()


def _bytes(op, *args):
    """workspace_bytes in a process of its own: a size must not end it."""
    r = subprocess.run([sys.executable, "-c",
                        "import fp8_grouped_expert_gb300 as f; print(f.workspace_bytes(%s))"
                        % ", ".join(map(str, (op,) + args))],
                       cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    return int(r.stdout)


@pytest.mark.parametrize("heads,n_kv", [(2, 4), (1, 64), (6, 4), (0, 4), (4, 0), (4, -1),
                                        ((1 << 32) + 4, 4)])
def test_heads_that_are_no_groups_need_no_scratch(heads, n_kv):
    for op in (fge.OP_ATTENTION_DECODE, fge.OP_ATTENTION_DECODE_SHARED):
        assert _bytes(op, 2, heads, 128, n_kv) == HEADER


@pytest.mark.parametrize("t,h,inter,e,k", [(65, 256, 128, 8, 2), (1 << 20, 4096, 1536, 128, 8),
                                           (4, 256, 128, 8, 1 << 30), (4, 256, 128, 8, 9),
                                           (4, 1 << 40, 128, 8, 2), (4, 256, 8320, 8, 2),
                                           (4, 256, 128, 513, 2)])
def test_layers_that_are_refused_need_no_scratch(t, h, inter, e, k):
    # the binding allocates a workspace before the call looks at the shape
    assert fge.workspace_bytes(fge.OP_MOE_DECODE, t, h, inter, e, k) == HEADER


def test_batches_that_are_refused_need_no_scratch():
    for op in (fge.OP_ATTENTION_DECODE, fge.OP_ATTENTION_DECODE_SHARED):
        assert fge.workspace_bytes(op, 65537, 16, 128, 4) == HEADER
        assert fge.workspace_bytes(op, 65536, 256, 128, 4) == HEADER
        assert fge.workspace_bytes(op, 65535, 256, 128, 4) > HEADER
