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
