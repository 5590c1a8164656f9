"""When and how the package loads its two compiled parts, in processes of their own."""

import subprocess
import sys

import pytest

from conftest import ROOT


@pytest.fixture(scope="module", autouse=True)
def built():
    from fp8_grouped_expert_gb300 import build
    build.build()


def _python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-2000:]
    return r.stdout


def test_importing_loads_no_library():
    # build() may replace both after the import; what is loaded before it would stay
    _python("import fp8_grouped_expert_gb300 as f\n"
            "maps = open('/proc/self/maps').read()\n"
            "assert 'libfge.so' not in maps and '_decode.so' not in maps\n"
            "f.lib()\n"
            "maps = open('/proc/self/maps').read()\n"
            "assert 'libfge.so' in maps and '_decode.so' in maps\n")


def test_a_decode_call_loads_what_it_needs():
    _python("import inspect, fp8_grouped_expert_gb300 as f\n"
            "early = f.kv_cache_read\n"
            "for call in (early, f.kv_cache_read, early):\n"
            "    try:\n"
            "        call(1, 2)\n"
            "        raise SystemExit('not refused')\n"
            "    except f.FgeError as e:\n"
            "        assert 'cache' in str(e), e\n"
            "assert inspect.isbuiltin(f.kv_cache_read) and inspect.isbuiltin(f.moe_layer_decode)\n")


def test_calls_through_ctypes_do_without_the_binding():
    # as where it was built for another torch
    out = _python(
        "import sys, torch\n"
        "sys.modules['fp8_grouped_expert_gb300._decode'] = None     # importing it fails\n"
        "import fp8_grouped_expert_gb300 as f\n"
        "assert f.lib().fge_version() > 0 and f.workspace_bytes(f.OP_MOE_LAYER, 1, 128, 128, 1, 1)\n"
        "x = torch.zeros((1, 128), dtype=torch.bfloat16)\n"
        "for call in (lambda: f.fp8_quant_act(x), lambda: f.moe_layer_decode(1, x),\n"
        "             lambda: f.kv_cache_read(x, None), lambda: f.attention_decode(q=x)):\n"
        "    try:\n"
        "        call()\n"
        "        raise SystemExit('not refused')\n"
        "    except f.FgeError as e:\n"
        "        print(e)\n").splitlines()
    assert "CUDA" in out[0] and len(out) == 4
    assert all("_decode" in line and "torch" in line for line in out[1:])
