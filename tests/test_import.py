"""Importing the binding does not import torch: programs that call the C entry points alone do not wait
for it, and the wrappers look it up when they are called."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def child(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_binding_alone(kvattn):
    child("import sys, numpy as np\n"
          "from kv_cache_decode_02_gb300 import kvattn as K\n"
          "assert 'torch' not in sys.modules\n"
          "plan, lens = K.build_cell_plan([np.arange(5)], 8)\n"
          "assert K.kvattn_rope_table(64, 1e4, 0, 1.0, 0, np.zeros(32, np.uint64)) == 1.0\n"
          "assert K.lib.kvattn_rope(None, 0, 0, None, 0, 0, None, None, 1.0, 0, 0, 0, 128, None, 0, None, 0, None) == 0\n"
          "assert 'torch' not in sys.modules\n")


def test_a_wrapper_as_the_first_call(kvattn):
    child("from kv_cache_decode_02_gb300 import kvattn as K\n"
          "import torch\n"
          "h = lambda *s: torch.zeros(s, dtype=torch.float16)\n"
          "i = torch.arange(4, dtype=torch.int32)\n"
          "calls = [lambda: K.rope(h(4, 4, 128), None, i, K.RopeTable(i, 1.0, 128), q_out=h(4, 4, 128)),\n"
          "         lambda: K.cache_write(h(4, 2, 128), h(4, 2, 128), i, h(9, 2, 128), h(9, 2, 128)),\n"
          "         lambda: K.cache_read(h(9, 2, 128), h(9, 2, 128), i, head_dim=128),\n"
          "         lambda: K.prefill(h(4, 4, 128), h(4, 2, 128), h(4, 2, 128), i[:2]),\n"
          "         lambda: K.prefill_chunk(h(4, 4, 128), i[:2], h(9, 2, 128), h(9, 2, 128), i[:1])]\n"
          "for call in calls:\n"
          "    K._torch = None\n"
          "    try:\n"
          "        call()\n"
          "    except ValueError as e:\n"
          "        assert 'current CUDA device' in str(e), e\n"
          "    else:\n"
          "        raise AssertionError\n")
