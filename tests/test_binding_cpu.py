"""The layer's own functions reach the library through ctypes: they need no
binding that is built for one torch."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
sys.modules["rotation_bit_ptq_amd._binding"] = None
import rotation_bit_ptq_amd as rbp
assert rbp.packed_row_bytes(256, 4) == 128
assert len(rbp.fit_codebook(256, 4).centroids_f64) == 16
for call in (lambda: rbp.block_norm(None), lambda: rbp.adapter_add(*[None] * 5), lambda: rbp.kv_append(*[None] * 5),
             lambda: rbp.kv_read(*[None] * 3), lambda: rbp.paged_attention(*[None] * 5)):
    try:
        call()
    except ImportError as e:
        assert "__graft_entry__.build()" in str(e)
    else:
        raise AssertionError("no error")
print("fine")
"""

WITH = """
import rotation_bit_ptq_amd as rbp
try:
    rbp.block_norm(None)
except rbp.OrbitError as e:
    assert "x must be a torch tensor" in str(e)
print("fine")
"""


def _run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr


def test_the_layer_without_the_binding():
    _run(WITHOUT)


def test_the_operators_with_it():
    _run(WITH)
