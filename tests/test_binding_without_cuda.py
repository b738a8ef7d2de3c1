"""The binding over a torch without CUDA: it imports, its host calls run, and calls on tensors
say what they need.  (Such a build lacks torch's CUDA functions; here they are taken away.)"""
import subprocess
import sys

from conftest import ROOT

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import bit_rotated_kv_tq_b200 as tq
assert tq.lloyd_max_table(128).shape == (16,) and tq.record_bytes(64) == 1184
assert tq.decode_weights_workspace_bytes(1, 8, 128, 256) > 0
c = tq.Cache(1, 2, 128, data=torch.zeros((1, 2, tq.record_bytes(128)), dtype=torch.uint8))
w, lens = torch.zeros((1, 2, 16)), torch.zeros(1, dtype=torch.int32)
bt, q = torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 4, 128), dtype=torch.bfloat16)
for call in (lambda: tq.evict_select(w, lens, 16, 8), lambda: tq.decode_attention(q, c, bt, lens, 16, 0.1),
             lambda: tq.decode_attention_weights(q, c, bt, lens, 16, 0.1, w), lambda: tq.dequantize(c, bt, lens, 16)):
    try:
        call()
    except ValueError as e:
        assert "must be a CUDA tensor" in str(e), e
    else:
        raise AssertionError("not refused")
print("ok")
"""


def test_binding_without_cuda():
    p = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "ok", p.stderr
