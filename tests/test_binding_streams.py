"""The binding's device and stream handles on a torch without its non-public functions for them."""
import subprocess
import sys

PROGRAM = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import encoder_decoder_document_b200 as kalm
class Stream:
    cuda_stream = 77
torch.cuda.current_device = lambda: 0
torch.cuda.current_stream = lambda dev=None: Stream() if dev in (0, 1) else None
assert kalm._stream(None) == 77 and kalm._stream(None, 1) == 77
assert kalm._stream(Stream()) == 77
assert kalm._current_device is not None
print("ok")
"""


def test_public_calls_take_their_place():
    out = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stderr
