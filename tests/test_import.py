"""What importing the package asks of torch."""
import subprocess
import sys

from conftest import ROOT

SCRIPT = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream   # as in a torch built without GPUs
import moe_layer_gating_amd as moe
s = moe.make_shape(16, 256, 8, 2, 256, moe.MOE_INT8)
assert moe.moe_check_shape(s) == 0 and moe.moe_workspace_bytes(s) > 0
class Stream:
    cuda_stream = 77
torch.cuda.current_stream = lambda dev: Stream if dev == 3 else None
assert moe._raw_stream(3) == 77
print("fine")
"""


def test_host_calls_need_no_private_name_of_torch():
    """The binding's short way to the current stream is a name that a torch
    without it need not have: imports and host-only calls work there."""
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr
