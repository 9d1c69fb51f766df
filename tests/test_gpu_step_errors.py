"""What a call leaves behind when the runtime refuses its launch."""
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

# The legacy stream may not be used while a stream that waits for it is captured: the runtime refuses
# the launch (and gives the capture up), so nothing runs on the device.  The runtime keeps
# a thread's last error until it is asked for; one that a call has reported must not come up
# again in the next library's check.
REFUSED = """
import sys; sys.path[:0] = [{root!r}, {root!r} + '/tests']
import ctypes
import torch
from bit_weight_only_packed_gb300 import qmv as q
from test_gpu_step import make_w4, F16
lib, rt = q.lib(), ctypes.CDLL('libcudart.so.13')
p, _, _ = make_w4(64, 256, 128, True, F16, 1)
x = torch.ones(4, 256, device='cuda', dtype=F16)
one = torch.ones(256, device='cuda', dtype=F16)
out, y = torch.empty(4, 256, device='cuda'), torch.empty(4, 64, device='cuda')
h = torch.empty(4, 256, device='cuda', dtype=F16)
tok, acc = torch.empty(1, 2, device='cuda', dtype=torch.int32), torch.empty(1, device='cuda', dtype=torch.int32)
d, u = torch.zeros(1, device='cuda', dtype=torch.int32), torch.zeros(1, device='cuda')
pr = torch.ones(2, 64, device='cuda')
a = lambda t: t.data_ptr()
CALLS = {{
    'softmax': lambda s: lib.qmv_softmax(4, 256, a(x), 256, q.QMV_F16, None, 1.0, a(out), 256, s),
    'norm': lambda s: lib.qmv_block_norm(4, 256, a(x), 256, q.QMV_F16, a(x), 256, None, None, 0, 1.0, 1.0, a(one), 0.0,
                                         1e-6, None, 0, a(h), 256, q.QMV_F16, s),
    'verify': lambda s: lib.qmv_verify_draft(1, 1, 64, a(pr), None, a(d), None, a(u), a(u), a(tok), a(acc), s),
    'w4': lambda s: lib.qmv_w4_gemv(p.handle, 4, a(x), 256, q.QMV_F16, a(y), 64, q.QMV_F32, s),
}}
call = CALLS[{name!r}]
assert call(torch.cuda.current_stream().cuda_stream) == 0
torch.cuda.synchronize()
side, graph = ctypes.c_void_p(), ctypes.c_void_p()
assert rt.cudaStreamCreate(ctypes.byref(side)) == 0             # one that waits for the legacy stream
assert rt.cudaStreamBeginCapture(side, 0) == 0
rc = call(None)
left = rt.cudaPeekAtLastError()
rt.cudaStreamEndCapture(side, ctypes.byref(graph))              # the capture was given up
assert rc == q.QMV_ERR_CUDA and q.qmv_last_cuda_error() != 0, rc
print('left', left)
"""


@pytest.mark.parametrize("name", ["softmax", "norm", "verify", "w4"])
def test_a_refused_launch_leaves_no_error_behind(name):
    r = subprocess.run([sys.executable, "-c", REFUSED.format(root=ROOT, name=name)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "left 0" in r.stdout, r.stdout
