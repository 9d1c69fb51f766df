"""A chain made by a host thread whose first call to the GPU it is."""
import threading

import pytest
import torch

from gpu_util import qmv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("no_alloc", [False, True])
def test_a_chain_is_made_on_a_fresh_host_thread(no_alloc):
    q = qmv()
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(-2, 2, (64, 4096), generator=g, device="cuda", dtype=torch.int8)
    p = q.Pack(64, 4096, 2, 32).pack_weights(codes, torch.ones(64, 128, device="cuda", dtype=torch.float16))
    x = torch.randint(-2, 3, (4096,), generator=g, device="cuda").half()
    y = torch.zeros(64, device="cuda")
    torch.cuda.synchronize()
    failed = []

    def body():
        try:
            c = q.Chain(1, no_alloc=no_alloc)
            c.add_gemv(p, x, y)
            c.run()
            torch.cuda.synchronize()
        except Exception as e:
            failed.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    assert not failed
    assert torch.equal(y.double(), codes.double() @ x.double())
