"""Weights that change between steps, under programmatic launch with early weights:
what is packed two calls before a matvec is what it multiplies by."""
import pytest
import torch

from gpu_util import qmv
from test_gpu_step import BF16, F16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("between", ["norm", "softmax", "verify", "w4"])
@pytest.mark.parametrize("kind", ["w4", "int2"])
def test_weights_packed_before_the_call_before(kind, between):
    q = qmv()
    g = torch.Generator(device="cuda").manual_seed(9)
    N, K = 4096, 2048
    ones = torch.ones(K, device="cuda", dtype=F16)
    x = torch.randint(-2, 3, (1, K), generator=g, device="cuda").to(F16)
    y = torch.zeros(1, K, device="cuda")
    if kind == "w4":
        codes = [torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        scales = torch.ones(N, K // 128, device="cuda", dtype=F16)
        p = q.W4Pack(N, K, 128, F16, False).pack_weights(codes[0], scales)
        ref = [x.double() @ (c.double() - 8).t() for c in codes]
        pack = lambda i, s: q.lib().qmv_w4_pack(p.handle, codes[i].data_ptr(), scales.data_ptr(), None,
                                                p.packed.data_ptr(), s)
        mul = lambda: q.qmv_w4_gemv(p, x)
    else:
        codes = [torch.randint(-2, 2, (N, K), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
        scales = torch.ones(N, K // 32, device="cuda", dtype=F16)
        p = q.Pack(N, K, 2, 32).pack_weights(codes[0], scales)
        ref = [x.double() @ c.double().t() for c in codes]
        pack = lambda i, s: q.lib().qmv_pack_weights(p.handle, codes[i].data_ptr(), scales.data_ptr(),
                                                     p.words.data_ptr(), p.scales.data_ptr(), s)
        mul = lambda: q.qmv_gemv(p, x)
    other = q.W4Pack(64, K, 128, F16, False).pack_weights(codes[0][:64].clone().to(torch.uint8) & 15, torch.ones(64, K // 128, device="cuda", dtype=F16))
    pr, d = torch.full((1, 2, 64), 1 / 64, device="cuda"), torch.zeros(1, 1, device="cuda", dtype=torch.int32)
    u = torch.rand(1, 1, device="cuda")
    call = {"norm": lambda: q.qmv_block_norm(y, x, ones), "softmax": lambda: q.qmv_softmax(x),
            "verify": lambda: q.qmv_verify_draft(pr, None, d, u, u[0]), "w4": lambda: q.qmv_w4_gemv(other, x)}[between]
    st = torch.cuda.current_stream().cuda_stream
    q.qmv_set_pdl(True)
    try:
        outs = []
        for i in range(40):
            assert pack(i & 1, st) == 0
            call()
            outs.append(mul())
        torch.cuda.synchronize()
    finally:
        q.qmv_set_pdl(False)
    # whole numbers below 2 * 15 * 2048: exact
    for i, o in enumerate(outs):
        assert torch.equal(o.double(), ref[i & 1]), i
    assert q.qmv_device_error(clear=True) == 0
