"""qmv_verify_draft where nothing was drafted: draft and u_accept may be left out."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def q():
    from bit_weight_only_packed_gb300 import build
    build.build()
    from bit_weight_only_packed_gb300 import qmv
    return qmv


def test_refusals(q):
    p, us = torch.full((3, 1, 8), 0.125), torch.rand(3)
    with pytest.raises(ValueError, match="CUDA"):
        q.qmv_verify_draft(p, None, None, None, us)
    with pytest.raises(ValueError, match="u_sample"):
        q.qmv_verify_draft(p, None, None, None, us[:2])
    p = torch.full((3, 3, 8), 0.125)
    d, ua = torch.zeros(3, 2, dtype=torch.int32), torch.rand(3, 2)
    with pytest.raises(ValueError, match="draft"):
        q.qmv_verify_draft(p, None, None, ua, us)
    with pytest.raises(ValueError, match="u_accept"):
        q.qmv_verify_draft(p, None, d, None, us)


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_the_token_is_drawn_from_p(q, given):
    from test_gpu_step import probs, ref_verify
    rng = np.random.default_rng(2)
    p, us = probs(rng, 5, 1, 4099), rng.random(5, dtype=np.float32)
    e = torch.empty(5, 0, device="cuda")
    d, ua, dq = (e.to(torch.int32), e, torch.empty(5, 0, 4099, device="cuda")) if given else (None, None, None)
    tok, acc = q.qmv_verify_draft(torch.from_numpy(p).cuda(), dq, d, ua, torch.from_numpy(us).cuda())
    rt, ra = ref_verify(p, None, np.empty((5, 0), np.int32), None, np.empty((5, 0), np.float32), us)
    assert np.array_equal(tok.cpu().numpy(), rt) and np.array_equal(acc.cpu().numpy(), ra)
