"""Calls whose kernels take an amount of shared memory that follows the sizes: a
smaller call, by the same host thread through another path or by another host
thread, never lowers what a larger one was allowed."""
import threading

import pytest
import torch

from gpu_util import qmv

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def in_thread(fn):
    """fn() on a host thread of its own; what it raised, or None."""
    out = []

    def body():
        try:
            torch.cuda.synchronize()
            fn()
            torch.cuda.synchronize()
            out.append(None)
        except Exception as e:
            out.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    return out[0]


def norm(D, lead=0):
    y = torch.randn(2, D + lead, generator=torch.Generator(device="cuda").manual_seed(D), device="cuda").to(BF16)[:, lead:]
    r = torch.full((2, D), 0.5, device="cuda", dtype=BF16)
    return lambda: qmv().qmv_block_norm(y, r, torch.ones(D, device="cuda", dtype=BF16))[1]


def softmax(V):
    x = torch.randn(400, V, generator=torch.Generator(device="cuda").manual_seed(V), device="cuda").to(F16)
    return lambda: qmv().qmv_softmax(x, 0.7)


def pack(K, bits):
    g = torch.Generator(device="cuda").manual_seed(K)
    codes = torch.randint(-2, 2, (64, K), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randn(4, K, generator=g, device="cuda").to(F16)
    return qmv().Pack(64, K, bits, 32).pack_weights(codes, torch.ones(64, K // 32, device="cuda", dtype=F16)), x


def gemv(K, bits=2):
    p, x = pack(K, bits)
    return lambda: qmv().qmv_gemv(p, x[:1])


def small(K):
    p, x = pack(K, 2)
    r, one = torch.zeros(4, K, device="cuda", dtype=F16), torch.ones(K, device="cuda", dtype=F16)
    return lambda: qmv().qmv_fused_rmsnorm_gemv(p, x, r, one)


def chain(K):
    p, x = pack(K, 2)
    y = torch.empty(64, device="cuda")

    def run():
        c = qmv().Chain(1)
        c.add_gemv(p, x[0], y)
        c.run()
        torch.cuda.synchronize()
        return y.clone()

    return run


def test_long_norms_of_one_thread_through_two_paths():
    # 128 KB of h for rows that begin aligned, then 60 KB for rows that do not
    large, less = norm(65536), norm(30000, lead=1)
    ref = large()
    assert bool(torch.isfinite(less()).all())
    assert torch.equal(large(), ref)


@pytest.mark.parametrize("make,large,less", [
    (norm, 65536, 40000), (softmax, 56001, 27001), (gemv, 32768, 8192), (small, 16384 + 64, 8192 + 64),
    (small, 32768, 16384), (chain, 16384, 4096)])
def test_a_smaller_call_on_another_host_thread(make, large, less):
    big, little = make(large), make(less)
    ref = big()
    torch.cuda.synchronize()
    assert in_thread(little) is None
    assert torch.equal(big(), ref)
    assert in_thread(big) is None and in_thread(little) is None
    assert torch.equal(big(), ref)
