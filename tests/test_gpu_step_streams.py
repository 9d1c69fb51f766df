"""Calls on a stream of their own (stream=): fresh results and the inputs' memory
are not used by other work while the call may still read or write them."""
import pytest
import torch

from gpu_util import qmv
from test_gpu_step import BF16, F16, make_w4

pytestmark = pytest.mark.gpu

BUSY = 200_000_000            # cycles, about 0.1 s: work still queued when the call below has long been made


def calls():
    """name -> a call on stream s with fresh results."""
    q = qmv()
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    p, _, _ = make_w4(4096, 1024, 64, True, F16, 5)
    x = rn(64, 1024).to(F16)
    one = torch.ones(1024, device="cuda", dtype=F16)
    pr = torch.softmax(rn(64, 3, 4096), 2)
    d = torch.zeros(64, 2, device="cuda", dtype=torch.int32)
    ua, us = torch.rand(64, 2, device="cuda"), torch.rand(64, device="cuda")
    p2 = q.Pack(4096, 1024, 2, 32).pack_weights(
        torch.randint(-2, 2, (4096, 1024), generator=g, device="cuda", dtype=torch.int8),
        torch.ones(4096, 32, device="cuda", dtype=F16))
    r0 = torch.zeros(64, 1024, device="cuda", dtype=F16)
    return {
        "w4": lambda s: (q.qmv_w4_gemv(p, x, stream=s),),
        "norm": lambda s: q.qmv_block_norm(x, x, one, stream=s),
        "softmax": lambda s: (q.qmv_softmax(x, stream=s),),
        "verify": lambda s: q.qmv_verify_draft(pr, None, d, ua, us, stream=s),
        "unpack": lambda s: (p.unpack_codes(stream=s),),
        "gemv": lambda s: (q.qmv_gemv(p2, x[:1], stream=s),),
        "chunk": lambda s: (q.qmv_gemv(p2, x[:8], stream=s),),
        "fused": lambda s: (q.qmv_fused_rmsnorm_gemv(p2, x[:8], r0[:8], one, stream=s),),
        "unpack2": lambda s: (q.qmv_unpack_codes(p2, stream=s),),
        "argmax": lambda s: q.qmv_gemv_argmax(p2, x[0], q.qmv_argmax_workspace(), stream=s),
    }


@pytest.mark.parametrize("as_int", [False, True])
@pytest.mark.parametrize("name", ["w4", "norm", "softmax", "verify", "unpack", "gemv", "chunk", "fused", "unpack2", "argmax"])
def test_fresh_results_are_not_written_by_work_queued_before(name, as_int):
    # blocks of the results' sizes are freed while the current stream has yet to write them
    call = calls()[name]
    side = torch.cuda.Stream()
    ref = [t.clone() for t in call(None)]
    sizes = [(t.shape, t.dtype) for t in ref]
    torch.cuda.synchronize()
    held = [torch.empty(s, dtype=dt, device="cuda") for s, dt in sizes for _ in range(3)]
    torch.cuda._sleep(BUSY)
    for t in held:
        t.fill_(77)
    del held, t
    out = call(side.cuda_stream if as_int else side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("name", ["softmax", "norm", "w4", "verify"])
def test_inputs_freed_after_the_call_keep_their_memory(name):
    q = qmv()
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(64, 4096, generator=g, device="cuda")
    h = x.to(BF16)
    one = torch.ones(4096, device="cuda", dtype=BF16)
    p, _, _ = make_w4(96, 4096, 64, True, BF16, 6)
    pr = torch.softmax(x.view(32, 2, 4096), 2)
    d, ua, us = torch.zeros(32, 1, device="cuda", dtype=torch.int32), torch.rand(32, 1, device="cuda"), torch.rand(32, device="cuda")
    f = {"softmax": (x, lambda t, s: (q.qmv_softmax(t, stream=s),)),
         "norm": (h, lambda t, s: q.qmv_block_norm(t, h, one, stream=s)),
         "w4": (h, lambda t, s: (q.qmv_w4_gemv(p, t, stream=s),)),
         "verify": (pr, lambda t, s: q.qmv_verify_draft(t, None, d, ua, us, stream=s))}[name]
    side = torch.cuda.Stream()
    ref = [t.clone() for t in f[1](f[0], None)]
    copy = f[0].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    out = f[1](copy, side)
    del copy
    for _ in range(4):
        torch.empty_like(f[0]).fill_(0)       # takes the freed block, if it was given back
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_results_freed_on_their_stream_and_on_the_current_one():
    # a result used on the current stream after a join, freed there, while the current
    # stream still reads it: the next call on the side stream must not be given its memory
    q = qmv()
    x = torch.randn(64, 4096, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    zero = torch.full_like(x, 3.0)
    side, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    y = q.qmv_softmax(x, stream=side)
    cur.wait_stream(side)
    ref = y.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    z = y + 0
    del y
    for _ in range(4):
        q.qmv_softmax(zero, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(z, ref)


def test_streams_of_their_own_in_a_capture():
    # a step whose calls go to a forked stream by stream=, results freed on the way
    q = qmv()
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(5, 1024, generator=g, device="cuda").to(F16)
    one = torch.ones(1024, device="cuda", dtype=F16)
    p, _, _ = make_w4(4099, 1024, 64, True, F16, 8)
    side = torch.cuda.Stream()

    def run(main):
        side.wait_stream(main)
        z = q.qmv_block_norm(x, x, one, stream=side)[1]
        lo = q.qmv_w4_gemv(p, z, stream=side)
        main.wait_stream(side)
        return q.qmv_softmax(lo, 0.7)

    ref = run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    main = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        cap = run(main)
    for _ in range(3):
        cap.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap, ref)


def test_steps_on_several_host_threads_at_once():
    import threading

    from test_gpu_step_edges import case, same
    runs = [case(seed=5 + 45 * i, M=3 + i, V=(4099, 70001, 515)[i]) for i in range(3)]
    ref = [r() for r in runs]
    torch.cuda.synchronize()
    wrong = []

    def body(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(30):
                    out = runs[i]()
                    s.synchronize()
                    if not same(out, ref[i]):
                        wrong.append(i)
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=body, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
