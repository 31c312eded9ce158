"""A pipeline wait that gives up leaves no gradient that could be taken for one: dH and dW are NaN, and the workspace
says why.  The wait is not made to give up here: while the call's products run, another stream sets the status word
that a wait would have set."""

import time

import pytest
import torch

from test_token_logprobs_gpu import kd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunk,dW_dtype,given", [(1024, torch.float32, False), (1024, torch.bfloat16, False),
                                                  (8192, torch.bfloat16, False), (8192, torch.float32, True),
                                                  (1024, None, False)])
def test_a_timeout_makes_the_gradients_nan(kd, chunk, dW_dtype, given):      # noqa: F811
    from chunked_top_kl_b200 import _abi
    N, d, V = 8192, 2048, 128256
    gen = torch.Generator(device="cuda").manual_seed(1)
    H = torch.randn(N, d, device="cuda", generator=gen).bfloat16()
    W = (torch.randn(V, d, device="cuda", generator=gen) * d ** -0.5).bfloat16()
    y = torch.randint(0, V, (N,), device="cuda", generator=gen)
    y[:500] = -1
    lse, g = torch.full((N,), 12.0, device="cuda"), torch.full((N,), 1.0, device="cuda")
    n = kd.kd_token_logp_backward_workspace_size(N, d, V, chunk, int(dW_dtype == torch.bfloat16))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    status = ws[:8].view(torch.int32)
    one = torch.ones(1, dtype=torch.int32).pin_memory()
    side = torch.cuda.Stream(priority=-1)
    start, done, end = (torch.cuda.Event(enable_timing=True) for _ in range(3))

    def call():
        kw = dict(dW=torch.zeros(V, d, device="cuda"), accumulate_dW=True) if given else dict(dW_dtype=dW_dtype)
        return kd.token_logprobs_backward(H, W, y, lse, g, chunk=chunk, workspace=ws, **kw)
    dH, dW = call()
    assert kd.check(ws) == (_abi.KD_OK, 0) and bool(torch.isfinite(dH).all())
    assert dW is None or bool(torch.isfinite(dW).all())
    for _ in range(10):
        torch.cuda.synchronize()
        start.record()
        dH, dW = call()
        end.record()
        time.sleep(0.002)                                     # the call, of 10 ms and more, has cleared the word
        with torch.cuda.stream(side):
            status[1:].copy_(one, non_blocking=True)
            done.record()
        torch.cuda.synchronize()
        if start.elapsed_time(done) < 0.8 * start.elapsed_time(end):
            break                                             # ... and was still at its products (no pause of the host)
    else:
        pytest.skip("the host never set the word in time")
    assert kd.check(ws)[0] == _abi.KD_ERR_TIMEOUT
    assert bool(torch.isnan(dH).all())
    assert dW is None or bool(torch.isnan(dW).all())
    # the next call on the workspace is a call like any other
    dH, dW = call()
    assert kd.check(ws) == (_abi.KD_OK, 0) and bool(torch.isfinite(dH).all())
    assert dW is None or bool(torch.isfinite(dW).all())
