"""Label log-probabilities: the oracle against closed forms and differences,
the schedules, and what the calls refuse (no GPU needed: the refusals come
before any CUDA call)."""

import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle

HERE = os.path.dirname(os.path.abspath(__file__))
P = 1 << 20          # a fake, well aligned device address: never dereferenced here


@pytest.fixture(scope="module")
def kd():
    from chunked_top_kl_b200 import build
    build.build()
    import chunked_top_kl_b200 as k
    return k


def _inputs(seed, N=9, d=5, V=11):
    rng = np.random.default_rng(seed)
    y = rng.integers(0, V, N)
    y[::4] = -100
    return rng.standard_normal((N, d)), rng.standard_normal((V, d)), y, rng.standard_normal(N), rng.standard_normal(N)


@pytest.mark.parametrize("T", [1.0, 0.6])
@pytest.mark.parametrize("ent", [False, True])
def test_oracle_gradient_is_that_of_differences(T, ent):
    H, W, y, g, h = _inputs(1)

    def f(H, W):
        logp, _, e = oracle.token_logprobs(H, W, y, T)
        return float((g * logp).sum() + ((h * e).sum() if ent else 0.0))
    dH, dW, _ = oracle.token_logprobs_grad(H, W, y, g, h if ent else None, T)
    eps = 1e-6
    for X, dX in ((H, dH), (W, dW)):
        for i in np.ndindex(X.shape):
            keep = X[i]
            X[i] = keep + eps
            up = f(H, W)
            X[i] = keep - eps
            down = f(H, W)
            X[i] = keep
            assert abs((up - down) / (2 * eps) - dX[i]) < 1e-7
    assert np.all(dH[y < 0] == 0)


def test_oracle_matches_torch_and_closed_forms():
    H, W, y, _, _ = _inputs(2)
    z = torch.tensor(H @ W.T / 0.8)
    logp, lse, ent = oracle.token_logprobs(H, W, y, 0.8)
    ref = -torch.nn.functional.cross_entropy(z, torch.tensor(y), ignore_index=-100, reduction="none").numpy()
    assert np.allclose(logp, ref, atol=1e-12)
    assert np.allclose(ent[y >= 0], torch.distributions.Categorical(logits=z).entropy().numpy()[y >= 0], atol=1e-12)
    logp, lse, ent = oracle.token_logprobs(H, 0 * W, np.abs(y) % 11)          # W = 0: the uniform distribution
    assert np.allclose(logp, -np.log(11)) and np.allclose(ent, np.log(11)) and np.allclose(lse, np.log(11))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_schedules_stay_in_their_slots(tmp_path):
    exe = tmp_path / "logp_schedule_check"
    subprocess.run(["g++", "-std=c++17", "-O2", "-o", str(exe), os.path.join(HERE, "native", "logp_schedule_check.cpp")],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and out.stdout.startswith("OK"), out.stdout + out.stderr


def test_workspace_sizes(kd):
    f, b = kd.kd_token_logp_forward_workspace_size, kd.kd_token_logp_backward_workspace_size
    assert f(0, 64, 100) > 0 and f(10, 64, 100) > 0
    for bad in ((-1, 64, 100), (1, 60, 100), (1, 0, 100), (1, 64, 0), (1 << 31, 64, 100), (1, 64, 1 << 31)):
        assert f(*bad) == 0 and b(*bad, 128, 0) == 0
    assert b(10, 64, 100, 0, 0) == 0 and b(10, 64, 100, 128, 2) == 0
    # linear in N: the gathered rows, 4 partials of 16 ranges, the token list, labels and their logits, pacing counters
    d = 2048
    per = 2 * d + 4 * 4 * 16 + 12 + 4 * 2 // 8
    assert abs((f(1 << 16, d, 128256) - f(1 << 15, d, 128256)) / (1 << 15) - per) < 0.1
    # one chunk writes a bf16 dW directly; several need an fp32 one
    assert b(4096, d, 128256, 4096, 1) == b(4096, d, 128256, 4096, 0)
    assert b(8192, d, 128256, 4096, 1) - b(8192, d, 128256, 4096, 0) == 4 * 128256 * d


def _fwd(kd, **kw):
    a = dict(H=P, W=P, labels=P, i64=1, N=100, d=64, V=1000, T=1.0, logp=P, lse=P, ent=None, ws=P, nb=1 << 40)
    a.update(kw)
    return kd.kd_token_logp_forward(*a.values(), None)


def _bwd(kd, **kw):
    a = dict(H=P, W=P, labels=P, i64=1, N=100, d=64, V=1000, T=1.0, chunk=128, lse=P, ent=None, dlogp=P, dent=None,
             dH=P, dW=P, half=0, acc=0, ws=P, nb=1 << 40)
    a.update(kw)
    return kd.kd_token_logp_backward(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(H=None), dict(H=P + 8), dict(W=None), dict(W=P + 2), dict(labels=None),
                                 dict(labels=P + 4), dict(i64=2), dict(N=-1), dict(d=0), dict(V=0), dict(T=0.0),
                                 dict(T=-1.0), dict(T=float("nan")), dict(ws=None), dict(ws=P + 128)])
def test_refusals_of_both_passes(kd, bad):
    from chunked_top_kl_b200 import _abi
    assert _fwd(kd, **bad) == _abi.KD_ERR_INVALID_ARG
    assert _bwd(kd, **bad) == _abi.KD_ERR_INVALID_ARG


def test_refusals_of_one_pass(kd):
    from chunked_top_kl_b200 import _abi
    for bad in (dict(logp=None), dict(lse=None), dict(logp=P + 2), dict(ent=P + 1)):
        assert _fwd(kd, **bad) == _abi.KD_ERR_INVALID_ARG
    for bad in (dict(chunk=0), dict(lse=None), dict(dlogp=None), dict(dH=None), dict(dH=P + 8), dict(dW=P + 8),
                dict(dent=P), dict(half=2), dict(half=1, acc=1), dict(dlogp=P + 2)):
        assert _bwd(kd, **bad) == _abi.KD_ERR_INVALID_ARG
    for bad in (dict(d=60), dict(T=1e-7), dict(T=float("inf")), dict(N=1 << 31), dict(V=1 << 31),
                dict(N=(1 << 31) - 1000), dict(V=(1 << 31) - 1000)):
        assert _fwd(kd, **bad) == _abi.KD_ERR_UNSUPPORTED
        assert _bwd(kd, **bad) == _abi.KD_ERR_UNSUPPORTED
    assert _fwd(kd, nb=kd.kd_token_logp_forward_workspace_size(100, 64, 1000) - 1) == _abi.KD_ERR_WORKSPACE
    assert _bwd(kd, nb=kd.kd_token_logp_backward_workspace_size(100, 64, 1000, 128, 0) - 1) == _abi.KD_ERR_WORKSPACE


def test_binding_refuses_cpu_tensors(kd):
    H, W, y = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(9, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        kd.token_logprobs(H, W, y)
