"""What follows a call on its stream starts when the call is over, even a kernel that is launched to start early
(programmatic dependent launch): no public call's last kernel lets it.

The follower notes the time when it starts and when the wait for its predecessor returns.  A predecessor that lets it
start early runs for milliseconds more; one that does not is over by then."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from test_token_logprobs_gpu import kd  # noqa: F401

pytestmark = pytest.mark.gpu

NVCC = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
SOURCE = r"""
#include <cuda_runtime.h>
__device__ unsigned long long now() { unsigned long long t; asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t)); return t; }
__global__ void follower(unsigned long long* out) {
  out[0] = now();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  out[1] = now();
}
extern "C" int follow(unsigned long long* out, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(1, 1, 1);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, follower, out);
}
"""


@pytest.fixture(scope="module")
def follow(tmp_path_factory):
    if not (os.path.exists(NVCC) or shutil.which("nvcc")):
        pytest.skip("needs nvcc")
    where = tmp_path_factory.mktemp("follower")
    (where / "follower.cu").write_text(SOURCE)
    lib = where / "follower.so"
    subprocess.run([NVCC if os.path.exists(NVCC) else "nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                    "-Xcompiler", "-fPIC", "-o", str(lib), str(where / "follower.cu")], check=True)
    f = ctypes.CDLL(str(lib)).follow
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    return f


N, D, V, K = 2048, 1024, 64000, 16


def _calls(kd):                                                              # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(2)
    H = torch.randn(N, D, device="cuda", generator=gen).bfloat16()
    W = (torch.randn(V, D, device="cuda", generator=gen) * D ** -0.5).bfloat16()
    y = torch.randint(0, V, (N,), device="cuda", generator=gen)
    idx = torch.stack([torch.randperm(V, device="cuda", generator=gen)[:K] for _ in range(16)]).int().repeat(N // 16, 1)
    top = torch.randn(N, K, device="cuda", generator=gen)
    lse, one = torch.full((N,), 12.0, device="cuda"), torch.ones(N, device="cuda")
    long = -torch.rand(1000, 8000, device="cuda", generator=gen)
    few = -torch.rand(4, 1000, device="cuda", generator=gen)
    return {
        "loss forward": lambda: kd.forward(H, W, idx, top),
        "loss backward": lambda: kd.backward(H, W, idx, top, None, 1.0, 4096, lse),
        "loss backward, chunks": lambda: kd.backward(H, W, idx, top, None, 1.0, 700, lse),
        "loss backward, rows skipped": lambda: kd.backward(H, W, idx, top, None, 1.0, 4096, lse, skip_masked_rows=True),
        "loss forward and backward": lambda: kd.forward_backward(H, W, idx, top),
        "teacher top-K": lambda: kd.teacher_topk(H, W, K),
        "logprobs": lambda: kd.token_logprobs_forward(H, W, y, entropy=True),
        "logprobs, few": lambda: kd.token_logprobs_forward(H[:4], W, y[:4]),
        "logprobs backward": lambda: kd.token_logprobs_backward(H, W, y, lse, one),
        "logprobs backward, chunks": lambda: kd.token_logprobs_backward(H, W, y, lse, one, chunk=700, dW_dtype=torch.bfloat16),
        "logprobs backward, dH": lambda: kd.token_logprobs_backward(H, W, y, lse, one, dW_dtype=None),
        "preference": lambda: kd.preference_loss_forward_backward(long, long),
        "preference, few": lambda: kd.preference_loss_forward_backward(few, few),
        "policy": lambda: kd.policy_loss_forward_backward(long, long, long),
        "policy, sequences": lambda: kd.policy_loss_forward_backward(long, long, long, reduce="sequence"),
        "policy, few": lambda: kd.policy_loss_forward_backward(few, few, few),
    }


def test_followers_start_after_the_call(kd, follow):                         # noqa: F811
    early = {}
    for name, call in _calls(kd).items():
        call()
        waits = []
        for _ in range(3):
            out = torch.zeros(2, dtype=torch.int64, device="cuda")
            torch.cuda.synchronize()
            keep = call()
            assert follow(out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
            torch.cuda.synchronize()
            del keep
            started, over = out.tolist()
            assert 0 < started <= over
            waits.append(over - started)
        if min(waits) > 20_000:                    # ns; a wait that has nothing to wait for takes about a thousand
            early[name] = waits
    assert not early
