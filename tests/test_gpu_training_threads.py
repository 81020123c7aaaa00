"""GPU: training calls from several host threads, each on its own stream and tensors."""
import ctypes
import threading

import pytest
import torch

import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_layernorm_from_threads_with_different_sizes():
    """The norm's kernels are shared by sizes with different needs of shared memory: calls with the small need do
    not take the large one's leave away between its set-up and its launch.

    The library is called directly, as a thread of a C program does (ctypes lets the other threads run)."""
    lib = mk.load_library()
    calls, results = 4000, {}
    start = threading.Barrier(4, timeout=60)  # a thread that fails before it ends the others

    def work(i, T, d):
        x, dy = torch.randn((T, d), device=DEV), torch.randn((T, d), device=DEV).to(torch.bfloat16)
        gamma, beta = torch.ones(d, device=DEV), torch.zeros(d, device=DEV)
        y, mean, rstd = mk.mk_moe_layernorm(x, gamma, beta)
        want = mk.mk_moe_layernorm_bwd(dy, x, gamma, mean, rstd)
        dx, dgamma, dbeta = (torch.zeros_like(t) for t in want)
        ws = torch.empty(lib.mk_moe_layernorm_bwd_workspace_size(T, d), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        p = [ctypes.c_void_p(t.data_ptr()) for t in (x, gamma, beta, y, mean, rstd, dy, dx, dgamma, dbeta, ws)]
        x_, g_, b_, y_, m_, r_, dy_, dx_, dg_, db_, ws_ = p
        raw, size = ctypes.c_void_p(s.cuda_stream), ws.numel()
        start.wait()
        bad = 0
        for _ in range(calls):
            bad += lib.mk_moe_layernorm(x_, mk.MK_TYPE_FP32, g_, b_, T, d, 1e-5, y_, m_, r_, raw) != mk.MK_OK
            bad += lib.mk_moe_layernorm_bwd(dy_, x_, mk.MK_TYPE_FP32, g_, m_, r_, None, T, d, dx_, dg_, db_, ws_, size,
                                            raw) != mk.MK_OK
        s.synchronize()
        results[i] = bad, all(torch.equal(a, b) for a, b in zip((dx, dgamma, dbeta), want))

    # both sizes run the same kernels, on rings for 16 and for 12 warps
    threads = [threading.Thread(target=work, args=(i, *((152, 16384) if i % 2 else (1, 12288)))) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert results == {i: (0, True) for i in range(4)}
