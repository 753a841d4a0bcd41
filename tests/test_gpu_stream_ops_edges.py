"""Streaming-block operators on the GPU: ends of the ranges, host threads, autograd and the kernel forms of large calls.

Tolerances are derived as in test_gpu_stream_ops, with u = 2^-24 and an output's rounding of half a step."""
import ctypes
import threading

import numpy as np
import pytest

import oracle
from conformer_speech_recognition_b200 import gam
from test_gpu_stream_ops import (U, _dt, _torch, conv_check, dev, host, inside, linear_check, linear_inputs, norm_check,
                                 normal, scan_call, scan_check, scan_inputs)

pytestmark = pytest.mark.gpu


def test_linear_calls_of_several_threads():
    """The C entry called by host threads with different numbers of rows, each on a stream of its own."""
    torch = _torch()
    n, k, calls = 4104, 6208, 6000                     # just enough weights for the form that sizes its shared memory by the call
    _, _, q, scale, _ = linear_inputs(1, 1, n, k, "bf16", False)
    w, s = dev(gam.gam_quant_linear_pack(q)), dev(scale)
    entry = gam.lib().gam_quant_linear
    jobs = []
    for rows in (1, 8, 1, 8):
        x, _ = normal(np.random.default_rng(rows), rows, k, dtype="bf16")
        jobs.append((x, gam.gam_quant_linear(x, w, s), torch.zeros(rows, n, dtype=x.dtype, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(jobs))

    def work(x, want, y, stream):
        args = (x.data_ptr(), gam.DTYPE_BF16, k, w.data_ptr(), s.data_ptr(), None, 0, len(x), n, k, y.data_ptr(), n,
                ctypes.c_void_p(stream.cuda_stream))
        start.wait()
        for i in range(calls):
            st = entry(*args)
            if st:
                bad.append(st)
            if i % 100 == 99:
                stream.synchronize()

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, f"{len(bad)} of {len(jobs) * calls} calls failed: {gam.STATUS[bad[0]]}"
    for _, want, y, _ in jobs:
        assert torch.equal(y, want)
