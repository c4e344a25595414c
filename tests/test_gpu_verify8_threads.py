"""Calls of the 8-bit attention from several host threads at once, each on a stream and with outputs of its own."""
import threading

import pytest
import torch

from speculative_tree_verify_mla_b200 import kdv
from tests import plain8
from tests.test_gpu_verify8 import Run, tree

pytestmark = pytest.mark.gpu


def test_cuda_core_calls_of_different_dims():
    """The kernel's shared memory, and with it the limit that a launch needs, goes by D_c: threads with small and large
    ones launch side by side and none fails."""
    runs = [Run(plain8.Attn(70 + k, [20], [tree(2)], 1, D_c=D_c, D_r=8, q_dtype=t), kdv.KDV_IMPL_SIMT)
            for k, (D_c, t) in enumerate([(512, "f32"), (32, "f32"), (512, "bf16"), (32, "bf16")])]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(runs)), []

    def work(run, stream):
        start.wait()
        for _ in range(4000):
            try:
                run.go(stream)
            except kdv.KdvError as e:
                failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(runs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, (len(failed), failed[0])
    for run in runs:
        run.check()
