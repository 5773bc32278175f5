"""Calls from host threads other than the main one: as a thread's first CUDA call, which finds no context, and from two at once."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import gated_deltanet_linear_mtp_gb300 as gdn
from test_gpu_kv4 import I32, attend

pytestmark = pytest.mark.gpu


def in_thread(call):
    """call() in a thread that has made no CUDA call."""
    failed = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed


@pytest.mark.parametrize("T", [1, 40])
def test_attention_as_a_threads_first_call(T):
    r = attend(np.random.default_rng(T), [T, T], [T + 200, T], 4, 2, 128, 64, cu=False)
    tables, kv, ws = torch.tensor(r["tables"], **I32), torch.tensor(r["kvlens"], **I32), gdn.kv4_attention_workspace(2, T, 4, 2, 128)
    o = torch.full_like(r["o"], 9.0)
    in_thread(lambda: gdn.gdn_kv4_attention(r["q"], r["cache"], tables, kv, o, ws))
    assert torch.equal(o, r["o"])


class InProj:
    """A call of gdn_in_proj_conv on B rows, and its outputs from the main thread."""

    def __init__(self, B):
        H, HK, HV, DK, DV, K = 256, 1, 2, 64, 64, 4
        key, val = HK * DK, HV * DV
        g = torch.Generator(device="cuda").manual_seed(B)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.x = torch.randn((B, 1, H), generator=g, device="cuda").bfloat16()
        self.W = (torch.randn((2 * key + 2 * val + 2 * HV, H), generator=g, device="cuda") / 16).bfloat16()
        self.w = torch.randn((2 * key + val, K), generator=g, device="cuda")
        self.bias, self.idx = torch.zeros(2 * key + val, device="cuda"), torch.arange(B, **I32)
        self.state = torch.zeros((B, K - 1, 2 * key + val), **bf)

        def outputs():
            shapes = ((HK, DK), (HK, DK), (HV, DV), (HV, DV), (HV,), (HV,))
            return gdn.InProjOut(*(torch.zeros((B, 1, *n), **bf) for n in shapes)), torch.zeros((B, 1, 2 * key + val), **bf)

        self.want, self.got = outputs(), outputs()
        self.call(self.want)

    def call(self, out=None):
        out, records = out or self.got
        gdn.gdn_in_proj_conv(self.x, self.W, self.w, self.bias, self.state, self.idx, out, False, records)

    def same(self):
        return torch.equal(self.want[1], self.got[1]) and all(torch.equal(getattr(self.want[0], n), getattr(self.got[0], n)) for n in "qkvzba")


def test_in_proj_conv_as_a_threads_first_call():
    a = InProj(8)
    in_thread(a.call)
    assert a.same()


def test_in_proj_conv_of_two_row_counts_from_two_threads(monkeypatch):
    """8 rows and 64, whose rings differ: a kernel's limit of shared memory belongs to all threads, so neither may lower it
    between the other's setting and launch.  The binding marshals each call once; the threads repeat it."""
    failed, start, streams = [], threading.Barrier(2), [torch.cuda.Stream() for _ in range(2)]
    a, made = [InProj(8), InProj(64)], []
    with monkeypatch.context() as m:
        m.setattr(gdn, "_launch", lambda device, stream, fn, args, what: made.append((fn, args)))
        for x in a:
            x.call()
    torch.cuda.synchronize()

    def work(i):
        fn, args = made[i]
        s = ctypes.c_void_p(streams[i].cuda_stream)
        start.wait()
        for n in range(20000):
            status = fn(*args, s)
            if status != 0:
                failed.append((i, n, status, gdn.lib().gdn_last_cuda_error()))
                break

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and all(x.same() for x in a), failed
