"""Calls on several streams and from several host threads (B200): scratch that a call allocates for itself belongs to the
stream it runs on, and threads with workspaces of their own do not disturb one another."""
import ctypes
import threading

import pytest
import torch

from fine_grained_mixture_route_b200 import moe
from fine_grained_mixture_route_b200 import workloads as W

pytestmark = pytest.mark.gpu


class _Recorder:
    """The library, with one entry point replaced by one that launches nothing and keeps its arguments."""

    def __init__(self, lib, name):
        self.lib, self.name, self.args = lib, name, None

    def __getattr__(self, n):
        return self._record if n == self.name else getattr(self.lib, n)

    def _record(self, *args):
        self.args = args
        return moe.MOE_OK


def _check_scratch(rec, where, n, side, call):
    # 2 MB and more: the allocator gives such a buffer a block of its own, and again to the next request of its size
    assert n >= 2 << 20
    torch.cuda.empty_cache()
    kept = call()                                               # outputs stay alive
    p = rec.args[where]
    mine = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert not p <= mine.data_ptr() < p + n and not mine.data_ptr() <= p < mine.data_ptr() + n
    with torch.cuda.stream(side):                               # it went back to the stream that used it
        again = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == p
    del kept
    torch.cuda.synchronize()


def test_norm_backward_scratch_belongs_to_its_stream(monkeypatch):
    rows, d, side = 300, 7168, torch.cuda.Stream()
    s = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    w, r = s[0].clone(), torch.ones(rows, device="cuda")
    rec = _Recorder(moe.lib_handle(), "moe_rmsnorm_backward")
    monkeypatch.setattr(moe, "_lib", lambda: rec)
    n = rec.moe_rmsnorm_backward_workspace_bytes(moe.MOE_BF16, rows, d)
    _check_scratch(rec, 10, n, side, lambda: moe.rmsnorm_backward(s, s, w, r, stream=side))


def test_balance_scratch_belongs_to_its_stream(monkeypatch):
    T, d, E, side = 16384, 256, 64, torch.cuda.Stream()
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    c, counts = x[:E].clone(), torch.zeros(E, dtype=torch.int32, device="cuda")
    shape = moe.make_shape(T, d, E, 64, 4)
    rec = _Recorder(moe.lib_handle(), "moe_balance_stats")
    monkeypatch.setattr(moe, "_lib", lambda: rec)
    n = rec.moe_balance_workspace_bytes(shape)
    _check_scratch(rec, 9, n, side, lambda: moe.balance_stats(shape, x, c, counts, stream=side))


def test_norm_backward_on_a_side_stream():
    rows, d, side = 2000, 2048, torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(0)
    dy, s = (torch.randn(rows, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    rstd = moe.rmsnorm(s, w)["rstd"]
    want = moe.rmsnorm_backward(dy, s, w, rstd)
    n = int(moe.lib_handle().moe_rmsnorm_backward_workspace_bytes(moe.MOE_BF16, rows, d))
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):                                         # the current stream goes on with buffers of the scratch's size
        got = moe.rmsnorm_backward(dy, s, w, rstd, stream=side)
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        side.wait_stream(torch.cuda.current_stream())


def test_few_token_layers_from_two_host_threads():
    # the same kernel with shared memory of two sizes (T and E differ), each thread with a stream and a workspace of its own.
    # The C entry point, without the interpreter's work between calls, so that the threads' calls overlap
    lib, work = moe.lib_handle(), []
    for T, E, k in ((1, 4, 1), (8, 1024, 32)):
        cfg = W.LayerConfig("few", T, 64, E, 32, k, 0, 0, True, torch.bfloat16, "normal_inv_sqrt_d")
        L = W.make_layer(cfg, "cuda", T)
        shape = moe.shape_of(L["x"], L["centroids"], L["routed"], k, None)
        ws = moe.new_few_workspace(shape)
        want = moe.layer_forward_few(shape, L["x"], L["centroids"], L["routed"], None, ws)
        out, stream, w = torch.empty_like(want), torch.cuda.Stream(), moe._weights(L["routed"])
        args = (ctypes.byref(shape), L["x"].data_ptr(), L["centroids"].data_ptr(), None, ctypes.byref(w), None, out.data_ptr(),
                None, None, None, ws.data_ptr(), ws.numel(), stream.cuda_stream)
        work.append(dict(args=args, keep=(shape, L, w), ws=ws, want=want, out=out, stream=stream, status=[]))
    torch.cuda.synchronize()
    go = threading.Barrier(2)

    def run(w):
        go.wait(30)
        w["status"] += [lib.moe_layer_forward_few(*w["args"]) for _ in range(5000)]

    threads = [threading.Thread(target=run, args=(w,)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    for w in work:
        assert len(w["status"]) == 5000 and set(w["status"]) == {moe.MOE_OK}
        assert torch.equal(w["out"], w["want"]) and moe.check_device_error(w["ws"]) == 0
