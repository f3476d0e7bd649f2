"""Which stream the buffers of a call belong to when it is given a stream that is
not the current one.  New results come from that stream's memory pool (the block
may otherwise still be in use by earlier work of the current stream), inputs are
kept until the stream is done with them, results until the current stream is, and
everything the call enqueues goes to the given stream.

On the CPU the streams, the pool that an allocation comes from and the C calls are
fakes; the GPU tests put work in the way of a reused block."""
import inspect

import pytest
import torch

import w4a4_gemm_nvfp4_b200 as nv
from w4a4_gemm_nvfp4_b200 import _lib as L


class Stream:
    def __init__(self, name, device):
        self.name, self.device, self.cuda_stream = name, device, len(name)


class Machine:
    """One fake device: the current stream, the pool of each allocation and the
    streams that each tensor's memory is recorded on."""

    def __init__(self, monkeypatch):
        self.device = torch.device("cpu")  # where the fake's tensors are
        self.main, self.side = Stream("main", self.device), Stream("side stream", self.device)
        self.current, self.pool, self.recorded, self.copies, self.calls = self.main, {}, {}, [], []
        machine = self

        class Under:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.before, machine.current = machine.current, self.stream

            def __exit__(self, *exc):
                machine.current = self.before

        empty, new_empty, copy = torch.empty, torch.Tensor.new_empty, torch.Tensor.copy_

        def owned(t):
            self.pool[t.data_ptr()] = self.current
            return t

        def copy_to(t, src):
            self.copies.append(self.current)
            return copy(t, src)

        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch.cuda, "stream", Under)
        monkeypatch.setattr(torch, "empty", lambda *a, **k: owned(empty(*a, **k)))
        monkeypatch.setattr(torch.Tensor, "new_empty", lambda t, *a, **k: owned(new_empty(t, *a, **k)))
        monkeypatch.setattr(torch.Tensor, "copy_", copy_to)
        monkeypatch.setattr(torch.Tensor, "is_cuda", True)
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: self.recorded.setdefault(t.data_ptr(), set()).add(s))
        monkeypatch.setattr(L, "_launch_on", lambda index, stream: (self.stream_of(stream), None))
        for name in ("nvfp4_quantize", "nvfp4_quantize_with_scale", "nvfp4_quantize_arc", "nvfp4_quantize_t",
                     "nvfp4_quantize_arc_rmsnorm", "nvfp4_gemm", "nvfp4_gemm_quantized", "nvfp4_gemm_segmented",
                     "nvfp4_quantize_gemm", "nvfp4_quantize_arc_gemm", "nvfp4_quantize_arc_rmsnorm_gemm"):
            monkeypatch.setattr(L, name, lambda *a: self.calls.append(a[-1]) or 0)
        monkeypatch.setattr(L, "_call", lambda fn, what, switch, *a: self.calls.append(a[-1]))

    def stream_of(self, stream):
        return (stream or self.current).cuda_stream


M, N, K, S = 4, 128, 128, 64


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def operand(rows, k):
    return nv.NVFP4Tensor(torch.zeros(rows, k // 2, dtype=torch.uint8),
                          torch.zeros(nv.nvfp4_scales_bytes(rows, k), dtype=torch.uint8), torch.ones(1),
                          torch.zeros(nv.nvfp4_quantize_workspace_bytes(rows, k), dtype=torch.uint8), rows, k)


def perm(k):
    return torch.arange(k, dtype=torch.int32)


def checkpoint():
    return nv.GatedCheckpoint(torch.zeros(2, M, N, dtype=torch.int8), bf16(2, M, N // 32), M, N, "silu")


CALLS = {
    "gemv": lambda **s: (nv.gemv, (bf16(M, K), operand(N, K)), s),
    "gemv_gated": lambda **s: (nv.gemv_gated, (bf16(M, K), operand(N, K), operand(N, K)), s),
    "gemm_gated": lambda **s: (nv.gemm_gated, (operand(M, K), operand(N, K), operand(N, K)), s),
    "gemm_gated kept": lambda **s: (nv.gemm_gated, (operand(M, K), operand(N, K), operand(N, K)),
                                    dict(checkpoint=True, **s)),
    "gemm_gated into": lambda **s: (nv.gemm_gated, (operand(M, K), operand(N, K), operand(N, K)),
                                    dict(checkpoint=checkpoint(), **s)),
    "gated_backward": lambda **s: (nv.gated_backward, (bf16(M, N), checkpoint()), dict(recompute=True, **s)),
    "quantize": lambda **s: (nv.quantize, (bf16(M, K),), s),
    "quantize with a scale": lambda **s: (nv.quantize, (bf16(M, K),), dict(global_scale=torch.ones(1), **s)),
    "quantize_arc": lambda **s: (nv.quantize_arc, (bf16(M, K), perm(K), S), s),
    "quantize_arc_rmsnorm": lambda **s: (nv.quantize_arc_rmsnorm, (bf16(M, K), bf16(K), 1e-6, perm(K), S), s),
    "quantize_t": lambda **s: (nv.quantize_t, (bf16(64, K),), s),
    "gemm": lambda **s: (nv.gemm, (operand(M, K), operand(N, K)), s),
    "quantize_gemm": lambda **s: (nv.quantize_gemm, (bf16(M, K), operand(N, K)), s),
    "quantize_arc_gemm": lambda **s: (nv.quantize_arc_gemm, (bf16(M, K), perm(K), S, operand(N, K + S)), s),
    "gemm_quantized": lambda **s: (nv.gemm_quantized, (operand(M, K), operand(N, K), torch.ones(1)), s),
    "gemm_segmented": lambda **s: (nv.gemm_segmented, (operand(M, K), operand(N, K), torch.ones(2), (64, N)), s),
}


def tensors(value):
    if isinstance(value, torch.Tensor):
        return [value]
    if isinstance(value, (nv.NVFP4Tensor, nv.GatedCheckpoint)):
        value = list(vars(value).values())
    if isinstance(value, dict):
        value = list(value.values())
    return [t for v in value for t in tensors(v)] if isinstance(value, (list, tuple)) else []


def test_every_call_with_a_stream_is_listed():
    takes = {n for n in dir(nv) if not n.startswith(("_", "nvfp4_")) and inspect.isfunction(getattr(nv, n))
             and "stream" in inspect.signature(getattr(nv, n)).parameters}
    assert takes - {"device_status"} == {c.split()[0] for c in CALLS}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_of_a_call_on_another_stream(name, monkeypatch):
    given = {}
    fn, args, kw = CALLS[name]()
    m = Machine(monkeypatch)
    given = {t.data_ptr() for t in tensors(args) + tensors(kw)}
    result = fn(*args, **kw, stream=m.side)
    new = [t for t in tensors(result) if t.data_ptr() not in given]
    assert m.calls == [m.side.cuda_stream] and m.current is m.main
    assert new and all(m.pool[t.data_ptr()] is m.side for t in new)
    assert all(m.main in m.recorded[t.data_ptr()] for t in new), "kept while the current stream uses them"
    assert all(m.side in m.recorded[p] for p in given), "kept while the given stream reads them"


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_the_current_stream_records_nothing(name, monkeypatch):
    fn, args, kw = CALLS[name]()
    m = Machine(monkeypatch)
    fn(*args, **kw, stream=m.main)
    assert m.calls == [m.main.cuda_stream] and not m.recorded and set(m.pool.values()) <= {m.main}


def test_a_scale_is_copied_on_the_calls_stream(monkeypatch):
    x, out, alpha = bf16(M, K), operand(M, K), torch.ones(1)
    m = Machine(monkeypatch)
    nv.quantize(x, "six", "max", None, out, m.side, alpha)  # (the stream by position)
    assert m.copies == [m.side] and m.calls == [m.side.cuda_stream]


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(name, monkeypatch):
    fn, args, kw = CALLS[name]()
    m = Machine(monkeypatch)
    m.side.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        fn(*args, **kw, stream=m.side)
    assert not m.calls


@pytest.mark.parametrize("name", [n for n in CALLS if n.startswith(("quantize", "gemm")) and "gated" not in n])
def test_a_stream_may_be_any_object_with_a_handle(name, monkeypatch):
    """(The decode and gated calls ask for the stream's device.)"""
    class Handle:
        cuda_stream = 11

    fn, args, kw = CALLS[name]()
    m = Machine(monkeypatch)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle: m.side if handle == m.side.cuda_stream else m.main)
    assert m.side.cuda_stream == Handle.cuda_stream
    fn(*args, **kw, stream=Handle())
    assert m.calls == [m.side.cuda_stream] and set(m.pool.values()) <= {m.side}


# ------------------------------------------------------------- on the GPU --

def weight(rows, k):
    return nv.quantize(torch.randn(rows, k, device="cuda").to(torch.bfloat16))


@pytest.mark.gpu
def test_a_freed_block_that_the_current_stream_still_reads_is_not_given_to_another():
    """The current stream is held up, then reads a block whose tensor is gone by
    the time a call on another stream allocates its result."""
    w, x = weight(4096, 512), torch.randn(16, 512, device="cuda").to(torch.bfloat16)
    ref = nv.gemv(x, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = torch.full((16, 4096), 3.0, dtype=torch.bfloat16, device="cuda")
    seen = torch.empty_like(held)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    seen.copy_(held)
    del held
    results = [nv.gemv(x, w, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert bool((seen == 3.0).all()) and all(torch.equal(y, ref) for y in results)


@pytest.mark.gpu
def test_an_input_dropped_after_the_call_is_kept_for_its_stream():
    """The other stream is held up ahead of the call; by the time it reads, the
    tensors are gone and the current stream has allocated and written blocks of
    their sizes."""
    dh = torch.randn(64, 320, device="cuda").to(torch.bfloat16)
    a, wg, wu = weight(64, 512), weight(320, 512), weight(320, 512)
    h, ck = nv.gemm_gated(a, wg, wu, checkpoint=True)
    ref = nv.gated_backward(dh, ck)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = nv.gated_backward(dh, ck, stream=side)
    shapes = [(t.shape, t.dtype) for t in (ck.codes, ck.scales)]
    del ck
    for _ in range(8):
        for shape, dtype in shapes:
            torch.ones(shape, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(got, ref)


@pytest.mark.gpu
def test_captured_on_a_forked_stream():
    """A capture that forks to another stream and joins it again, results and
    temporaries dropped inside it."""
    a, wg, wu = weight(64, 512), weight(320, 512), weight(320, 512)
    x, dh = (torch.randn(64, n, device="cuda").to(torch.bfloat16) for n in (512, 320))
    side = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        h, ck = nv.gemm_gated(a, wg, wu, checkpoint=True, stream=side)
        dgu = nv.gated_backward(dh, ck, stream=side)
        del ck
        q = nv.quantize(x, stream=side)
        y = nv.gemm(q, wg, stream=side)
        del q
        z = nv.gemv(x[:5], wu, stream=side)
        main.wait_stream(side)
        return h, dgu, y, z

    ref = [t.clone() for t in work()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, ref))
