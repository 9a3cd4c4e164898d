"""The workspace contract of the layer entry points: a workspace zeroed once serves calls of
any shape and either kernel, because every call that completes leaves the workspace header
at zero again: the tensor-core kernel's split-K counters (64 KiB) and the decode kernel's
split-K exchange area after them (10 MiB of tagged partial sums, where 0 means "not posted").
Checked after calls whose bands or tiles are split between CTAs (decode split-K,
tensor-core split tiles), with every epilogue, and with one workspace shared by consecutive
calls of different shapes; each output against the float64 oracle, so a counter or a
partial sum left behind (which would make a later call skip, double or mix up a reduction)
shows up as a wrong result too."""
import numpy as np
import pytest

from bit_weight_quantized_wq_gb300 import inputs
from oracle import int4_g128, linear, mxfp4, swiglu
from tests._util import assert_close, to_dev, x_to_dev, y_to_host

pytestmark = pytest.mark.gpu

HEADER = 64 * 1024 + 2 * 160 * 32 * 256 * 4   # counters + the decode exchange area


@pytest.fixture(scope="module")
def B():
    import torch
    from bit_weight_quantized_wq_gb300 import binding
    binding.check_device()
    torch.cuda.init()
    return binding


def _pack(fmt, W):
    return int4_g128.quantize(W) if fmt == "int4_g128" else mxfp4.quantize(W)


def _dev(fmt, pk):
    d = [to_dev(a) for a in pk]
    return d[0], d[1], (d[2] if fmt == "int4_g128" else None)


def _header_zero(ws):
    import torch
    torch.cuda.synchronize()
    head = ws[:HEADER].cpu().numpy()
    return int(np.count_nonzero(head))


# (fmt, M, K, N, entry): decode with bands shared between CTAs (M = 1, 16, 40 -- two row
# slices), the tensor-core kernel with every tile split along K (M = 64) and with a split
# last wave (M = 300).
CASES = [("int4_g128", 1, 4096, 4096, "gemv"), ("mxfp4", 16, 4096, 6144, "gemv"), ("int4_g128", 40, 2048, 3072, "gemv"),
         ("int4_g128", 64, 4096, 256, "tc"), ("mxfp4", 300, 1024, 1024, "tc")]


@pytest.mark.parametrize("fmt,M,K,N,entry", CASES)
def test_counters_back_at_zero_after_a_call(B, fmt, M, K, N, entry):
    import torch
    pk = _pack(fmt, inputs.weights(M + K + N, N, K, 0.05))
    xb, xf = inputs.activations(M * 3 + K, M, K)
    ws = torch.zeros(max(B.gemm_workspace_bytes(fmt, M, K, N), HEADER), dtype=torch.uint8, device="cuda")
    fn = B.gemv_w4a16 if entry == "gemv" else B.gemm_tc_w4a16
    Y = fn(fmt, x_to_dev(xb), *_dev(fmt, pk), workspace=ws)
    assert _header_zero(ws) == 0, "split-K counters or partial sums left non-zero"
    assert_close(y_to_host(Y), linear.linear_w4a16(fmt, xf, *pk), "%s %s M=%d" % (entry, fmt, M))
    assert B.read_error_flags() == 0


def test_one_workspace_across_shapes_and_epilogues(B):
    """Decode, tensor-core, SwiGLU and QKV calls in a row on one workspace, zeroed once."""
    import torch
    calls = [("gemv", "int4_g128", 1, 4096, 4096), ("tc", "int4_g128", 64, 4096, 256), ("gemv", "mxfp4", 16, 4096, 2048),
             ("swiglu", "int4_g128", 4, 4096, 2048), ("qkv", "int4_g128", 300, 1024, 1536), ("gemv", "int4_g128", 1, 4096, 4096)]
    need = max(B.gemm_workspace_bytes(f, M, K, N) for _, f, M, K, N in calls)
    ws = torch.zeros(max(need, HEADER), dtype=torch.uint8, device="cuda")
    for i, (kind, fmt, M, K, N) in enumerate(calls):
        pk = _pack(fmt, inputs.weights(900 + i, N, K, 0.05))
        xb, xf = inputs.activations(950 + i, M, K)
        X = x_to_dev(xb)
        ref = linear.linear_w4a16(fmt, xf, *pk)
        if kind == "gemv":
            got = y_to_host(B.gemv_w4a16(fmt, X, *_dev(fmt, pk), workspace=ws))
            assert_close(got, ref, "call %d" % i)
        elif kind == "tc":
            got = y_to_host(B.gemm_tc_w4a16(fmt, X, *_dev(fmt, pk), workspace=ws))
            assert_close(got, ref, "call %d" % i)
        elif kind == "swiglu":
            # the fused gate+up weight in the interleaved row order; SiLU(gate) * up against
            # the float64 product of the same rows
            d = [B.interleave_gate_up(t) for t in (to_dev(a) for a in pk)]
            got = y_to_host(B.gemv_w4a16_swiglu(fmt, X, d[0], d[1], d[2], workspace=ws))
            assert_close(got, swiglu.swiglu_w4a16(fmt, xf, *pk), "call %d (SwiGLU)" % i)
        else:
            Nkv = (N - 1024) // 2
            q, k, v = B.gemm_w4a16_qkv(fmt, X, *_dev(fmt, pk), Nq=1024, Nkv=Nkv, workspace=ws)
            for t, (lo, hi) in zip((q, k, v), ((0, 1024), (1024, 1024 + Nkv), (1024 + Nkv, N))):
                assert_close(y_to_host(t), ref[:, lo:hi], "call %d (QKV)" % i)
        assert _header_zero(ws) == 0, "call %d left split-K counters or partial sums non-zero" % i
    assert B.read_error_flags() == 0


def test_a_captured_graph_keeps_its_workspace(B):
    """A layer captured in a graph, then a call that needs a larger workspace on the same stream: the
    graph's replay gives the same bits and writes to nothing that was allocated since."""
    import torch
    pk = _pack("int4_g128", inputs.weights(31, 256, 4096, 0.05))
    q, s, z = _dev("int4_g128", pk)
    xb, _ = inputs.activations(32, 2, 4096)
    X = x_to_dev(xb)
    Xl = x_to_dev(inputs.activations(33, 900, 4096)[0])
    small, large = B.gemm_workspace_bytes("int4_g128", 2, 4096, 256), B.gemm_workspace_bytes("int4_g128", 900, 4096, 256)
    assert 0 < small < large
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        want = B.gemm_w4a16("int4_g128", X, q, s, z).clone()
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        got = B.gemm_w4a16("int4_g128", X, q, s, z)
    with torch.cuda.stream(stream):
        B.gemm_w4a16("int4_g128", Xl, q, s, z)
        others = [torch.full(((small + 255) // 256 * 256,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(4)]
    stream.synchronize()
    got.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all((t == 0xA5).all() for t in others)
    assert B.read_error_flags() == 0


def test_a_replaced_workspace_is_given_back_unless_a_capture_took_it(B):
    import weakref
    import torch
    ws = B.Workspace()
    first = weakref.ref(ws.get(4096))
    ws.get(8192)
    assert first() is None
    second = weakref.ref(ws.buf)
    stream = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        ws.get(8192).add_(1)
    ws.get(1 << 20)
    assert second() is not None and ws.buf is not second()


def test_calls_on_a_given_stream_have_scratch_of_their_own(B):
    """stream=...: the workspace kept is that stream's, and what a call allocates for itself is not handed out
    again on the current stream while the call still runs."""
    import torch
    pk = _pack("int4_g128", inputs.weights(41, 256, 4096, 0.05))
    q, s, z = _dev("int4_g128", pk)
    X = x_to_dev(inputs.activations(42, 2, 4096)[0])
    want = B.gemm_w4a16("int4_g128", X, q, s, z)
    W8, sw = B.quantize_fp8_weights(torch.randn(256, 4096, generator=torch.Generator().manual_seed(1)).cuda())
    want8 = B.gemm_w8a8_fp8(X, W8, sw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = B.gemm_w4a16("int4_g128", X, q, s, z, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    kept = {k[1]: w.buf.data_ptr() for k, w in B._default_ws.items() if w.buf is not None}
    assert kept[side.cuda_stream] != kept[torch.cuda.current_stream().cuda_stream]
    y = torch.empty_like(want8)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20000000)                          # the call's kernels wait; its scratch is given up at once
    B.gemm_w8a8_fp8(X, W8, sw, out=y, stream=side)
    size = B.load_library().wq_gemm_w8a8_fp8_workspace_bytes(2, 4096)
    others = [torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(y, want8) and all((t == 0xA5).all() for t in others)
    assert B.read_error_flags() == 0


def test_a_workspace_made_during_a_capture_serves_that_capture_only(B):
    """Its zeros are written when the graph is replayed: another capture, or a call at once, that took it
    would find whatever the memory held."""
    import torch
    ws, stream = B.Workspace(), torch.cuda.Stream()
    taken = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            first, second, larger = ws.get(4096), ws.get(2048), ws.get(8192)
            larger.add_(1)
        assert second.data_ptr() == first.data_ptr() and larger.data_ptr() != first.data_ptr()
        taken.append((g, first.data_ptr(), larger.data_ptr()))
    now = ws.get(4096)
    assert len({p for t in taken for p in t[1:]} | {now.data_ptr()}) == 5 and int(now.count_nonzero()) == 0
    # a layer captured without a call before it, then called at once, then replayed
    q, s, z = _dev("int4_g128", _pack("int4_g128", inputs.weights(51, 256, 4096, 0.05)))
    X = x_to_dev(inputs.activations(52, 2, 4096)[0])
    want = B.gemm_w4a16("int4_g128", X, q, s, z)
    torch.cuda.synchronize()
    fresh, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    B._default_ws.pop((X.get_device(), fresh.cuda_stream), None)
    with torch.cuda.graph(g, stream=fresh):
        y = B.gemm_w4a16("int4_g128", X, q, s, z)
    with torch.cuda.stream(fresh):
        at_once = B.gemm_w4a16("int4_g128", X, q, s, z)
    fresh.synchronize()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(at_once, want) and torch.equal(y, want)
    assert B.read_error_flags() == 0
