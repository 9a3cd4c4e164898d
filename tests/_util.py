"""Helpers shared by the tests: device transfer and the tolerance check."""
import numpy as np

TOL = 1e-2  # max |y - ref| <= TOL * (1 + |ref|), elementwise (float64 oracle, same dequantized weights)


def to_dev(a, dev="cuda"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def x_to_dev(xbits, dev="cuda"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(xbits).view(np.int16)).to(dev).view(torch.bfloat16)


def y_to_host(Y):
    return Y.float().cpu().numpy().astype(np.float64)


def assert_close(y, ref, what="", extra=None):
    """|y - ref| <= TOL (1 + |ref|) (+ ``extra``, an elementwise allowance derived by the caller)."""
    y = np.asarray(y, np.float64)
    err = np.abs(y - ref)
    lim = TOL * (1 + np.abs(ref))
    if extra is not None:
        lim = lim + extra
    bad = ~(err <= lim)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err / lim, 0)), err.shape)
        raise AssertionError("%s: %d of %d outputs outside tolerance; worst at %s: y=%r ref=%r"
                             % (what, int(bad.sum()), bad.size, i, y[i], ref[i]))
    return float((err / lim).max()) if err.size else 0.0


def kernels_of(graph):
    """Names of the kernels that a captured torch.cuda.CUDAGraph(keep_graph=True) launches, from CUDA's
    graph queries."""
    import ctypes

    cu = ctypes.CDLL("libcuda.so.1")

    class Params(ctypes.Structure):               # CUDA_KERNEL_NODE_PARAMS_v2
        _fields_ = ([("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "smem")]
                    + [(n, ctypes.c_void_p) for n in ("params", "extra", "kern", "ctx")])

    def call(name, *args):
        assert getattr(cu, name)(*args) == 0, name

    g, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    call("cuGraphGetNodes", g, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    call("cuGraphGetNodes", g, nodes, ctypes.byref(n))
    names = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        call("cuGraphNodeGetType", ctypes.c_void_p(node), ctypes.byref(kind))
        if kind.value != 0:
            continue
        p, s = Params(), ctypes.c_char_p()
        call("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node), ctypes.byref(p))
        if p.kern:
            call("cuKernelGetName", ctypes.byref(s), ctypes.c_void_p(p.kern))
        else:
            call("cuFuncGetName", ctypes.byref(s), ctypes.c_void_p(p.func))
        names.append(s.value.decode())
    return names
