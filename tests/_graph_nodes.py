"""What a call puts into a CUDA graph, by the CUDA driver's C interface: which
kernels in which grids, which memsets."""
import ctypes

import torch

KERNEL, MEMSET = 0, 2       # CUgraphNodeType
RELAXED = 2                 # CUstreamCaptureMode


class _KernelParams(ctypes.Structure):      # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


class Kernel:
    def __init__(self, name, grid, block):
        self.name, self.grid, self.block, self.ints = name, grid, block, ()


def _ok(result):
    assert result == 0, f"CUDA driver error {result}"


def nodes(call, ints=None):
    """Kernels of the graph that ``call()`` is captured in (on the current stream, which it has to use), and the
    number of its memsets.  The graph is not run.  ``ints``: (part of a kernel's name, index of a parameter, count)
    reads the first so many 32-bit integers of that parameter of such kernels."""
    cu = ctypes.CDLL("libcuda.so.1")
    p, ref = ctypes.c_void_p, ctypes.byref
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = p()
    with torch.cuda.stream(s):
        _ok(cu.cuStreamBeginCapture_v2(p(s.cuda_stream), RELAXED))
        try:
            kept = call()       # its tensors live until the capture has ended
        finally:
            ended = cu.cuStreamEndCapture(p(s.cuda_stream), ref(graph))
    _ok(ended)
    del kept
    count = ctypes.c_size_t()
    _ok(cu.cuGraphGetNodes(graph, None, ref(count)))
    array = (p * count.value)()
    _ok(cu.cuGraphGetNodes(graph, array, ref(count)))
    kernels, memsets = [], 0
    for node in array:
        kind = ctypes.c_int()
        _ok(cu.cuGraphNodeGetType(p(node), ref(kind)))
        if kind.value == MEMSET:
            memsets += 1
        elif kind.value == KERNEL:
            k, name = _KernelParams(), ctypes.c_char_p()
            _ok(cu.cuGraphKernelNodeGetParams_v2(p(node), ref(k)))
            if k.func:
                _ok(cu.cuFuncGetName(ref(name), p(k.func)))
            else:
                _ok(cu.cuKernelGetName(ref(name), p(k.kern)))
            kernels.append(Kernel(name.value.decode(), tuple(k.grid), tuple(k.block)))
            if ints is not None and ints[0] in kernels[-1].name:
                params = ctypes.cast(k.params, ctypes.POINTER(p))
                kernels[-1].ints = tuple(ctypes.cast(params[ints[1]], ctypes.POINTER(ctypes.c_int))[:ints[2]])
    _ok(cu.cuGraphDestroy(graph))
    return kernels, memsets
