"""Which instantiations of the library's kernels a call launches, read from a graph that it is captured into. Test
infrastructure."""
import ctypes
import re

import torch


class _Node(ctypes.Structure):   # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("dims", ctypes.c_uint * 7), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launched(call):
    """Names of the kernels with their template arguments, e.g. 'ragged_kernel<true, false, 16, true>'. Nothing runs."""
    cu = ctypes.CDLL("libcuda.so.1")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call()
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    found = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value != 0:   # a kernel
            continue
        p, name = _Node(), ctypes.c_char_p()
        assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        get, handle = (cu.cuFuncGetName, p.func) if p.func else (cu.cuKernelGetName, p.kern)
        assert get(ctypes.byref(name), ctypes.c_void_p(handle)) == 0
        for m in re.finditer(r"(?=(\d\d)([a-z][a-z0-9_]*?_kernel)(?:I((?:L[bi]\d+E)+)E)?)", name.value.decode()):
            if len(m.group(2)) == int(m.group(1)):   # an identifier behind its length
                args = [("false", "true")[int(v)] if t == "b" else v for t, v in re.findall(r"L([bi])(\d+)E", m.group(3) or "")]
                found.append(m.group(2) + ("<%s>" % ", ".join(args) if args else ""))
    return found


def expect(call, name):
    """Runs `call`, which has to launch the kernel `name`."""
    found = launched(call)
    assert name in found, (name, found)
    call()
