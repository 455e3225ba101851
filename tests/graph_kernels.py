"""Which kernels a call launches: the call is captured into a graph, whose nodes name them."""
import ctypes
import re


class _Dim(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint), ("y", ctypes.c_uint), ("z", ctypes.c_uint)]


class _KernelParams(ctypes.Structure):
    """hipKernelNodeParams"""
    _fields_ = [("block", _Dim), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", _Dim),
                ("params", ctypes.c_void_p), ("shared", ctypes.c_uint)]


def _readable(symbol):
    """A kernel of the library with its template arguments, as "k_name<1, 0>"."""
    m = re.match(r"_ZN9bitlinear(\d+)", symbol)
    if not m:
        return symbol
    end = m.end() + int(m.group(1))
    name, args = symbol[m.end():end], re.match(r"I((?:L[a-z]n?\d+E)+)E", symbol[end:])
    if not args:
        return name
    return name + "<" + ", ".join(re.findall(r"L[a-z](n?\d+)E", args.group(1))) + ">"


def kernels(torch, call):
    """Names of the kernels that `call` launches on the current stream, in their order.  The call is not run."""
    hip = ctypes.CDLL("libamdhip64.so")
    hip.hipKernelNameRefByPtr.restype = ctypes.c_char_p
    hip.hipKernelNameRefByPtr.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    raw, count = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert hip.hipGraphGetNodes(raw, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert hip.hipGraphGetNodes(raw, nodes, ctypes.byref(count)) == 0
    names = []
    for node in nodes:
        params = _KernelParams()
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(params)) == 0
        names.append(_readable(hip.hipKernelNameRefByPtr(params.func, None).decode()))
    return names
