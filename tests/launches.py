"""What a call launches, read from a graph that it is captured into (nothing runs)."""
import ctypes

import torch


class _Params(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


class _Attribute(ctypes.Structure):  # CUlaunchAttribute
    _fields_ = [("id", ctypes.c_int), ("pad", ctypes.c_int), ("value", ctypes.c_uint * 16)]


class _Config(ctypes.Structure):  # CUlaunchConfig
    _fields_ = [("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint), ("stream", ctypes.c_void_p),
                ("attrs", ctypes.POINTER(_Attribute)), ("count", ctypes.c_uint)]


_CLUSTER = 4  # CU_LAUNCH_ATTRIBUTE_CLUSTER_DIMENSION


def kernels(call):
    """The kernels that ``call`` launches, in order of the graph's nodes: dicts of name, grid (CTAs in x, y, z),
    cluster (CTAs of one) and resident (CTAs that the device holds at once, in whole clusters)."""
    cuda = ctypes.CDLL("libcuda.so.1")

    def ask(name, *args):
        rc = getattr(cuda, name)(*args)
        assert rc == 0, (name, rc)

    graph = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = call()
    del out
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    ask("cuGraphGetNodes", raw, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    ask("cuGraphGetNodes", raw, nodes, ctypes.byref(n))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    found = []
    for node in nodes:
        node, kind = ctypes.c_void_p(node), ctypes.c_int()
        ask("cuGraphNodeGetType", node, ctypes.byref(kind))
        if kind.value != 0:  # CU_GRAPH_NODE_TYPE_KERNEL
            continue
        p, attr, func = _Params(), _Attribute(), ctypes.c_void_p()
        ask("cuGraphKernelNodeGetParams_v2", node, ctypes.byref(p))
        func.value = p.func
        if p.kern:
            ask("cuKernelGetFunction", ctypes.byref(func), ctypes.c_void_p(p.kern))
        name = ctypes.c_char_p()
        ask("cuFuncGetName", ctypes.byref(name), func)
        value = (ctypes.c_uint * 16)()
        ask("cuGraphKernelNodeGetAttribute", node, _CLUSTER, ctypes.byref(value))
        cluster, held = max(1, value[0]) * max(1, value[1]) * max(1, value[2]), ctypes.c_int()
        threads = p.block[0] * p.block[1] * p.block[2]
        if cluster == 1:
            ask("cuOccupancyMaxActiveBlocksPerMultiprocessor", ctypes.byref(held), func, threads, ctypes.c_size_t(p.shared))
            resident = held.value * sms
        else:
            attr.id, attr.value = _CLUSTER, value
            cfg = _Config(p.grid, p.block, p.shared, None, ctypes.pointer(attr), 1)
            ask("cuOccupancyMaxActiveClusters", ctypes.byref(held), func, ctypes.byref(cfg))
            resident = held.value * cluster
        found.append(dict(name=name.value.decode(), grid=tuple(p.grid), cluster=cluster, resident=resident))
    return found
