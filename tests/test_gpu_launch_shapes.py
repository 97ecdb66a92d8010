"""The launches that calls make, read from a captured graph: which kernel, on how
many CTAs of how many threads."""
import ctypes
import re
import subprocess

import numpy as np
import pytest

from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


class _KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launches(call):
    """[(kernel's name, CTAs, threads per CTA)] of call(stream), which runs once captured
    and never replayed."""
    torch = _torch()
    cu = ctypes.CDLL("libcuda.so.1")

    def ok(status):
        assert status == 0, status

    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    ok(cu.cuStreamBeginCapture_v2(handle, 2))
    try:
        call(stream)
    finally:
        ok(cu.cuStreamEndCapture(handle, ctypes.byref(graph)))
    n = ctypes.c_size_t(0)
    ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
    nodes = (ctypes.c_void_p * max(n.value, 1))()
    ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
    found = []
    for node in nodes[:n.value]:
        kind, p, name = ctypes.c_int(), _KernelNode(), ctypes.c_char_p()
        ok(cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)))
        assert kind.value == 0                                     # kernels only
        ok(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)))
        if p.func:
            ok(cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)))
        else:
            ok(cu.cuKernelGetName(ctypes.byref(name), ctypes.c_void_p(p.kern)))
        full = subprocess.run(["c++filt", name.value.decode()], capture_output=True, text=True).stdout
        full = full.replace("photon::", "").replace("(anonymous namespace)::", "").replace("void ", "")
        found.append((full.split("(DecodeArgs")[0].split("(NormRopeArgs")[0].split("(photon")[0].strip(),
                      int(np.prod(list(p.grid))), int(np.prod(list(p.block)))))
    ok(cu.cuGraphDestroy(graph))
    return found


@pytest.mark.parametrize("d,per_sm", [(64, 2), (128, 1)])
def test_tiles_of_the_8_bit_write(d, per_sm):
    """A tile's tokens are the fewest, of 1, 2, 4, 8 and 16, whose whole tiles do not outnumber
    the resident CTAs; each CTA has a tile, and one may have a ragged second one."""
    torch = _torch()
    pk = ensure_built()
    room = torch.cuda.get_device_properties(0).multi_processor_count * per_sm
    for T in (1, room - 1, room, room + 1, 2 * room - 1, 2 * room, 2 * room + 1, 2 * room + 2, 4 * room + 3, 8 * room + 7, 8 * room + 8,
              16 * room, 16 * room + 15, 16 * room + 16, 40 * room):
        k = torch.zeros(T, 1, d, dtype=torch.bfloat16, device="cuda")
        pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda")
        pool = torch.zeros(-(-T // 16), 1, 32 * d + 16, dtype=torch.uint8, device="cuda")
        (name, ctas, threads), = launches(lambda st: pk.photon_kv_cache_write_int8(k, k, pos, slots, pool, 1e4, stream=st))
        tile = next(n for n in (1, 2, 4, 8, 16) if T // n <= room or n == 16)
        assert re.match(r"kv_cache_write_int8_kernel<BF16Tag, %d, false>" % d, name) and threads == 256
        assert ctas == min(room, -(-T // tile)), T


