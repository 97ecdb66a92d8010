"""The launches that calls make, read from a captured graph: which kernel, on how
many CTAs of how many threads."""
import ctypes
import re
import subprocess

import numpy as np
import pytest

from tests import test_gpu_int8
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
    return [(name, ctas, threads) for name, ctas, threads, _, _ in _captured(call)]


def _captured(call):
    """The same with the shared memory of a CTA and the kernel's handle."""
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
                      int(np.prod(list(p.grid))), int(np.prod(list(p.block))), p.shared, p.func or p.kern))
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


def _decode_launches(pk, B, H, G, d, max_ctx, part, out):
    torch = _torch()
    W = -(-max(max_ctx, 1) // 16)
    n = pk.photon_paged_attention_workspace_size(B, H * G, d, max_ctx, part)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    q = torch.zeros(B, H * G, d, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(B, H * G, d, dtype=out, device="cuda")
    pool = torch.zeros(1, H, 32 * d + 16, dtype=torch.uint8, device="cuda")
    bt, cl = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((B, W), (B,)))
    call = lambda st: pk.photon_paged_attention_decode_int8(q, pool, bt, cl, 0.1, o, max_ctx, part, ws, stream=st)
    call(None)                                                     # sets the kernels' attributes up
    return _captured(call)


# Whole contexts as items, too many for clusters: one piece per row and no merge.
WHOLE_ITEMS = [(320, 1, 4500, 8, 1, 64, 8192, "f32"), (320, 1, 4500, 8, 2, 128, 8192, "bf16"), (64, 1, 6000, 8, 1, 128, 8192, "f32")]


@pytest.mark.parametrize("B,lo,hi,H,G,d,part,out", WHOLE_ITEMS)
def test_whole_contexts_as_items(B, lo, hi, H, G, d, part, out):
    test_gpu_int8.test_decode_grids(B, lo, hi, H, G, d, part, out)


def test_every_launch_shape_of_the_8_bit_decode_is_tested():
    """The batches of test_decode_grids and of WHOLE_ITEMS, and the small ones declared as
    they are and as long, take between them every kernel that the launcher can choose:
    (head_dim, pages of a step, warps of a CTA, pieces by the page stream, how a CTA's warps share items)."""
    torch = _torch()
    pk = ensure_built()
    parameters = lambda test: [m.args[1] for m in test.pytestmark if m.name == "parametrize"]
    batches = []
    for B, lo, hi, H, G, d, part, out in parameters(test_gpu_int8.test_decode_grids)[0] + WHOLE_ITEMS:
        ctx = np.random.default_rng(B + hi).integers(lo, hi + 1, B)
        if B > 2:
            ctx[B // 2], ctx[B // 3] = 0, 1
        batches.append((B, H, G, d, int(max(ctx.max(), 1)), part))
    for ctx, part in test_gpu_int8.CONTEXTS:
        for H, G in parameters(test_gpu_int8.test_decode_matches_the_oracle)[2]:
            for declared in test_gpu_int8.DECLARED:
                batches += [(len(ctx), H, G, d, declared or max(ctx), part) for d in (64, 128)]
    seen = set()
    for batch in batches:
        for out in (torch.bfloat16, torch.float32):
            first, *rest = _decode_launches(pk, *batch, out)
            m = re.fullmatch(r"paged_decode_int8_kernel<(\d+), (\d+), 2, (\d+), \d, (true|false), \(Mode\)(\d)>", first[0])
            d, pages, warps, pieces, mode = (int(x) if x.isdigit() else x == "true" for x in m.groups())
            seen.add((d, pages, warps, pieces, ("warps", "team", "cluster")[mode]))
            # pieces are merged by a second launch, whole rows by none
            assert [n[0].split("<")[0] for n in rest] == (["fp4_merge_kernel"] if pieces else [])
    assert seen == {(64, 2, 8, False, "cluster"), (64, 2, 4, False, "cluster"), (128, 2, 8, False, "cluster"),
                    (128, 2, 4, False, "cluster"), (128, 1, 4, False, "cluster"),
                    (64, 2, 4, True, "team"), (64, 2, 4, False, "team"), (128, 2, 4, True, "team"), (128, 2, 4, False, "team"),
                    (64, 2, 12, True, "warps"), (64, 2, 4, True, "warps"), (64, 2, 4, False, "warps"), (128, 2, 8, True, "warps"),
                    (128, 2, 8, False, "warps")}


class _Attribute(ctypes.Structure):  # CUlaunchAttribute
    _fields_ = [("id", ctypes.c_int), ("pad", ctypes.c_int), ("dim", ctypes.c_uint * 3), ("rest", ctypes.c_char * 52)]


class _Config(ctypes.Structure):  # CUlaunchConfig
    _fields_ = [("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint), ("stream", ctypes.c_void_p),
                ("attrs", ctypes.POINTER(_Attribute)), ("n", ctypes.c_uint)]


def _resident_clusters(func, size, threads, shared):
    attr = _Attribute(id=4, dim=(size, 1, 1))                      # CU_LAUNCH_ATTRIBUTE_CLUSTER_DIMENSION
    cfg = _Config(grid=(size, 1, 1), block=(threads, 1, 1), shared=shared, attrs=ctypes.pointer(attr), n=1)
    n = ctypes.c_int()
    status = ctypes.CDLL("libcuda.so.1").cuOccupancyMaxActiveClusters(ctypes.byref(n), ctypes.c_void_p(func), ctypes.byref(cfg))
    assert status == 0, status
    return n.value


@pytest.mark.parametrize("d", [64, 128])
def test_clusters_of_several_ctas_are_resident_at_once(d):
    """A second round of clusters costs a whole one: 16 pairs of sequence and KV head took 15
    clusters of 8 CTAs and then one more."""
    torch = _torch()
    pk = ensure_built()
    several = 0
    for H in (1, 2, 8):
        for B in list(range(1, 41)) + [75, 76, 80, 147, 152]:
            for max_ctx in (256, 1024, 2048, 4096, 8192):
                (name, ctas, threads, shared, func), *_ = _decode_launches(pk, B, H, 1, d, max_ctx, 64, torch.bfloat16)
                if name.endswith("(Mode)2>") and ctas > B * H:
                    assert B * H <= _resident_clusters(func, ctas // (B * H), threads, shared), (B, H, max_ctx)
                    several += 1
    assert several > 100
