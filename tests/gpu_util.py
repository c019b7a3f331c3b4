"""Host <-> device marshalling for the GPU parity tests (no arithmetic here)."""

import ctypes as C

import numpy as np
import torch

DEV = "cuda:0"


def dev_bf16(bits: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def dev_u8(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint8)).to(DEV)


def dev_f32(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.float32))).to(DEV)


def host_bf16_bits(t: torch.Tensor) -> np.ndarray:
    return t.detach().view(torch.int16).cpu().numpy().view(np.uint16)


def host(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().numpy()


def status_word() -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def sample_rows(M: int, tile: int = 128):
    """Rows that touch every M tile: the first and last row of each tile and the ragged tail."""
    rows = set()
    for t0 in range(0, M, tile):
        rows.update({t0, min(M - 1, t0 + tile - 1), min(M - 1, t0 + 37)})
    rows.add(M - 1)
    return sorted(rows)


class _KernelNode(C.Structure):
    """CUDA_KERNEL_NODE_PARAMS of the driver API."""
    _fields_ = [("func", C.c_void_p), ("grid", C.c_uint * 3), ("block", C.c_uint * 3), ("smem", C.c_uint),
                ("params", C.c_void_p), ("extra", C.c_void_p), ("kern", C.c_void_p), ("ctx", C.c_void_p)]


def kernels_of(call):
    """(mangled name, grid, block) of every kernel that `call` launches, in no order: captured, not run."""
    cu = C.CDLL("libcuda.so.1")

    def ok(error):
        assert error == 0, f"driver call failed: {error}"
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw, n = C.c_void_p(graph.raw_cuda_graph()), C.c_size_t(0)
    ok(cu.cuGraphGetNodes(raw, None, C.byref(n)))
    nodes = (C.c_void_p * n.value)()
    ok(cu.cuGraphGetNodes(raw, nodes, C.byref(n)))
    found = []
    for node in map(C.c_void_p, nodes):
        kind, p, name = C.c_int(-1), _KernelNode(), C.c_char_p()
        ok(cu.cuGraphNodeGetType(node, C.byref(kind)))
        if kind.value != 0:  # not a kernel
            continue
        ok(cu.cuGraphKernelNodeGetParams_v2(node, C.byref(p)))
        if p.func:
            ok(cu.cuFuncGetName(C.byref(name), C.c_void_p(p.func)))
        else:
            ok(cu.cuKernelGetName(C.byref(name), C.c_void_p(p.kern)))
        found.append((name.value.decode(), tuple(p.grid), tuple(p.block)))
    return found
