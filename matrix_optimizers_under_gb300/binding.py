"""Thin Python binding of libmfsdp.so (the C ABI declared in include/mfsdp.h).

Argument marshalling only: every step of the owner-local optimizer step runs in
the library's CUDA kernels.  Device buffers are torch tensors (PyTorch supplies
device memory and streams); the library never allocates.  Importing this
module raises if the library has not been built -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import List, Optional, Sequence, Tuple

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libmfsdp.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libmfsdp.so is not built ({_LIB_PATH}); run __graft_entry__.build()")
_lib = ctypes.CDLL(_LIB_PATH)

OK = 0
ERR_INVALID_ARG = -1
ERR_MISALIGNED = -2
ERR_OVERLAP = -3
ERR_OUT_OF_BOUNDS = -4
ERR_UNSUPPORTED_DTYPE = -5
ERR_UNSUPPORTED_SHAPE = -6
ERR_WORKSPACE_TOO_SMALL = -7
ERR_CUDA = -8
ERR_DEVICE_TIMEOUT = -9
ERR_IO = -10
ERR_FORMAT = -11

DTYPE_F32 = 0
DTYPE_BF16 = 1
KIND_MATRIX = 0
KIND_TAIL = 1

PHASE_MOMENTUM = 1
PHASE_NEWTON_SCHULZ = 2

EXPORTED = ("mfsdp_plan_owners", "mfsdp_muon_workspace_bytes", "mfsdp_muon_owner_step", "mfsdp_muon_owner_step_phases",
            "mfsdp_muon_device_status", "mfsdp_muon_workspace_layout", "mfsdp_adamw_tail_step",
            "mfsdp_status_string", "mfsdp_version", "mfsdp_muon_owner_step_static_scratch",
            "mfsdp_muon_step_flops", "mfsdp_muon_owner_step_host", "mfsdp_muon_owner_step_apply",
            "mfsdp_model_layout", "mfsdp_placement_segments", "mfsdp_segment_copy", "mfsdp_test_inject_stall",
            "mfsdp_host_step_groups", "mfsdp_muon_static_scratch_status", "mfsdp_checkpoint_bytes",
            "mfsdp_checkpoint_write", "mfsdp_checkpoint_read_header", "mfsdp_checkpoint_read",
            "mfsdp_muon_gram_space_layout", "mfsdp_grad_clip_workspace_bytes", "mfsdp_grad_norm", "mfsdp_grad_clip",
            "mfsdp_sort_ids_workspace_bytes", "mfsdp_sort_ids", "mfsdp_embedding_lookup",
            "mfsdp_embedding_grad_workspace_bytes", "mfsdp_embedding_grad", "mfsdp_expert_workspace_bytes",
            "mfsdp_expert_matmul", "mfsdp_expert_weight_grad", "mfsdp_op_device_status", "mfsdp_adamw_set_step",
            "mfsdp_token_logprob", "mfsdp_token_logprob_grad", "mfsdp_block_norm",
            "mfsdp_block_norm_grad_workspace_bytes", "mfsdp_block_norm_grad")

SEGMENT_REDUCE = 0
SEGMENT_GATHER = 1

SCALE_NONE = 0      # scale = 1
SCALE_MUON = 1      # scale = sqrt(max(1, rows/cols))
SCALE_RMS = 2       # scale = 0.2 * sqrt(max(rows, cols))

STATIC_SCRATCH_BYTES = 64 << 20


class CParam(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("kind", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MatrixShard(ctypes.Structure):
    _fields_ = [("param_id", ctypes.c_int32), ("owner", ctypes.c_int32), ("offset", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("transposed", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("cost", ctypes.c_uint64)]

    def as_dict(self) -> dict:
        return dict(param_id=self.param_id, owner=self.owner, offset=self.offset, rows=self.rows,
                    cols=self.cols, transposed=self.transposed, cost=self.cost)


class TailShard(ctypes.Structure):
    _fields_ = [("param_id", ctypes.c_int32), ("owner", ctypes.c_int32), ("offset", ctypes.c_int64),
                ("numel", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return dict(param_id=self.param_id, owner=self.owner, offset=self.offset, numel=self.numel)


_i32, _i64, _u64, _d, _vp, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_double,
                                  ctypes.c_void_p, ctypes.c_size_t)
_lib.mfsdp_plan_owners.argtypes = [ctypes.POINTER(CParam), _i32, _i32, _i32, _i64, ctypes.POINTER(MatrixShard),
                                   ctypes.POINTER(_i32), ctypes.POINTER(TailShard), ctypes.POINTER(_i32),
                                   ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
_lib.mfsdp_plan_owners.restype = ctypes.c_int
_lib.mfsdp_muon_workspace_bytes.argtypes = [ctypes.POINTER(MatrixShard), _i32]
_lib.mfsdp_muon_workspace_bytes.restype = _sz
_lib.mfsdp_muon_workspace_layout.argtypes = [ctypes.POINTER(MatrixShard), _i32, ctypes.POINTER(_i64)]
_lib.mfsdp_muon_workspace_layout.restype = ctypes.c_int
_lib.mfsdp_muon_gram_space_layout.argtypes = [ctypes.POINTER(MatrixShard), _i32, _i32, ctypes.POINTER(_i64)]
_lib.mfsdp_muon_gram_space_layout.restype = ctypes.c_int
_STEP_ARGS = [ctypes.POINTER(MatrixShard), _i32, _vp, _i32, _vp, _vp, _i32, _i64, _d, _i32, _i32, _d, _d, _d, _d,
              _vp, _sz, _vp]
_lib.mfsdp_muon_owner_step.argtypes = _STEP_ARGS
_lib.mfsdp_muon_owner_step.restype = ctypes.c_int
_lib.mfsdp_muon_owner_step_phases.argtypes = _STEP_ARGS + [_i32]
_lib.mfsdp_muon_owner_step_phases.restype = ctypes.c_int
_lib.mfsdp_muon_owner_step_host.argtypes = [ctypes.POINTER(MatrixShard), _i32, _vp, _vp, _i32, _vp, _vp, _vp, _i32,
                                            _i64, _d, _i32, _i32, _d, _d, _d, _d, _vp, _sz, _i32, _vp]
_lib.mfsdp_muon_owner_step_host.restype = ctypes.c_int
_lib.mfsdp_host_step_groups.argtypes = [ctypes.POINTER(MatrixShard), _i32, _i32, _i32, _i32,
                                        ctypes.POINTER(_i32)]
_lib.mfsdp_host_step_groups.restype = _i32
_lib.mfsdp_muon_owner_step_apply.argtypes = [ctypes.POINTER(MatrixShard), _i32, _vp, _i32, _vp, _vp, _i32, _vp, _i32,
                                             _i64, _d, _i32, _i32, _d, _d, _d, _d, _d, _d, _i32, _vp, _sz, _vp]
_lib.mfsdp_muon_owner_step_apply.restype = ctypes.c_int
_lib.mfsdp_muon_owner_step_static_scratch.argtypes = _STEP_ARGS[:15] + [_vp]
_lib.mfsdp_muon_owner_step_static_scratch.restype = ctypes.c_int
_lib.mfsdp_muon_step_flops.argtypes = [ctypes.POINTER(MatrixShard), _i32, _i32, ctypes.POINTER(_u64),
                                       ctypes.POINTER(_u64)]
_lib.mfsdp_muon_step_flops.restype = ctypes.c_int
_lib.mfsdp_muon_device_status.argtypes = [_vp, _vp, ctypes.POINTER(_i32)]
_lib.mfsdp_muon_device_status.restype = ctypes.c_int
_lib.mfsdp_muon_static_scratch_status.argtypes = [_vp, ctypes.POINTER(_i32)]
_lib.mfsdp_muon_static_scratch_status.restype = ctypes.c_int
_lib.mfsdp_test_inject_stall.argtypes = [_i32]
_lib.mfsdp_test_inject_stall.restype = ctypes.c_int
_lib.mfsdp_adamw_tail_step.argtypes = [_vp, _vp, _vp, _vp, _i64, _d, _d, _d, _d, _d, _i64, _vp]
_lib.mfsdp_adamw_tail_step.restype = ctypes.c_int
_lib.mfsdp_status_string.argtypes = [ctypes.c_int]
_lib.mfsdp_status_string.restype = ctypes.c_char_p
_lib.mfsdp_version.argtypes = []
_lib.mfsdp_version.restype = ctypes.c_char_p


class MfsdpError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


def status_string(status: int) -> str:
    return _lib.mfsdp_status_string(int(status)).decode()


def version() -> str:
    return _lib.mfsdp_version().decode()


def _current_stream() -> int:
    """The current CUDA stream's handle.  Making a torch.cuda.Stream object for it takes 3 us of a call
    that may take 5; torch hands out the plain handle too."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None or not torch.cuda.is_initialized():
        return int(torch.cuda.current_stream().cuda_stream)
    return raw(torch._C._cuda_getDevice())


def _check(status: int, what: str) -> None:
    if status != OK:
        raise MfsdpError(status, what)


@dataclasses.dataclass
class Plan:
    matrix_shards: List[MatrixShard]
    tail_shards: List[TailShard]
    rank_matrix_elems: List[int]
    rank_tail_elems: List[int]

    def rank_matrices(self, r: int) -> List[MatrixShard]:
        return [s for s in self.matrix_shards if s.owner == r]

    def rank_tails(self, r: int) -> List[TailShard]:
        return [s for s in self.tail_shards if s.owner == r]


def plan_owners(params: Sequence[Tuple[int, int, int]], world: int, ns_steps: int = 5,
                align_elems: int = 128) -> Plan:
    """Balance-aware owner plan: params are (rows, cols, kind) in declaration order."""
    n = len(params)
    arr = (CParam * max(n, 1))()
    for i, (r, c, k) in enumerate(params):
        arr[i].rows, arr[i].cols, arr[i].kind = int(r), int(c), int(k)
    nm = sum(1 for p in params if p[2] == KIND_MATRIX)
    nt = n - nm
    out_m = (MatrixShard * max(nm, 1))()
    out_t = (TailShard * max(nt, 1))()
    cm, ct = _i32(0), _i32(0)
    world_i = int(world)
    rme = (_i64 * max(world_i, 1))()
    rte = (_i64 * max(world_i, 1))()
    _check(_lib.mfsdp_plan_owners(arr, n, world_i, int(ns_steps), int(align_elems), out_m, ctypes.byref(cm), out_t,
                                  ctypes.byref(ct), rme, rte), "plan_owners")
    return Plan([out_m[i] for i in range(cm.value)], [out_t[i] for i in range(ct.value)],
                list(rme[:world_i]), list(rte[:world_i]))


def _shard_array(shards: Sequence[MatrixShard]):
    arr = (MatrixShard * max(len(shards), 1))()
    for i, s in enumerate(shards):
        arr[i] = s
    return arr


class Placement(ctypes.Structure):
    _fields_ = [("param_id", ctypes.c_int32), ("owner", ctypes.c_int32), ("offset", ctypes.c_int64),
                ("numel", ctypes.c_int64)]


class Segment(ctypes.Structure):
    _fields_ = [("src_offset", ctypes.c_int64), ("dst_offset", ctypes.c_int64), ("numel", ctypes.c_int64),
                ("src_index", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return dict(src_index=self.src_index, src_offset=self.src_offset, dst_offset=self.dst_offset,
                    numel=self.numel)


def placements(plan: "Plan") -> Tuple[List[Placement], List[Placement]]:
    """The plan's matrix shards and tail shards as placements (param, owner, offset, numel)."""
    def mk(pid, owner, off, n):
        p = Placement()
        p.param_id, p.owner, p.offset, p.numel = pid, owner, off, n
        return p
    return ([mk(s.param_id, s.owner, s.offset, s.rows * s.cols) for s in plan.matrix_shards],
            [mk(s.param_id, s.owner, s.offset, s.numel) for s in plan.tail_shards])


def model_layout(params: Sequence[Tuple[int, int, int]], align_elems: int = 128) -> Tuple[List[int], int]:
    """Offsets of the parameters in the unsharded flat layout, and its extent."""
    n = len(params)
    arr = (CParam * max(n, 1))()
    for i, (r, c, k) in enumerate(params):
        arr[i].rows, arr[i].cols, arr[i].kind = int(r), int(c), int(k)
    offs = (ctypes.c_int64 * max(n, 1))()
    total = ctypes.c_int64(0)
    _check(_lib.mfsdp_model_layout(arr, n, int(align_elems), offs, ctypes.byref(total)), "model_layout")
    return list(offs[:n]), int(total.value)


def model_placements(params: Sequence[Tuple[int, int, int]], align_elems: int = 128) -> List[Placement]:
    """Every parameter in the unsharded layout, as placements with owner 0."""
    offs, _ = model_layout(params, align_elems)
    out = []
    for i, (r, c, _) in enumerate(params):
        p = Placement()
        p.param_id, p.owner, p.offset, p.numel = i, 0, offs[i], r * c
        out.append(p)
    return out


def placement_segments(src: Sequence[Placement], dst: Sequence[Placement], dst_owner: int) -> List[Segment]:
    """Segments that fill dst_owner's buffer of `dst` from `src` (see include/mfsdp.h)."""
    a = (Placement * max(len(src), 1))(*src)
    b = (Placement * max(len(dst), 1))(*dst)
    out = (Segment * max(len(dst), 1))()
    n = ctypes.c_int32(0)
    _check(_lib.mfsdp_placement_segments(a, len(src), b, len(dst), int(dst_owner), out, ctypes.byref(n)),
           "placement_segments")
    return [out[i] for i in range(n.value)]


def segment_copy(srcs, segs: Sequence[Segment], mode: int, dst, stream=None) -> None:
    """REDUCE (sum of all sources in order) or GATHER the segments into dst."""
    n = len(srcs)
    ptrs = (ctypes.c_void_p * max(n, 1))(*[_ptr(t) for t in srcs])
    sizes = (ctypes.c_int64 * max(n, 1))(*[int(t.numel()) for t in srcs])
    arr = (Segment * max(len(segs), 1))(*segs)
    _check(_lib.mfsdp_segment_copy(ptrs, sizes, n, _dtype_code(srcs[0]), arr, len(segs), int(mode), _ptr(dst),
                                   _dtype_code(dst), int(dst.numel()), _stream(stream)), "segment_copy")


def make_shard(offset: int, rows: int, cols: int, param_id: int = 0, owner: int = 0) -> MatrixShard:
    s = MatrixShard()
    s.param_id, s.owner, s.offset, s.rows, s.cols = param_id, owner, offset, rows, cols
    s.transposed = int(rows > cols)
    return s


def muon_workspace_bytes(shards: Sequence[MatrixShard]) -> int:
    return int(_lib.mfsdp_muon_workspace_bytes(_shard_array(shards), len(shards)))


def muon_workspace_layout(shards: Sequence[MatrixShard]) -> List[Tuple[int, ...]]:
    out = (_i64 * max(8 * len(shards), 1))()
    _check(_lib.mfsdp_muon_workspace_layout(_shard_array(shards), len(shards), out), "muon_workspace_layout")
    return [tuple(out[8 * i: 8 * i + 8]) for i in range(len(shards))]


def muon_gram_space_layout(shards: Sequence[MatrixShard], ns_steps: int = 5) -> List[Tuple[int, ...]]:
    """Per shard (1 if the Gram-space form runs else 0, offset of C, of Q_even,
    of Q_odd) for ns_steps (see include/mfsdp.h)."""
    out = (_i64 * max(4 * len(shards), 1))()
    _check(_lib.mfsdp_muon_gram_space_layout(_shard_array(shards), len(shards), int(ns_steps), out),
           "muon_gram_space_layout")
    return [tuple(out[4 * i: 4 * i + 4]) for i in range(len(shards))]


def muon_step_flops(shards: Sequence[MatrixShard], ns_steps: int = 5) -> Tuple[int, int]:
    """(dense, executed) FLOPs of one owner step (see include/mfsdp.h)."""
    dn, ex = _u64(0), _u64(0)
    _check(_lib.mfsdp_muon_step_flops(_shard_array(shards), len(shards), int(ns_steps), ctypes.byref(dn),
                                      ctypes.byref(ex)), "muon_step_flops")
    return int(dn.value), int(ex.value)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_dtype_codes: dict = {}   # torch dtype -> code, filled once torch is there
_id_codes: dict = {}


def _fill_codes() -> None:
    import torch
    _dtype_codes.update({torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16})
    _id_codes.update({torch.int32: ID_I32, torch.int64: ID_I64})


def _dtype_code(t) -> int:
    if not _dtype_codes:
        _fill_codes()
    return _dtype_codes.get(t.dtype, 99)   # 99: rejected by the library as UNSUPPORTED_DTYPE


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    return int(stream) if isinstance(stream, int) else int(stream.cuda_stream)


def muon_owner_step(shards: Sequence[MatrixShard], grad, momentum, update, workspace, *, beta: float = 0.95,
                    nesterov: bool = False, ns_steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315),
                    eps: float = 1e-7, numel: Optional[int] = None, stream=None,
                    phases: int = PHASE_MOMENTUM | PHASE_NEWTON_SCHULZ) -> None:
    """One owner-local Muon step over the shards of one rank (see include/mfsdp.h).

    grad: flat fp32/bf16 CUDA tensor; momentum: flat fp32; update: flat fp32/bf16;
    workspace: CUDA uint8 tensor of at least muon_workspace_bytes(shards) bytes.
    phases: both (default, mfsdp_muon_owner_step) or one of PHASE_MOMENTUM /
    PHASE_NEWTON_SCHULZ (mfsdp_muon_owner_step_phases)."""
    arr = _shard_array(shards)
    n = int(numel if numel is not None else grad.numel())
    a, b, c = coeffs
    args = (arr, len(shards), _ptr(grad), _dtype_code(grad), _ptr(momentum), _ptr(update), _dtype_code(update), n,
            float(beta), int(bool(nesterov)), int(ns_steps), float(a), float(b), float(c), float(eps),
            _ptr(workspace), int(workspace.numel() if workspace is not None else 0), _stream(stream))
    if phases == PHASE_MOMENTUM | PHASE_NEWTON_SCHULZ:
        _check(_lib.mfsdp_muon_owner_step(*args), "muon_owner_step")
    else:
        _check(_lib.mfsdp_muon_owner_step_phases(*args, int(phases)), "muon_owner_step_phases")


def muon_owner_step_apply(shards: Sequence[MatrixShard], grad, momentum, update, weights, workspace, *, lr: float,
                          weight_decay: float = 0.0, scale_mode: int = SCALE_MUON, beta: float = 0.95,
                          nesterov: bool = False, ns_steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315),
                          eps: float = 1e-7, numel: Optional[int] = None, stream=None) -> None:
    """The owner step, then W <- W*(1 - lr*wd) - lr*scale*O fused into the last
    epilogue (see include/mfsdp.h).  update may be None."""
    arr = _shard_array(shards)
    n = int(numel if numel is not None else grad.numel())
    a, b, c = coeffs
    _check(_lib.mfsdp_muon_owner_step_apply(arr, len(shards), _ptr(grad), _dtype_code(grad), _ptr(momentum),
                                            _ptr(update), _dtype_code(update) if update is not None else DTYPE_BF16,
                                            _ptr(weights), _dtype_code(weights), n, float(beta), int(bool(nesterov)),
                                            int(ns_steps), float(a), float(b), float(c), float(eps), float(lr),
                                            float(weight_decay), int(scale_mode), _ptr(workspace),
                                            int(workspace.numel() if workspace is not None else 0), _stream(stream)),
           "muon_owner_step_apply")


def muon_owner_step_host(shards: Sequence[MatrixShard], grad_host, grad_dev, momentum, update_dev, update_host,
                         workspace, *, groups: int = 0, beta: float = 0.95, nesterov: bool = False,
                         ns_steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                         numel: Optional[int] = None, stream=None) -> None:
    """The owner step with the gradient read from and the update written to pinned
    host tensors, the copies of each shard group overlapped with the compute of
    its neighbours (see include/mfsdp.h).  grad_dev/update_dev are device staging
    tensors of the same length.  groups = 0: the count host_step_groups gives."""
    arr = _shard_array(shards)
    n = int(numel if numel is not None else grad_dev.numel())
    a, b, c = coeffs
    _check(_lib.mfsdp_muon_owner_step_host(arr, len(shards), _ptr(grad_host), _ptr(grad_dev), _dtype_code(grad_dev),
                                           _ptr(momentum), _ptr(update_dev), _ptr(update_host), _dtype_code(update_dev),
                                           n, float(beta), int(bool(nesterov)), int(ns_steps), float(a), float(b),
                                           float(c), float(eps), _ptr(workspace),
                                           int(workspace.numel() if workspace is not None else 0), int(groups),
                                           _stream(stream)),
           "muon_owner_step_host")


def host_step_groups(shards: Sequence[MatrixShard], grad_dtype=None, update_dtype=None,
                     groups: int = 0) -> Tuple[int, List[int]]:
    """(number of groups, each shard's group) of the host-buffer step for
    `groups` (0 = the library's choice); host only.  The dtypes are torch
    dtypes, bf16 gradient and update by default."""
    import torch
    g = torch.bfloat16 if grad_dtype is None else grad_dtype
    u = torch.bfloat16 if update_dtype is None else update_dtype
    code = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
    out = (_i32 * max(len(shards), 1))()
    ng = int(_lib.mfsdp_host_step_groups(_shard_array(shards), len(shards), code.get(g, 99), code.get(u, 99),
                                         int(groups), out))
    return ng, [int(out[i]) for i in range(len(shards))] if ng else []


def muon_owner_step_static_scratch(shards: Sequence[MatrixShard], grad, momentum, update, *, beta: float = 0.95,
                                   nesterov: bool = False, ns_steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315),
                                   eps: float = 1e-7, numel: Optional[int] = None, stream=None) -> None:
    """The owner step for callers that cannot allocate device memory: no
    workspace argument; the library's fixed STATIC_SCRATCH_BYTES device array
    serves as scratch (see include/mfsdp.h).  Calls that overlap on the GPU race."""
    arr = _shard_array(shards)
    n = int(numel if numel is not None else grad.numel())
    a, b, c = coeffs
    _check(_lib.mfsdp_muon_owner_step_static_scratch(arr, len(shards), _ptr(grad), _dtype_code(grad), _ptr(momentum),
                                                     _ptr(update), _dtype_code(update), n, float(beta),
                                                     int(bool(nesterov)), int(ns_steps), float(a), float(b), float(c),
                                                     float(eps), _stream(stream)),
           "muon_owner_step_static_scratch")


def test_inject_stall(tile: int) -> None:
    """Testing only: the next Newton-Schulz launch's tile `tile` waits for a
    dependency that is never satisfied, so its bounded wait runs out (see
    include/mfsdp.h)."""
    _check(_lib.mfsdp_test_inject_stall(int(tile)), "test_inject_stall")


def muon_device_status(workspace, stream=None) -> Tuple[int, int]:
    detail = _i32(0)
    st = _lib.mfsdp_muon_device_status(_ptr(workspace), _stream(stream), ctypes.byref(detail))
    return st, detail.value


def muon_static_scratch_status(stream=None) -> Tuple[int, int]:
    """(status, raw word) of the last static-scratch step on the current device
    (synchronises the stream; see include/mfsdp.h)."""
    detail = _i32(0)
    st = _lib.mfsdp_muon_static_scratch_status(_stream(stream), ctypes.byref(detail))
    return st, detail.value


def adamw_tail_step(p, g, m, v, *, lr: float, beta1: float, beta2: float, eps: float, wd: float, step: int,
                    stream=None) -> None:
    """Fused AdamW over one rank's packed fp32 tail (see include/mfsdp.h)."""
    n = int(p.numel())
    _check(_lib.mfsdp_adamw_tail_step(_ptr(p), _ptr(g), _ptr(m), _ptr(v), n, float(lr), float(beta1), float(beta2),
                                      float(eps), float(wd), int(step), _stream(stream)), "adamw_tail_step")


_lib.mfsdp_model_layout.argtypes = [ctypes.POINTER(CParam), _i32, _i64, ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
_lib.mfsdp_model_layout.restype = ctypes.c_int
_lib.mfsdp_placement_segments.argtypes = [ctypes.POINTER(Placement), _i32, ctypes.POINTER(Placement), _i32, _i32,
                                          ctypes.POINTER(Segment), ctypes.POINTER(_i32)]
_lib.mfsdp_placement_segments.restype = ctypes.c_int
_lib.mfsdp_segment_copy.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(_i64), _i32, _i32,
                                    ctypes.POINTER(Segment), _i32, _i32, _vp, _i32, _i64, _vp]
_lib.mfsdp_segment_copy.restype = ctypes.c_int


class CheckpointHeader(ctypes.Structure):
    _fields_ = [("world", ctypes.c_int32), ("rank", ctypes.c_int32), ("ns_steps", ctypes.c_int32),
                ("n_matrix", ctypes.c_int32), ("n_tail", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("align_elems", ctypes.c_int64), ("matrix_elems", ctypes.c_int64), ("tail_elems", ctypes.c_int64),
                ("adam_step", ctypes.c_int64)]


_lib.mfsdp_checkpoint_bytes.argtypes = [ctypes.POINTER(CheckpointHeader)]
_lib.mfsdp_checkpoint_bytes.restype = _sz
_lib.mfsdp_checkpoint_write.argtypes = [ctypes.c_char_p, ctypes.POINTER(CheckpointHeader), ctypes.POINTER(MatrixShard),
                                        ctypes.POINTER(TailShard), _vp, _vp, _vp, _vp]
_lib.mfsdp_checkpoint_write.restype = ctypes.c_int
_lib.mfsdp_checkpoint_read_header.argtypes = [ctypes.c_char_p, ctypes.POINTER(CheckpointHeader)]
_lib.mfsdp_checkpoint_read_header.restype = ctypes.c_int
_lib.mfsdp_checkpoint_read.argtypes = [ctypes.c_char_p, ctypes.POINTER(CheckpointHeader), ctypes.POINTER(MatrixShard),
                                       _i32, ctypes.POINTER(TailShard), _i32, _vp, _i64, _vp, _vp, _vp, _i64]
_lib.mfsdp_checkpoint_read.restype = ctypes.c_int


@dataclasses.dataclass
class Checkpoint:
    """One rank's owner-shard checkpoint: its header, tables and host buffers
    (NumPy float32 arrays)."""
    header: CheckpointHeader
    matrix_shards: List[MatrixShard]
    tail_shards: List[TailShard]
    momentum: "object"
    tail_p: "object"
    tail_m: "object"
    tail_v: "object"


def _host_f32(x, n: int):
    """A C-contiguous float32 NumPy copy of a tensor or array of n elements."""
    import numpy as np
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").numpy()
    a = np.ascontiguousarray(np.asarray(x, dtype=np.float32))
    if a.size != n:
        raise ValueError(f"buffer has {a.size} elements, the header says {n}")
    return a


def checkpoint_save(path: str, world: int, rank: int, ns_steps: int, align_elems: int,
                    matrix_shards: Sequence[MatrixShard], tail_shards: Sequence[TailShard], momentum, tail_p, tail_m,
                    tail_v, adam_step: int) -> None:
    """Writes one rank's state (momentum and the AdamW tail's p, m, v, as
    tensors or arrays; copied to host memory here) with its tables (see
    include/mfsdp.h)."""
    h = CheckpointHeader()
    h.world, h.rank, h.ns_steps = int(world), int(rank), int(ns_steps)
    h.n_matrix, h.n_tail, h.align_elems = len(matrix_shards), len(tail_shards), int(align_elems)
    h.matrix_elems = int(momentum.numel() if hasattr(momentum, "numel") and callable(momentum.numel)
                         else len(momentum))
    h.tail_elems = int(tail_p.numel() if hasattr(tail_p, "numel") and callable(tail_p.numel) else len(tail_p))
    h.adam_step = int(adam_step)
    bufs = [_host_f32(momentum, h.matrix_elems)] + [_host_f32(t, h.tail_elems) for t in (tail_p, tail_m, tail_v)]
    marr = _shard_array(matrix_shards)
    tarr = (TailShard * max(len(tail_shards), 1))(*tail_shards)
    _check(_lib.mfsdp_checkpoint_write(os.fsencode(path), ctypes.byref(h), marr, tarr,
                                       *[b.ctypes.data for b in bufs]), "checkpoint_write")


def checkpoint_load(path: str) -> Checkpoint:
    """Reads one rank's checkpoint into host memory (see include/mfsdp.h)."""
    import numpy as np
    h = CheckpointHeader()
    _check(_lib.mfsdp_checkpoint_read_header(os.fsencode(path), ctypes.byref(h)), "checkpoint_read_header")
    marr = (MatrixShard * max(h.n_matrix, 1))()
    tarr = (TailShard * max(h.n_tail, 1))()
    mom = np.empty(h.matrix_elems, np.float32)
    tail = [np.empty(h.tail_elems, np.float32) for _ in range(3)]
    _check(_lib.mfsdp_checkpoint_read(os.fsencode(path), ctypes.byref(h), marr, h.n_matrix, tarr, h.n_tail,
                                      mom.ctypes.data, h.matrix_elems, *[t.ctypes.data for t in tail], h.tail_elems),
           "checkpoint_read")
    return Checkpoint(h, [marr[i] for i in range(h.n_matrix)], [tarr[i] for i in range(h.n_tail)], mom, *tail)


# --------------------------------------------------- operators next to the step
ID_I32 = 0
ID_I64 = 1
MAX_EXPERTS = 1024


class GradTensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("src_dtype", ctypes.c_int32), ("dst_dtype", ctypes.c_int32)]


_lib.mfsdp_grad_clip_workspace_bytes.argtypes = [_i32]
_lib.mfsdp_grad_clip_workspace_bytes.restype = _sz
for _f in (_lib.mfsdp_grad_norm, _lib.mfsdp_grad_clip):
    _f.argtypes = [ctypes.POINTER(GradTensor), _i32, _d, _d, _vp, _vp, _sz, _vp]
    _f.restype = ctypes.c_int
_lib.mfsdp_sort_ids_workspace_bytes.argtypes = [_i64, _i64]
_lib.mfsdp_sort_ids_workspace_bytes.restype = _sz
_lib.mfsdp_sort_ids.argtypes = [_vp, _i32, _i64, _i64, _vp, _vp, _vp, _sz, _vp]
_lib.mfsdp_sort_ids.restype = ctypes.c_int
_lib.mfsdp_embedding_lookup.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _i64, _d, _vp, _i32, _i64, _vp]
_lib.mfsdp_embedding_lookup.restype = ctypes.c_int
_lib.mfsdp_embedding_grad_workspace_bytes.argtypes = [_i64, _i64, _i64]
_lib.mfsdp_embedding_grad_workspace_bytes.restype = _sz
_lib.mfsdp_embedding_grad.argtypes = [_vp, _i32, _i64, _vp, _i32, _i64, _d, _vp, _i32, _i64, _i64, _i64, _i32, _vp,
                                      _sz, _vp]
_lib.mfsdp_embedding_grad.restype = ctypes.c_int
_lib.mfsdp_expert_workspace_bytes.argtypes = [_i32, _i64, _i64, _i64, _i64, _i64, _i64]
_lib.mfsdp_expert_workspace_bytes.restype = _sz
_lib.mfsdp_expert_matmul.argtypes = [_vp, _i64, _vp, _i64, _i32, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _i32, _i64,
                                     _vp, _sz, _vp]
_lib.mfsdp_expert_matmul.restype = ctypes.c_int
_lib.mfsdp_expert_weight_grad.argtypes = [_vp, _i64, _vp, _i64, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _i64,
                                          _i32, _vp, _sz, _vp]
_lib.mfsdp_expert_weight_grad.restype = ctypes.c_int
_lib.mfsdp_op_device_status.argtypes = [_vp, _vp, ctypes.POINTER(_i32)]
_lib.mfsdp_op_device_status.restype = ctypes.c_int


def _flat(t, what: str):
    """A contiguous CUDA tensor (any shape), as the library reads it."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _rows_of(t, what: str) -> int:
    """Leading dimension of a 2D CUDA tensor with contiguous rows."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"{what} must be 2D with contiguous rows")
    return stride[0] if shape[0] > 1 else max(stride[0], shape[1])


def _id_code(t) -> int:
    if not _id_codes:
        _fill_codes()
    return _id_codes.get(t.dtype, 99)


def _int32(t, n: int, what: str):
    _flat(t, what)
    if _id_code(t) != ID_I32 or t.numel() != n:
        raise ValueError(f"{what} must be {n} int32 elements")
    return t


def _ws(workspace):
    """Address and bytes of a workspace (None: the library says whether it needs one)."""
    if workspace is None:
        return None, 0
    return _ptr(_flat(workspace, "workspace")), workspace.numel() * workspace.element_size()


class GradSet:
    """The tensors of a gradient set with their clipped copies, marshalled once
    (the tensors are kept alive; their addresses must not change)."""

    def __init__(self, srcs, dsts=None):
        self.srcs = list(srcs)
        self.dsts = list(dsts) if dsts is not None else self.srcs
        if len(self.srcs) != len(self.dsts):
            raise ValueError("as many destinations as sources")
        self.array = (GradTensor * max(len(self.srcs), 1))()
        for a, s, d in zip(self.array, self.srcs, self.dsts):
            _flat(s, "a gradient tensor")
            _flat(d, "a clipped tensor")
            if s.numel() != d.numel():
                raise ValueError("a clipped tensor must be as long as its source")
            a.src, a.dst, a.numel = _ptr(s), _ptr(d), int(s.numel())
            a.src_dtype, a.dst_dtype = _dtype_code(s), _dtype_code(d)

    def __len__(self) -> int:
        return len(self.srcs)


def grad_set(srcs, dsts=None) -> GradSet:
    """A gradient set from contiguous CUDA tensors; dsts (default: srcs, in
    place) receive the clipped gradients."""
    return GradSet(srcs, dsts)


def grad_clip_workspace_bytes(tensors: GradSet) -> int:
    return int(_lib.mfsdp_grad_clip_workspace_bytes(len(tensors)))


def _norm_out(out):
    _flat(out, "out")
    if _dtype_code(out) != DTYPE_F32 or out.numel() < 2:
        raise ValueError("out must be two float32 elements")
    return _ptr(out)


def grad_norm(tensors: GradSet, out, workspace, *, max_norm: float = float("inf"), eps: float = 1e-6,
              stream=None) -> None:
    """out[0] = the global norm of the set's sources, out[1] = the clipping
    coefficient min(1, max_norm / (norm + eps)) (see include/mfsdp.h)."""
    _check(_lib.mfsdp_grad_norm(tensors.array, len(tensors), float(max_norm), float(eps), _norm_out(out),
                                *_ws(workspace), _stream(stream)), "grad_norm")


def grad_clip(tensors: GradSet, out, workspace, *, max_norm: float, eps: float = 1e-6, stream=None) -> None:
    """grad_norm, then every destination = coefficient * source."""
    _check(_lib.mfsdp_grad_clip(tensors.array, len(tensors), float(max_norm), float(eps), _norm_out(out),
                                *_ws(workspace), _stream(stream)), "grad_clip")


def sort_ids_workspace_bytes(n: int, n_keys: int) -> int:
    return int(_lib.mfsdp_sort_ids_workspace_bytes(int(n), int(n_keys)))


def sort_ids(ids, n_keys: int, order, starts, workspace, *, stream=None) -> None:
    """Stable sort of positions by id (int32 or int64): order[n] and starts[n_keys + 1],
    both int32; ids outside [0, n_keys) come last (see include/mfsdp.h)."""
    n = int(_flat(ids, "ids").numel())
    _check(_lib.mfsdp_sort_ids(_ptr(ids), _id_code(ids), n, int(n_keys), _ptr(_int32(order, n, "order")),
                               _ptr(_int32(starts, int(n_keys) + 1, "starts")), *_ws(workspace), _stream(stream)),
           "sort_ids")


def embedding_lookup(weight, ids, out, *, scale: float = 1.0, stream=None) -> None:
    """out[t, :] = scale * weight[ids[t], :]; zeros for an id outside the vocabulary."""
    w_ld, o_ld = _rows_of(weight, "weight"), _rows_of(out, "out")
    n, (vocab, dim) = int(_flat(ids, "ids").numel()), weight.shape
    if out.shape != (n, dim):
        raise ValueError(f"out must be {n} x {dim}")
    _check(_lib.mfsdp_embedding_lookup(_ptr(weight), _dtype_code(weight), vocab, dim, w_ld, _ptr(ids), _id_code(ids),
                                       n, float(scale), _ptr(out), _dtype_code(out), o_ld, _stream(stream)),
           "embedding_lookup")


def embedding_grad_workspace_bytes(n: int, vocab: int, dim: int) -> int:
    return int(_lib.mfsdp_embedding_grad_workspace_bytes(int(n), int(vocab), int(dim)))


def embedding_grad(dout, ids, grad, workspace, *, scale: float = 1.0, accumulate: bool = False,
                   stream=None) -> None:
    """grad[v, :] = (grad[v, :] +) scale * sum of dout[t, :] over ids[t] = v (see include/mfsdp.h)."""
    d_ld, g_ld = _rows_of(dout, "dout"), _rows_of(grad, "grad")
    n, (vocab, dim) = int(_flat(ids, "ids").numel()), grad.shape
    if dout.shape != (n, dim):
        raise ValueError(f"dout must be {n} x {dim}")
    _check(_lib.mfsdp_embedding_grad(_ptr(dout), _dtype_code(dout), d_ld, _ptr(ids), _id_code(ids), n, float(scale),
                                     _ptr(grad), _dtype_code(grad), vocab, dim, g_ld, int(bool(accumulate)),
                                     *_ws(workspace), _stream(stream)), "embedding_grad")


def expert_workspace_bytes(n_experts: int, rows: int, cols: int, n_rows: int, *, w_stride: Optional[int] = None,
                           rows_ld: Optional[int] = None, cols_ld: Optional[int] = None) -> int:
    """Workspace of the grouped products; strides default to contiguous tensors."""
    return int(_lib.mfsdp_expert_workspace_bytes(int(n_experts), int(n_rows), int(rows), int(cols),
                                                 int(rows * cols if w_stride is None else w_stride),
                                                 int(rows if rows_ld is None else rows_ld),
                                                 int(cols if cols_ld is None else cols_ld)))


def _stack(t, what: str) -> int:
    """Element stride between the matrices of a 3D CUDA tensor, each contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (shape[2] > 1 and stride[2] != 1) or (shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError(f"{what} must be 3D with contiguous matrices")
    return stride[0] if shape[0] > 1 else shape[1] * shape[2]


def expert_matmul(x, w, starts, y, workspace, *, input_grad: bool = False, stream=None) -> None:
    """y[t, :] = W_e x[t, :] (input_grad: W_e^T x[t, :]) for the rows t of each expert e, with w of
    shape (experts, rows, cols) and starts int32 (see include/mfsdp.h)."""
    x_ld, y_ld, w_stride = _rows_of(x, "x"), _rows_of(y, "y"), _stack(w, "w")
    e, rows, cols = w.shape
    n = x.shape[0]
    xw, yw = (rows, cols) if input_grad else (cols, rows)
    if x.shape[1] != xw or y.shape != (n, yw):
        raise ValueError(f"x must be n x {xw} and y n x {yw}")
    in_dtype = _dtype_code(x) if x.dtype == w.dtype else 99
    _check(_lib.mfsdp_expert_matmul(_ptr(x), x_ld, _ptr(w), w_stride, in_dtype, _ptr(_int32(starts, e + 1, "starts")),
                                    e, n, rows, cols, int(bool(input_grad)), _ptr(y), _dtype_code(y), y_ld,
                                    *_ws(workspace), _stream(stream)), "expert_matmul")


def expert_weight_grad(dy, x, starts, dw, workspace, *, accumulate: bool = False, stream=None) -> None:
    """dw[e] = (dw[e] +) dy_e^T x_e over each expert's rows (see include/mfsdp.h)."""
    dy_ld, x_ld, dw_stride = _rows_of(dy, "dy"), _rows_of(x, "x"), _stack(dw, "dw")
    e, rows, cols = dw.shape
    n = x.shape[0]
    if dy.shape != (n, rows) or x.shape[1] != cols:
        raise ValueError(f"dy must be n x {rows} and x n x {cols}")
    in_dtype = _dtype_code(x) if x.dtype == dy.dtype else 99
    _check(_lib.mfsdp_expert_weight_grad(_ptr(dy), dy_ld, _ptr(x), x_ld, in_dtype,
                                         _ptr(_int32(starts, e + 1, "starts")), e, n, rows, cols, _ptr(dw),
                                         _dtype_code(dw), dw_stride, int(bool(accumulate)), *_ws(workspace),
                                         _stream(stream)), "expert_weight_grad")


def op_device_status(workspace, stream=None) -> Tuple[int, int]:
    """(status, raw word) of the last grouped product or embedding gradient that ran with this
    workspace (synchronises)."""
    detail = _i32(0)
    st = _lib.mfsdp_op_device_status(_ws(workspace)[0], _stream(stream), ctypes.byref(detail))
    return st, detail.value


# ------------------------------------------ the loss, norms and AdamW over a set
STATE_F32 = 0
STATE_E4M3 = 1
STATE_BLOCK = 256


class AdamwTensor(ctypes.Structure):
    _fields_ = [("p", _vp), ("g", _vp), ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp), ("copy", _vp),
                ("numel", _i64), ("lr_scale", _d), ("wd", _d), ("p_dtype", _i32), ("g_dtype", _i32), ("state", _i32),
                ("reserved", _i32)]


_lib.mfsdp_adamw_set_step.argtypes = [ctypes.POINTER(AdamwTensor), _i32, _d, _d, _d, _d, _i64, _vp, _vp]
_lib.mfsdp_adamw_set_step.restype = ctypes.c_int


def adamw_scales(numel: int) -> int:
    """Scales of an 8-bit moment of numel elements: one for 256."""
    return -(-int(numel) // STATE_BLOCK)


class AdamwSet:
    """The tensors of an AdamW set, marshalled once (they are kept alive; their addresses must not
    change).  The state of each is 32-bit (m and v float32) or 8-bit (m and v float8_e4m3fn or
    uint8, with float32 scales); a set may hold both."""

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, m_scales=None, v_scales=None, copies=None, lr_scales=None,
                 weight_decays=None):
        import torch
        n = len(params)
        none = [None] * n

        def listed(x, what):
            x = none if x is None else list(x)
            if len(x) != n:
                raise ValueError(f"as many {what} as parameters")
            return x

        self.params = list(params)
        self.tensors = [self.params] + [listed(x, what) for x, what in (
            (grads, "gradients"), (exp_avgs, "first moments"), (exp_avg_sqs, "second moments"), (m_scales, "m_scales"),
            (v_scales, "v_scales"), (copies, "copies"))]
        lr_scales = [1.0] * n if lr_scales is None else listed(lr_scales, "lr_scales")
        weight_decays = [0.0] * n if weight_decays is None else listed(weight_decays, "weight_decays")
        self.array = (AdamwTensor * max(n, 1))()
        eight = (torch.float8_e4m3fn, torch.uint8)
        for a, p, g, m, v, ms, vs, c, lr, wd in zip(self.array, *self.tensors, lr_scales, weight_decays):
            numel = int(p.numel())
            for t, what in ((p, "a parameter"), (g, "a gradient"), (m, "a moment"), (v, "a moment"), (c, "a copy")):
                if t is not None and _flat(t, what).numel() != numel:
                    raise ValueError(f"{what} must be as long as its parameter")
            a.state = STATE_E4M3 if m.dtype in eight else STATE_F32
            if m.dtype not in eight + (torch.float32,) or v.dtype != m.dtype:
                raise ValueError("moments must both be float32, float8_e4m3fn or uint8")
            if a.state == STATE_E4M3:
                for t, what in ((ms, "m_scales"), (vs, "v_scales")):
                    if t is None or t.dtype != torch.float32 or _flat(t, what).numel() != adamw_scales(numel):
                        raise ValueError(f"{what}: {adamw_scales(numel)} float32 elements for 8-bit moments")
                a.m_scale, a.v_scale = _ptr(ms), _ptr(vs)
            if c is not None and c.dtype != torch.bfloat16:
                raise ValueError("a copy must be bfloat16")
            a.p, a.g, a.m, a.v, a.copy = _ptr(p), _ptr(g), _ptr(m), _ptr(v), (_ptr(c) if c is not None else None)
            a.numel, a.lr_scale, a.wd = numel, float(lr), float(wd)
            a.p_dtype, a.g_dtype = _dtype_code(p), _dtype_code(g)

    def __len__(self) -> int:
        return len(self.params)


def adamw_set(params, grads, exp_avgs, exp_avg_sqs, m_scales=None, v_scales=None, copies=None, lr_scales=None,
              weight_decays=None) -> AdamwSet:
    """An AdamW set from contiguous CUDA tensors; lr_scales (default 1) and weight_decays (default 0)
    give each tensor's own rate and decay, copies receive the new weights in bfloat16."""
    return AdamwSet(params, grads, exp_avgs, exp_avg_sqs, m_scales, v_scales, copies, lr_scales, weight_decays)


def adamw_set_step(tensors: AdamwSet, *, lr: float, beta1: float, beta2: float, eps: float, step: int, norm=None,
                   stream=None) -> None:
    """One AdamW step over the set (see include/mfsdp.h); norm: what grad_norm left, to clip on the way."""
    _check(_lib.mfsdp_adamw_set_step(tensors.array, len(tensors), float(lr), float(beta1), float(beta2), float(eps),
                                     int(step), _norm_out(norm) if norm is not None else None, _stream(stream)),
           "adamw_set_step")


MAX_TOP = 32

_lib.mfsdp_token_logprob.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _d, _vp, _vp, _vp, _i32, _vp, _vp, _vp]
_lib.mfsdp_token_logprob.restype = ctypes.c_int
_lib.mfsdp_token_logprob_grad.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _d, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
_lib.mfsdp_token_logprob_grad.restype = ctypes.c_int


def _floats(t, n: int, what: str) -> Optional[int]:
    """Address of a contiguous float32 CUDA tensor of n elements (None: not wanted)."""
    if t is None:
        return None
    if t.numel() != n or _dtype_code(t) != DTYPE_F32 or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{what} must be {n} contiguous float32 elements of CUDA memory")
    return t.data_ptr()


def _targets(targets, n: int):
    """Address and type code of n targets (None: no targets)."""
    if targets is None:
        return None, ID_I64
    if _flat(targets, "targets").numel() != n:
        raise ValueError(f"targets must be {n} ids")
    return targets.data_ptr(), _id_code(targets)


def token_logprob(logits, targets, logprob=None, *, lse=None, entropy=None, top_ids=None, top_logprob=None,
                  scale: float = 1.0, stream=None) -> None:
    """Log-probabilities of targets (int32 or int64; outside the vocabulary: masked, 0) under
    softmax(scale * logits), with the rows' log-sum-exp, entropy, and the largest logits' ids and
    log-probabilities (n x k, int32 and float32); outputs that are None are not computed
    (see include/mfsdp.h)."""
    ld = _rows_of(logits, "logits")
    n, vocab = logits.shape
    k = 0
    for t in (top_ids, top_logprob):
        if t is not None:
            if len(t.shape) != 2 or t.shape[0] != n or (k and t.shape[1] != k):
                raise ValueError(f"top_ids and top_logprob must both be {n} x k")
            k = int(t.shape[1])
    ids = _ptr(_int32(top_ids, n * k, "top_ids")) if top_ids is not None else None
    y, id_type = _targets(targets, n)
    _check(_lib.mfsdp_token_logprob(_ptr(logits), _dtype_code(logits), n, vocab, ld, y, id_type, float(scale),
                                    _floats(logprob, n, "logprob"), _floats(lse, n, "lse"),
                                    _floats(entropy, n, "entropy"), k, ids, _floats(top_logprob, n * k, "top_logprob"),
                                    _stream(stream)), "token_logprob")


def token_logprob_grad(logits, targets, lse, dlogits, *, dlogprob=None, entropy=None, dentropy=None,
                       scale: float = 1.0, stream=None) -> None:
    """dlogits from the gradients of the log-probabilities and entropies, with lse and entropy as
    token_logprob left them; dlogits may be logits (see include/mfsdp.h)."""
    ld, d_ld = _rows_of(logits, "logits"), _rows_of(dlogits, "dlogits")
    n, vocab = logits.shape
    if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype:
        raise ValueError(f"dlogits must be {n} x {vocab} of the logits' type")
    y, id_type = _targets(targets, n)
    _check(_lib.mfsdp_token_logprob_grad(_ptr(logits), _dtype_code(logits), n, vocab, ld, y, id_type, float(scale),
                                         _floats(lse, n, "lse"), _floats(entropy, n, "entropy"),
                                         _floats(dlogprob, n, "dlogprob"), _floats(dentropy, n, "dentropy"),
                                         _ptr(dlogits), d_ld, _stream(stream)), "token_logprob_grad")


NORM_NONE = 0
NORM_RMS = 1
NORM_LAYER = 2
MAX_NORM_DIM = 16384


class BlockNormSpec(ctypes.Structure):
    _fields_ = [("dim", _i64), ("post_norm", _i32), ("pre_norm", _i32), ("residual_dtype", _i32),
                ("branch_dtype", _i32), ("weight_dtype", _i32), ("reserved", _i32), ("eps", _d),
                ("residual_scale", _d), ("branch_scale", _d), ("post_weight", _vp), ("post_bias", _vp), ("gate", _vp),
                ("gate_rows", _i64), ("pre_weight", _vp), ("pre_bias", _vp)]


class BlockNormGrads(ctypes.Structure):
    _fields_ = [("d_post_weight", _vp), ("d_post_bias", _vp), ("d_gate", _vp), ("d_pre_weight", _vp),
                ("d_pre_bias", _vp), ("accumulate", _i32), ("reserved", _i32)]


_SPEC = ctypes.POINTER(BlockNormSpec)
_lib.mfsdp_block_norm.argtypes = [_SPEC, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp]
_lib.mfsdp_block_norm.restype = ctypes.c_int
_lib.mfsdp_block_norm_grad_workspace_bytes.argtypes = [_SPEC, _i64]
_lib.mfsdp_block_norm_grad_workspace_bytes.restype = _sz
_lib.mfsdp_block_norm_grad.argtypes = [_SPEC, _i64] + [_vp, _i64] * 2 + [_vp] + [_vp, _i64] * 4 + [
    ctypes.POINTER(BlockNormGrads), _vp, _sz, _vp]
_lib.mfsdp_block_norm_grad.restype = ctypes.c_int


class BlockNorm:
    """The norms around a block, marshalled once: norm kinds and their vectors (kept alive; their
    addresses must not change).  gate: contiguous rows of dim, one for every gate_rows rows.  All
    vectors have one type."""

    def __init__(self, dim: int, *, post: int = NORM_NONE, post_weight=None, post_bias=None, gate=None,
                 gate_rows: int = 0, pre: int = NORM_NONE, pre_weight=None, pre_bias=None, eps: float = 1e-6,
                 residual_scale: float = 1.0, branch_scale: float = 1.0):
        self.dim, self.gate_rows = int(dim), int(gate_rows)
        self.vectors = dict(post_weight=post_weight, post_bias=post_bias, gate=gate, pre_weight=pre_weight,
                            pre_bias=pre_bias)
        self.spec = s = BlockNormSpec()
        s.dim, s.post_norm, s.pre_norm, s.gate_rows = self.dim, int(post), int(pre), self.gate_rows
        s.eps, s.residual_scale, s.branch_scale = float(eps), float(residual_scale), float(branch_scale)
        kinds = {t.dtype for t in self.vectors.values() if t is not None}
        if len(kinds) > 1:
            raise ValueError("weights, biases and gate must have one type")
        for name, t in self.vectors.items():
            if t is None:
                continue
            if _flat(t, name).numel() % self.dim if name == "gate" else _flat(t, name).numel() != self.dim:
                raise ValueError(f"{name} must have {self.dim} columns")
            setattr(s, name, _ptr(t))
            s.weight_dtype = _dtype_code(t)
        if gate is not None and self.gate_rows < 1:
            raise ValueError("gate_rows must be positive with a gate")
        self.gate_numel = int(gate.numel()) if gate is not None else None
        self.refs = {}

    def gates(self, n: int) -> int:
        """Rows of the gate for n rows."""
        return -(-n // self.gate_rows) if self.gate_numel is not None else 0

    def _rows(self, t, n: int, like):
        """Address and leading dimension of a tensor of n rows of `like`'s type (None: not there)."""
        if t is None:
            return None, 0
        shape, stride = t.shape, t.stride()
        if len(shape) != 2 or shape[0] != n or shape[1] != self.dim:
            raise ValueError(f"every tensor of rows must be {n} x {self.dim}")
        if t.dtype != like.dtype:
            raise ValueError("residual, its output and their gradients must have one type, branch, normed and "
                             "their gradients one")
        if not t.is_cuda:
            raise ValueError("a tensor of rows must be a CUDA tensor")
        if stride[1] != 1 and shape[1] > 1:
            raise ValueError("a tensor of rows must have contiguous rows")
        return t.data_ptr(), stride[0] if n > 1 else max(stride[0], shape[1])

    def _call(self, residual, side):
        """The specification for a call's types (side: any tensor of the branch's side, or None) and its
        number of rows, with which the gate has to agree.  One is made for each pair of types, so
        that calls of several threads share none that changes."""
        n, key = residual.shape[0], (residual.dtype, side.dtype if side is not None else None)
        ref = self.refs.get(key)
        if ref is None:
            spec = BlockNormSpec.from_buffer_copy(self.spec)
            spec.residual_dtype = _dtype_code(residual)
            spec.branch_dtype = _dtype_code(side if side is not None else residual)
            ref = self.refs[key] = ctypes.byref(spec)
        if n and self.gate_numel is not None and self.gate_numel != self.gates(n) * self.dim:
            raise ValueError(f"gate must have {self.gates(n)} rows for {n} rows")
        return ref, n


def block_norm(norm: BlockNorm, residual, *, branch=None, residual_out=None, normed=None, stats=None,
               stream=None) -> None:
    """residual_out = residual_scale * residual + branch_scale * gate * post_norm(branch) and
    normed = pre_norm(residual_out), in one pass; stats (n x 4 float32) is what the gradient takes
    (see include/mfsdp.h)."""
    side = branch if branch is not None else normed
    (spec, n), rows = norm._call(residual, side), norm._rows
    _check(_lib.mfsdp_block_norm(spec, n, *rows(residual, n, residual), *rows(branch, n, side),
                                 *rows(residual_out, n, residual), *rows(normed, n, side),
                                 _floats(stats, 4 * n, "stats"), _stream(stream)), "block_norm")


def block_norm_grad_workspace_bytes(norm: BlockNorm, n: int) -> int:
    return int(_lib.mfsdp_block_norm_grad_workspace_bytes(ctypes.byref(norm.spec), int(n)))


def block_norm_grad(norm: BlockNorm, residual, stats, *, branch=None, d_residual_out=None, d_normed=None,
                    d_residual=None, d_branch=None, d_post_weight=None, d_post_bias=None, d_gate=None,
                    d_pre_weight=None, d_pre_bias=None, accumulate: bool = False, workspace, stream=None) -> None:
    """Gradients of block_norm's inputs from d_residual_out and d_normed; those that are None are
    not wanted (or zero).  Vectors' gradients are float32 (see include/mfsdp.h)."""
    side = branch if branch is not None else d_normed
    (spec, n), rows = norm._call(residual, side), norm._rows
    dim = norm.dim
    gates = norm.gates(n) * dim if n or d_gate is None else d_gate.numel()       # without rows no gate is touched
    g = BlockNormGrads(_floats(d_post_weight, dim, "d_post_weight"), _floats(d_post_bias, dim, "d_post_bias"),
                       _floats(d_gate, gates, "d_gate"), _floats(d_pre_weight, dim, "d_pre_weight"),
                       _floats(d_pre_bias, dim, "d_pre_bias"), 1 if accumulate else 0)
    _check(_lib.mfsdp_block_norm_grad(spec, n, *rows(residual, n, residual), *rows(branch, n, side),
                                      _floats(stats, 4 * n, "stats"), *rows(d_residual_out, n, residual),
                                      *rows(d_normed, n, side), *rows(d_residual, n, residual),
                                      *rows(d_branch, n, side), ctypes.byref(g), *_ws(workspace), _stream(stream)),
           "block_norm_grad")


def library_path() -> str:
    """Path of the loaded libmfsdp.so."""
    return _LIB_PATH


def raw_lib() -> ctypes.CDLL:
    """The loaded library, for callers that marshal raw pointers themselves."""
    return _lib
