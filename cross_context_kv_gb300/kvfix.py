"""ctypes binding of libkvfix (include/kvfix.h).

Argument marshalling only: every function checks tensor dtypes/devices, builds the
plane descriptors from tensor shapes and strides, allocates outputs with torch on the
tensors' device, which has to be the current one, and calls the C entry point of the
same name on the current CUDA stream.  All arithmetic runs in the library's CUDA kernels.  If libkvfix.so is
missing, importing this module raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

# Two parts of torch that its releases do not promise, for their host time alone: a small
# shared_attend call allocates three tensors (2 us each beside a launch, 4.5 by empty_strided).
# Without them the public ways are taken.
try:
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None
_raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvfix.so")

OK, EINVAL, ENOSPACE, ECUDA, ETIMEOUT, EDEVICE = range(6)
STATUS_NAMES = {0: "KVFIX_OK", 1: "KVFIX_EINVAL", 2: "KVFIX_ENOSPACE", 3: "KVFIX_ECUDA",
                4: "KVFIX_ETIMEOUT", 5: "KVFIX_EDEVICE"}


class KvfixError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class KvDesc(ctypes.Structure):
    _fields_ = [("chunks", ctypes.c_int32), ("layers", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("stride_chunk", ctypes.c_int64), ("stride_layer", ctypes.c_int64),
                ("stride_token", ctypes.c_int64)]


class PoolDesc(ctypes.Structure):
    """kvfix_pool: strides in bytes."""
    _fields_ = [("format", ctypes.c_int32), ("layers", ctypes.c_int32), ("slots", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("stride_layer", ctypes.c_int64), ("stride_slot", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


class RopeDesc(ctypes.Structure):
    """kvfix_rope."""
    _fields_ = [("layout", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("original_tokens", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("attention", ctypes.c_double)]


# name -> (restype, argtypes); mirrors include/kvfix.h
P, I32, I64, F64, SZ, D = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double,
                           ctypes.c_size_t, KvDesc)
PD, RD = PoolDesc, RopeDesc
SIGNATURES = {
    "kvfix_version": (ctypes.c_int, []),
    "kvfix_last_error": (ctypes.c_char_p, []),
    "kvfix_check_status": (ctypes.c_int, [P]),
    "kvfix_rerope": (ctypes.c_int, [P, D, P, D, P, F64, P]),
    "kvfix_score_topk": (ctypes.c_int, [P, P, D, P, P, D, I32, P, F64, I32, P, P, P, P, P, P, P, P, P, P]),
    "kvfix_mean_correct": (ctypes.c_int, [P, P, D, P, P, D, P, P, D, I32, P, F64, P, P, I32, P, P, P, P, P]),
    "kvfix_lowrank_apply": (ctypes.c_int, [P, D, P, P, I32, P, D, P]),
    "kvfix_draft_rank_workspace_bytes": (SZ, [D, I32]),
    "kvfix_draft_rank": (ctypes.c_int, [P, D, P, I32, I32, I32, I32, P, P, P, P, D, P, P, P, SZ, P]),
    "kvfix_draft_rank_noalloc": (ctypes.c_int, [P, D, P, I32, I32, I32, I32, P, P, P, P, D, P, P, P]),
    "kvfix_lowrank_draft_workspace_bytes": (SZ, [D, I32]),
    "kvfix_lowrank_draft": (ctypes.c_int, [P, D, P, P, I32, P, D, P, I32, I32, I32, I32, P, P, P, P, D, P, P, SZ, P]),
    "kvfix_diff_encode": (ctypes.c_int, [P, P, D, P, P, D, I32, P, P, P, I64, P, P]),
    "kvfix_diff_gather": (ctypes.c_int, [P, P, D, P, P, P, I64, I32, I32, P, P, D, P]),
    "kvfix_diff_restore": (ctypes.c_int, [P, P, D, P, P, P, I64, I32, I32, P, F64, P, P, P, D, P]),
    "kvfix_repair_layout": (ctypes.c_int, [P, I32, I32, I32, I32, I32, I32, F64, I32, P, I32, P, P]),
    "kvfix_master_select": (ctypes.c_int, [P, P, I32, I32, I32, P, P, P]),
    "kvfix_selftest_wait": (ctypes.c_int, [I64, P, P]),
    "kvfix_anchor_gate_correct": (ctypes.c_int, [P, P, D, P, P, P, P, P, P, P, P, I32, I32, I32, F64, F64, P, F64, P,
                                                 P, P, P, P, P, P, P, D, P, SZ, P]),
    "kvfix_diff_encode_split": (ctypes.c_int, [P, P, D, P, P, D, I32, P, P, P, P, P, P, I64, I64, P, P]),
    "kvfix_diff_gather_split": (ctypes.c_int, [P, P, D, P, P, P, P, P, P, I64, I64, I32, I32, P, P, D, P]),
    "kvfix_diff_restore_split": (ctypes.c_int, [P, P, D, P, P, P, P, P, P, I64, I64, I32, I32, P, F64, P, P, P, D,
                                                P]),
    "kvfix_pool_write": (ctypes.c_int, [P, P, D, P, F64, P, PD, P]),
    "kvfix_pool_read": (ctypes.c_int, [PD, P, P, F64, P, P, D, P]),
    "kvfix_shared_attend_workspace_bytes": (SZ, [I32, I32, I32, I32, I32, I32]),
    "kvfix_shared_attend": (ctypes.c_int, [P, D, PD, I32, P, I32, P, P, I32, P, I32, P, F64, P, D, P, P, SZ, P]),
    "kvfix_rotary": (ctypes.c_int, [P, D, P, D, P, RD, P, D, P, D, P]),
    "kvfix_tree_attend": (ctypes.c_int, [P, D, PD, I32, P, I32, P, P, I32, P, I32, P, P, P, F64, P, D, P, P, SZ, P]),
    "kvfix_pages_extend_workspace_bytes": (SZ, [I32, I32]),
    "kvfix_pages_extend": (ctypes.c_int, [PD, I32, P, P, I32, P, I32, P, P, P, SZ, P]),
    "kvfix_pages_cut": (ctypes.c_int, [PD, I32, P, P, I32, P, I32, P, P, I32, P, P]),
    "kvfix_pages_compact_workspace_bytes": (SZ, [I32]),
    "kvfix_pages_compact": (ctypes.c_int, [PD, I32, P, P, I32, P, I32, P, P, SZ, P]),
    "kvfix_repair_rows": (ctypes.c_int, [P, P, D, P, P, D, P, I32, P, P]),
    "kvfix_anchor_gate_workspace_bytes": (SZ, [D, I32, I32]),
    "kvfix_anchor_gate": (ctypes.c_int, [P, D, P, P, I32, I32, I32, F64, F64, P, P, P, P, P, SZ, P]),
    "kvfix_anchor_correct": (ctypes.c_int, [P, P, D, P, P, P, P, P, P, P, P, I32, I32, F64, P, F64, P, P, P, P, P,
                                            D, P]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _check(status: int):
    if status != OK:
        raise KvfixError(status, lib.kvfix_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _launch_device(dev: int):
    """Refuses tensors of a device that is not current: the library launches on the current one,
    and another device's default stream looks the same to it."""
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")


def _stream(t) -> ctypes.c_void_p:
    _launch_device(t.get_device())
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _bf16(t, name):
    if t is None:
        return
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor (got {t.dtype} on {t.device})")


def plane_desc(t: torch.Tensor) -> KvDesc:
    """Descriptor of a [chunks][layers][tokens][heads][dim] (or [chunks][tokens][heads][dim],
    read as one layer) bf16 view whose heads and dims are contiguous."""
    if t.dim() == 4:
        t = t.unsqueeze(1)
    if t.dim() != 5:
        raise ValueError(f"KV plane must be 4-D or 5-D, got shape {tuple(t.shape)}")
    C, L, n, H, Dh = t.shape
    sc, sl, st, sh, sd = t.stride()
    if (sd != 1 or sh != Dh) and H * Dh > 1:
        raise ValueError("KV plane views need contiguous heads and dims (stride(-1) == 1, "
                         "stride(-2) == head_dim)")
    return KvDesc(C, L, n, H, Dh, sc if C > 1 else 0, sl if L > 1 else 0, st if n > 1 else H * Dh)


def _i32(t, name):
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA int32 tensor")


_INT32 = torch.int32


def _ints(dev: int, tensors) -> bool:
    """Whether all are contiguous int32 tensors of CUDA device `dev` (None is skipped): what a call
    wants, in one pass; where it is false, the checks one by one say what is wrong."""
    for t in tensors:
        if t is not None and (t.dtype is not _INT32 or t.get_device() != dev or not t.is_contiguous()):
            return False
    return True


def _f32(t, name):
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA float32 tensor")


def version() -> int:
    return lib.kvfix_version()


def check_status(stream_of: torch.Tensor | None = None) -> int:
    """Synchronise the current stream and raise if the device flagged a condition."""
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    _check(lib.kvfix_check_status(s))
    return OK


# --------------------------------------------------------------------- calls

def rerope(k: torch.Tensor, delta: torch.Tensor, rope_base: float, out: torch.Tensor | None = None):
    _bf16(k, "k")
    _i32(delta, "delta")
    out = torch.empty_like(k) if out is None else out
    _bf16(out, "out")
    _check(lib.kvfix_rerope(_ptr(k), plane_desc(k), _ptr(out), plane_desc(out), _ptr(delta),
                            float(rope_base), _stream(k)))
    return out


def score_topk(k_reuse, v_reuse, k_fresh, v_fresh, agents: int, delta, rope_base: float, b: int,
               masks: bool = False):
    """Check-layer views: reuse [R](1)[n][H][D], fresh [agents*R](1)[n][H][D]."""
    for t, nm in ((k_reuse, "k_reuse"), (v_reuse, "v_reuse"), (k_fresh, "k_fresh"), (v_fresh, "v_fresh")):
        _bf16(t, nm)
    _i32(delta, "delta")
    rd, fd = plane_desc(k_reuse), plane_desc(k_fresh)
    units, n = fd.chunks, fd.tokens
    dev = k_reuse.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"d_k": torch.empty(units, n, **f32), "d_v": torch.empty(units, n, **f32),
           "w_k": torch.empty(units, n, **f32), "w_v": torch.empty(units, n, **f32),
           "idx_k": torch.empty(units, max(b, 0), dtype=torch.int32, device=dev),
           "idx_v": torch.empty(units, max(b, 0), dtype=torch.int32, device=dev)}
    words = (n + 31) // 32
    if masks:
        for nm in ("mask_k", "mask_v", "mask_union"):
            out[nm] = torch.empty(units, words, dtype=torch.int32, device=dev)
    _check(lib.kvfix_score_topk(_ptr(k_reuse), _ptr(v_reuse), rd, _ptr(k_fresh), _ptr(v_fresh), fd,
                                int(agents), _ptr(delta), float(rope_base), int(b),
                                _ptr(out["d_k"]), _ptr(out["d_v"]), _ptr(out["w_k"]), _ptr(out["w_v"]),
                                _ptr(out["idx_k"]) if b > 0 else None, _ptr(out["idx_v"]) if b > 0 else None,
                                _ptr(out.get("mask_k")), _ptr(out.get("mask_v")),
                                _ptr(out.get("mask_union")), _stream(k_reuse)))
    return out


def mean_correct(k_reuse, v_reuse, k_fresh, v_fresh, agents: int, delta, rope_base: float,
                 idx_k, idx_v, w_k, w_v, k_out=None, v_out=None, mu_k=None, mu_v=None):
    """reuse [R][L][n][H][D]; fresh/out [agents*R][L][n][H][D]; idx [agents*R][b]."""
    for t, nm in ((k_reuse, "k_reuse"), (v_reuse, "v_reuse"), (k_fresh, "k_fresh"), (v_fresh, "v_fresh")):
        _bf16(t, nm)
    _i32(delta, "delta")
    _i32(idx_k, "idx_k")
    _i32(idx_v, "idx_v")
    _f32(w_k, "w_k")
    _f32(w_v, "w_v")
    if idx_k.shape != idx_v.shape:
        raise ValueError("idx_k and idx_v must have the same shape")
    b = idx_k.shape[-1] if idx_k.dim() else 0
    k_out = torch.empty_like(k_fresh) if k_out is None else k_out
    v_out = torch.empty_like(v_fresh) if v_out is None else v_out
    rd, fd, od = plane_desc(k_reuse), plane_desc(k_fresh), plane_desc(k_out)
    units, L, H, Dh = fd.chunks, fd.layers, fd.kv_heads, fd.head_dim
    if mu_k is None:
        mu_k = torch.empty(units, L, H * Dh, dtype=torch.float32, device=k_reuse.device)
    if mu_v is None:
        mu_v = torch.empty(units, L, H * Dh, dtype=torch.float32, device=k_reuse.device)
    _check(lib.kvfix_mean_correct(_ptr(k_reuse), _ptr(v_reuse), rd, _ptr(k_fresh), _ptr(v_fresh), fd,
                                  _ptr(k_out), _ptr(v_out), od, int(agents), _ptr(delta),
                                  float(rope_base), _ptr(idx_k), _ptr(idx_v), int(b), _ptr(w_k),
                                  _ptr(w_v), _ptr(mu_k), _ptr(mu_v), _stream(k_reuse)))
    return k_out, v_out, mu_k, mu_v


def lowrank_apply(x, A, B, out=None):
    """x [C][L][n][H][D]; A [C][L][H][n][r]; B [C][L][H][r][D] (A, B contiguous)."""
    _bf16(x, "x")
    _bf16(A, "A")
    _bf16(B, "B")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous")
    out = torch.empty_like(x) if out is None else out
    _bf16(out, "out")
    _check(lib.kvfix_lowrank_apply(_ptr(x), plane_desc(x), _ptr(A), _ptr(B), int(A.shape[-1]), _ptr(out),
                                   plane_desc(out), _stream(x)))
    return out


def draft_rank_workspace_bytes(k, layer_begin: int) -> int:
    return int(lib.kvfix_draft_rank_workspace_bytes(plane_desc(k), int(layer_begin)))


def draft_rank(k, q, layer_begin: int, k_rows: int, k_fresh=None, v_fresh=None, k_io=None,
               v_io=None, workspace=None):
    """k [C][L][n][Hkv][D]; q [C][L][T][Hq][D] contiguous.  Returns (idx, scores)."""
    _bf16(k, "k")
    _bf16(q, "q")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    d = plane_desc(k)
    C, n = d.chunks, d.tokens
    ws_bytes = draft_rank_workspace_bytes(k, layer_begin)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=k.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    idx = torch.empty(C, max(k_rows, 0), dtype=torch.int32, device=k.device)
    scores = torch.empty(C, n, dtype=torch.float64, device=k.device)
    fd = plane_desc(k_fresh) if k_fresh is not None else (plane_desc(v_fresh) if v_fresh is not None else d)
    _check(lib.kvfix_draft_rank(_ptr(k), d, _ptr(q), int(q.shape[2]), int(q.shape[3]), int(layer_begin),
                                int(k_rows), _ptr(idx), _ptr(scores), _ptr(k_fresh), _ptr(v_fresh), fd,
                                _ptr(k_io), _ptr(v_io), _ptr(workspace), workspace.numel(), _stream(k)))
    return idx, scores


def lowrank_draft_workspace_bytes(k, layer_begin: int) -> int:
    return int(lib.kvfix_lowrank_draft_workspace_bytes(plane_desc(k), int(layer_begin)))


def lowrank_draft(x, A, B, q, layer_begin: int, k_rows: int, out=None, k_fresh=None, v_fresh=None, v_io=None,
                  workspace=None):
    """out = x + A B (the key plane) and the draft ranking of out in one pass; with k_fresh
    the selected rows of out, with v_fresh/v_io those of v_io, are overwritten.  x, out
    [C][L][n][Hkv][D]; A [C][L][Hkv][n][r]; B [C][L][Hkv][r][D]; q [C][L][T][Hq][D].
    Returns (out, idx, scores)."""
    for t, nm in ((x, "x"), (A, "A"), (B, "B"), (q, "q")):
        _bf16(t, nm)
    if not (A.is_contiguous() and B.is_contiguous() and q.is_contiguous()):
        raise ValueError("A, B and q must be contiguous")
    out = torch.empty_like(x) if out is None else out
    _bf16(out, "out")
    d, od = plane_desc(x), plane_desc(out)
    C, n = d.chunks, d.tokens
    ws_bytes = lowrank_draft_workspace_bytes(out, layer_begin)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    idx = torch.empty(C, max(k_rows, 0), dtype=torch.int32, device=x.device)
    scores = torch.empty(C, n, dtype=torch.float64, device=x.device)
    fd = plane_desc(k_fresh) if k_fresh is not None else (plane_desc(v_fresh) if v_fresh is not None else d)
    _check(lib.kvfix_lowrank_draft(_ptr(x), d, _ptr(A), _ptr(B), int(A.shape[-1]), _ptr(out), od, _ptr(q),
                                   int(q.shape[2]), int(q.shape[3]), int(layer_begin), int(k_rows), _ptr(idx),
                                   _ptr(scores), _ptr(k_fresh), _ptr(v_fresh), fd, _ptr(v_io), _ptr(workspace),
                                   workspace.numel(), _stream(x)))
    return out, idx, scores


def diff_encode(master_k, master_v, sib_k, sib_v, block_tokens: int, capacity: int | None = None,
                sync: bool = True):
    """master [L][n][H][D] (or [1][L][n][H][D]); siblings [S][L][n][H][D].
    Returns (mask int32 words, offsets int64, payload [cap][2][bt][H][D], entries or None)."""
    for t, nm in ((master_k, "master_k"), (master_v, "master_v"), (sib_k, "sib_k"), (sib_v, "sib_v")):
        _bf16(t, nm)
    mk = master_k.unsqueeze(0) if master_k.dim() == 4 else master_k
    mv = master_v.unsqueeze(0) if master_v.dim() == 4 else master_v
    md, sd = plane_desc(mk), plane_desc(sib_k)
    S, L, n, H, Dh = sd.chunks, sd.layers, sd.tokens, sd.kv_heads, sd.head_dim
    bt = int(block_tokens)
    E = S * L * (n // bt)
    dev = sib_k.device
    mask = torch.empty((E + 31) // 32, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int64, device=dev)
    cap = E if capacity is None else int(capacity)
    payload = torch.empty(max(cap, 1), 2, bt, H, Dh, dtype=torch.bfloat16, device=dev)
    entries = ctypes.c_int64(-1)
    st = lib.kvfix_diff_encode(_ptr(mk), _ptr(mv), md, _ptr(sib_k), _ptr(sib_v), sd, bt, _ptr(mask),
                               _ptr(offsets), _ptr(payload), cap, ctypes.byref(entries) if sync else None,
                               _stream(sib_k))
    _check(st)
    return mask, offsets, payload, (entries.value if sync else None)


def diff_gather(master_k, master_v, mask, offsets, payload, siblings: int, block_tokens: int,
                out_k=None, out_v=None, payload_entries: int | None = None):
    _bf16(master_k, "master_k")
    _bf16(master_v, "master_v")
    mk = master_k.unsqueeze(0) if master_k.dim() == 4 else master_k
    mv = master_v.unsqueeze(0) if master_v.dim() == 4 else master_v
    md = plane_desc(mk)
    shape = (int(siblings),) + tuple(mk.shape[1:])
    out_k = torch.empty(shape, dtype=torch.bfloat16, device=mk.device) if out_k is None else out_k
    out_v = torch.empty(shape, dtype=torch.bfloat16, device=mk.device) if out_v is None else out_v
    pe = payload.shape[0] if payload_entries is None else int(payload_entries)
    _check(lib.kvfix_diff_gather(_ptr(mk), _ptr(mv), md, _ptr(mask), _ptr(offsets), _ptr(payload), pe,
                                 int(siblings), int(block_tokens), _ptr(out_k), _ptr(out_v),
                                 plane_desc(out_k), _stream(mk)))
    return out_k, out_v


def diff_restore(master_k, master_v, mask, offsets, payload, siblings: int, block_tokens: int,
                 delta, rope_base: float, slot_mapping, pool_k, pool_v,
                 payload_entries: int | None = None):
    """Restore every sibling into the paged pool pool_k/pool_v [layers][slots][heads][dim]
    (written in place): token t of sibling s goes to row slot_mapping[s][t] (< 0: not
    restored), keys rotated by delta[s]."""
    _bf16(master_k, "master_k")
    _bf16(master_v, "master_v")
    _bf16(pool_k, "pool_k")
    _bf16(pool_v, "pool_v")
    _i32(delta, "delta")
    _i32(slot_mapping, "slot_mapping")
    mk = master_k.unsqueeze(0) if master_k.dim() == 4 else master_k
    mv = master_v.unsqueeze(0) if master_v.dim() == 4 else master_v
    if pool_k.dim() != 4 or pool_v.shape != pool_k.shape:
        raise ValueError("pool_k and pool_v must both be [layers][slots][heads][dim]")
    if delta.numel() != int(siblings) or slot_mapping.numel() != int(siblings) * mk.shape[2]:
        raise ValueError("delta must hold one shift per sibling and slot_mapping one slot per "
                         "(sibling, token)")
    pe = payload.shape[0] if payload_entries is None else int(payload_entries)
    _check(lib.kvfix_diff_restore(_ptr(mk), _ptr(mv), plane_desc(mk), _ptr(mask), _ptr(offsets),
                                  _ptr(payload), pe, int(siblings), int(block_tokens), _ptr(delta),
                                  float(rope_base), _ptr(slot_mapping), _ptr(pool_k), _ptr(pool_v),
                                  plane_desc(pool_k.unsqueeze(0)), _stream(mk)))
    return pool_k, pool_v


def _factor(t, name, shape):
    _bf16(t, name)
    if not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}, got {tuple(t.shape)}")


def anchor_gate(v_src, a_c, b_ct, prefix: int, temperature: float = 1.0, tau: float = 0.5):
    """Reliability gate per segment.  v_src [C][L][n][H][D]; a_c [C][V][L][n][r];
    b_ct [C][V][L][H*D][r].  Returns (d [C][V] f64, g [C][V] f64, hbar [C] f64, accept [C] i32)."""
    _bf16(v_src, "v_src")
    x = v_src if v_src.dim() == 5 else v_src.unsqueeze(0)
    C, L, n, H, Dh = x.shape
    V, r = a_c.shape[1], a_c.shape[-1]
    _factor(a_c, "a_c", (C, V, L, n, r))
    _factor(b_ct, "b_ct", (C, V, L, H * Dh, r))
    dev = x.device
    d = torch.empty((C, V), dtype=torch.float64, device=dev)
    g = torch.empty_like(d)
    hbar = torch.empty(C, dtype=torch.float64, device=dev)
    acc = torch.empty(C, dtype=torch.int32, device=dev)
    desc = plane_desc(x)
    nbytes = lib.kvfix_anchor_gate_workspace_bytes(desc, V, int(prefix))
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _check(lib.kvfix_anchor_gate(_ptr(x), desc, _ptr(a_c), _ptr(b_ct), V, r, int(prefix), float(temperature),
                                 float(tau), _ptr(d), _ptr(g), _ptr(hbar), _ptr(acc), _ptr(ws), ws.numel(),
                                 _stream(x)))
    return d, g, hbar, acc


def anchor_correct(k_src, v_src, factors: dict, delta, rope_base: float, temperature: float = 1.0,
                   accept=None, out_k=None, out_v=None, w_k=None, w_v=None):
    """Token-weighted anchor correction of both planes.  k_src/v_src [C][L][n][H][D];
    factors: a_c_k, b_ct_k, a_c_v, b_ct_v, a_d_k, b_dt_k, a_d_v, b_dt_v ([C][V][L][n][r] and
    [C][V][L][H*D][r]).  Returns (out_k, out_v, w_k, w_v); w_* [C][L][n][V] float32."""
    _bf16(k_src, "k_src")
    _bf16(v_src, "v_src")
    _i32(delta, "delta")
    C, L, n, H, Dh = k_src.shape
    V, r = factors["a_c_k"].shape[1], factors["a_c_k"].shape[-1]
    names = ("a_c_k", "b_ct_k", "a_c_v", "b_ct_v", "a_d_k", "b_dt_k", "a_d_v", "b_dt_v")
    for nm in names:
        _factor(factors[nm], nm, (C, V, L, n, r) if nm.startswith("a_") else (C, V, L, H * Dh, r))
    dev = k_src.device
    out_k = torch.empty_like(k_src) if out_k is None else out_k
    out_v = torch.empty_like(v_src) if out_v is None else out_v
    w_k = torch.empty((C, L, n, V), dtype=torch.float32, device=dev) if w_k is None else w_k
    w_v = torch.empty((C, L, n, V), dtype=torch.float32, device=dev) if w_v is None else w_v
    _f32(w_k, "w_k")
    _f32(w_v, "w_v")
    if accept is not None:
        _i32(accept, "accept")
    _check(lib.kvfix_anchor_correct(_ptr(k_src), _ptr(v_src), plane_desc(k_src),
                                    *[_ptr(factors[nm]) for nm in names], V, r, float(temperature), _ptr(delta),
                                    float(rope_base), _ptr(accept), _ptr(w_k), _ptr(w_v), _ptr(out_k), _ptr(out_v),
                                    plane_desc(out_k), _stream(k_src)))
    return out_k, out_v, w_k, w_v


LAYOUT_SINGLE, LAYOUT_CHUNK, LAYOUT_GROW = 0, 1, 2


def _round_half_even(p: int, q: int) -> int:
    f, r = divmod(p, q)
    return f + (1 if 2 * r > q or (2 * r == q and f % 2) else 0)


def layout_max_rows(tokens: int, layout: int, chunk_tokens: int = 64, budget=(1, 5)) -> int:
    """The most rows a layout can choose (the size idx needs per unit)."""
    num, den = budget
    if layout == LAYOUT_CHUNK:
        nch = -(-tokens // chunk_tokens)
        c = min(nch, max(1, _round_half_even(num * tokens, den * chunk_tokens)))
        return max(1, min(tokens, c * chunk_tokens))
    return max(1, _round_half_even(num * tokens, den))


def repair_layout(scores, layout: int, chunk_tokens: int = 64, budget=(1, 5), tau: float = 0.25,
                  skip_rule: bool = True, max_rows: int | None = None):
    """scores [units][tokens] float64 (CUDA) -> (idx [units][max_rows] int32, counts [units] int32)."""
    if scores.dtype != torch.float64 or not scores.is_cuda or not scores.is_contiguous():
        raise TypeError("scores must be a contiguous CUDA float64 tensor")
    sc = scores if scores.dim() == 2 else scores.unsqueeze(0)
    U, n = sc.shape
    mr = layout_max_rows(n, layout, chunk_tokens, budget) if max_rows is None else int(max_rows)
    idx = torch.empty((U, mr), dtype=torch.int32, device=sc.device)
    counts = torch.empty(U, dtype=torch.int32, device=sc.device)
    _check(lib.kvfix_repair_layout(_ptr(sc), U, n, int(layout), int(chunk_tokens), int(budget[0]), int(budget[1]),
                                   float(tau), int(bool(skip_rule)), _ptr(idx), mr, _ptr(counts), _stream(sc)))
    return idx, counts


def repair_rows(k_io, v_io, k_fresh, v_fresh, idx, counts):
    """Overwrite rows idx[c][:counts[c]] of k_io / v_io ([C][L][n][H][D]) with the fresh rows."""
    for t, nm in ((k_io, "k_io"), (v_io, "v_io"), (k_fresh, "k_fresh"), (v_fresh, "v_fresh")):
        _bf16(t, nm)
    _i32(idx, "idx")
    _i32(counts, "counts")
    ref = k_io if k_io is not None else v_io
    fref = k_fresh if k_fresh is not None else v_fresh
    _check(lib.kvfix_repair_rows(_ptr(k_io), _ptr(v_io), plane_desc(ref), _ptr(k_fresh), _ptr(v_fresh),
                                 plane_desc(fref), _ptr(idx), idx.shape[-1], _ptr(counts), _stream(ref)))


def master_select(d_k, d_v, agents: int):
    """d_k, d_v [agents*R][n] float32 (CUDA; either may be None) -> (master int32 [1], totals [agents] f64)."""
    ref = d_k if d_k is not None else d_v
    for t, nm in ((d_k, "d_k"), (d_v, "d_v")):
        if t is not None:
            _f32(t, nm)
    A = int(agents)
    R = ref.shape[0] // A
    totals = torch.empty(A, dtype=torch.float64, device=ref.device)
    master = torch.empty(1, dtype=torch.int32, device=ref.device)
    _check(lib.kvfix_master_select(_ptr(d_k), _ptr(d_v), A, R, ref.shape[-1], _ptr(totals), _ptr(master),
                                   _stream(ref)))
    return master, totals


def diff_encode_split(master_k, master_v, sib_k, sib_v, block_tokens: int, capacity=None, sync: bool = True):
    """Per-plane block lists.  Returns ((mask_k, offsets_k, payload_k), (mask_v, offsets_v, payload_v),
    (entries_k, entries_v) or None); payload_P [cap][bt][H][D]."""
    for t, nm in ((master_k, "master_k"), (master_v, "master_v"), (sib_k, "sib_k"), (sib_v, "sib_v")):
        _bf16(t, nm)
    mk = master_k.unsqueeze(0) if master_k.dim() == 4 else master_k
    mv = master_v.unsqueeze(0) if master_v.dim() == 4 else master_v
    md, sd = plane_desc(mk), plane_desc(sib_k)
    S, L, n, H, Dh = sd.chunks, sd.layers, sd.tokens, sd.kv_heads, sd.head_dim
    bt = int(block_tokens)
    E = S * L * (n // bt)
    dev = sib_k.device
    caps = (E, E) if capacity is None else tuple(int(c) for c in capacity)
    lists = []
    for cap in caps:
        lists.append((torch.empty((E + 31) // 32, dtype=torch.int32, device=dev),
                      torch.empty(E + 1, dtype=torch.int64, device=dev),
                      torch.empty(max(cap, 1), bt, H, Dh, dtype=torch.bfloat16, device=dev)))
    entries = (ctypes.c_int64 * 2)(-1, -1)
    (mk_, ok_, pk_), (mv_, ov_, pv_) = lists
    _check(lib.kvfix_diff_encode_split(_ptr(mk), _ptr(mv), md, _ptr(sib_k), _ptr(sib_v), sd, bt, _ptr(mk_), _ptr(mv_),
                                       _ptr(ok_), _ptr(ov_), _ptr(pk_), _ptr(pv_), caps[0], caps[1],
                                       entries if sync else None, _stream(sib_k)))
    return lists[0], lists[1], ((entries[0], entries[1]) if sync else None)


def diff_gather_split(master_k, master_v, k_list, v_list, siblings: int, block_tokens: int, out_k=None,
                      out_v=None, entries=None):
    _bf16(master_k, "master_k")
    _bf16(master_v, "master_v")
    mk = master_k.unsqueeze(0) if master_k.dim() == 4 else master_k
    mv = master_v.unsqueeze(0) if master_v.dim() == 4 else master_v
    md = plane_desc(mk)
    shape = (int(siblings),) + tuple(mk.shape[1:])
    out_k = torch.empty(shape, dtype=torch.bfloat16, device=mk.device) if out_k is None else out_k
    out_v = torch.empty(shape, dtype=torch.bfloat16, device=mk.device) if out_v is None else out_v
    ek, ev = (k_list[2].shape[0], v_list[2].shape[0]) if entries is None else entries
    _check(lib.kvfix_diff_gather_split(_ptr(mk), _ptr(mv), md, _ptr(k_list[0]), _ptr(v_list[0]), _ptr(k_list[1]),
                                       _ptr(v_list[1]), _ptr(k_list[2]), _ptr(v_list[2]), int(ek), int(ev),
                                       int(siblings), int(block_tokens), _ptr(out_k), _ptr(out_v), plane_desc(out_k),
                                       _stream(mk)))
    return out_k, out_v


def diff_restore_split(master_k, master_v, k_list, v_list, siblings: int, block_tokens: int, delta,
                       rope_base: float, slot_mapping, pool_k, pool_v, entries=None):
    """diff_restore from the per-plane lists of diff_encode_split (written in place)."""
    for t, name in ((master_k, "master_k"), (master_v, "master_v"), (pool_k, "pool_k"), (pool_v, "pool_v")):
        _bf16(t, name)
    _i32(delta, "delta")
    _i32(slot_mapping, "slot_mapping")
    mk = master_k.unsqueeze(0) if master_k.dim() == 4 else master_k
    mv = master_v.unsqueeze(0) if master_v.dim() == 4 else master_v
    if pool_k.dim() != 4 or pool_v.shape != pool_k.shape:
        raise ValueError("pool_k and pool_v must both be [layers][slots][heads][dim]")
    if delta.numel() != int(siblings) or slot_mapping.numel() != int(siblings) * mk.shape[2]:
        raise ValueError("delta must hold one shift per sibling and slot_mapping one slot per "
                         "(sibling, token)")
    ek, ev = (k_list[2].shape[0], v_list[2].shape[0]) if entries is None else entries
    _check(lib.kvfix_diff_restore_split(_ptr(mk), _ptr(mv), plane_desc(mk), _ptr(k_list[0]), _ptr(v_list[0]),
                                        _ptr(k_list[1]), _ptr(v_list[1]), _ptr(k_list[2]), _ptr(v_list[2]),
                                        int(ek), int(ev), int(siblings), int(block_tokens), _ptr(delta),
                                        float(rope_base), _ptr(slot_mapping), _ptr(pool_k), _ptr(pool_v),
                                        plane_desc(pool_k.unsqueeze(0)), _stream(mk)))
    return pool_k, pool_v


def selftest_wait(limit_cycles: int, flag=None):
    """Launch the bounded-wait self test on the current stream (see kvfix_selftest_wait)."""
    if flag is not None:
        _i32(flag, "flag")
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    _check(lib.kvfix_selftest_wait(int(limit_cycles), _ptr(flag), s))


def anchor_gate_correct(k_src, v_src, factors: dict, prefix: int, delta, rope_base: float,
                        temperature: float = 1.0, tau: float = 0.5, out_k=None, out_v=None):
    """The gate and the correction in one pass (see kvfix_anchor_gate_correct).  Returns
    (out_k, out_v, w_k, w_v, d, g, hbar, accept)."""
    _bf16(k_src, "k_src")
    _bf16(v_src, "v_src")
    _i32(delta, "delta")
    C, L, n, H, Dh = k_src.shape
    V, r = factors["a_c_k"].shape[1], factors["a_c_k"].shape[-1]
    names = ("a_c_k", "b_ct_k", "a_c_v", "b_ct_v", "a_d_k", "b_dt_k", "a_d_v", "b_dt_v")
    for nm in names:
        _factor(factors[nm], nm, (C, V, L, n, r) if nm.startswith("a_") else (C, V, L, H * Dh, r))
    dev = k_src.device
    out_k = torch.empty_like(k_src) if out_k is None else out_k
    out_v = torch.empty_like(v_src) if out_v is None else out_v
    w_k = torch.empty((C, L, n, V), dtype=torch.float32, device=dev)
    w_v = torch.empty_like(w_k)
    d = torch.empty((C, V), dtype=torch.float64, device=dev)
    g = torch.empty_like(d)
    hbar = torch.empty(C, dtype=torch.float64, device=dev)
    acc = torch.empty(C, dtype=torch.int32, device=dev)
    desc = plane_desc(k_src)
    nbytes = lib.kvfix_anchor_gate_workspace_bytes(desc, V, n)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _check(lib.kvfix_anchor_gate_correct(_ptr(k_src), _ptr(v_src), desc, *[_ptr(factors[nm]) for nm in names], V, r,
                                         int(prefix), float(temperature), float(tau), _ptr(delta), float(rope_base),
                                         _ptr(d), _ptr(g), _ptr(hbar), _ptr(acc), _ptr(w_k), _ptr(w_v), _ptr(out_k),
                                         _ptr(out_v), plane_desc(out_k), _ptr(ws), ws.numel(), _stream(k_src)))
    return out_k, out_v, w_k, w_v, d, g, hbar, acc


# --------------------------------------------------------------------- paged pools

POOL_FORMATS = {"bf16": 0, "e4m3": 1, "int4": 2}


class Pool(NamedTuple):
    """A paged pool's planes (or some consecutive layers of them).
    format    "bf16", "e4m3" or "int4"
    k, v      bf16: bfloat16 [layers][slots][heads][dim]; e4m3: uint8 of that shape;
              int4: uint8 [layers][slots][heads][dim/2]
    *_scales  bf16: None; e4m3: uint8 [layers][heads][slots]; int4: bfloat16
              [layers][heads][slots][dim/32][2] (scale, zero)"""
    format: str
    k: torch.Tensor
    v: torch.Tensor
    k_scales: torch.Tensor | None = None
    v_scales: torch.Tensor | None = None

    def layer(self, i: int) -> "Pool":
        """The pool's layer i alone, as shared_attend takes it (views)."""
        one = lambda t: None if t is None else t[i:i + 1]  # noqa: E731
        return Pool(self.format, self.k[i:i + 1], self.v[i:i + 1], one(self.k_scales), one(self.v_scales))


def pool_empty(format: str, layers: int, slots: int, kv_heads: int, head_dim: int, device="cuda") -> Pool:
    """A pool of `slots` rows per layer, its contents zero."""
    if format not in POOL_FORMATS:
        raise ValueError(f"unknown pool format {format!r}")
    z = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device=device)  # noqa: E731

    def plane():
        if format == "bf16":
            return z(layers, slots, kv_heads, head_dim, dtype=torch.bfloat16), None
        if format == "e4m3":
            return (z(layers, slots, kv_heads, head_dim, dtype=torch.uint8),
                    z(layers, kv_heads, slots, dtype=torch.uint8))
        return (z(layers, slots, kv_heads, head_dim // 2, dtype=torch.uint8),
                z(layers, kv_heads, slots, head_dim // 32, 2, dtype=torch.bfloat16))

    (k, ks), (v, vs) = plane(), plane()
    return Pool(format, k, v, ks, vs)


def _raw_stream(t) -> int:
    """The current stream of a CUDA tensor's device, as an address (no Stream object on the way)."""
    if _raw_stream_of is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return _raw_stream_of(t.get_device())


def _empty(shape, stride, dtype):
    """torch.empty_strided on the current CUDA device."""
    if _empty_strided_cuda is None:
        return torch.empty_strided(shape, stride, dtype=dtype, device="cuda")
    return _empty_strided_cuda(shape, stride, dtype)


def pool_desc(pool: Pool) -> PoolDesc:
    """Descriptor of a pool; checks dtypes, devices, shapes and strides."""
    format, k, v, ks, vs = pool
    fmt = POOL_FORMATS.get(format)
    if fmt is None:
        raise ValueError(f"unknown pool format {format!r}")
    code = torch.uint8 if fmt else torch.bfloat16
    dev = k.device
    if k.dtype != code or v.dtype != code or not k.is_cuda or dev != v.device:
        raise TypeError(f"pool planes of a {format} pool must be CUDA {code} tensors on one device")
    shape, stride = k.shape, k.stride()
    if len(shape) != 4 or shape != v.shape or stride != v.stride():
        raise ValueError("pool planes must be [layers][slots][heads][width], of one shape and strides")
    L, n, H, W = shape
    sl, ss, sh, sw = stride
    if (sw != 1 or sh != W) and H * W > 1:
        raise ValueError("a pool slot's heads must be contiguous")
    if not fmt:
        return PoolDesc(0, L, n, H, W, 2 * sl if L > 1 else 0, 2 * ss if n > 1 else 2 * H * W,
                        k.data_ptr(), v.data_ptr(), None, None)
    dim = 2 * W if fmt == 2 else W
    want, kind = ((L, H, n), torch.uint8) if fmt == 1 else ((L, H, n, dim // 32, 2), torch.bfloat16)
    for s in (ks, vs):
        if s is None or s.dtype != kind or s.shape != want or not s.is_contiguous() or s.device != dev:
            raise TypeError(f"scales of this {format} pool must be contiguous {kind} tensors {want} "
                            "on the planes' device")
    return PoolDesc(fmt, L, n, H, dim, sl if L > 1 else 0, ss if n > 1 else H * W,
                    k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr())


def _rows_desc(t: torch.Tensor, name: str) -> KvDesc:
    """plane_desc of a CUDA bf16 tensor (one layer if 4-D), without a view on the way."""
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor (got {t.dtype} on {t.device})")
    shape, stride = t.shape, t.stride()
    if len(shape) == 5:
        C, L, n, H, Dh = shape
        sc, sl, st, sh, sd = stride
    elif len(shape) == 4:
        C, n, H, Dh = shape
        sc, st, sh, sd = stride
        L, sl = 1, 0
    else:
        raise ValueError(f"{name} must be 4-D or 5-D, got shape {tuple(shape)}")
    if (sd != 1 or sh != Dh) and H * Dh > 1:
        raise ValueError(f"{name} needs contiguous heads and dims (stride(-1) == 1, stride(-2) == head_dim)")
    return KvDesc(C, L, n, H, Dh, sc if C > 1 else 0, sl if L > 1 else 0, st if n > 1 else H * Dh)


def _pool_rows(k, v, slot_mapping, delta, pool):
    d = _rows_desc(k, "k")
    _launch_device(k.get_device())
    if v.dtype != torch.bfloat16 or not v.is_cuda:
        raise TypeError(f"v must be a CUDA bfloat16 tensor (got {v.dtype} on {v.device})")
    if k.shape != v.shape or k.stride() != v.stride():
        raise ValueError("k and v must have the same shape and strides")
    _i32(slot_mapping, "slot_mapping")
    if slot_mapping.numel() != d.chunks * d.tokens:
        raise ValueError(f"slot_mapping must hold {d.chunks} x {d.tokens} slots")
    if delta is not None:
        _i32(delta, "delta")
        if delta.numel() != d.chunks:
            raise ValueError(f"delta must hold {d.chunks} shifts")
    if k.device != pool.k.device or v.device != k.device or slot_mapping.device != k.device or \
            (delta is not None and delta.device != k.device):
        raise ValueError("the pool, the rows, slot_mapping and delta must be on one device")
    return d


def pool_write(pool: Pool, k, v, slot_mapping, delta=None, rope_base: float = 0.0):
    """Write rows k, v [C][L][n][H][D] (L, H, D the pool's) to pool rows slot_mapping [C][n]
    (< 0: not kept), in the pool's format, keys rotated by delta [C] first (None: as they are)."""
    pd = pool_desc(pool)
    d = _pool_rows(k, v, slot_mapping, delta, pool)
    _check(lib.kvfix_pool_write(k.data_ptr(), v.data_ptr(), d, None if delta is None else delta.data_ptr(),
                                float(rope_base), slot_mapping.data_ptr(), pd, _raw_stream(k)))


def pool_read(pool: Pool, slot_mapping, delta=None, rope_base: float = 0.0, k_out=None, v_out=None):
    """The values of pool rows slot_mapping [C][n] as bf16 planes [C][L][n][H][D], keys rotated
    by delta [C] (None: as stored).  Rows with a negative slot keep what the outputs held (zero
    in outputs allocated here)."""
    pd = pool_desc(pool)
    if k_out is None or v_out is None:
        if slot_mapping.dim() != 2:
            raise ValueError("slot_mapping must be [chunks][tokens]")
        shape = (slot_mapping.shape[0], pd.layers, slot_mapping.shape[1], pd.kv_heads, pd.head_dim)
        new = lambda: torch.zeros(shape, dtype=torch.bfloat16, device=pool.k.device)  # noqa: E731
        k_out, v_out = new() if k_out is None else k_out, new() if v_out is None else v_out
    d = _pool_rows(k_out, v_out, slot_mapping, delta, pool)
    _check(lib.kvfix_pool_read(pd, slot_mapping.data_ptr(), None if delta is None else delta.data_ptr(),
                               float(rope_base), k_out.data_ptr(), v_out.data_ptr(), d, _raw_stream(k_out)))
    return k_out, v_out


def shared_attend_workspace_bytes(q, pool: Pool, groups: int) -> int:
    A, T, Hq, D = q.shape
    return int(lib.kvfix_shared_attend_workspace_bytes(A, T, Hq, pool.k.shape[2], D, groups))


def shared_attend(q, pool: Pool, page_tokens: int, suffix_pages, suffix_len, prefix_pages=None, prefix_len=None,
                  group_begin=None, scale: float | None = None, out=None, return_lse: bool = False, workspace=None):
    """Attention of queries q [agents][T][q_heads][dim] over one layer of a pool (pool.layer(i)):
    agent a's keys are its group's prefix (the first prefix_len[g] keys on prefix_pages[g]), then
    the first suffix_len[a] on suffix_pages[a], the T newest of them its own queries' places.
    Groups are the runs of agents group_begin[g] .. group_begin[g+1].  scale: dim^-1/2 if None.
    Returns out, shaped like q, or (out, lse [agents][T][q_heads])."""
    return _attend(lib.kvfix_shared_attend, (), q, pool, page_tokens, suffix_pages, suffix_len, prefix_pages, prefix_len,
                   group_begin, scale, out, return_lse, workspace)


def tree_attend(q, pool: Pool, page_tokens: int, suffix_pages, suffix_len, tree_mask, nodes=None, prefix_pages=None,
                prefix_len=None, group_begin=None, scale: float | None = None, out=None, return_lse: bool = False,
                workspace=None):
    """shared_attend of a tree of drafts: the last nodes[a] (T if nodes is None) of agent a's own
    keys are the nodes that its first queries stand for, and node t sees of them those j <= t whose
    bit is set in tree_mask [agents][T][ceil(T/32)] int32 (see tree_masks).  Queries past nodes[a]
    give 0, and -inf.  The workspace is shared_attend's."""
    if q.dim() != 4:
        raise ValueError("q must be [agents][new tokens][heads][dim]")
    A, T, dev = q.shape[0], q.shape[1], q.get_device()
    if not _ints(dev, (tree_mask, nodes)):
        _i32(tree_mask, "tree_mask")
        if nodes is not None:
            _i32(nodes, "nodes")
        raise ValueError("tree_mask and nodes must be on q's device")
    if tree_mask.shape != (A, T, (T + 31) // 32):
        raise ValueError(f"tree_mask must be [{A}][{T}][{(T + 31) // 32}]")
    if nodes is not None and nodes.numel() != A:
        raise ValueError(f"nodes must hold {A} numbers")
    tree = (None if nodes is None else nodes.data_ptr(), tree_mask.data_ptr())
    return _attend(lib.kvfix_tree_attend, tree, q, pool, page_tokens, suffix_pages, suffix_len, prefix_pages, prefix_len,
                   group_begin, scale, out, return_lse, workspace)


def tree_masks(parents, device="cpu"):
    """Masks and depths of drafted trees from their nodes' parents (each before its children; -1:
    the node hangs on the context).  parents: a list of nodes for each agent, of any lengths.
    Returns (tree_mask int32 [agents][T][ceil(T/32)], depth int32 [agents][T], nodes int32 [agents]):
    node t of agent a stands at its context's length + depth[a][t]."""
    T = max([len(p) for p in parents], default=0)
    W = (T + 31) // 32
    mask, depth = [], []
    for p in parents:
        line, deep = [], []
        for t, up in enumerate(p):
            if not -1 <= up < t:
                raise ValueError(f"node {t} hangs on {up}: a parent comes before its children")
            line.append((line[up] if up >= 0 else 0) | 1 << t)
            deep.append(deep[up] + 1 if up >= 0 else 0)
        line += [0] * (T - len(line))
        # (bit 31 of a word is an int32's sign)
        mask.append([[((x >> 32 * w & 0xffffffff) ^ 0x80000000) - 0x80000000 for w in range(W)] for x in line])
        depth.append(deep + [0] * (T - len(deep)))
    i32 = lambda x, *shape: torch.tensor(x, dtype=torch.int32).view(*shape).to(device)  # noqa: E731
    return (i32(mask, len(parents), T, W), i32(depth, len(parents), T), i32([len(p) for p in parents], len(parents)))


def _attend(call, tree, q, pool, page_tokens, suffix_pages, suffix_len, prefix_pages, prefix_len, group_begin, scale, out,
            return_lse, workspace):
    if q.dim() != 4:
        raise ValueError("q must be [agents][new tokens][heads][dim]")
    qd, pd, dev = _rows_desc(q, "q"), pool_desc(pool), q.get_device()
    _launch_device(dev)
    A, T, Hq, Dh = q.shape
    if prefix_len is None and not (prefix_pages is None and group_begin is None):
        raise ValueError("prefix_len is required with prefix_pages and group_begin")
    groups = 0 if prefix_len is None else prefix_len.numel()
    if not _ints(dev, (suffix_pages, suffix_len)) or pool.k.get_device() != dev:
        _i32(suffix_pages, "suffix_pages")
        _i32(suffix_len, "suffix_len")
        raise ValueError("q, the pool, pages and lengths must be on one device")
    if suffix_pages.dim() != 2 or suffix_pages.shape[0] != A or suffix_len.numel() != A:
        raise ValueError(f"suffix_pages must be [{A}][pages] and suffix_len hold {A} lengths")
    shared = (None, 0, None, None)
    if groups:
        if prefix_pages is None or group_begin is None:
            raise ValueError("prefix_pages and group_begin are required with prefix_len")
        if not _ints(dev, (prefix_pages, prefix_len, group_begin)):
            _i32(prefix_pages, "prefix_pages")
            _i32(prefix_len, "prefix_len")
            _i32(group_begin, "group_begin")
            raise ValueError("q, the pool, pages and lengths must be on one device")
        if prefix_pages.dim() != 2 or prefix_pages.shape[0] != groups or group_begin.numel() != groups + 1:
            raise ValueError(f"prefix_pages must be [{groups}][pages] and group_begin hold {groups + 1} bounds")
        shared = (prefix_pages.data_ptr(), prefix_pages.shape[1], prefix_len.data_ptr(), group_begin.data_ptr())
    if out is None:
        row = Hq * Dh
        out = _empty((A, T, Hq, Dh), (T * row, row, Dh, 1), torch.bfloat16)
        od = KvDesc(A, 1, T, Hq, Dh, T * row if A > 1 else 0, 0, row)
    else:
        od = _rows_desc(out, "out")
        if out.get_device() != dev:
            raise ValueError("out and workspace must be on q's device")
    lse = _empty((A, T, Hq), (T * Hq, Hq, 1), torch.float32) if return_lse else None
    if workspace is None:
        size = lib.kvfix_shared_attend_workspace_bytes(A, T, Hq, pd.kv_heads, Dh, groups)
        workspace = _empty((size,), (1,), torch.uint8)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    else:
        size = workspace.numel() * workspace.element_size()
        if workspace.get_device() != dev:
            raise ValueError("out and workspace must be on q's device")
    _check(call(
        q.data_ptr(), qd, pd, int(page_tokens), *shared, groups, suffix_pages.data_ptr(), suffix_pages.shape[1],
        suffix_len.data_ptr(), *tree, Dh ** -0.5 if scale is None else float(scale), out.data_ptr(), od,
        None if lse is None else lse.data_ptr(), workspace.data_ptr(), size, _raw_stream(q)))
    return (out, lse) if return_lse else out


# --------------------------------------------------------------------- rotary positions

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "bands": 2, "yarn": 3}


class Rope(NamedTuple):
    """How a model turns its queries and keys (kvfix_rope).
    rotary_dim  the first values of a head that turn (None: all)
    layout      "half" (pairs i, i + rotary_dim/2) or "interleaved" (pairs 2i, 2i + 1)
    scaling     "none", "linear", "bands" or "yarn", with factor, and for the last two low, high
                (turns over the original context) and original (its tokens)
    attention   factor of cos and sin"""
    base: float
    rotary_dim: int | None = None
    layout: str = "half"
    scaling: str = "none"
    factor: float = 1.0
    low: float = 0.0
    high: float = 0.0
    original: int = 0
    attention: float = 1.0


def rope_desc(rope: Rope, head_dim: int) -> RopeDesc:
    layout, scaling = ROPE_LAYOUTS.get(rope.layout), ROPE_SCALINGS.get(rope.scaling)
    if layout is None or scaling is None:
        raise ValueError(f"unknown rope layout {rope.layout!r} or scaling {rope.scaling!r}")
    return RopeDesc(layout, head_dim if rope.rotary_dim is None else rope.rotary_dim, scaling, rope.original, rope.base,
                    rope.factor, rope.low, rope.high, rope.attention)


def rotary(q, k, positions, rope: Rope, q_out=None, k_out=None):
    """Rows q and k ([C][T][heads][dim] or [C][L][T][heads][dim]; either may be None) turned to
    positions int32 [C][T], the same in every layer.  q_out, k_out: where to (the inputs
    themselves for in place).  Returns (q_out, k_out)."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("neither queries nor keys")
    dev = ref.get_device()
    _launch_device(dev)
    if not _ints(dev, (positions,)):
        _i32(positions, "positions")
        raise ValueError("q, k, positions and outputs must be on one device")
    qi, qd, q_out, qo, qod = _turned(q, q_out, "q", dev, positions)
    ki, kd, k_out, ko, kod = _turned(k, k_out, "k", dev, positions)
    _check(lib.kvfix_rotary(qi, qd, ki, kd, positions.data_ptr(), rope_desc(rope, ref.shape[-1]), qo, qod, ko, kod,
                            _raw_stream(ref)))
    return q_out, k_out


_NO_ROWS = KvDesc()


def _turned(x, y, name, dev, positions):
    """A plane of a rotary call and where it goes: (address, descriptor, output, its address, its
    descriptor)."""
    if x is None:
        if y is not None:
            raise ValueError(f"{name}_out without {name}")
        return None, _NO_ROWS, None, None, _NO_ROWS
    d = _rows_desc(x, name)
    if positions.numel() != d.chunks * d.tokens:
        raise ValueError(f"positions must hold {d.chunks} x {d.tokens} numbers")
    if y is None:
        y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    elif y.shape != x.shape:
        raise ValueError(f"{name}_out must have {name}'s shape")
    if x.get_device() != dev or y.get_device() != dev:
        raise ValueError("q, k, positions and outputs must be on one device")
    return x.data_ptr(), d, y, y.data_ptr(), d if y is x else _rows_desc(y, name + "_out")


# --------------------------------------------------------------------- page books

def _books(pool, page_tokens, refs, pages, lens, names, more):
    """Checks the books of a pool and the call's other int32 arrays; returns the first arguments of
    the page calls."""
    pd, dev = pool_desc(pool), pool.k.get_device()
    _launch_device(dev)
    if not _ints(dev, (refs, pages, lens, *more)):
        for t, name in zip((refs, pages, lens, *more), ("refs", "pages", "lens", *names)):
            if t is not None:
                _i32(t, name)
        raise ValueError("the pool, the books and their arguments must be on one device")
    shape, lists = pages.shape, lens.numel()
    if len(shape) != 2 or lists != shape[0]:
        raise ValueError("pages must be [lists][pages] and lens hold a length for each list")
    if page_tokens < 1 or refs.numel() != pd.slots // page_tokens:
        raise ValueError(f"refs must hold a count for each of the pool's {pd.slots} / {page_tokens} pages")
    for t, name in zip(more, names):
        if t is not None and t.numel() != lists:
            raise ValueError(f"{name} must hold a number for each list")
    return pd, page_tokens, refs.data_ptr(), pages.data_ptr(), shape[1], lens.data_ptr(), lists


def _workspace(given, need, like):
    """A workspace and its bytes: the given one, or a new one beside `like`."""
    if given is None:
        return _empty((need,), (1,), torch.uint8), need
    if not given.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if given.get_device() != like.get_device():
        raise ValueError("workspace must be on the pool's device")
    return given, given.numel() * given.element_size()


def pages_extend(pool: Pool, page_tokens: int, refs, pages, lens, extra, parent=None, workspace=None):
    """Room for extra [lists] tokens behind each list of pages [lists][max_pages] with lengths lens
    [lists], all int32 and changed in place, refs [pages of the pool] the lists that hold each page.
    parent [lists]: a list of which list i, empty until now, becomes a fork first (itself: it
    grows; below 0: nothing happens).  Last pages that others hold are copied."""
    books = _books(pool, page_tokens, refs, pages, lens, ("extra", "parent"), (extra, parent))
    ws, size = _workspace(workspace, lib.kvfix_pages_extend_workspace_bytes(refs.numel(), books[-1]), refs)
    _check(lib.kvfix_pages_extend(*books, None if parent is None else parent.data_ptr(), extra.data_ptr(), ws.data_ptr(),
                                  size, _raw_stream(refs)))


def pages_cut(pool: Pool, page_tokens: int, refs, pages, lens, base, path=None, kept=None):
    """Each list keeps its first base [lists] tokens (below 0: all of it) and behind them the tokens
    base + path[i][j], j < kept[i] (path [lists][most], ascending); pages behind its new end are
    given back.  All int32, the books changed in place."""
    if (path is None) != (kept is None):
        raise ValueError("path and kept come together")
    books = _books(pool, page_tokens, refs, pages, lens, ("base", "kept"), (base, kept))
    most = 0
    if path is not None:
        if not _ints(pool.k.get_device(), (path,)):
            _i32(path, "path")
            raise ValueError("the pool, the books and their arguments must be on one device")
        if path.dim() != 2 or path.shape[0] != books[-1]:
            raise ValueError("path must be [lists][most]")
        if path.shape[1] == 0:
            # no column to keep from: one that none may be kept of, so that lists which ask for some
            # are left alone and flagged
            path = _empty((books[-1], 1), (1, 1), torch.int32)
            path.fill_(-1)
        most = path.shape[1]
    _check(lib.kvfix_pages_cut(*books, base.data_ptr(), None if path is None else path.data_ptr(), most,
                               None if kept is None else kept.data_ptr(), _raw_stream(refs)))


def pages_compact(pool: Pool, page_tokens: int, refs, pages, lens, workspace=None):
    """Pages in use move to the front of the pool, refs and the lists follow.  Returns the number of
    pages in use, int32 [1] on the device."""
    books = _books(pool, page_tokens, refs, pages, lens, (), ())
    live = _empty((1,), (1,), torch.int32)
    ws, size = _workspace(workspace, lib.kvfix_pages_compact_workspace_bytes(refs.numel()), refs)
    _check(lib.kvfix_pages_compact(*books, live.data_ptr(), ws.data_ptr(), size, _raw_stream(refs)))
    return live
