"""ctypes binding of libsn.so (include/sn.h).

Argument marshalling only: every stage of the energy/force path runs in the
HIP library.  PyTorch supplies device memory and the current stream.  If the
compiled library is missing, loading fails loudly; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsn.so")

SN_OK = 0
SN_ERR_INVALID = -1
SN_ERR_CAPACITY = -2
SN_ERR_BOX = -3
SN_ERR_HIP = -4
SN_ERR_NONFINITE = -5
SN_ERR_WORKSPACE = -6
SN_ERR_ROW = -7
SN_MAX_ROW = 2048
SN_MD_GRAPH = 1
SN_F32 = 0
SN_BF16 = 1
SN_ACT_NONE = 0
SN_ACT_SSP = 1
SN_ACT_SILU = 2
SN_MAX_HEAD_DIM = 128
SN_MAX_BUCKETS = 64
SN_MAX_BUCKET_SPAN = 2046
SN_MAX_AXES = 8
SN_CODES_NONE = 0
SN_CODES_INT8 = 1
SN_CODES_E4M3 = 2

EXPORTED = (
    "sn_param_count", "sn_param_offsets", "sn_quantize_filter_weights", "sn_workspace_bytes",
    "sn_status_string", "sn_version", "sn_build_csr_neighbors", "sn_energy_forces", "sn_verlet_step",
    "sn_filter_forward", "sn_read_status", "sn_profile_enable", "sn_profile_classes", "sn_profile_name",
    "sn_profile_collect", "sn_energy_forces_static",
    "sn_relative_thresholds", "sn_cross_attention_workspace_bytes", "sn_cross_attention_forward",
    "sn_cross_attention_forward_train", "sn_cross_attention_backward", "sn_group_norm_workspace_bytes", "sn_group_norm_forward",
    "sn_group_norm_backward",
    "sn_rotary_frequencies", "sn_head_rotary_workspace_bytes", "sn_head_rotary_forward", "sn_head_rotary_backward",
    "sn_cache_workspace_bytes", "sn_cache_write", "sn_cache_read", "sn_cache_attend",
)
SN_STATIC_SCRATCH_BYTES = 64 << 20


class SnSystem(ctypes.Structure):
    _fields_ = [("n_atoms", ctypes.c_int32), ("n_replicas", ctypes.c_int32),
                ("replica_ptr", ctypes.c_void_p), ("types", ctypes.c_void_p),
                ("periodic", ctypes.c_int32), ("box", ctypes.c_float * 3)]


class SnModel(ctypes.Structure):
    _fields_ = [("n_types", ctypes.c_int32), ("n_interactions", ctypes.c_int32),
                ("n_features", ctypes.c_int32), ("n_rbf", ctypes.c_int32),
                ("cutoff", ctypes.c_float), ("rbf_lo", ctypes.c_float), ("rbf_hi", ctypes.c_float),
                ("rbf_gamma", ctypes.c_float), ("filter_format", ctypes.c_int32),
                ("params", ctypes.c_void_p), ("qweights", ctypes.c_void_p), ("qscales", ctypes.c_void_p),
                ("filter_math", ctypes.c_int32)]


class SnCrossAttention(ctypes.Structure):
    _fields_ = [("n_segments", ctypes.c_int32), ("n_q", ctypes.c_int32), ("n_k", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("max_k", ctypes.c_int32),
                ("q_ptr", ctypes.c_void_p), ("k_ptr", ctypes.c_void_p),
                ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("keep", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("n_buckets", ctypes.c_int32),
                ("thresholds", ctypes.c_void_p), ("q_pos", ctypes.c_void_p), ("k_pos", ctypes.c_void_p)]


class SnGroupNorm(ctypes.Structure):
    _fields_ = [("n_segments", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("row_ptr", ctypes.c_void_p), ("n_channels", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p)]


class SnHeadRotary(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("eps", ctypes.c_float), ("n_pairs", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("freqs", ctypes.c_void_p), ("axes", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p)]


class SnCache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("codes", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("n_sequences", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("row_ptr", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("n_heads", ctypes.c_int32), ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("window", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64)]


class SnError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_LIB = None


def lib() -> ctypes.CDLL:
    """Load libsn.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m schnet_cfconv_force_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    P64 = ctypes.POINTER(ctypes.c_int64)
    PS, PM = ctypes.POINTER(SnSystem), ctypes.POINTER(SnModel)
    sig = {
        "sn_param_count": (i64, [i32, i32, i32, i32]),
        "sn_param_offsets": (i32, [i32, i32, i32, i32, P64, i32]),
        "sn_quantize_filter_weights": (i32, [i32, i32, i32, i32, vp, vp, vp]),
        "sn_workspace_bytes": (sz, [PM, PS, i64]),
        "sn_status_string": (ctypes.c_char_p, [i32]),
        "sn_version": (i32, []),
        "sn_build_csr_neighbors": (i32, [PS, vp, f32, vp, vp, vp, i64, P64, vp, sz, vp]),
        "sn_energy_forces": (i32, [PM, PS, vp, vp, vp, vp, i64, vp, vp, vp, sz, vp]),
        "sn_energy_forces_static": (i32, [PM, PS, vp, vp, vp, vp, i64, vp, vp, vp, vp]),
        "sn_verlet_step": (i32, [PM, PS, vp, vp, vp, vp, f32, f32, i32, i32, f32, vp, vp, vp, i64, P64, vp, vp, vp,
                                 ctypes.POINTER(ctypes.c_int32), ctypes.c_uint32, vp, sz, vp]),
        "sn_filter_forward": (i32, [PM, i32, vp, i64, vp, vp, sz, vp]),
        "sn_read_status": (i32, [vp, vp]),
        "sn_profile_enable": (None, [i32]),
        "sn_profile_classes": (i32, []),
        "sn_profile_name": (ctypes.c_char_p, [i32]),
        "sn_profile_collect": (i32, [ctypes.POINTER(ctypes.c_double), P64]),
        "sn_relative_thresholds": (i32, [i32, i32, vp]),
        "sn_cross_attention_workspace_bytes": (sz, [vp]),
        "sn_cross_attention_forward": (i32, [vp, vp, vp, vp, sz, vp]),
        "sn_cross_attention_forward_train": (i32, [vp, vp, vp, vp, vp, sz, vp]),
        "sn_cross_attention_backward": (i32, [vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, vp, sz, vp]),
        "sn_group_norm_workspace_bytes": (sz, [vp]),
        "sn_group_norm_forward": (i32, [vp, vp, vp, vp, vp, sz, vp]),
        "sn_group_norm_backward": (i32, [vp, vp, vp, vp, i64, vp, vp, vp, vp, sz, vp]),
        "sn_rotary_frequencies": (i32, [i32, vp, ctypes.c_double, i32, vp, vp]),
        "sn_head_rotary_workspace_bytes": (sz, [vp]),
        "sn_head_rotary_forward": (i32, [vp, vp, vp, vp, sz, vp]),
        "sn_head_rotary_backward": (i32, [vp, vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, vp, sz, vp]),
        "sn_cache_workspace_bytes": (sz, [vp]),
        "sn_cache_write": (i32, [vp, vp, i64, i64, vp, i64, i64, vp, sz, vp]),
        "sn_cache_read": (i32, [vp, vp, vp, vp, sz, vp]),
        "sn_cache_attend": (i32, [vp, vp, vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = L
    return L


def status_string(st: int) -> str:
    return lib().sn_status_string(st).decode()


def _check(st: int, what: str):
    if st != SN_OK:
        raise SnError(st, what)


# ------------------------------------------------------------------ host helpers

def param_offsets(n_types: int, n_interactions: int, n_features: int, n_rbf: int) -> np.ndarray:
    n = 9 * n_interactions + 6
    buf = (ctypes.c_int64 * n)()
    got = lib().sn_param_offsets(n_types, n_interactions, n_features, n_rbf, buf, n)
    if got != n:
        raise SnError(SN_ERR_INVALID, "sn_param_offsets")
    return np.frombuffer(buf, dtype=np.int64).copy()


def pack_params(params: dict, hyper: dict) -> np.ndarray:
    """Place named float32 weights into the packed layout the library reports."""
    T, I, F, K = (hyper[k] for k in ("n_types", "n_interactions", "n_features", "n_rbf"))
    off = param_offsets(T, I, F, K)
    out = np.zeros(off[-1], np.float32)
    keys = ("W_in", "A1", "b1", "A2", "b2", "Wo1", "bo1", "Wo2", "bo2")
    arrays = [params["emb"]]
    for blk in params["interactions"]:
        arrays += [blk[k] for k in keys]
    arrays += [params["R1"], params["c1"], params["R2"], np.reshape(params["c2"], (1,))]
    for k, a in enumerate(arrays):
        a = np.asarray(a, np.float32).ravel()
        if off[k] + a.size != off[k + 1]:
            raise ValueError(f"parameter {k} has {a.size} values, layout expects {off[k + 1] - off[k]}")
        out[off[k]:off[k + 1]] = a
    return out


def quantize_filter_weights(packed: np.ndarray, hyper: dict):
    """Host int16 per-output-channel quantisation of every A1, A2 (sn_quantize_filter_weights)."""
    T, I, F, K = (hyper[k] for k in ("n_types", "n_interactions", "n_features", "n_rbf"))
    packed = np.ascontiguousarray(packed, np.float32)
    q = np.zeros(I * (K * F + F * F), np.int16)
    s = np.zeros(I * 2 * F, np.float32)
    _check(lib().sn_quantize_filter_weights(T, I, F, K, packed.ctypes.data, q.ctypes.data, s.ctypes.data),
           "sn_quantize_filter_weights")
    return q, s


# ------------------------------------------------------------------ device objects

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


class Model:
    """Device copy of the packed weights plus the hyper-parameters (sn_model)."""

    def __init__(self, params: dict, hyper: dict, filter_format: int = 0, filter_math: int = 0, device="cuda"):
        torch = _torch()
        self.hyper = dict(hyper)
        self.filter_format = int(filter_format)
        self.filter_math = int(filter_math)
        packed = pack_params(params, hyper)
        self.params = torch.from_numpy(packed).to(device)
        self.qweights = self.qscales = None
        if self.filter_format == 1:
            q, s = quantize_filter_weights(packed, hyper)
            self.qweights = torch.from_numpy(q).to(device)
            self.qscales = torch.from_numpy(s).to(device)
        h = self.hyper
        self.c = SnModel(h["n_types"], h["n_interactions"], h["n_features"], h["n_rbf"], h["cutoff"],
                         h["rbf_lo"], h["rbf_hi"], h["rbf_gamma"], self.filter_format, _ptr(self.params),
                         _ptr(self.qweights), _ptr(self.qscales), self.filter_math)


class System:
    """Device copy of replica_ptr and types plus the box (sn_system)."""

    def __init__(self, replica_ptr, types, box=None, device="cuda"):
        torch = _torch()
        self.replica_ptr = torch.as_tensor(np.asarray(replica_ptr, np.int32)).to(device)
        self.types = torch.as_tensor(np.asarray(types, np.int32)).to(device)
        self.n_atoms = int(self.types.numel())
        self.n_replicas = int(self.replica_ptr.numel()) - 1
        self.box = None if box is None else [float(v) for v in box]
        b = (ctypes.c_float * 3)(*(self.box or [0.0, 0.0, 0.0]))
        self.c = SnSystem(self.n_atoms, self.n_replicas, _ptr(self.replica_ptr), _ptr(self.types),
                          1 if box is not None else 0, b)


def workspace_bytes(model: Optional[Model], system: System, max_edges: int) -> int:
    mp = ctypes.byref(model.c) if model is not None else None
    return int(lib().sn_workspace_bytes(mp, ctypes.byref(system.c), int(max_edges)))


def workspace(model: Optional[Model], system: System, max_edges: int, device="cuda"):
    torch = _torch()
    n = workspace_bytes(model, system, max_edges)
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    pad = (-ws.data_ptr()) % 256
    return ws[pad:pad + n]


def build_csr_neighbors(system: System, pos, r_list: float, capacity: int, ws, stream=None):
    """sn_build_csr_neighbors -> (row_ptr, col_idx, rev_idx, n_edges); raises SnError on failure."""
    torch = _torch()
    dev = pos.device
    row_ptr = torch.empty(system.n_atoms + 1, dtype=torch.int32, device=dev)
    col = torch.empty(max(capacity, 1), dtype=torch.int32, device=dev)
    rev = torch.empty(max(capacity, 1), dtype=torch.int32, device=dev)
    ne = ctypes.c_int64(0)
    st = lib().sn_build_csr_neighbors(ctypes.byref(system.c), pos.data_ptr(), float(r_list), row_ptr.data_ptr(),
                                      col.data_ptr(), rev.data_ptr(), int(capacity), ctypes.byref(ne),
                                      ws.data_ptr(), ws.numel(), _stream(stream))
    if st != SN_OK:
        err = SnError(st, "sn_build_csr_neighbors")
        err.n_edges = ne.value
        raise err
    E = ne.value
    return row_ptr, col[:E], rev[:E], E


def build_csr_status(system: System, pos, r_list: float, capacity: int, ws, stream=None):
    """Like build_csr_neighbors but returns (status, n_edges) instead of raising."""
    torch = _torch()
    dev = pos.device
    row_ptr = torch.empty(system.n_atoms + 1, dtype=torch.int32, device=dev)
    col = torch.empty(max(capacity, 1), dtype=torch.int32, device=dev)
    rev = torch.empty(max(capacity, 1), dtype=torch.int32, device=dev)
    ne = ctypes.c_int64(0)
    st = lib().sn_build_csr_neighbors(ctypes.byref(system.c), pos.data_ptr(), float(r_list), row_ptr.data_ptr(),
                                      col.data_ptr(), rev.data_ptr(), int(capacity), ctypes.byref(ne),
                                      ws.data_ptr(), ws.numel(), _stream(stream))
    return st, ne.value


def energy_forces(model: Model, system: System, pos, row_ptr, col, rev, n_edges: int, ws, energy=None,
                  forces=None, stream=None):
    """sn_energy_forces -> (energy[B], forces[N,3]) device tensors."""
    torch = _torch()
    dev = pos.device
    if energy is None:
        energy = torch.empty(system.n_replicas, dtype=torch.float32, device=dev)
    if forces is None:
        forces = torch.empty((system.n_atoms, 3), dtype=torch.float32, device=dev)
    st = lib().sn_energy_forces(ctypes.byref(model.c), ctypes.byref(system.c), pos.data_ptr(), row_ptr.data_ptr(),
                                col.data_ptr(), rev.data_ptr(), int(n_edges), energy.data_ptr(), forces.data_ptr(),
                                ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "sn_energy_forces")
    return energy, forces


def energy_forces_static(model: Model, system: System, pos, row_ptr, col, rev, n_edges: int, energy=None,
                         forces=None, status=None, stream=None):
    """sn_energy_forces_static (no workspace, nothing allocated by the library) -> (energy[B], forces[N,3]).
    status (optional int32 device tensor [1]) receives the call's device status in stream order."""
    torch = _torch()
    dev = pos.device
    if energy is None:
        energy = torch.empty(system.n_replicas, dtype=torch.float32, device=dev)
    if forces is None:
        forces = torch.empty((system.n_atoms, 3), dtype=torch.float32, device=dev)
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1 or status.device != dev):
        raise ValueError("status must be an int32 tensor on the device with at least one value")
    st = lib().sn_energy_forces_static(ctypes.byref(model.c), ctypes.byref(system.c), pos.data_ptr(),
                                       row_ptr.data_ptr(), col.data_ptr(), rev.data_ptr(), int(n_edges),
                                       energy.data_ptr(), forces.data_ptr(), _ptr(status), _stream(stream))
    _check(st, "sn_energy_forces_static")
    return energy, forces


def verlet_step(model: Model, system: System, pos, vel, forces, inv_mass, dt: float, force_to_accel: float,
                n_steps: int, r_list: float, capacity: int, ws, epot_log=None, ekin_log=None, csr=None,
                stream=None, edge_log=None, rebuild_every: int = 1, graph: bool = False):
    """sn_verlet_step; pos, vel, forces are updated in place.  Returns (row_ptr, col, rev, n_edges).
    epot_log, ekin_log (optional float64 device tensors [n_steps, B]) receive each step's replica energies,
    edge_log (optional int32 device tensor [n_steps]) each step's edge count.
    rebuild_every != 1 keeps a list built at r_list = cutoff + skin across steps (rebuilt on schedule
    and when an atom drifts beyond skin/2); graph=True replays one rebuild interval as a HIP graph."""
    torch = _torch()
    dev = pos.device
    if csr is None:
        row_ptr = torch.empty(system.n_atoms + 1, dtype=torch.int32, device=dev)
        col = torch.empty(max(capacity, 1), dtype=torch.int32, device=dev)
        rev = torch.empty(max(capacity, 1), dtype=torch.int32, device=dev)
    else:
        row_ptr, col, rev = csr
    # the logs are written by the device: wrong types or sizes would be written out of bounds
    for name, t, dt_ in (("epot_log", epot_log, torch.float64), ("ekin_log", ekin_log, torch.float64),
                         ("edge_log", edge_log, torch.int32)):
        need = n_steps * (system.n_replicas if name != "edge_log" else 1)
        if t is not None and (t.dtype != dt_ or t.numel() < need or not t.is_contiguous() or t.device != dev):
            raise ValueError(f"{name} must be a contiguous {dt_} tensor on {dev} with at least {need} values")
    ne = ctypes.c_int64(0)
    done = ctypes.c_int32(0)
    st = lib().sn_verlet_step(ctypes.byref(model.c), ctypes.byref(system.c), pos.data_ptr(), vel.data_ptr(),
                              forces.data_ptr(), inv_mass.data_ptr(), float(dt), float(force_to_accel),
                              int(n_steps), int(rebuild_every), float(r_list), row_ptr.data_ptr(), col.data_ptr(),
                              rev.data_ptr(), int(capacity), ctypes.byref(ne), _ptr(epot_log), _ptr(ekin_log),
                              _ptr(edge_log), ctypes.byref(done), SN_MD_GRAPH if graph else 0, ws.data_ptr(),
                              ws.numel(), _stream(stream))
    if st != SN_OK:
        err = SnError(st, "sn_verlet_step")
        err.steps_done = done.value
        err.n_edges = ne.value
        raise err
    return row_ptr, col[:ne.value], rev[:ne.value], ne.value


def filter_forward(model: Model, interaction: int, d, ws, phi=None, stream=None):
    """sn_filter_forward: phi[n, F] = ssp(rbf(d) A1 + b1) A2 + b2 (no envelope); ws: a workspace."""
    torch = _torch()
    n = d.numel()
    if phi is None:
        phi = torch.empty((n, model.hyper["n_features"]), dtype=torch.float32, device=d.device)
    _check(lib().sn_filter_forward(ctypes.byref(model.c), int(interaction), d.data_ptr(), n, phi.data_ptr(),
                                   ws.data_ptr(), ws.numel(), _stream(stream)), "sn_filter_forward")
    return phi


def read_status(ws, stream=None) -> int:
    return int(lib().sn_read_status(ws.data_ptr(), _stream(stream)))


# ------------------------------------------------------------------ context operators
#
# `stream` of the calls below: None is the current stream.  Another one waits for the current stream's work so far, so
# inputs and workspaces that were made there are ready; what uses the outputs elsewhere has to wait for it.
# The calls record no graph, whether or not an input requires a gradient: the backward calls are the caller's to make
# (examples/context_embedding.py wraps both in autograd functions).

_ACTIVATIONS = {"none": SN_ACT_NONE, "ssp": SN_ACT_SSP, "silu": SN_ACT_SILU}


def _row_type(dtype) -> int:
    torch = _torch()
    if dtype == torch.float32:
        return SN_F32
    if dtype == torch.bfloat16:
        return SN_BF16
    raise ValueError(f"dtype must be torch.float32 or torch.bfloat16, not {dtype}")


def _ragged(ptr, name: str):
    """Checked host copy of a segment pointer array and its longest segment."""
    ptr = np.asarray(ptr, np.int64).ravel()
    if ptr.size < 2 or ptr[0] != 0 or np.any(np.diff(ptr) < 0) or ptr[-1] > np.iinfo(np.int32).max:
        raise ValueError(f"{name} must be a non-decreasing array of B + 1 >= 2 row offsets that begins with 0")
    return ptr.astype(np.int32), int(np.diff(ptr).max())


def _int32(value, name: str) -> int:
    """A whole number that a descriptor holds in 32 bits (ctypes keeps the lowest 32 of a larger one, silently)."""
    n = int(value)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name} must be within 32 bits, not {n}")
    return n


def _int32s(values, name: str):
    """The same for an array: its own int32 copy, flat."""
    wide = np.asarray(values, np.int64).ravel()
    narrow = wide.astype(np.int32)
    if not np.array_equal(wide, narrow):
        raise ValueError(f"{name} must be within 32 bits")
    return narrow


def _rows(t, name: str, shape, dtype, device):
    """Check a row tensor (its last index contiguous); returns its strides."""
    strides = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.device != device or (strides[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must be a {dtype} tensor {tuple(shape)} on {device} whose last index is contiguous, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device} with strides {strides}")
    return strides


def _gradient(t):
    """A gradient as it came, or laid out anew where its last index is not contiguous: the backward pass of a sum hands
    down one number in every place, with strides of zero."""
    strides = t.stride()
    return t.contiguous() if strides and strides[-1] != 1 else t


def _flat(t, name: str, shape, dtypes, device) -> int:
    """Check an optional contiguous tensor; returns its address or 0."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype not in dtypes or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtypes[0]} tensor {tuple(shape)} on {device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _launch(plan, entry, stream, ws, tensors, *args):
    """Call an entry point with `args`, the workspace and the stream, on the plan's device.

    An explicit stream waits for what the current one has been given so far (the outputs' memory may still be in use
    there, and the inputs or the workspace's zeroing on their way), and `tensors`, all of the call's, are tied to it."""
    index = plan.index
    # the kernels write the workspace: a host address there would fault (get_device() is -1 for a host tensor)
    if index is None or ws.get_device() != index or ws.dtype is not plan.byte or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous torch.uint8 tensor on the plan's GPU, not {ws.dtype} on {ws.device} "
                         f"(the plan lies on {plan.device})")
    raw = plan.current_stream(index)
    if stream is not None and stream.cuda_stream != raw:
        if stream.device != plan.device:
            raise ValueError(f"the stream belongs to {stream.device}, the plan to {plan.device}")
        stream.wait_stream(_torch().cuda.current_stream(index))
        for t in (ws, *plan.pointers, *tensors):
            if t is not None:
                t.record_stream(stream)
        raw = stream.cuda_stream
    if plan.current_device() == index:
        st = entry(*args, ws.data_ptr(), ws.numel(), raw)
    else:
        with _torch().cuda.device(index):
            st = entry(*args, ws.data_ptr(), ws.numel(), raw)
    if st != SN_OK:
        raise SnError(st, entry.__name__)


def _current_getters():
    """A function from a device index to its current raw stream, and one to the current device's index (torch's own
    accessors where it has them: short calls are bound by the host)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    return raw or (lambda index: torch.cuda.current_stream(index).cuda_stream), device or torch.cuda.current_device


def _zeroed_workspace(plan):
    torch = _torch()
    ws = torch.empty(plan.workspace_bytes + 256, dtype=torch.uint8, device=plan.device)
    ws = ws[(-ws.data_ptr()) % 256:][:plan.workspace_bytes]
    ws[:256].zero_()      # the status words
    return ws


def relative_thresholds(n_buckets: int = 32, max_distance: int = 128) -> np.ndarray:
    """sn_relative_thresholds: int32 [n_buckets - 1]; bucket(rel) = number of thresholds <= rel.

    Logarithmic by -rel for rel <= 0 and by rel - 1 for rel > 0.  For a table trained with |rel| on both sides, lower
    the thresholds above 1 by one (thr[thr > 1] -= 1) and put its columns in order of rel."""
    out = np.zeros(max(int(n_buckets) - 1, 1), np.int32)
    _check(lib().sn_relative_thresholds(int(n_buckets), int(max_distance), out.ctypes.data), "sn_relative_thresholds")
    return out


# the fields of SnCrossAttention and SnGroupNorm that a call fills in: everything from q and from x on
_ATTENTION_CALL = struct.Struct("@PPP6qPPiPPP")
_NORM_CALL = struct.Struct("@PqPP")


class CrossAttention:
    """Segment pointers, head layout and position buckets of a cross attention (sn_cross_attention).

    q_ptr, k_ptr: host row offsets [B + 1] of the query and the key/value segments.
    thresholds: int32 [n_buckets - 1] (see relative_thresholds), needed where a bias is given.
    scale: default 1 / sqrt(head_dim)."""

    def __init__(self, q_ptr, k_ptr, n_heads: int, n_kv_heads: int, head_dim: int, dtype=None, scale=None,
                 thresholds=None, device="cuda"):
        torch = _torch()
        self.dtype = torch.float32 if dtype is None else dtype
        code = _row_type(self.dtype)
        qp, max_q = _ragged(q_ptr, "q_ptr")
        kp, max_k = _ragged(k_ptr, "k_ptr")
        if qp.size != kp.size:
            raise ValueError(f"q_ptr has {qp.size - 1} segments, k_ptr {kp.size - 1}")
        self.thresholds = None if thresholds is None else _int32s(thresholds, "thresholds")
        self.n_buckets = 0 if self.thresholds is None else self.thresholds.size + 1
        self.q_ptr = torch.from_numpy(qp).to(device)
        self.k_ptr = torch.from_numpy(kp).to(device)
        self.device = self.q_ptr.device
        self.n_q, self.n_k = int(qp[-1]), int(kp[-1])
        self.n_heads, self.n_kv_heads = _int32(n_heads, "n_heads"), _int32(n_kv_heads, "n_kv_heads")
        self.head_dim = _int32(head_dim, "head_dim")
        self.scale = float(head_dim) ** -0.5 if scale is None else float(scale)
        # sizes are checked with the bias slot set, so that the bucket count is checked too
        self.c = SnCrossAttention(qp.size - 1, self.n_q, self.n_k, max_q, max_k, _ptr(self.q_ptr), _ptr(self.k_ptr),
                                  self.n_heads, self.n_kv_heads, self.head_dim, code, self.scale)
        self.c.n_buckets = self.n_buckets
        self.c.thresholds = None if self.thresholds is None else self.thresholds.ctypes.data
        self.c.bias = 16 if self.n_buckets else None
        self.workspace_bytes = int(lib().sn_cross_attention_workspace_bytes(ctypes.byref(self.c)))
        self.c.bias = None
        if self.workspace_bytes == 0:
            raise SnError(SN_ERR_INVALID, "sn_cross_attention")
        self.head = bytes(self.c)[:SnCrossAttention.q.offset]
        self.pointers = (self.q_ptr, self.k_ptr)
        self.index, self.byte = self.device.index, torch.uint8
        self.current_stream, self.current_device = _current_getters()
        self.q_shape = torch.Size((self.n_q, self.n_heads, self.head_dim))
        self.k_shape = torch.Size((self.n_k, self.n_kv_heads, self.head_dim))

    def _bind(self, q, k, v, bias, q_pos, k_pos, keep) -> bytes:
        """The descriptor of one call (its own bytes: calls from several threads share nothing)."""
        torch, device, dtype = _torch(), self.device, self.dtype
        qs, qh, _ = _rows(q, "q", self.q_shape, dtype, device)
        ks, kh, _ = _rows(k, "k", self.k_shape, dtype, device)
        vs, vh, _ = _rows(v, "v", self.k_shape, dtype, device)
        if bias is not None and not self.n_buckets:
            raise ValueError("a bias needs the plan's thresholds")
        return self.head + _ATTENTION_CALL.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, qh, ks, kh, vs, vh,
            _flat(keep, "keep", (self.n_k,), (torch.bool, torch.uint8), device),
            _flat(bias, "bias", (self.n_heads, self.n_buckets), (torch.float32,), device),
            self.n_buckets, self.c.thresholds or 0,
            _flat(q_pos, "q_pos", (self.n_q,), (torch.int32,), device),
            _flat(k_pos, "k_pos", (self.n_k,), (torch.int32,), device))


def cross_attention_workspace(plan: CrossAttention):
    """A workspace (status words zeroed) for the plan's calls; calls that share one must be ordered on a stream."""
    return _zeroed_workspace(plan)


def cross_attention_forward(plan: CrossAttention, q, k, v, ws, bias=None, q_pos=None, k_pos=None, keep=None,
                            save: bool = False, stream=None):
    """sn_cross_attention_forward -> o [n_q, H, D]; with save=True -> (o, saved), saved = (o before its rounding, lse)
    for the backward pass (sn_cross_attention_forward_train).  q [n_q, H, D], k and v [n_k, Hkv, D]; bias float32
    [H, n_buckets]; q_pos [n_q] and k_pos [n_k] int32 (default: the index in the segment); keep bool [n_k], False:
    the key is absent."""
    torch = _torch()
    op = plan._bind(q, k, v, bias, q_pos, k_pos, keep)
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    inputs = (q, k, v, bias, q_pos, k_pos, keep)
    if not save:
        _launch(plan, lib().sn_cross_attention_forward, stream, ws, (*inputs, o), op, o.data_ptr(), None)
        return o
    lse = torch.empty(plan.q_shape[:2], dtype=torch.float32, device=plan.device)
    rows = o if plan.dtype == torch.float32 else torch.empty(plan.q_shape, dtype=torch.float32, device=plan.device)
    _launch(plan, lib().sn_cross_attention_forward_train, stream, ws, (*inputs, o, rows, lse), op, o.data_ptr(),
            rows.data_ptr(), lse.data_ptr())
    return o, (rows, lse)


def cross_attention_backward(plan: CrossAttention, q, k, v, saved, d_o, ws, bias=None, q_pos=None, k_pos=None,
                             keep=None, stream=None):
    """sn_cross_attention_backward -> (dq, dk, dv, dbias) from the forward's `saved` and the gradient d_o of o (any
    strides; copied if its last index is not contiguous); dbias is None without a bias.  The other arguments are the
    forward's."""
    torch = _torch()
    op = plan._bind(q, k, v, bias, q_pos, k_pos, keep)
    rows, lse = saved
    d_o = _gradient(d_o)
    gs, gh, _ = _rows(d_o, "d_o", plan.q_shape, plan.dtype, plan.device)
    dq = torch.empty_like(q, memory_format=torch.contiguous_format)
    dk = torch.empty_like(k, memory_format=torch.contiguous_format)
    dv = torch.empty_like(v, memory_format=torch.contiguous_format)
    dbias = None if bias is None else torch.empty_like(bias)
    _launch(plan, lib().sn_cross_attention_backward, stream, ws,
            (q, k, v, rows, lse, d_o, bias, q_pos, k_pos, keep, dq, dk, dv, dbias), op,
            _flat(rows, "saved[0]", plan.q_shape, (torch.float32,), plan.device),
            _flat(lse, "saved[1]", plan.q_shape[:2], (torch.float32,), plan.device), d_o.data_ptr(), gs, gh,
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(dbias))
    return dq, dk, dv, dbias


class GroupNorm:
    """Segment pointers, groups and activation of a group norm (sn_group_norm); row_ptr: host row offsets [B + 1]."""

    def __init__(self, row_ptr, n_channels: int, n_groups: int, activation: str = "none", eps: float = 1e-5,
                 dtype=None, device="cuda"):
        torch = _torch()
        self.dtype = torch.float32 if dtype is None else dtype
        code = _row_type(self.dtype)
        if activation not in _ACTIVATIONS:
            raise ValueError(f"activation must be one of {tuple(_ACTIVATIONS)}, not {activation!r}")
        rp, longest = _ragged(row_ptr, "row_ptr")
        self.row_ptr = torch.from_numpy(rp).to(device)
        self.device = self.row_ptr.device
        self.n_segments, self.n_rows = rp.size - 1, int(rp[-1])
        self.n_channels, self.n_groups = _int32(n_channels, "n_channels"), _int32(n_groups, "n_groups")
        self.c = SnGroupNorm(self.n_segments, self.n_rows, longest, _ptr(self.row_ptr), self.n_channels,
                             self.n_groups, _ACTIVATIONS[activation], code, float(eps))
        self.workspace_bytes = int(lib().sn_group_norm_workspace_bytes(ctypes.byref(self.c)))
        if self.workspace_bytes == 0:
            raise SnError(SN_ERR_INVALID, "sn_group_norm")
        self.head = bytes(self.c)[:SnGroupNorm.x.offset]
        self.pointers = (self.row_ptr,)
        self.index, self.byte = self.device.index, torch.uint8
        self.current_stream, self.current_device = _current_getters()
        self.shape = torch.Size((self.n_rows, self.n_channels))

    def _bind(self, x, gamma, beta) -> bytes:
        """The descriptor of one call (its own bytes: calls from several threads share nothing)."""
        f32 = (_torch().float32,)
        stride, _ = _rows(x, "x", self.shape, self.dtype, self.device)
        return self.head + _NORM_CALL.pack(x.data_ptr(), stride,
                                           _flat(gamma, "gamma", (self.n_channels,), f32, self.device),
                                           _flat(beta, "beta", (self.n_channels,), f32, self.device))


def group_norm_workspace(plan: GroupNorm):
    """A workspace (status words zeroed) for the plan's calls; calls that share one must be ordered on a stream."""
    return _zeroed_workspace(plan)


def group_norm_forward(plan: GroupNorm, x, gamma, beta, ws, save: bool = False, stream=None):
    """sn_group_norm_forward -> y [n_rows, C]; with save=True -> (y, saved), saved = (mean, rstd) [B, n_groups].
    gamma, beta: float32 [C], or None for 1 and 0."""
    torch = _torch()
    op = plan._bind(x, gamma, beta)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    mean = rstd = None
    if save:
        mean, rstd = torch.empty((2, plan.n_segments, plan.n_groups), dtype=torch.float32, device=plan.device).unbind(0)
    _launch(plan, lib().sn_group_norm_forward, stream, ws, (x, gamma, beta, y, mean, rstd), op, y.data_ptr(), _ptr(mean),
            _ptr(rstd))
    return (y, (mean, rstd)) if save else y


def group_norm_backward(plan: GroupNorm, x, gamma, beta, saved, dy, ws, stream=None):
    """sn_group_norm_backward -> (dx, dgamma, dbeta) from the forward's `saved` and the gradient dy of y (any strides;
    copied if its last index is not contiguous)."""
    torch = _torch()
    op = plan._bind(x, gamma, beta)
    dy = _gradient(dy)
    dy_stride, _ = _rows(dy, "dy", plan.shape, plan.dtype, plan.device)
    stats = (plan.n_segments, plan.n_groups)
    dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    dgamma, dbeta = torch.empty((2, plan.n_channels), dtype=torch.float32, device=plan.device).unbind(0)
    _launch(plan, lib().sn_group_norm_backward, stream, ws, (x, gamma, beta, *saved, dy, dx, dgamma, dbeta), op,
            _flat(saved[0], "saved[0]", stats, (torch.float32,), plan.device),
            _flat(saved[1], "saved[1]", stats, (torch.float32,), plan.device), dy.data_ptr(), dy_stride, dx.data_ptr(),
            dgamma.data_ptr(), dbeta.data_ptr())
    return dx, dgamma, dbeta


def _shaped(shape, dtype, device):
    """A tensor of a shape without its memory, for torch.empty_like (three times as fast as torch.empty with a shape)."""
    return _torch().empty((1,) * len(shape), dtype=dtype, device=device).expand(shape)


# ------------------------------------------------------------------ rotation of heads
#
# The streams, workspaces and autograd conventions of the calls below are the context operators'.

_ROTARY_CALL = struct.Struct("@PPP4qPP")


def rotary_frequencies(sections, base: float = 10000.0, shared: bool = True):
    """sn_rotary_frequencies -> (freqs float64, axes int32), a value for each pair: sections[a] pairs turn by axis a.

    shared: one ladder base^(-j/n) falls over all n pairs; else every axis has a ladder of its own."""
    sections = _int32s(sections, "sections")
    n = max(int(np.clip(sections, 0, None).sum(dtype=np.int64)), 1)
    freqs, axes = np.zeros(min(n, SN_MAX_HEAD_DIM), np.float64), np.zeros(min(n, SN_MAX_HEAD_DIM), np.int32)
    _check(lib().sn_rotary_frequencies(sections.size, sections.ctypes.data, float(base), int(shared), freqs.ctypes.data,
                                       axes.ctypes.data), "sn_rotary_frequencies")
    return freqs, axes


class HeadRotary:
    """Head layout, norm and rotation of query and key rows (sn_head_rotary).

    freqs, axes: host arrays with a value for each pair (see rotary_frequencies); None: nothing turns.  axes defaults
    to one axis.  interleaved: pairs are adjacent elements instead of the halves of the part that turns.
    norm: heads are divided by their root mean square (and multiplied by a weight) first."""

    def __init__(self, n_rows: int, n_heads: int, head_dim: int, n_kv_heads: int = 0, freqs=None, axes=None,
                 interleaved: bool = False, norm: bool = True, eps: float = 1e-6, dtype=None, device="cuda"):
        torch = _torch()
        self.dtype = torch.float32 if dtype is None else dtype
        code = _row_type(self.dtype)
        self.freqs = np.ascontiguousarray([] if freqs is None else freqs, np.float64).ravel().copy()
        self.n_pairs = self.freqs.size
        self.axes = np.zeros(self.n_pairs, np.int32) if axes is None else _int32s(axes, "axes")
        if self.axes.size != self.n_pairs:
            raise ValueError(f"{self.n_pairs} frequencies and {self.axes.size} axes")
        self.n_axes = int(self.axes.max()) + 1 if self.n_pairs else 0
        if self.n_pairs and (self.axes.min() < 0 or not (np.abs(self.freqs) < 2.0 ** 52).all()):
            raise ValueError("axes must not be negative, and frequencies have to be within +-2^52")
        self.norm = bool(norm)
        if self.norm and not np.finfo(np.float32).tiny <= eps <= np.finfo(np.float32).max:
            raise ValueError(f"eps must be a positive normal number of 32 bits, not {eps}")
        self.n_rows, self.n_heads = _int32(n_rows, "n_rows"), _int32(n_heads, "n_heads")
        self.n_kv_heads, self.head_dim = _int32(n_kv_heads, "n_kv_heads"), _int32(head_dim, "head_dim")
        self.c = SnHeadRotary(self.n_rows, self.n_heads, self.n_kv_heads, self.head_dim, code, int(self.norm), float(eps),
                              self.n_pairs, self.n_axes, int(bool(interleaved)), self.freqs.ctypes.data, self.axes.ctypes.data)
        self.workspace_bytes = int(lib().sn_head_rotary_workspace_bytes(ctypes.byref(self.c)))
        if self.workspace_bytes == 0:
            raise SnError(SN_ERR_INVALID, "sn_head_rotary")
        self.head = bytes(self.c)[:SnHeadRotary.positions.offset]
        self.device = torch.empty(0, device=device).device
        self.pointers = ()
        self.index, self.byte = self.device.index, torch.uint8
        self.current_stream, self.current_device = _current_getters()
        self.q_shape = torch.Size((self.n_rows, self.n_heads, self.head_dim))
        self.k_shape = torch.Size((self.n_rows, self.n_kv_heads, self.head_dim))
        self.weight_like = _shaped((self.head_dim,), torch.float32, self.device)

    def _rows(self, q, k, names):
        """The strides of a query and a key tensor (k None where the plan has no key heads)."""
        qs, qh, _ = _rows(q, names[0], self.q_shape, self.dtype, self.device)
        if self.n_kv_heads == 0:
            if k is not None:
                raise ValueError(f"{names[1]} must be None: the plan has no key heads")
            return qs, qh, 0, 0
        if k is None:
            raise ValueError(f"{names[1]} is missing: the plan has {self.n_kv_heads} key heads")
        ks, kh, _ = _rows(k, names[1], self.k_shape, self.dtype, self.device)
        return qs, qh, ks, kh

    def _bind(self, q, k, positions, q_weight, k_weight) -> bytes:
        """The descriptor of one call (its own bytes: calls from several threads share nothing)."""
        strides = self._rows(q, k, ("q", "k"))
        if not self.norm and (q_weight is not None or k_weight is not None):
            raise ValueError("a weight needs the plan's norm")
        f32, shape = (_torch().float32,), (self.head_dim,)
        if self.n_pairs and positions is None:
            raise ValueError("positions are missing: the plan turns pairs")
        at = _flat(positions, "positions", (self.n_axes, self.n_rows), (_torch().int32,), self.device) if self.n_pairs else 0
        return self.head + _ROTARY_CALL.pack(at, q.data_ptr(), _ptr(k) or 0, *strides,
                                             _flat(q_weight, "q_weight", shape, f32, self.device),
                                             _flat(k_weight, "k_weight", shape, f32, self.device))


def head_rotary_workspace(plan: HeadRotary):
    """A workspace (status words zeroed) for the plan's calls; calls that share one must be ordered on a stream."""
    return _zeroed_workspace(plan)


def head_rotary_forward(plan: HeadRotary, q, k, positions, ws, q_weight=None, k_weight=None, stream=None):
    """sn_head_rotary_forward -> (q, k) normed and turned.  q [n_rows, H, D], k [n_rows, Hkv, D] (None without key
    heads, and returned so); positions int32 [n_axes, n_rows]; weights float32 [D], None for 1."""
    torch = _torch()
    op = plan._bind(q, k, positions, q_weight, k_weight)
    q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    k_out = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
    _launch(plan, lib().sn_head_rotary_forward, stream, ws, (q, k, positions, q_weight, k_weight, q_out, k_out), op,
            q_out.data_ptr(), _ptr(k_out))
    return q_out, k_out


def head_rotary_backward(plan: HeadRotary, q, k, positions, d_q, d_k, ws, q_weight=None, k_weight=None, stream=None):
    """sn_head_rotary_backward -> (dq, dk, dq_weight, dk_weight) from the gradients of the turned rows (any strides;
    copied if their last index is not contiguous).  The other arguments are the forward's.  The weights' gradients are
    returned with a norm, also where a weight was None; without one they are None."""
    torch = _torch()
    op = plan._bind(q, k, positions, q_weight, k_weight)
    d_q, d_k = _gradient(d_q), None if d_k is None else _gradient(d_k)
    gs, gh, ks, kh = plan._rows(d_q, d_k, ("d_q", "d_k"))
    dq = torch.empty_like(q, memory_format=torch.contiguous_format)
    dk = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
    dqw = dkw = None
    if plan.norm:
        dqw, dkw = (torch.empty_like(plan.weight_like, memory_format=torch.contiguous_format) for _ in range(2))
    _launch(plan, lib().sn_head_rotary_backward, stream, ws,
            (q, k, positions, d_q, d_k, q_weight, k_weight, dq, dk, dqw, dkw), op, d_q.data_ptr(), gs, gh, _ptr(d_k), ks, kh,
            dq.data_ptr(), _ptr(dk), _ptr(dqw), _ptr(dkw))
    return dq, dk, dqw, dkw if plan.n_kv_heads else None


# ------------------------------------------------------------------ state cache

_CODES = {None: SN_CODES_NONE, "int8": SN_CODES_INT8, "e4m3": SN_CODES_E4M3}
_CACHE_TABLE = struct.Struct("@PP")
_CACHE_QUERY = struct.Struct("@P2q")


class StateCache:
    """Pages for the keys and values of sequences (the first part of sn_cache), zeroed.

    codes: None holds rows in dtype; "int8" and "e4m3" hold 8-bit codes with a float32 scale for each row of a head.
    k, v [n_pages, n_kv_heads, page_size, head_dim] and (with codes) k_scale, v_scale [n_pages, n_kv_heads, page_size]
    are the storage itself, viewed without the rows' padding."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, dtype=None, codes=None, device="cuda"):
        torch = _torch()
        self.dtype = torch.float32 if dtype is None else dtype
        code = _row_type(self.dtype)
        if codes not in _CODES:
            raise ValueError(f"codes must be one of {tuple(_CODES)}, not {codes!r}")
        self.codes = codes
        self.n_pages, self.page_size = _int32(n_pages, "n_pages"), _int32(page_size, "page_size")
        self.n_kv_heads, self.head_dim = _int32(n_kv_heads, "n_kv_heads"), _int32(head_dim, "head_dim")
        self.c = SnCache(self.n_pages, self.page_size, self.n_kv_heads, self.head_dim, code, _CODES[codes])
        probe = SnCache.from_buffer_copy(self.c)
        probe.n_sequences = probe.max_pages = 1
        probe.n_heads = self.n_kv_heads
        if lib().sn_cache_workspace_bytes(ctypes.byref(probe)) == 0:
            raise SnError(SN_ERR_INVALID, "sn_cache")
        shape = (self.n_pages, self.n_kv_heads, self.page_size, (self.head_dim + 15) // 16 * 16)
        kind = self.dtype if codes is None else torch.int8
        pages = [torch.zeros(shape, dtype=kind, device=device) for _ in range(2)]
        self.k_scale = self.v_scale = None
        if codes is not None:
            self.k_scale, self.v_scale = (torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
        self.c.k, self.c.v, self.c.k_scale, self.c.v_scale = (_ptr(t) for t in (*pages, self.k_scale, self.v_scale))
        if codes == "e4m3":
            pages = [t.view(torch.float8_e4m3fn) for t in pages]
        self.k, self.v = (t[..., :self.head_dim] for t in pages)
        self.device = self.k.device
        self.tensors = (self.k, self.v) if codes is None else (self.k, self.v, self.k_scale, self.v_scale)


class CacheRows:
    """The rows of a cache's sequences that a call writes, reads back or attends from (sn_cache).

    row_ptr: host row offsets [B + 1]; the rows of sequence b are its last ones, at positions lengths[b] - count on.
    max_pages: entries of a sequence in the page table.  For cache_attend: n_heads (default: the cache's), scale
    (default 1 / sqrt(head_dim)), causal (a row sees the positions up to its own, else all) and window (> 0: only the
    last `window` of them).  A plan of more rows than an attention's launch holds (sn_cache_workspace_bytes) writes and
    reads alone."""

    def __init__(self, cache: StateCache, row_ptr, max_pages: int, n_heads=None, scale=None, causal: bool = True,
                 window: int = 0):
        torch = _torch()
        self.cache, self.dtype, self.device = cache, cache.dtype, cache.device
        rp, most = _ragged(row_ptr, "row_ptr")
        self.row_ptr = torch.from_numpy(rp).to(self.device)
        self.n_sequences, self.n_rows, self.max_pages = rp.size - 1, int(rp[-1]), _int32(max_pages, "max_pages")
        self.n_heads = cache.n_kv_heads if n_heads is None else _int32(n_heads, "n_heads")
        self.scale = cache.head_dim ** -0.5 if scale is None else float(scale)
        if not abs(self.scale) <= float(np.finfo(np.float32).max):
            raise ValueError(f"scale must be finite in 32 bits, not {scale}")
        self.c = SnCache.from_buffer_copy(cache.c)
        self.c.n_sequences, self.c.n_rows, self.c.max_rows, self.c.max_pages = self.n_sequences, self.n_rows, most, self.max_pages
        self.c.row_ptr = _ptr(self.row_ptr)
        self.c.n_heads, self.c.scale, self.c.causal, self.c.window = self.n_heads, self.scale, int(bool(causal)), _int32(window, "window")
        self.workspace_bytes = int(lib().sn_cache_workspace_bytes(ctypes.byref(self.c)))
        if self.workspace_bytes == 0:
            raise SnError(SN_ERR_INVALID, "sn_cache")
        raw = bytes(self.c)
        self.head, self.middle = raw[:SnCache.table.offset], raw[SnCache.n_heads.offset:SnCache.q.offset]
        self.pointers = (self.row_ptr, *cache.tensors)
        self.index, self.byte = self.device.index, torch.uint8
        self.current_stream, self.current_device = _current_getters()
        self.q_shape = torch.Size((self.n_rows, self.n_heads, cache.head_dim))
        self.k_shape = torch.Size((self.n_rows, cache.n_kv_heads, cache.head_dim))
        self.k_like = _shaped(self.k_shape, self.dtype, self.device)

    def _bind(self, table, lengths, q=None) -> bytes:
        """The descriptor of one call (its own bytes: calls from several threads share nothing)."""
        i32 = (_torch().int32,)
        if table is None or lengths is None:
            raise ValueError("the page table and the lengths are needed")
        at = _flat(table, "table", (self.n_sequences, self.max_pages), i32, self.device)
        held = _flat(lengths, "lengths", (self.n_sequences,), i32, self.device)
        query = (0, 0, 0)
        if q is not None:
            qs, qh, _ = _rows(q, "q", self.q_shape, self.dtype, self.device)
            query = (q.data_ptr(), qs, qh)
        return self.head + _CACHE_TABLE.pack(at, held) + self.middle + _CACHE_QUERY.pack(*query)


def cache_workspace(plan: CacheRows):
    """A workspace (status words zeroed) for the plan's calls; calls that share one must be ordered on a stream."""
    return _zeroed_workspace(plan)


def cache_write(plan: CacheRows, k, v, table, lengths, ws, stream=None):
    """sn_cache_write: the rows k and v [n_rows, Hkv, D] to their places.  table int32 [B, max_pages] holds the pages
    of each sequence in order, lengths int32 [B] its rows with these among them."""
    op = plan._bind(table, lengths)
    ks, kh, _ = _rows(k, "k", plan.k_shape, plan.dtype, plan.device)
    vs, vh, _ = _rows(v, "v", plan.k_shape, plan.dtype, plan.device)
    _launch(plan, lib().sn_cache_write, stream, ws, (k, v, table, lengths), op, k.data_ptr(), ks, kh, v.data_ptr(), vs, vh)


def cache_read(plan: CacheRows, table, lengths, ws, stream=None):
    """sn_cache_read -> (k, v) [n_rows, Hkv, D]: the plan's rows as the pages hold them."""
    torch = _torch()
    op = plan._bind(table, lengths)
    k = torch.empty_like(plan.k_like, memory_format=torch.contiguous_format)
    v = torch.empty_like(plan.k_like, memory_format=torch.contiguous_format)
    _launch(plan, lib().sn_cache_read, stream, ws, (k, v, table, lengths), op, k.data_ptr(), v.data_ptr())
    return k, v


def cache_attend(plan: CacheRows, q, table, lengths, ws, save: bool = False, stream=None):
    """sn_cache_attend -> o [n_rows, H, D]: attention of the plan's rows q over their sequences' pages; with save=True
    -> (o, lse), lse float32 [n_rows, H] the logarithm of the sum of exp of the scores, by which parts over different
    keys can be joined."""
    torch = _torch()
    op = plan._bind(table, lengths, q)
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = torch.empty(plan.q_shape[:2], dtype=torch.float32, device=plan.device) if save else None
    _launch(plan, lib().sn_cache_attend, stream, ws, (q, table, lengths, o, lse), op, o.data_ptr(), _ptr(lse))
    return (o, lse) if save else o


# ------------------------------------------------------------------ timing

def profile_enable(on: bool = True):
    lib().sn_profile_enable(1 if on else 0)


def profile_collect() -> dict:
    """Per kernel class: (total ms, launches) of the launches since the last collect."""
    n = lib().sn_profile_classes()
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    _check(lib().sn_profile_collect(ms, cnt), "sn_profile_collect")
    return {lib().sn_profile_name(k).decode(): (ms[k], cnt[k]) for k in range(n) if cnt[k] > 0}
