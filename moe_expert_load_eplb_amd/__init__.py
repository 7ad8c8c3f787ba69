"""Python binding of libeplb (the EPLB hot path on MI355X).

Argument marshalling only: every step of the path runs in the HIP kernels of
``libeplb.so``; this module checks dtypes, devices and contiguity, passes raw
device pointers and the current HIP stream through the C ABI declared in
``include/eplb.h``, ``include/eplb_experts.h`` and ``include/eplb_layer.h``, and raises :class:`EplbError` on a non-zero
return code.
PyTorch supplies device memory and streams.

Importing this package loads the library; if it has not been built
(``python moe_expert_load_eplb_amd/build.py``) the import fails loudly.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libeplb.so")

EPLB_OK = 0
EPLB_E_ARG = 1
EPLB_E_DIV = 2
EPLB_E_REDUNDANCY = 3
EPLB_E_CAPACITY = 4
EPLB_E_LIMIT = 5
EPLB_E_RANGE = 6
EPLB_E_HIP = 7
EPLB_S_OK = 0
EPLB_S_BAD_LOAD = 16
EPLB_S_OVERFLOW = 17
EPLB_S_BAD_MAP = 18
EPLB_S_BAD_TOPOLOGY = 19
EPLB_DTYPE_F32 = 0
EPLB_DTYPE_BF16 = 1
EPLB_DTYPE_F16 = 2
EPLB_SCORE_SIGMOID = 0
EPLB_SCORE_SOFTMAX = 1

EXPORTS = ("eplb_load_hist", "eplb_rebalance", "eplb_redirect", "eplb_hist_redirect",
           "eplb_load_ema", "eplb_ema_redirect", "eplb_placement_load", "eplb_rearrange", "eplb_lp_solve", "eplb_lp_redirect",
           "eplb_lp_redirect_workspace_bytes", "eplb_status_string",
           "eplb_rebalance_lds_bytes", "eplb_rebalance_max_count", "eplb_lp_redirect_noalloc",
           "eplb_gate", "eplb_gate_loss", "eplb_gate_loss_workspace_bytes", "eplb_balance_loss", "eplb_gate_backward",
           "eplb_group_rows", "eplb_group_rows_workspace_bytes", "eplb_quantize_rows", "eplb_quantize_columns",
           "eplb_quantize_weights", "eplb_expert_matmul", "eplb_expert_wgrad",
           "eplb_expert_matmul16", "eplb_expert_wgrad16", "eplb_quantize_weights4", "eplb_expert_matmul4",
           "eplb_combine_rows", "eplb_combine_rows_backward")


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with "
                          "`python moe_expert_load_eplb_amd/build.py` (hipcc, gfx950)")
    lib = ctypes.CDLL(_LIB_PATH)
    missing = [f for f in EXPORTS if not hasattr(lib, f)]
    if missing:
        raise ImportError(f"{_LIB_PATH} lacks {missing}: rebuild it with "
                          "`python moe_expert_load_eplb_amd/build.py`")
    p, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.eplb_load_hist.argtypes = [p, i64, i64, i32, i32, p, i32, i64, p, p, p]
    lib.eplb_load_hist.restype = i32
    lib.eplb_rebalance.argtypes = [p, i64, i32, i32, i32, i32, i32, i32, p, p, p, p, p]
    lib.eplb_rebalance.restype = i32
    lib.eplb_redirect.argtypes = [p, i64, i64, i32, i32, p, p, i32, p, p]
    lib.eplb_redirect.restype = i32
    lib.eplb_hist_redirect.argtypes = [p, i64, i64, i32, i32, p, i32, i64, p, p, p, p, i32, p, p]
    lib.eplb_hist_redirect.restype = i32
    lib.eplb_load_ema.argtypes = [p, i64, i64, i32, i32, p, i32, p, p, p]
    lib.eplb_load_ema.restype = i32
    lib.eplb_ema_redirect.argtypes = [p, i64, i64, i32, i32, p, i32, p, p, p, p, i32, p, p]
    lib.eplb_ema_redirect.restype = i32
    lib.eplb_placement_load.argtypes = [p, p, p, i64, i32, i32, i32, p, p, p]
    lib.eplb_placement_load.restype = i32
    lib.eplb_rearrange.argtypes = [p, p, p, i64, i32, i32, i32, i32, i32, p, p, p, p, p, p]
    lib.eplb_rearrange.restype = i32
    lib.eplb_lp_solve.argtypes = [p, p, p, i64, i32, i32, i32, p, p, p, p, p]
    lib.eplb_lp_solve.restype = i32
    lib.eplb_lp_redirect.argtypes = [p, i64, i64, i32, i32, p, p, i32, i32, p, i64, p, p]
    lib.eplb_lp_redirect.restype = i32
    lib.eplb_lp_redirect_workspace_bytes.argtypes = [i64, i64, i32, i32]
    lib.eplb_lp_redirect_workspace_bytes.restype = i64
    lib.eplb_status_string.argtypes = [i32]
    lib.eplb_status_string.restype = ctypes.c_char_p
    lib.eplb_rebalance_lds_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.eplb_rebalance_lds_bytes.restype = i64
    lib.eplb_rebalance_max_count.argtypes = [i32, i32, i32, i32]
    lib.eplb_rebalance_max_count.restype = i32
    lib.eplb_lp_redirect_noalloc.argtypes = [p, i64, i64, i32, i32, p, p, i32, i32, p, p]
    lib.eplb_lp_redirect_noalloc.restype = i32
    f32 = ctypes.c_float
    choice = [i32, i32, i32, i32, f32, p]     # G, top_groups, group_top, normalize, scale, mask
    lib.eplb_gate.argtypes = [p, i32, i64, i64, i32, i32, i32, p, *choice, p, p, p]
    lib.eplb_gate.restype = i32
    lib.eplb_gate_loss.argtypes = [p, i32, i64, i64, i32, i32, i32, p, *choice, p, i64, f32, p, i64,
                                   p, p, p, p, p, p, p]
    lib.eplb_gate_loss.restype = i32
    lib.eplb_gate_loss_workspace_bytes.argtypes = [i64, i32, i64]
    lib.eplb_gate_loss_workspace_bytes.restype = i64
    lib.eplb_balance_loss.argtypes = [p, i32, i64, i64, i32, p, i32, i32, p, p, i64, f32, p, i64, p, p, p, p, p]
    lib.eplb_balance_loss.restype = i32
    lib.eplb_gate_backward.argtypes = [p, i32, i64, i64, i32, p, i32, i32, i32, f32, p, p, p, i64, f32, p, p, p, p, p]
    lib.eplb_gate_backward.restype = i32
    lib.eplb_group_rows.argtypes = [p, i64, i64, i32, i32, p, i64, p, p, p, p]
    lib.eplb_group_rows.restype = i32
    lib.eplb_group_rows_workspace_bytes.argtypes = [i64, i64, i32]
    lib.eplb_group_rows_workspace_bytes.restype = i64
    lib.eplb_quantize_rows.argtypes = [p, i32, i64, i64, i64, p, p, p]
    lib.eplb_quantize_rows.restype = i32
    lib.eplb_quantize_columns.argtypes = [p, i32, i64, i64, i64, p, i64, i32, p, i32, i64, p, p, p]
    lib.eplb_quantize_columns.restype = i32
    lib.eplb_quantize_weights.argtypes = [p, i32, i32, i64, i64, p, p, p, p, p]
    lib.eplb_quantize_weights.restype = i32
    lib.eplb_expert_matmul.argtypes = [p, p, i64, p, p, p, i32, p, i64, i32, i64, i64, i32, p, p]
    lib.eplb_expert_matmul.restype = i32
    lib.eplb_expert_wgrad.argtypes = [p, p, p, p, p, i32, i64, i64, i64, i64, i32, p, p]
    lib.eplb_expert_wgrad.restype = i32
    lib.eplb_expert_matmul16.argtypes = [p, i32, i64, i64, p, p, i32, p, i64, i32, i64, i64, i32, i32, p, p]
    lib.eplb_expert_matmul16.restype = i32
    lib.eplb_expert_wgrad16.argtypes = [p, i32, i64, i64, p, i64, i64, p, i32, p, i32, i64, i64, i32, p, p]
    lib.eplb_expert_wgrad16.restype = i32
    lib.eplb_quantize_weights4.argtypes = [p, i32, i32, i64, i64, p, p, p]
    lib.eplb_quantize_weights4.restype = i32
    lib.eplb_expert_matmul4.argtypes = [p, i32, i64, i64, p, p, p, i32, p, i64, i32, i64, i64, i32, p, p]
    lib.eplb_expert_matmul4.restype = i32
    lib.eplb_combine_rows.argtypes = [p, i32, i64, i64, p, p, i64, i32, i32, p, p]
    lib.eplb_combine_rows.restype = i32
    lib.eplb_combine_rows_backward.argtypes = [p, i32, p, i32, i64, p, p, p, i64, i32, p, p, p]
    lib.eplb_combine_rows_backward.restype = i32
    return lib


lib = _load()


class EplbError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {lib.eplb_status_string(code).decode()} (code {code})")


def status_string(code: int) -> str:
    return lib.eplb_status_string(int(code)).decode()


def _check(code: int, where: str) -> None:
    if code != EPLB_OK:
        raise EplbError(code, where)


def _dev(t: torch.Tensor, dtype: torch.dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# torch's own accessor of the current stream's handle where it has one (0.1 us
# a call; the Stream object of the public call costs 1.9 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    if _raw_stream is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def load_hist(idx: torch.Tensor, E: int, ring: torch.Tensor, step: int,
              load: torch.Tensor | None = None, n_invalid: torch.Tensor | None = None):
    """Count one step's routing ids into ring[step % W] and sum the window.

    idx [L, T, K] int32; ring [W, L, E] int32 (zeroed once by the caller).
    Returns (load [L, E] int64, n_invalid [L] int64).
    """
    if idx.dim() != 3:
        raise ValueError("idx must be [L, T, K]")
    L, T, K = idx.shape
    if ring.dim() != 3 or ring.shape[1] != L or ring.shape[2] != E:
        raise ValueError(f"ring must be [W, {L}, {E}], got {tuple(ring.shape)}")
    W = ring.shape[0]
    dev = idx.device
    if load is None:
        load = torch.empty((L, E), dtype=torch.int64, device=dev)
    if n_invalid is None:
        n_invalid = torch.empty((L,), dtype=torch.int64, device=dev)
    if tuple(load.shape) != (L, E) or tuple(n_invalid.shape) != (L,):
        raise ValueError("load must be [L, E] and n_invalid [L]")
    rc = lib.eplb_load_hist(_dev(idx, torch.int32, "idx"), L, T, K, E,
                            _dev(ring, torch.int32, "ring"), W, int(step),
                            _dev(load, torch.int64, "load"), _dev(n_invalid, torch.int64, "n_invalid"),
                            _stream(dev))
    _check(rc, "eplb_load_hist")
    return load, n_invalid


def max_count(E: int, P: int, G: int, N: int) -> int:
    """Largest replica count a placement can give one expert (the least
    log2phy width rebalance accepts), from eplb_rebalance_max_count."""
    n = lib.eplb_rebalance_max_count(int(E), int(P), int(G), int(N))
    if n < 0:
        raise EplbError(-n, "eplb_rebalance_max_count")
    return n


def rebalance(load: torch.Tensor, P: int, G: int, N: int, RK: int, X: int | None = None,
              out: tuple | None = None):
    """Replica placement for every row of ``load`` ([B, E] int64).

    Returns (phy2log [B, P], log2phy [B, E, X], logcnt [B, E], status [B]),
    all int32.  X defaults to the largest possible count.
    """
    if load.dim() != 2:
        raise ValueError("load must be [B, E]")
    B, E = load.shape
    if X is None:
        X = max_count(E, P, G, N)
    dev = load.device
    if out is None:
        out = (torch.empty((B, P), dtype=torch.int32, device=dev),
               torch.empty((B, E, X), dtype=torch.int32, device=dev),
               torch.empty((B, E), dtype=torch.int32, device=dev),
               torch.empty((B,), dtype=torch.int32, device=dev))
    phy2log, log2phy, logcnt, status = out
    if (tuple(phy2log.shape) != (B, P) or tuple(log2phy.shape) != (B, E, X)
            or tuple(logcnt.shape) != (B, E) or tuple(status.shape) != (B,)):
        raise ValueError("output shapes must be [B, P], [B, E, X], [B, E], [B]")
    rc = lib.eplb_rebalance(_dev(load, torch.int64, "load"), B, E, P, G, N, RK, X,
                            _dev(phy2log, torch.int32, "phy2log"), _dev(log2phy, torch.int32, "log2phy"),
                            _dev(logcnt, torch.int32, "logcnt"), _dev(status, torch.int32, "status"),
                            _stream(dev))
    _check(rc, "eplb_rebalance")
    return phy2log, log2phy, logcnt, status


def rebalance_experts(weight: torch.Tensor, num_replicas: int, num_groups: int, num_nodes: int, num_gpus: int):
    """The pages' interface to the rebalance (EPLB README translation,
    «DualPipe и EPLB», Part 2, section "Интерфейс и пример"): the same
    arguments and the same three maps, for a caller switching from it.

    weight [layers, E]: token counts per logical expert, any integer dtype or
    a floating dtype holding whole numbers, on the GPU or the host (a host
    tensor is copied to the current GPU).  Returns int64 (phy2log [layers,
    num_replicas], log2phy [layers, E, max logcnt], logcnt [layers, E]) on
    weight's device; log2phy is as wide as the largest replica count, as the
    pages' function returns it, which costs one device-to-host read.  A load
    outside [0, 2^40] raises EplbError.
    """
    if weight.dim() != 2:
        raise ValueError("weight must be [layers, experts]")
    if weight.is_floating_point() and not bool(torch.equal(weight, torch.trunc(weight))):
        raise ValueError("weight must hold whole token counts")
    if weight.is_floating_point() and weight.numel() and float(weight.abs().max()) >= 2.0 ** 62:
        raise ValueError("weight holds values that do not convert to int64")
    dev = weight.device if weight.device.type == "cuda" else torch.device("cuda", torch.cuda.current_device())
    load = weight.to(device=dev, dtype=torch.int64).contiguous()
    phy2log, log2phy, logcnt, status = rebalance(load, num_replicas, num_groups, num_nodes, num_gpus)
    bad = status.ne(0).nonzero()
    if bad.numel():
        raise EplbError(int(status[bad[0, 0]]), f"eplb_rebalance (layer {int(bad[0, 0])})")
    width = int(logcnt.max()) if logcnt.numel() else 1
    out = (phy2log.long(), log2phy[:, :, :width].long(), logcnt.long())
    return tuple(t.to(weight.device) for t in out)


def redirect(idx: torch.Tensor, log2phy: torch.Tensor, logcnt: torch.Tensor,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """Physical replica of every routed (token, k): [L, T, K] int32."""
    if idx.dim() != 3 or log2phy.dim() != 3 or logcnt.dim() != 2:
        raise ValueError("idx [L, T, K], log2phy [L, E, X], logcnt [L, E] expected")
    L, T, K = idx.shape
    _, E, X = log2phy.shape
    if log2phy.shape[0] != L or tuple(logcnt.shape) != (L, E):
        raise ValueError("log2phy / logcnt do not match idx's layers")
    if out is None:
        out = torch.empty_like(idx)
    if out.shape != idx.shape:
        raise ValueError("out must have idx's shape")
    rc = lib.eplb_redirect(_dev(idx, torch.int32, "idx"), L, T, K, E,
                           _dev(log2phy, torch.int32, "log2phy"), _dev(logcnt, torch.int32, "logcnt"), X,
                           _dev(out, torch.int32, "out"), _stream(idx.device))
    _check(rc, "eplb_redirect")
    return out


def hist_redirect(idx: torch.Tensor, E: int, ring: torch.Tensor, step: int,
                  log2phy: torch.Tensor, logcnt: torch.Tensor, load: torch.Tensor | None = None,
                  n_invalid: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """load_hist and redirect in one pass over idx (the placement given is the
    one in force for this step).  Returns (load, n_invalid, out)."""
    if idx.dim() != 3 or log2phy.dim() != 3 or logcnt.dim() != 2:
        raise ValueError("idx [L, T, K], log2phy [L, E, X], logcnt [L, E] expected")
    L, T, K = idx.shape
    if ring.dim() != 3 or ring.shape[1] != L or ring.shape[2] != E:
        raise ValueError(f"ring must be [W, {L}, {E}], got {tuple(ring.shape)}")
    if tuple(log2phy.shape[:2]) != (L, E) or tuple(logcnt.shape) != (L, E):
        raise ValueError("log2phy / logcnt do not match idx's layers and E")
    W, X = ring.shape[0], log2phy.shape[2]
    dev = idx.device
    if load is None:
        load = torch.empty((L, E), dtype=torch.int64, device=dev)
    if n_invalid is None:
        n_invalid = torch.empty((L,), dtype=torch.int64, device=dev)
    if out is None:
        out = torch.empty_like(idx)
    if tuple(load.shape) != (L, E) or tuple(n_invalid.shape) != (L,) or out.shape != idx.shape:
        raise ValueError("load [L, E], n_invalid [L], out like idx expected")
    rc = lib.eplb_hist_redirect(_dev(idx, torch.int32, "idx"), L, T, K, E, _dev(ring, torch.int32, "ring"), W,
                                int(step), _dev(load, torch.int64, "load"),
                                _dev(n_invalid, torch.int64, "n_invalid"), _dev(log2phy, torch.int32, "log2phy"),
                                _dev(logcnt, torch.int32, "logcnt"), X, _dev(out, torch.int32, "out"),
                                _stream(dev))
    _check(rc, "eplb_hist_redirect")
    return load, n_invalid, out


def load_ema(idx: torch.Tensor, E: int, ema: torch.Tensor, shift: int,
             count: torch.Tensor | None = None, n_invalid: torch.Tensor | None = None):
    """Count one step's routing ids and fold them into an integer moving
    average: ema <- ema - (ema >> shift) + count, in place.

    idx [L, T, K] int32; ema [L, E] int64 (zeroed once by the caller).
    Returns (ema, count [L, E] int32, n_invalid [L] int64).
    """
    if idx.dim() != 3:
        raise ValueError("idx must be [L, T, K]")
    L, T, K = idx.shape
    if tuple(ema.shape) != (L, E):
        raise ValueError(f"ema must be [{L}, {E}], got {tuple(ema.shape)}")
    dev = idx.device
    if count is None:
        count = torch.empty((L, E), dtype=torch.int32, device=dev)
    if n_invalid is None:
        n_invalid = torch.empty((L,), dtype=torch.int64, device=dev)
    if tuple(count.shape) != (L, E) or tuple(n_invalid.shape) != (L,):
        raise ValueError("count must be [L, E] and n_invalid [L]")
    rc = lib.eplb_load_ema(_dev(idx, torch.int32, "idx"), L, T, K, E, _dev(count, torch.int32, "count"),
                           int(shift), _dev(ema, torch.int64, "ema"), _dev(n_invalid, torch.int64, "n_invalid"),
                           _stream(dev))
    _check(rc, "eplb_load_ema")
    return ema, count, n_invalid


def ema_redirect(idx: torch.Tensor, E: int, ema: torch.Tensor, shift: int, log2phy: torch.Tensor,
                 logcnt: torch.Tensor, count: torch.Tensor | None = None, n_invalid: torch.Tensor | None = None,
                 out: torch.Tensor | None = None):
    """load_ema and redirect in one pass over idx (the placement given is the
    one in force for this step).  Returns (ema, count, n_invalid, out)."""
    if idx.dim() != 3 or log2phy.dim() != 3 or logcnt.dim() != 2:
        raise ValueError("idx [L, T, K], log2phy [L, E, X], logcnt [L, E] expected")
    L, T, K = idx.shape
    if tuple(ema.shape) != (L, E):
        raise ValueError(f"ema must be [{L}, {E}], got {tuple(ema.shape)}")
    if tuple(log2phy.shape[:2]) != (L, E) or tuple(logcnt.shape) != (L, E):
        raise ValueError("log2phy / logcnt do not match idx's layers and E")
    X = log2phy.shape[2]
    dev = idx.device
    if count is None:
        count = torch.empty((L, E), dtype=torch.int32, device=dev)
    if n_invalid is None:
        n_invalid = torch.empty((L,), dtype=torch.int64, device=dev)
    if out is None:
        out = torch.empty_like(idx)
    if tuple(count.shape) != (L, E) or tuple(n_invalid.shape) != (L,) or out.shape != idx.shape:
        raise ValueError("count [L, E], n_invalid [L], out like idx expected")
    rc = lib.eplb_ema_redirect(_dev(idx, torch.int32, "idx"), L, T, K, E, _dev(count, torch.int32, "count"),
                               int(shift), _dev(ema, torch.int64, "ema"), _dev(n_invalid, torch.int64, "n_invalid"),
                               _dev(log2phy, torch.int32, "log2phy"), _dev(logcnt, torch.int32, "logcnt"), X,
                               _dev(out, torch.int32, "out"), _stream(dev))
    _check(rc, "eplb_ema_redirect")
    return ema, count, n_invalid, out


def placement_load(load: torch.Tensor, phy2log: torch.Tensor, logcnt: torch.Tensor, RK: int,
                   out: tuple | None = None):
    """Load of every rank under a placement and its max / mean.

    load [B, E] int64, phy2log [B, P] int32, logcnt [B, E] int32.
    Returns (rank_load [B, RK] float64, imbalance [B] float64); NaN marks a
    problem with an invalid load or map.
    """
    if load.dim() != 2 or phy2log.dim() != 2 or logcnt.dim() != 2:
        raise ValueError("load [B, E], phy2log [B, P], logcnt [B, E] expected")
    B, E = load.shape
    P = phy2log.shape[1]
    if phy2log.shape[0] != B or tuple(logcnt.shape) != (B, E):
        raise ValueError("phy2log / logcnt do not match load")
    dev = load.device
    if out is None:
        out = (torch.empty((B, RK), dtype=torch.float64, device=dev),
               torch.empty((B,), dtype=torch.float64, device=dev))
    rank_load, imbalance = out
    if tuple(rank_load.shape) != (B, RK) or tuple(imbalance.shape) != (B,):
        raise ValueError("outputs must be [B, RK] and [B]")
    rc = lib.eplb_placement_load(_dev(load, torch.int64, "load"), _dev(phy2log, torch.int32, "phy2log"),
                                 _dev(logcnt, torch.int32, "logcnt"), B, E, P, int(RK),
                                 _dev(rank_load, torch.float64, "rank_load"),
                                 _dev(imbalance, torch.float64, "imbalance"), _stream(dev))
    _check(rc, "eplb_placement_load")
    return rank_load, imbalance


def rearrange(old_phy2log: torch.Tensor, new_phy2log: torch.Tensor, new_log2phy: torch.Tensor, RK: int, N: int,
              out: tuple | None = None):
    """Plan of weight copies from the placement in force to a new one.

    old_phy2log, new_phy2log [B, P] int32; new_log2phy [B, E, X] int32.
    Returns (phy2log [B, P], log2phy [B, E, X], src [B, P], moves [B, 3],
    status [B]), all int32: the new placement permuted within ranks so that
    every replica that can stay does, and for each changed slot the old slot
    to copy from (-1 where nothing moves).
    """
    if old_phy2log.dim() != 2 or new_phy2log.dim() != 2 or new_log2phy.dim() != 3:
        raise ValueError("old_phy2log [B, P], new_phy2log [B, P], new_log2phy [B, E, X] expected")
    B, P = new_phy2log.shape
    _, E, X = new_log2phy.shape
    if tuple(old_phy2log.shape) != (B, P) or new_log2phy.shape[0] != B:
        raise ValueError("the three maps must describe the same B problems and P slots")
    dev = new_phy2log.device
    if out is None:
        out = (torch.empty((B, P), dtype=torch.int32, device=dev),
               torch.empty((B, E, X), dtype=torch.int32, device=dev),
               torch.empty((B, P), dtype=torch.int32, device=dev),
               torch.empty((B, 3), dtype=torch.int32, device=dev),
               torch.empty((B,), dtype=torch.int32, device=dev))
    phy2log, log2phy, src, moves, status = out
    if (tuple(phy2log.shape) != (B, P) or tuple(log2phy.shape) != (B, E, X) or tuple(src.shape) != (B, P)
            or tuple(moves.shape) != (B, 3) or tuple(status.shape) != (B,)):
        raise ValueError("output shapes must be [B, P], [B, E, X], [B, P], [B, 3], [B]")
    rc = lib.eplb_rearrange(_dev(old_phy2log, torch.int32, "old_phy2log"), _dev(new_phy2log, torch.int32, "new_phy2log"),
                            _dev(new_log2phy, torch.int32, "new_log2phy"), B, E, P, int(RK), int(N), X,
                            _dev(phy2log, torch.int32, "phy2log"), _dev(log2phy, torch.int32, "log2phy"),
                            _dev(src, torch.int32, "src"), _dev(moves, torch.int32, "moves"),
                            _dev(status, torch.int32, "status"), _stream(dev))
    _check(rc, "eplb_rearrange")
    return phy2log, log2phy, src, moves, status


def lp_solve(cnt: torch.Tensor, home: torch.Tensor, rep: torch.Tensor, out: tuple | None = None):
    """Per-batch redistribution of tokens over replica edges.

    cnt [B, E] int64 (tokens per expert in the batch), home [B, E] int32
    (rank of each expert's original), rep [B, RK, R] int32 (expert in each
    replica slot, or -1).  Returns (lam [B] int64, flow [B, RK, R] int64,
    rank_load [B, RK] int64, status [B] int32).
    """
    if cnt.dim() != 2 or home.dim() != 2 or rep.dim() != 3:
        raise ValueError("cnt [B, E], home [B, E], rep [B, RK, R] expected")
    B, E = cnt.shape
    _, RK, R = rep.shape
    if tuple(home.shape) != (B, E) or rep.shape[0] != B:
        raise ValueError("cnt, home and rep must describe the same B problems")
    dev = cnt.device
    if out is None:
        out = (torch.empty((B,), dtype=torch.int64, device=dev),
               torch.empty((B, RK, R), dtype=torch.int64, device=dev),
               torch.empty((B, RK), dtype=torch.int64, device=dev),
               torch.empty((B,), dtype=torch.int32, device=dev))
    lam, flow, rank_load, status = out
    if (tuple(lam.shape) != (B,) or tuple(flow.shape) != (B, RK, R) or tuple(rank_load.shape) != (B, RK)
            or tuple(status.shape) != (B,)):
        raise ValueError("output shapes must be [B], [B, RK, R], [B, RK], [B]")
    rc = lib.eplb_lp_solve(_dev(cnt, torch.int64, "cnt"), _dev(home, torch.int32, "home"),
                           _dev(rep, torch.int32, "rep"), B, E, RK, R, _dev(lam, torch.int64, "lam"),
                           _dev(flow, torch.int64, "flow"), _dev(rank_load, torch.int64, "rank_load"),
                           _dev(status, torch.int32, "status"), _stream(dev))
    _check(rc, "eplb_lp_solve")
    return lam, flow, rank_load, status


def lp_redirect_workspace_bytes(L: int, T: int, K: int, E: int) -> int:
    n = lib.eplb_lp_redirect_workspace_bytes(L, T, K, E)
    if n < 0:
        raise EplbError(-n, "eplb_lp_redirect_workspace_bytes")
    return n


def lp_redirect(idx: torch.Tensor, E: int, rep: torch.Tensor, flow: torch.Tensor,
                workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Physical expert of every (token, k) under the flows of lp_solve:
    [L, T, K] int32.  ``workspace`` (any dtype, contiguous, on the GPU) must
    hold lp_redirect_workspace_bytes(L, T, K, E) bytes; one is made if absent."""
    if idx.dim() != 3 or rep.dim() != 3 or flow.dim() != 3:
        raise ValueError("idx [L, T, K], rep [L, RK, R], flow [L, RK, R] expected")
    L, T, K = idx.shape
    _, RK, R = rep.shape
    if rep.shape[0] != L or tuple(flow.shape) != tuple(rep.shape):
        raise ValueError("rep and flow must be [L, RK, R] for idx's layers")
    need = lp_redirect_workspace_bytes(L, T, K, E)
    if workspace is None:
        workspace = torch.empty((max(need, 4),), dtype=torch.uint8, device=idx.device)
    if workspace.device.type != "cuda" or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    if out is None:
        out = torch.empty_like(idx)
    if out.shape != idx.shape:
        raise ValueError("out must have idx's shape")
    rc = lib.eplb_lp_redirect(_dev(idx, torch.int32, "idx"), L, T, K, E, _dev(rep, torch.int32, "rep"),
                              _dev(flow, torch.int64, "flow"), RK, R, workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _dev(out, torch.int32, "out"),
                              _stream(idx.device))
    _check(rc, "eplb_lp_redirect")
    return out


NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024


def lp_redirect_noalloc(idx: torch.Tensor, E: int, rep: torch.Tensor, flow: torch.Tensor,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """lp_redirect without a workspace: the counts live in the library's
    fixed per-GPU array (NOALLOC_SCRATCH_BYTES).  Calls that overlap in time
    on one GPU race; calls on one stream are safe."""
    if idx.dim() != 3 or rep.dim() != 3 or flow.dim() != 3:
        raise ValueError("idx [L, T, K], rep [L, RK, R], flow [L, RK, R] expected")
    L, T, K = idx.shape
    _, RK, R = rep.shape
    if rep.shape[0] != L or tuple(flow.shape) != tuple(rep.shape):
        raise ValueError("rep and flow must be [L, RK, R] for idx's layers")
    if out is None:
        out = torch.empty_like(idx)
    if out.shape != idx.shape:
        raise ValueError("out must have idx's shape")
    rc = lib.eplb_lp_redirect_noalloc(_dev(idx, torch.int32, "idx"), L, T, K, E, _dev(rep, torch.int32, "rep"),
                                      _dev(flow, torch.int64, "flow"), RK, R, _dev(out, torch.int32, "out"),
                                      _stream(idx.device))
    _check(rc, "eplb_lp_redirect_noalloc")
    return out


# ---------------------------------------------------------------- router
_DTYPES = {torch.float32: EPLB_DTYPE_F32, torch.bfloat16: EPLB_DTYPE_BF16, torch.float16: EPLB_DTYPE_F16}
_SCORING = {"sigmoid": EPLB_SCORE_SIGMOID, "softmax": EPLB_SCORE_SOFTMAX}
F8 = torch.float8_e4m3fn     # 1 sign, 4 exponent and 3 mantissa bits; largest value 448
BLOCK = 128                  # elements a scale covers along an axis


def _dtype(dtype: torch.dtype, name: str) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return _DTYPES[dtype]


def _rows(t: torch.Tensor, name: str) -> tuple[int, int, int]:
    """(pointer, dtype code, row stride) of a 2-D tensor whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _dtype(t.dtype, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {t.dim()}")
    if t.is_contiguous():
        return t.data_ptr(), code, t.shape[1]
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if (t.shape[1] > 1 and t.stride(1) != 1) or ld < t.shape[1]:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), code, ld


def _f8(t: torch.Tensor, name: str) -> int:
    if isinstance(t, torch.Tensor) and t.dtype == torch.uint8:
        return _dev(t, torch.uint8, name)
    return _dev(t, F8, name)


def _optional(t, dtype: torch.dtype, shape: tuple, name: str) -> int | None:
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return _dev(t, dtype, name)


def _mask(mask, T: int) -> int | None:
    if mask is not None and mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    return _optional(mask, torch.uint8, (T,), "mask")


def _scoring(scoring: str) -> int:
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {scoring!r}")
    return _SCORING[scoring]


def _workspace(workspace, need: int, device) -> torch.Tensor:
    if workspace is None:
        return torch.empty((max(need, 4),), dtype=torch.uint8, device=device)
    if workspace.device.type != "cuda" or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    return workspace


def _shapes(out: tuple, shapes: tuple, what: str) -> None:
    same = len(out) == len(shapes)
    for t, s in zip(out, shapes):
        same = same and t.shape == s
    if not same:
        raise ValueError(f"{what} must have the shapes {[list(s) for s in shapes]}")


def gate(logits: torch.Tensor, K: int, *, scoring: str = "sigmoid", bias: torch.Tensor | None = None, G: int = 1,
         top_groups: int | None = None, group_top: int = 1, normalize: bool = True, scale: float = 1.0,
         mask: torch.Tensor | None = None, out: tuple | None = None):
    """The K experts with the largest keys of every token, and their weights.

    logits [T, E] float32, bfloat16 or float16 (rows may be strided); bias [E]
    float32 is added to the key only; with G groups only the experts of the
    top_groups best groups may be chosen (a group's score: the sum of its
    group_top largest keys); mask [T] bool or uint8: rows to route.  Equal keys
    go to the lowest index.  Returns (ids [T, K] int32, weights [T, K]
    float32); id -1 with weight 0 where nothing is left to choose.
    """
    ptr, dt, ld = _rows(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    if out is None:
        out = (torch.empty((T, K), dtype=torch.int32, device=dev),
               torch.empty((T, K), dtype=torch.float32, device=dev))
    else:
        _shapes(out, ((T, K), (T, K)), "out")
    rc = lib.eplb_gate(ptr, dt, ld, T, E, K, _scoring(scoring), _optional(bias, torch.float32, (E,), "bias"), G,
                       G if top_groups is None else top_groups, group_top, int(normalize), scale, _mask(mask, T),
                       _dev(out[0], torch.int32, "ids"), _dev(out[1], torch.float32, "weights"), _stream(dev))
    _check(rc, "eplb_gate")
    return out


def gate_loss_workspace_bytes(T: int, E: int, S: int) -> int:
    n = lib.eplb_gate_loss_workspace_bytes(T, E, S)
    if n < 0:
        raise EplbError(-n, "eplb_gate_loss_workspace_bytes")
    return n


def _loss_out(out, S: int, E: int, dev, first: tuple) -> tuple:
    shapes = tuple(s for s, _ in first) + ((S,), (S, E), (S, E), (S,))
    if out is None:
        types = tuple(d for _, d in first) + (torch.float32, torch.int32, torch.float32, torch.int32)
        out = tuple(torch.empty(s, dtype=d, device=dev) for s, d in zip(shapes, types))
    _shapes(out, shapes, "out")
    return out


def gate_loss(logits: torch.Tensor, K: int, seg: torch.Tensor, alpha: float, *, scoring: str = "sigmoid",
              bias: torch.Tensor | None = None, G: int = 1, top_groups: int | None = None, group_top: int = 1,
              normalize: bool = True, scale: float = 1.0, mask: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, out: tuple | None = None):
    """gate with the balance loss of S segments of rows (seg [S + 1] int32:
    segment s holds rows seg[s] .. seg[s + 1] - 1).

    loss = alpha * sum over e of (E * counts / (K * tokens)) * prob, where prob
    is the mean share of an expert in the rows' scores.  Returns (ids [T, K]
    int32, weights [T, K] float32, loss [S] float32, counts [S, E] int32, prob
    [S, E] float32, tokens [S] int32).
    """
    ptr, dt, ld = _rows(logits, "logits")
    T, E = logits.shape
    if seg.dim() != 1 or seg.shape[0] < 2:
        raise ValueError("seg must be [S + 1]")
    S, dev = seg.shape[0] - 1, logits.device
    out = _loss_out(out, S, E, dev, (((T, K), torch.int32), ((T, K), torch.float32)))
    ids, weights, loss, counts, prob, tokens = out
    ws = _workspace(workspace, gate_loss_workspace_bytes(T, E, S), dev)
    rc = lib.eplb_gate_loss(ptr, dt, ld, T, E, K, _scoring(scoring), _optional(bias, torch.float32, (E,), "bias"), G,
                            G if top_groups is None else top_groups, group_top, int(normalize), scale, _mask(mask, T),
                            _dev(seg, torch.int32, "seg"), S, alpha, ws.data_ptr(), ws.numel() * ws.element_size(),
                            _dev(ids, torch.int32, "ids"), _dev(weights, torch.float32, "weights"),
                            _dev(loss, torch.float32, "loss"), _dev(counts, torch.int32, "counts"),
                            _dev(prob, torch.float32, "prob"), _dev(tokens, torch.int32, "tokens"), _stream(dev))
    _check(rc, "eplb_gate_loss")
    return out


def balance_loss(logits: torch.Tensor, ids: torch.Tensor, seg: torch.Tensor, alpha: float, *,
                 scoring: str = "sigmoid", mask: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 out: tuple | None = None):
    """gate_loss's loss for choices made elsewhere (ids [T, K] int32).
    Returns (loss [S], counts [S, E], prob [S, E], tokens [S])."""
    ptr, dt, ld = _rows(logits, "logits")
    T, E = logits.shape
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids must be [{T}, K]")
    if seg.dim() != 1 or seg.shape[0] < 2:
        raise ValueError("seg must be [S + 1]")
    S, dev = seg.shape[0] - 1, logits.device
    out = _loss_out(out, S, E, dev, ())
    loss, counts, prob, tokens = out
    ws = _workspace(workspace, gate_loss_workspace_bytes(T, E, S), dev)
    rc = lib.eplb_balance_loss(ptr, dt, ld, T, E, _dev(ids, torch.int32, "ids"), ids.shape[1], _scoring(scoring),
                               _mask(mask, T), _dev(seg, torch.int32, "seg"), S, alpha, ws.data_ptr(),
                               ws.numel() * ws.element_size(), _dev(loss, torch.float32, "loss"),
                               _dev(counts, torch.int32, "counts"), _dev(prob, torch.float32, "prob"),
                               _dev(tokens, torch.int32, "tokens"), _stream(dev))
    _check(rc, "eplb_balance_loss")
    return out


def gate_backward(logits: torch.Tensor, ids: torch.Tensor, d_weights: torch.Tensor | None, *,
                  scoring: str = "sigmoid", normalize: bool = True, scale: float = 1.0,
                  mask: torch.Tensor | None = None, seg: torch.Tensor | None = None, alpha: float = 0.0,
                  counts: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                  d_loss: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of sum(d_weights * weights) + sum(d_loss * loss) with respect
    to the logits: [T, E] in the logits' dtype.  Either term may be left out
    (d_weights or d_loss None); the loss's needs seg, counts and tokens."""
    ptr, dt, ld = _rows(logits, "logits")
    T, E = logits.shape
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids must be [{T}, K]")
    K, dev = ids.shape[1], logits.device
    S = 0
    if d_loss is not None:
        if seg is None or counts is None or tokens is None:
            raise ValueError("the loss's gradient needs seg, counts and tokens")
        S = d_loss.shape[0]
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=dev)
    else:
        _shapes((out,), ((T, E),), "out")
    given = d_loss is not None
    rc = lib.eplb_gate_backward(ptr, dt, ld, T, E, _dev(ids, torch.int32, "ids"), K, _scoring(scoring), int(normalize),
                                scale, _mask(mask, T), _optional(d_weights, torch.float32, (T, K), "d_weights"),
                                _optional(seg, torch.int32, (S + 1,), "seg") if given else None, S, alpha,
                                _optional(counts, torch.int32, (S, E), "counts") if given else None,
                                _optional(tokens, torch.int32, (S,), "tokens") if given else None,
                                _optional(d_loss, torch.float32, (S,), "d_loss"), _dev(out, logits.dtype, "out"),
                                _stream(dev))
    _check(rc, "eplb_gate_backward")
    return out


# ---------------------------------------------------------------- grouping
def group_rows_workspace_bytes(L: int, n: int, P: int) -> int:
    b = lib.eplb_group_rows_workspace_bytes(L, n, P)
    if b < 0:
        raise EplbError(-b, "eplb_group_rows_workspace_bytes")
    return b


def group_rows(ids: torch.Tensor, P: int, first: int = 0, workspace: torch.Tensor | None = None,
               out: tuple | None = None):
    """Rows (t, k) of every layer grouped by slot (slots first .. first + P - 1).

    ids [L, T, K] or [L, n] int32 (redirect's output).  Returns (offsets [L, P +
    1], order [L, n], place [L, n]), all int32: rows offsets[g] .. offsets[g +
    1] - 1 of the grouped order belong to slot g, order names the position of
    each in ids, place is its inverse.  Ids of no slot come last, in order.
    """
    if ids.dim() not in (2, 3):
        raise ValueError("ids must be [L, T, K] or [L, n]")
    L = ids.shape[0]
    n = ids.shape[1] * (ids.shape[2] if ids.dim() == 3 else 1)
    dev = ids.device
    if out is None:
        out = (torch.empty((L, P + 1), dtype=torch.int32, device=dev),
               torch.empty((L, n), dtype=torch.int32, device=dev),
               torch.empty((L, n), dtype=torch.int32, device=dev))
    else:
        _shapes(out, ((L, P + 1), (L, n), (L, n)), "out")
    need = group_rows_workspace_bytes(L, n, P)
    ws = _workspace(workspace, need, dev) if need > 0 or workspace is not None else None
    rc = lib.eplb_group_rows(_dev(ids, torch.int32, "ids"), L, n, first, P, None if ws is None else ws.data_ptr(),
                             0 if ws is None else ws.numel() * ws.element_size(),
                             _dev(out[0], torch.int32, "offsets"), _dev(out[1], torch.int32, "order"),
                             _dev(out[2], torch.int32, "place"), _stream(dev))
    _check(rc, "eplb_group_rows")
    return out


# ---------------------------------------------------------------- 8-bit blocks and products
def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def quantize_rows(x: torch.Tensor, out: tuple | None = None):
    """x [R, C] (rows may be strided) as 8-bit floating point with a scale for
    each 128 elements of a row: (q [R, C] float8_e4m3fn, scale [R, ceil(C /
    128)] float32)."""
    ptr, dt, ld = _rows(x, "x")
    R, C = x.shape
    if out is None:
        out = (torch.empty((R, C), dtype=F8, device=x.device),
               torch.empty((R, _blocks(C)), dtype=torch.float32, device=x.device))
    else:
        _shapes(out, ((R, C), (R, _blocks(C))), "out")
    rc = lib.eplb_quantize_rows(ptr, dt, ld, R, C, _f8(out[0], "q"), _dev(out[1], torch.float32, "scale"),
                                _stream(x.device))
    _check(rc, "eplb_quantize_rows")
    return out


def padded_rows(R: int, G: int) -> int:
    """Columns of quantize_columns' output: R rows in G groups, each group
    rounded up to a multiple of 128."""
    return (R + (BLOCK - 1) * G) // BLOCK * BLOCK


def _grouping(offsets: torch.Tensor, rows: torch.Tensor | None, R: int | None, X: int, K: int) -> tuple[int, int]:
    """(groups, grouped rows) of a grouping over an operand of X rows."""
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be [G + 1]")
    if rows is not None and rows.dim() != 1:
        raise ValueError("rows must be [R]")
    n = X if rows is None else rows.shape[0]
    if R is not None and R != n:
        raise ValueError(f"out has {R} rows for {n} grouped rows")
    return offsets.shape[0] - 1, n


def quantize_columns(x: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None, K: int = 1,
                     out: tuple | None = None):
    """Grouped rows of x [X, C] transposed, in 8 bits with a scale for each 128
    rows of a group: (q [C, Rp] float8_e4m3fn, scale [Rp / 128, C] float32)
    with Rp = padded_rows(R, G).  Grouped row r is row rows[r] // K of x
    (group_rows' order), or row r without rows."""
    ptr, dt, ld = _rows(x, "x")
    X, C = x.shape
    G, R = _grouping(offsets, rows, None, X, K)
    Rp = padded_rows(R, G)
    if out is None:
        out = (torch.empty((C, Rp), dtype=F8, device=x.device),
               torch.empty((Rp // BLOCK, C), dtype=torch.float32, device=x.device))
    else:
        _shapes(out, ((C, Rp), (Rp // BLOCK, C)), "out")
    rc = lib.eplb_quantize_columns(ptr, dt, ld, X, C, _optional(rows, torch.int32, (R,), "rows"), R, K,
                                   _dev(offsets, torch.int32, "offsets"), G, Rp, _f8(out[0], "q"),
                                   _dev(out[1], torch.float32, "scale"), _stream(x.device))
    _check(rc, "eplb_quantize_columns")
    return out


def quantize_weights(w: torch.Tensor, transpose: bool = False, out: tuple | None = None):
    """w [G, N, K] as 8-bit floating point with a scale for each 128 x 128
    block: (q [G, N, K], scale [G, ceil(N / 128), ceil(K / 128)]), and with
    transpose also (qt [G, K, N], scale_t), the same values transposed."""
    if w.dim() != 3:
        raise ValueError("w must be [G, N, K]")
    code = _dtype(w.dtype, "w")
    G, N, K = w.shape
    shapes = ((G, N, K), (G, _blocks(N), _blocks(K)), (G, K, N), (G, _blocks(K), _blocks(N)))[:4 if transpose else 2]
    if out is None:
        out = tuple(torch.empty(s, dtype=torch.float32 if i & 1 else F8, device=w.device)
                    for i, s in enumerate(shapes))
    _shapes(out, shapes, "out")
    rc = lib.eplb_quantize_weights(_dev(w, w.dtype, "w"), code, G, N, K, _f8(out[0], "q"),
                                   _dev(out[1], torch.float32, "scale"), _f8(out[2], "qt") if transpose else None,
                                   _dev(out[3], torch.float32, "scale_t") if transpose else None, _stream(w.device))
    _check(rc, "eplb_quantize_weights")
    return out


def expert_matmul(q: torch.Tensor, scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                  offsets: torch.Tensor, rows: torch.Tensor | None = None, K: int = 1,
                  dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Every grouped row times the transposed weights of its expert, both in 8
    bits with a scale for each block of 128.

    q [X, C], scale: quantize_rows' outputs; w [G, N, C], w_scale:
    quantize_weights'; offsets [G + 1] int32: rows offsets[g] .. offsets[g + 1]
    - 1 belong to expert g.  Grouped row r reads row rows[r] // K of q
    (group_rows' order), or row r without rows.  Returns [R, N] in ``dtype``
    (out's own type where out is given); rows of no expert are 0.  offsets = [0, R] is the plain product.
    """
    if q.dim() != 2 or w.dim() != 3 or w.shape[2] != q.shape[1]:
        raise ValueError("q [X, C] and w [G, N, C] expected")
    X, C = q.shape
    G, N, _ = w.shape
    g, R = _grouping(offsets, rows, None if out is None else out.shape[0], X, K)
    if g != G:
        raise ValueError(f"offsets must be [{G + 1}]")
    if out is None:
        out = torch.empty((R, N), dtype=dtype, device=q.device)
    _shapes((scale, w_scale, out), ((X, _blocks(C)), (G, _blocks(N), _blocks(C)), (R, N)), "scale, w_scale, out")
    rc = lib.eplb_expert_matmul(_f8(q, "q"), _dev(scale, torch.float32, "scale"), X, _f8(w, "w"),
                                _dev(w_scale, torch.float32, "w_scale"), _dev(offsets, torch.int32, "offsets"), G,
                                _optional(rows, torch.int32, (R,), "rows"), R, K, N, C, _dtype(out.dtype, "out"),
                                _dev(out, out.dtype, "out"), _stream(q.device))
    _check(rc, "eplb_expert_matmul")
    return out


def expert_wgrad(dy: torch.Tensor, dy_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor,
                 offsets: torch.Tensor, R: int | None = None, dtype: torch.dtype = torch.float32,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of expert_matmul with respect to the weights: [G, N, C].

    dy [N, Rp], dy_scale and x [C, Rp], x_scale: quantize_columns' outputs for
    the same offsets.  R: the grouped rows (offsets past it are clamped);
    default: as many as Rp allows."""
    if dy.dim() != 2 or x.dim() != 2 or dy.shape[1] != x.shape[1] or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("dy [N, Rp], x [C, Rp] and offsets [G + 1] expected")
    N, Rp = dy.shape
    C = x.shape[0]
    G = offsets.shape[0] - 1
    if R is None:
        R = max(0, Rp - (BLOCK - 1) * (G - 1)) if Rp else 0
    if out is None:
        out = torch.empty((G, N, C), dtype=dtype, device=dy.device)
    _shapes((dy_scale, x_scale, out), ((Rp // BLOCK, N), (Rp // BLOCK, C), (G, N, C)), "dy_scale, x_scale, out")
    rc = lib.eplb_expert_wgrad(_f8(dy, "dy"), _dev(dy_scale, torch.float32, "dy_scale"), _f8(x, "x"),
                               _dev(x_scale, torch.float32, "x_scale"), _dev(offsets, torch.int32, "offsets"), G, R,
                               Rp, N, C, _dtype(out.dtype, "out"), _dev(out, out.dtype, "out"), _stream(dy.device))
    _check(rc, "eplb_expert_wgrad")
    return out


# ---------------------------------------------------------------- 16-bit and 4-bit products, rows joined to tokens
SCALE_GROUP = 32             # 4-bit elements a scale covers along a row


def _launch(name: str, dev: torch.device, *args) -> None:
    """Calls the entry point on dev's current stream, with dev the current device."""
    fn = getattr(lib, name)
    if dev.index is None or dev.index == torch.cuda.current_device():
        rc = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(dev))
    _check(rc, name)


def _together(*tensors) -> torch.device:
    """The one device of the tensors that are given."""
    dev = tensors[0].device
    for t in tensors[1:]:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    return dev


def _short(t: torch.Tensor, name: str) -> tuple[int, int, int]:
    """_rows of a bfloat16 or float16 tensor."""
    if isinstance(t, torch.Tensor) and t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return _rows(t, name)


def expert_matmul16(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                    K: int = 1, transpose: bool = False, dtype: torch.dtype | None = None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Every grouped row times the transposed weights of its expert, both in 16
    bits; with transpose, times the weights as they are.

    x [X, C] bfloat16 or float16 (rows may be strided by multiples of 8); w [G,
    N, C] of the same type; offsets [G + 1] int32: rows offsets[g] .. offsets[g
    + 1] - 1 belong to expert g.  Grouped row r reads row rows[r] // K of x
    (group_rows' order), or row r without rows.  Returns [R, N] in ``dtype``
    (out's own type where out is given, else x's); rows of no expert are 0.
    With transpose x is [X, N] and the result [R, C]: the gradient of the rows
    from that of the product.  C is a multiple of 8, with transpose N too.
    """
    ptr, code, ld = _short(x, "x")
    if w.dim() != 3 or x.shape[1] != w.shape[1 if transpose else 2]:
        raise ValueError("x [X, N] and w [G, N, C] expected" if transpose else "x [X, C] and w [G, N, C] expected")
    X = x.shape[0]
    G, N, C = w.shape
    g, R = _grouping(offsets, rows, None if out is None else out.shape[0], X, K)
    if g != G:
        raise ValueError(f"offsets must be [{G + 1}]")
    dev = _together(x, w, offsets, rows, out)
    width = C if transpose else N
    if out is None:
        out = torch.empty((R, width), dtype=x.dtype if dtype is None else dtype, device=dev)
    else:
        _shapes((out,), ((R, width),), "out")
    _launch("eplb_expert_matmul16", dev, ptr, code, ld, X, _dev(w, x.dtype, "w"), _dev(offsets, torch.int32, "offsets"),
            G, _optional(rows, torch.int32, (R,), "rows"), R, K, N, C, int(transpose), _dtype(out.dtype, "out"),
            _dev(out, out.dtype, "out"))
    return out


def expert_wgrad16(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                   K: int = 1, dtype: torch.dtype | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of expert_matmul16 with respect to the weights: [G, N, C] in
    ``dtype`` (out's own type where out is given, else x's).

    dy [R, N]: the gradient of the product; x [X, C], offsets, rows and K: its
    arguments.  N and C are multiples of 8; rows may be strided by multiples of
    8.  An expert without rows gets zeros."""
    dptr, code, dy_ld = _short(dy, "dy")
    ptr, xcode, ld = _short(x, "x")
    if code != xcode:
        raise TypeError(f"dy must be {x.dtype}, got {dy.dtype}")
    X, C = x.shape
    N = dy.shape[1]
    G, R = _grouping(offsets, rows, None, X, K)
    if dy.shape[0] != R:
        raise ValueError(f"dy must be [{R}, N]")
    dev = _together(x, dy, offsets, rows, out)
    if out is None:
        out = torch.empty((G, N, C), dtype=x.dtype if dtype is None else dtype, device=dev)
    else:
        _shapes((out,), ((G, N, C),), "out")
    _launch("eplb_expert_wgrad16", dev, dptr, code, dy_ld, R, ptr, ld, X, _dev(offsets, torch.int32, "offsets"), G,
            _optional(rows, torch.int32, (R,), "rows"), K, N, C, _dtype(out.dtype, "out"), _dev(out, out.dtype, "out"))
    return out


def quantize_weights4(w: torch.Tensor, out: tuple | None = None):
    """w [G, N, C] as 4-bit floating point (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6)
    with a power of two for each 32 elements of a row: (q [G, N, C / 2] uint8,
    two codes to a byte, the even element in the low half; scale [G, N, C / 32]
    uint8, 2^(scale - 127), 255: NaN).  C is a multiple of 32."""
    if w.dim() != 3:
        raise ValueError("w must be [G, N, C]")
    G, N, C = w.shape
    shapes = ((G, N, C // 2), (G, N, C // SCALE_GROUP))
    if out is None:
        out = tuple(torch.empty(s, dtype=torch.uint8, device=w.device) for s in shapes)
    _shapes(out, shapes, "out")
    dev = _together(w, *out)
    _launch("eplb_quantize_weights4", dev, _dev(w, w.dtype, "w"), _dtype(w.dtype, "w"), G, N, C,
            _dev(out[0], torch.uint8, "q"), _dev(out[1], torch.uint8, "scale"))
    return out


def expert_matmul4(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, offsets: torch.Tensor,
                   rows: torch.Tensor | None = None, K: int = 1, dtype: torch.dtype | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """expert_matmul16 with 4-bit weights: x [X, C] bfloat16 or float16; w [G, N, C
    / 2], w_scale [G, N, C / 32]: quantize_weights4's outputs."""
    ptr, code, ld = _short(x, "x")
    X, C = x.shape
    if w.dim() != 3 or 2 * w.shape[2] != C:
        raise ValueError("x [X, C] and w [G, N, C / 2] expected")
    G, N, _ = w.shape
    g, R = _grouping(offsets, rows, None if out is None else out.shape[0], X, K)
    if g != G:
        raise ValueError(f"offsets must be [{G + 1}]")
    dev = _together(x, w, w_scale, offsets, rows, out)
    if out is None:
        out = torch.empty((R, N), dtype=x.dtype if dtype is None else dtype, device=dev)
    _shapes((w_scale, out), ((G, N, C // SCALE_GROUP), (R, N)), "w_scale, out")
    _launch("eplb_expert_matmul4", dev, ptr, code, ld, X, _dev(w, torch.uint8, "w"),
            _dev(w_scale, torch.uint8, "w_scale"), _dev(offsets, torch.int32, "offsets"), G,
            _optional(rows, torch.int32, (R,), "rows"), R, K, N, C, _dtype(out.dtype, "out"), _dev(out, out.dtype, "out"))
    return out


def _choices(place: torch.Tensor, weights: torch.Tensor | None) -> tuple[int, int]:
    """(tokens, choices of a token) of a grouping's place and the router's weights."""
    shaped = place if weights is None else weights
    if shaped.dim() != 2:
        raise ValueError("weights must be [T, K]" if weights is not None else "place must be [T, K] without weights")
    T, K = shaped.shape
    if place.numel() != T * K or place.dim() > 1 and (
            place.dim() > 2 or place.shape != (T, K) and max(place.shape) != T * K):
        raise ValueError(f"place must have {T * K} elements, as [{T}, {K}] or [{T * K}]")
    return T, K


def combine_rows(y: torch.Tensor, place: torch.Tensor, weights: torch.Tensor | None,
                 dtype: torch.dtype | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The experts' rows joined to tokens: out[t] = sum over k of weights[t, k] *
    y[place[t, k]], in 32 bits, rounded once.

    y [R, C] float32, bfloat16 or float16; place [T, K] (or [T * K]) int32:
    group_rows' place, outside [0, R): nothing is added; weights [T, K] float32
    (the router's), or None: ones, place being [T, K].  Returns [T, C] in
    ``dtype`` (out's own type where out is given, else y's)."""
    T, K = _choices(place, weights)
    if y.dim() != 2:
        raise ValueError("y must be [R, C]")
    R, C = y.shape
    dev = _together(y, place, weights, out)
    if out is None:
        out = torch.empty((T, C), dtype=y.dtype if dtype is None else dtype, device=dev)
    else:
        _shapes((out,), ((T, C),), "out")
    _launch("eplb_combine_rows", dev, _dev(y, y.dtype, "y"), _dtype(y.dtype, "y"), R, C,
            _dev(place, torch.int32, "place"), _optional(weights, torch.float32, (T, K), "weights"), T, K,
            _dtype(out.dtype, "out"), _dev(out, out.dtype, "out"))
    return out


def combine_rows_backward(d_out: torch.Tensor, y: torch.Tensor, place: torch.Tensor, order: torch.Tensor,
                          weights: torch.Tensor | None, out: tuple | None = None):
    """Gradients of combine_rows: (d_y [T * K, C] in y's type, d_weights [T, K]
    float32).

    d_out [T, C]; y [T * K, C]; place and order: group_rows', each the inverse of
    the other.  A choice whose place is outside y gets d_weights 0, a row that is
    not the place of its own order gets zeros.  Where d_weights is not wanted, y is
    one element expanded to its shape, y.new_empty(()).expand(T * K, C): only the
    type counts, no rows are read, and None stands for d_weights, in out too."""
    T, K = _choices(place, weights)
    if d_out.dim() != 2 or d_out.shape[0] != T:
        raise ValueError(f"d_out must be [{T}, C]")
    C = d_out.shape[1]
    _shapes((y,), ((T * K, C),), "y")
    if order.numel() != T * K:
        raise ValueError(f"order must have {T * K} elements")
    both = y.stride() != (0, 0) or y.is_contiguous()          # an expanded y of one element has it
    dev = _together(d_out, y, place, order, weights, *(out or ()))
    if out is None:
        out = (torch.empty((T * K, C), dtype=y.dtype, device=dev),
               torch.empty((T, K), dtype=torch.float32, device=dev) if both else None)
    elif both:
        _shapes(out, ((T * K, C), (T, K)), "out")
    else:
        _shapes(out[:1], ((T * K, C),), "out")
        if len(out) != 2 or out[1] is not None:
            raise ValueError("out must be (d_y, None) without y's rows")
    _launch("eplb_combine_rows_backward", dev, _dev(d_out, d_out.dtype, "d_out"), _dtype(d_out.dtype, "d_out"),
            _dev(y, y.dtype, "y") if both else None, _dtype(y.dtype, "y"), C, _dev(place, torch.int32, "place"),
            _dev(order, torch.int32, "order"), _optional(weights, torch.float32, (T, K), "weights"), T, K,
            _dev(out[0], y.dtype, "d_y"), _dev(out[1], torch.float32, "d_weights") if both else None)
    return out
