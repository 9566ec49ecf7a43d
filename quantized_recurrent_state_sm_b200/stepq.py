"""Python binding of the C ABI in include/stepq.h (libstepq.so, sm_100a).

Argument marshalling only: tensors are checked for dtype, device, shape and
contiguity, then their device pointers and torch's current CUDA stream are
passed to the library.  Every step of the computation runs in the library's
kernels; there is no fallback.  If the library has not been built the import of
this module raises.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# STEPQ_CHECK=1 in the environment selects the checking build (the kernels
# validate the pool's tables before touching memory; include/stepq.h).
CHECK_BUILD = os.environ.get("STEPQ_CHECK", "0") == "1"
LIB_PATH = os.path.join(_HERE, "libstepq_check.so" if CHECK_BUILD else "libstepq.so")

GDN, KDA, LINEAR = 0, 1, 2
SCALE_DUAL, SCALE_ROW, SCALE_COL, SCALE_HEAD = 0, 1, 2, 3
PIVOT_BITS = 16
DK = DV = 128
BLOCK = 64        # tokens of a block of a plan
STEP_TOKENS = 8   # prompts of at most this many tokens run token by token
MAX_BEAMS = 64
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_STATE = 0, 1, 2, 3, 4


class StepqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class Desc(C.Structure):
    _fields_ = [("variant", C.c_int), ("batch", C.c_int), ("heads", C.c_int), ("dk", C.c_int),
                ("dv", C.c_int), ("ls_iters", C.c_int), ("bits", C.c_void_p), ("rho", C.c_void_p)]


class Regions(C.Structure):
    _fields_ = [("states", C.c_size_t), ("state_bytes", C.c_size_t), ("head_records", C.c_size_t),
                ("head_offsets", C.c_size_t), ("item_sizes", C.c_size_t), ("status_word", C.c_size_t),
                ("item_order", C.c_size_t), ("staging_records", C.c_size_t), ("guards", C.c_size_t * 7),
                ("guard_bytes", C.c_size_t), ("total", C.c_size_t)]


class CalibDesc(C.Structure):
    _fields_ = [("variant", C.c_int), ("batch", C.c_int), ("heads", C.c_int), ("dk", C.c_int),
                ("dv", C.c_int), ("steps", C.c_int), ("sample_every", C.c_int), ("ls_iters", C.c_int),
                ("n_widths", C.c_int), ("widths", C.c_void_p), ("avg_bits", C.c_double),
                ("pivot_frac", C.c_double)]


class PlanDesc(C.Structure):
    _fields_ = [("requests", C.c_int), ("tokens", C.c_int), ("slots", C.c_int)]


class PlanRegions(C.Structure):
    _fields_ = [(f, C.c_size_t) for f in ("starts", "slot", "live", "fresh", "token_request", "token_position",
                                          "block_starts", "block_request", "block_first", "head", "scratch", "total")] + [("blocks", C.c_int)]


class PromptDesc(C.Structure):
    _fields_ = [(f, C.c_int) for f in ("variant", "dtype", "heads", "heads_qk", "dk", "dv", "max_length", "by_slot")] + [
        (f, C.c_longlong) for f in ("stride_q", "stride_k", "stride_v")]


EXPORTS = ("stepq_pool_bytes", "stepq_state_bytes", "stepq_pool_layout", "stepq_pool_check_guards", "stepq_pool_create", "stepq_pool_destroy",
           "stepq_pool_set_stream", "stepq_pack", "stepq_unpack", "stepq_decode_step",
           "stepq_fp32_step", "stepq_pool_check", "stepq_status_string", "stepq_last_error", "stepq_selftest_bounded_wait",
           "stepq_decode_step_noalloc", "stepq_decode_step_split", "stepq_pool_set_active",
           "stepq_pool_set_scale_mode", "stepq_calib_scratch_bytes", "stepq_calibrate", "stepq_calib_accumulate", "stepq_calib_row_error",
           "stepq_calib_reduce", "stepq_calib_rho", "stepq_calib_bits",
           "stepq_plan_layout", "stepq_plan_bytes", "stepq_plan_build", "stepq_plan_check", "stepq_prompt_scratch_bytes",
           "stepq_prompt", "stepq_pack_requests", "stepq_beam_scratch_bytes", "stepq_beam_select", "stepq_reorder_rows",
           "stepq_pool_reorder")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = C.CDLL(LIB_PATH)
    P, D = C.c_void_p, C.POINTER(Desc)
    L.stepq_pool_bytes.argtypes = [D]; L.stepq_pool_bytes.restype = C.c_size_t
    L.stepq_state_bytes.argtypes = [D]; L.stepq_state_bytes.restype = C.c_size_t
    L.stepq_pool_create.argtypes = [D, P, C.c_size_t, P, C.POINTER(P)]
    L.stepq_pool_destroy.argtypes = [P]
    L.stepq_pool_set_stream.argtypes = [P, P]
    L.stepq_pool_check.argtypes = [P]
    L.stepq_pool_check_guards.argtypes = [P]
    L.stepq_pool_layout.argtypes = [D, C.POINTER(Regions)]
    L.stepq_selftest_bounded_wait.argtypes = [P, C.c_longlong, C.c_int, P]
    L.stepq_pack.argtypes = [P, P]
    L.stepq_unpack.argtypes = [P, P]
    L.stepq_decode_step.argtypes = [P, P, P, P, P, P, P]
    L.stepq_fp32_step.argtypes = [D, P, P, P, P, P, P, P, P]
    L.stepq_decode_step_noalloc.argtypes = [D, P, C.c_size_t, P, P, P, P, P, P, P]
    L.stepq_decode_step_split.argtypes = [P, P, P, P, P, P, P, P, P]
    L.stepq_pool_set_active.argtypes = [P, P, C.c_int]
    L.stepq_pool_set_scale_mode.argtypes = [P, C.c_int]
    CD, i, dbl = C.POINTER(CalibDesc), C.c_int, C.c_double
    L.stepq_calib_scratch_bytes.argtypes = [CD]; L.stepq_calib_scratch_bytes.restype = C.c_size_t
    L.stepq_calibrate.argtypes = [CD, P, P, P, P, P, P, P, C.c_size_t, P, P, P]
    L.stepq_calib_accumulate.argtypes = [i, i, i, P, P, P, P, P]
    L.stepq_calib_row_error.argtypes = [i, i, P, P, i, P, i, P, P, P]
    L.stepq_calib_reduce.argtypes = [i, i, i, P, P, P]
    L.stepq_calib_rho.argtypes = [i, dbl, P, P]
    L.stepq_calib_bits.argtypes = [i, i, dbl, P, P, P, i, P, dbl, dbl, P]
    PD, z, ll = C.POINTER(PlanDesc), C.c_size_t, C.c_longlong
    L.stepq_plan_layout.argtypes = [PD, C.POINTER(PlanRegions)]
    L.stepq_plan_bytes.argtypes = [PD]; L.stepq_plan_bytes.restype = z
    L.stepq_plan_build.argtypes = [PD, P, z, i, P, P, P, P, i, P]
    L.stepq_plan_check.argtypes = [PD, P, z, P]
    L.stepq_prompt_scratch_bytes.argtypes = [PD, C.POINTER(PromptDesc)]; L.stepq_prompt_scratch_bytes.restype = z
    L.stepq_prompt.argtypes = [PD, P, z, C.POINTER(PromptDesc), P, P, P, P, P, P, P, P, z, P]
    L.stepq_pack_requests.argtypes = [P, PD, P, z, P, i]
    L.stepq_beam_scratch_bytes.argtypes = [i, i, i, i]; L.stepq_beam_scratch_bytes.restype = z
    L.stepq_beam_select.argtypes = [i, i, i, i, i, P, ll, P, P, P, P, P, z, P]
    L.stepq_reorder_rows.argtypes = [P, z, i, i, P, P]
    L.stepq_pool_reorder.argtypes = [P, i, i, i, P]
    for fn in ("stepq_plan_layout", "stepq_plan_build", "stepq_plan_check", "stepq_prompt", "stepq_pack_requests",
               "stepq_beam_select", "stepq_reorder_rows", "stepq_pool_reorder"):
        getattr(L, fn).restype = C.c_int
    for fn in ("stepq_pool_create", "stepq_pool_destroy", "stepq_pool_set_stream", "stepq_pool_check",
               "stepq_selftest_bounded_wait", "stepq_pack",
               "stepq_unpack", "stepq_decode_step", "stepq_fp32_step", "stepq_decode_step_noalloc",
               "stepq_decode_step_split", "stepq_pool_set_active", "stepq_pool_set_scale_mode", "stepq_calibrate", "stepq_calib_accumulate",
               "stepq_calib_row_error", "stepq_calib_reduce", "stepq_calib_rho", "stepq_calib_bits"):
        getattr(L, fn).restype = C.c_int
    L.stepq_status_string.argtypes = [C.c_int]; L.stepq_status_string.restype = C.c_char_p
    L.stepq_last_error.argtypes = []; L.stepq_last_error.restype = C.c_char_p
    return L


lib = _load()


def _check(status: int):
    if status != OK:
        msg = lib.stepq_last_error().decode(errors="replace")
        raise StepqError(status, f"{lib.stepq_status_string(status).decode()}: {msg}")


def _stream_ptr(stream=None):
    if stream is None:  # the raw handle: making a Stream object costs more than a small launch
        return C.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return C.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor, name: str, shape) -> C.c_void_p:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.float32 or not t.is_cuda:
        raise TypeError(f"{name} must be a float32 CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return C.c_void_p(t.data_ptr())


def make_desc(variant: int, batch: int, heads: int, bits: np.ndarray, rho: np.ndarray, ls_iters: int = 1):
    bits = np.ascontiguousarray(bits, dtype=np.uint8)
    rho = np.ascontiguousarray(rho, dtype=np.float32)
    if bits.shape != (heads, DK) or rho.shape != (heads, DK):
        raise ValueError("bits and rho must have shape [heads, 128]")
    d = Desc(variant, batch, heads, DK, DV, ls_iters, bits.ctypes.data_as(C.c_void_p),
             rho.ctypes.data_as(C.c_void_p))
    return d, (bits, rho)  # keep the host tables alive while the desc is used


def pool_bytes(variant, batch, heads, bits, rho, ls_iters=1) -> int:
    d, keep = make_desc(variant, batch, heads, bits, rho, ls_iters)
    n = lib.stepq_pool_bytes(C.byref(d))
    if n == 0:
        _check(ERR_INVALID_ARG)
    return int(n)


class PackedStatePool:
    """Packed recurrent states of batch x heads (request, head) items on one GPU.

    The device buffer is a torch uint8 tensor owned by this object; the library
    works in it in place.  Kernels run on torch's current CUDA stream.
    """

    def __init__(self, variant: int, batch: int, heads: int, bits, rho, ls_iters: int = 1,
                 device=None):
        self.variant, self.batch, self.heads, self.ls_iters = variant, batch, heads, ls_iters
        self._desc, self._keep = make_desc(variant, batch, heads, bits, rho, ls_iters)
        self.nbytes = int(lib.stepq_pool_bytes(C.byref(self._desc)))
        if self.nbytes == 0:
            _check(ERR_INVALID_ARG)
        self.state_nbytes = int(lib.stepq_state_bytes(C.byref(self._desc)))
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.buffer = torch.empty(self.nbytes, dtype=torch.uint8, device=dev)
        h = C.c_void_p()
        _check(lib.stepq_pool_create(C.byref(self._desc), C.c_void_p(self.buffer.data_ptr()),
                                     self.nbytes, _stream_ptr(), C.byref(h)))
        self._h = h
        self.n_active = batch

    @property
    def n_items(self) -> int:
        return self.batch * self.heads

    def set_scale_mode(self, mode: int):
        """The scale fit of later pack / decode calls: SCALE_DUAL (the method)
        or an ablation variant SCALE_ROW, SCALE_COL, SCALE_HEAD."""
        _check(lib.stepq_pool_set_scale_mode(self._h, int(mode)))

    def set_active(self, requests=None):
        """Restrict later decode steps to the listed requests (distinct slot
        indices in 0 .. batch-1); None = all.  decode_step keeps its
        [batch, heads, ...] shapes: it reads and writes only the listed
        requests' rows and updates only their states."""
        if requests is None:
            self._check_active(lib.stepq_pool_set_active(self._h, None, 0))
            self.n_active = self.batch
            return
        arr = np.ascontiguousarray(np.asarray(requests, dtype=np.int32).reshape(-1))
        self._sync_stream()
        self._check_active(lib.stepq_pool_set_active(self._h, arr.ctypes.data_as(C.c_void_p), int(arr.size)))
        self._active_host = arr  # the upload reads it on the stream
        self.n_active = int(arr.size)

    @staticmethod
    def _check_active(status):
        _check(status)

    @property
    def state(self) -> torch.Tensor:
        """The packed states (a view of the first state_nbytes bytes of the buffer)."""
        return self.buffer[: self.state_nbytes]

    def _sync_stream(self):
        _check(lib.stepq_pool_set_stream(self._h, _stream_ptr()))

    def pack(self, S: torch.Tensor):
        self._sync_stream()
        _check(lib.stepq_pack(self._h, _dev(S, "S", (self.batch, self.heads, DK, DV))))

    def unpack(self, out: torch.Tensor | None = None) -> torch.Tensor:
        if out is None:
            out = torch.empty((self.batch, self.heads, DK, DV), dtype=torch.float32, device=self.buffer.device)
        self._sync_stream()
        _check(lib.stepq_unpack(self._h, _dev(out, "S_out", (self.batch, self.heads, DK, DV))))
        return out

    def decode_step(self, q, k, v, alpha, beta, out=None) -> torch.Tensor:
        B, H = self.batch, self.heads
        if out is None:
            out = torch.empty((B, H, DV), dtype=torch.float32, device=self.buffer.device)
        ash = (B, H, DK) if self.variant == KDA else (B, H)
        self._sync_stream()
        _check(lib.stepq_decode_step(self._h, _dev(q, "q", (B, H, DK)), _dev(k, "k", (B, H, DK)),
                                     _dev(v, "v", (B, H, DV)), _dev(alpha, "alpha", ash),
                                     _dev(beta, "beta", (B, H)), _dev(out, "out", (B, H, DV))))
        return out

    def decode_step_split(self, q, k, v, alpha, beta, S_work, out=None, side_stream=None) -> torch.Tensor:
        """The same step as decode_step, split the way the pages' kernels split
        it: update + readout into S_work (fp32 [B, H, 128, 128]), then fit and
        packed writeback on side_stream (a torch.cuda.Stream; None = the
        current stream)."""
        B, H = self.batch, self.heads
        if out is None:
            out = torch.empty((B, H, DV), dtype=torch.float32, device=self.buffer.device)
        ash = (B, H, DK) if self.variant == KDA else (B, H)
        self._sync_stream()
        side = None if side_stream is None else C.c_void_p(side_stream.cuda_stream)
        _check(lib.stepq_decode_step_split(self._h, _dev(S_work, "S_work", (B, H, DK, DV)),
                                           _dev(q, "q", (B, H, DK)), _dev(k, "k", (B, H, DK)),
                                           _dev(v, "v", (B, H, DV)), _dev(alpha, "alpha", ash),
                                           _dev(beta, "beta", (B, H)), _dev(out, "out", (B, H, DV)), side))
        return out

    def pack_requests(self, plan: "RequestPlan", S: torch.Tensor, by_slot: bool = False):
        """Pack the states of the plan's live requests into their slots; the
        pool's other requests stay as they are.  S: [requests, heads, 128, 128]
        (state r of request r), or with by_slot [batch, heads, 128, 128]."""
        rows = self.batch if by_slot else plan.requests
        self._sync_stream()
        _check(lib.stepq_pack_requests(self._h, *plan._args, _dev(S, "S", (rows, self.heads, DK, DV)), int(by_slot)))

    def reorder(self, parents: torch.Tensor, first: int = 0):
        """Reorder packed states inside groups, in place: with parents [groups,
        beams] (int32 CUDA), request first + g * beams + i becomes what request
        first + g * beams + parents[g, i] was (a parent outside the group's
        beams, as -1, leaves it)."""
        if not isinstance(parents, torch.Tensor) or parents.dim() != 2:
            raise ValueError("parents must have shape [groups, beams]")
        G, B = parents.shape
        self._sync_stream()
        _check(lib.stepq_pool_reorder(self._h, int(first), G, B, _dev_any(parents, "parents", torch.int32, (G, B))))

    def beam_step(self, logits: torch.Tensor, scores: torch.Tensor, first: int = 0):
        """One step of a beam search over the pool: select the best `beams`
        continuations of each group (beam_select) and give each new beam the
        state of its parent (reorder).  logits [groups, beams, vocab], scores
        [groups, beams]; request first + g * beams + i holds the state of beam
        i of group g.  Returns (scores, parents, tokens), each [groups, beams]."""
        if not isinstance(logits, torch.Tensor) or logits.dim() != 3:
            raise ValueError("logits must have shape [groups, beams, vocab]")
        G, B = logits.shape[:2]
        if first < 0 or first + G * B > self.batch:
            raise ValueError(f"{G} groups of {B} beams from request {first} pass the pool's {self.batch} requests")
        got = beam_select(logits, scores)
        self.reorder(got[1], first)
        return got

    def check(self):
        """Synchronise the pool's stream and raise if a kernel reported an error."""
        self._sync_stream()
        _check(lib.stepq_pool_check(self._h))

    def check_guards(self):
        """Raise if a guard word after any region of the pool buffer changed."""
        self._sync_stream()
        _check(lib.stepq_pool_check_guards(self._h))

    @property
    def regions(self) -> dict:
        """Byte offsets of the buffer's regions (stepq_pool_layout)."""
        r = Regions()
        _check(lib.stepq_pool_layout(C.byref(self._desc), C.byref(r)))
        out = {f: getattr(r, f) for f, _ in Regions._fields_ if f != "guards"}
        out["guards"] = list(r.guards)
        return out

    def close(self):
        if getattr(self, "_h", None):
            lib.stepq_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fp32_step(variant: int, S: torch.Tensor, q, k, v, alpha, beta, out=None) -> torch.Tensor:
    """Unquantised fp32-state update + readout, in place on S [B, H, 128, 128]."""
    B, H = S.shape[0], S.shape[1]
    if out is None:
        out = torch.empty((B, H, DV), dtype=torch.float32, device=S.device)
    d = Desc(variant, B, H, DK, DV, 1, None, None)
    ash = (B, H, DK) if variant == KDA else (B, H)
    _check(lib.stepq_fp32_step(C.byref(d), _dev(S, "S", (B, H, DK, DV)), _dev(q, "q", (B, H, DK)),
                               _dev(k, "k", (B, H, DK)), _dev(v, "v", (B, H, DV)),
                               _dev(alpha, "alpha", ash), _dev(beta, "beta", (B, H)),
                               _dev(out, "out", (B, H, DV)), _stream_ptr()))
    return out


def decode_step_noalloc(variant: int, bits, rho, states: torch.Tensor, q, k, v, alpha, beta, out=None,
                        ls_iters: int = 1) -> torch.Tensor:
    """The fused decode step on packed states held in `states` (a uint8 CUDA
    tensor laid out as a pool's packed states), without a pool: the library
    keeps the kernel's tables in its own fixed device scratch and allocates
    nothing.  Calls must not overlap (one stream); see include/stepq.h."""
    bits = np.ascontiguousarray(bits, dtype=np.uint8)
    H = bits.shape[0]
    B = q.shape[0]
    d, keep = make_desc(variant, B, H, bits, rho, ls_iters)
    if not isinstance(states, torch.Tensor) or states.dtype != torch.uint8 or not states.is_cuda:
        raise TypeError("states must be a uint8 CUDA tensor")
    if not states.is_contiguous():
        raise ValueError("states must be contiguous")
    if out is None:
        out = torch.empty((B, H, DV), dtype=torch.float32, device=states.device)
    ash = (B, H, DK) if variant == KDA else (B, H)
    _check(lib.stepq_decode_step_noalloc(C.byref(d), C.c_void_p(states.data_ptr()), states.numel(),
                                         _dev(q, "q", (B, H, DK)), _dev(k, "k", (B, H, DK)),
                                         _dev(v, "v", (B, H, DV)), _dev(alpha, "alpha", ash),
                                         _dev(beta, "beta", (B, H)), _dev(out, "out", (B, H, DV)),
                                         _stream_ptr()))
    return out


def selftest_bounded_wait(limit_cycles: int, arrive: bool, device=None) -> tuple[int, int]:
    """Run the kernels' bounded barrier wait once (include/stepq.h,
    stepq_selftest_bounded_wait): (0 or 1 = gave up, cycles waited)."""
    res = torch.full((2,), -1, dtype=torch.int32, device=device or "cuda")
    _check(lib.stepq_selftest_bounded_wait(C.c_void_p(res.data_ptr()), int(limit_cycles), int(bool(arrive)),
                                           _stream_ptr()))
    torch.cuda.current_stream().synchronize()
    r = res.cpu().tolist()
    return r[0], r[1]


def _dev_any(t: torch.Tensor, name: str, dtype, shape) -> C.c_void_p:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a {dtype} CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return C.c_void_p(t.data_ptr())


# ---- serving: plans, prompts, beam search --------------------------------------

class RequestPlan:
    """The plan of a ragged batch: block table and slot map, built on the GPU.

    Holds room for `requests` requests with `tokens` token rows in all, whose
    states live in `slots` slots (default: one each).  After build() the int32
    views starts and block_starts [requests + 1], slots and live [requests], fresh [requests],
    token_request and token_position [tokens], block_request and block_first
    [blocks] describe the batch (include/stepq.h, stepq_plan_regions).
    """

    def __init__(self, requests: int, tokens: int, slots: int | None = None, device=None):
        self.requests, self.tokens = int(requests), int(tokens)
        self.n_slots = self.requests if slots is None else int(slots)
        self.max_length = self.tokens
        self._prompts = {}  # descriptor and scratch size of the prompts run over this plan, by their sizes
        self._desc = PlanDesc(self.requests, self.tokens, self.n_slots)
        r = PlanRegions()
        _check(lib.stepq_plan_layout(C.byref(self._desc), C.byref(r)))
        self.nbytes, self.blocks = int(r.total), int(r.blocks)
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.buffer = torch.empty(max(self.nbytes, 16), dtype=torch.uint8, device=dev)
        self._args = C.byref(self._desc), C.c_void_p(self.buffer.data_ptr()), self.nbytes
        ints = self.buffer[:self.nbytes].view(torch.int32)

        def view(offset, n):
            return ints[offset // 4: offset // 4 + n]

        self.head = view(r.head, 4)
        self.starts, self.block_starts = (view(o, self.requests + 1) for o in (r.starts, r.block_starts))
        self.slots, self.live, self.fresh = (view(o, self.requests) for o in (r.slot, r.live, r.fresh))
        self.token_request, self.token_position = (view(o, self.tokens) for o in (r.token_request, r.token_position))
        self.block_request, self.block_first = (view(o, self.blocks) for o in (r.block_request, r.block_first))

    def build(self, lengths: torch.Tensor, contexts: torch.Tensor | None = None, slots: torch.Tensor | None = None,
              busy: torch.Tensor | None = None, max_length: int | None = None) -> "RequestPlan":
        """Build the plan of a batch (stepq_plan_build), asynchronously on the
        current stream.  lengths, contexts, slots: int32 CUDA tensors of one
        entry a request; busy: uint8 CUDA map of the used slots, from which
        slots of -1 are served and which is updated; max_length: an upper bound
        of the lengths (default: the plan's tokens)."""
        n = lengths.shape[0] if isinstance(lengths, torch.Tensor) and lengths.dim() == 1 else -1
        bound = self.tokens if max_length is None else int(max_length)
        _check(lib.stepq_plan_build(*self._args, n, _dev_any(lengths, "lengths", torch.int32, (max(n, 0),)),
                                    None if contexts is None else _dev_any(contexts, "contexts", torch.int32, (n,)),
                                    None if slots is None else _dev_any(slots, "slots", torch.int32, (n,)),
                                    None if busy is None else _dev_any(busy, "busy", torch.uint8, (self.n_slots,)),
                                    bound, _stream_ptr()))
        self.max_length = bound
        return self

    def check(self):
        """Synchronise the current stream and raise if the plan refused a request."""
        _check(lib.stepq_plan_check(*self._args, _stream_ptr()))


def _rows(t: torch.Tensor, name: str, dtype, tokens: int, heads: int):
    """A [tokens, heads, 128] tensor whose rows of heads * 128 are contiguous: (pointer, token stride)."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a {dtype} CUDA tensor")
    if t.dim() != 3 or tuple(t.shape) != (tokens, heads, DK):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(tokens, heads, DK)}")
    if tokens > 0 and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != DK)):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return C.c_void_p(t.data_ptr()), (t.stride(0) if tokens > 1 else heads * DK)


def prompt(variant: int, plan: RequestPlan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
           beta: torch.Tensor, S: torch.Tensor, out: torch.Tensor | None = None, by_slot: bool = False) -> torch.Tensor:
    """The recurrence over all tokens of the plan's requests (stepq_prompt).

    variant GDN, KDA (the gated Delta rule) or LINEAR (decayed linear
    attention); q, k [tokens, heads_qk, 128] and v [tokens, heads, 128] in
    float32, float16 or bfloat16, token rows possibly strided, heads a multiple
    of heads_qk; alpha [tokens, heads] or [tokens, heads, 128] (KDA) and beta
    [tokens, heads] float32; S float32 [requests, heads, 128, 128], or with
    by_slot [slots, heads, 128, 128], updated in place.  Returns out [tokens,
    heads, 128] in the type of q; rows of no request keep what `out` held."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise TypeError("q must be a float32, float16 or bfloat16 CUDA tensor")
    if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("q and v must have shape [tokens, heads, 128]")
    T, Hk, H, dt = plan.tokens, q.shape[1], v.shape[1], q.dtype
    (qp, qs), (kp, ks) = _rows(q, "q", dt, T, Hk), _rows(k, "k", dt, T, Hk)
    vp, vs = _rows(v, "v", dt, T, H)
    ap = _dev(alpha, "alpha", (T, H, DK) if variant == KDA else (T, H))
    bp = _dev(beta, "beta", (T, H))
    Sp = _dev(S, "S", (plan.n_slots if by_slot else plan.requests, H, DK, DV))
    if out is None:
        out = torch.empty((T, H, DV), dtype=dt, device=q.device)
    op = _dev_any(out, "out", dt, (T, H, DV))
    key = (variant, dt, H, Hk, plan.max_length, by_slot, qs, ks, vs)
    if key not in plan._prompts:
        d = PromptDesc(variant, _DTYPES[dt], H, Hk, DK, DV, plan.max_length, int(by_slot), qs, ks, vs)
        need = lib.stepq_prompt_scratch_bytes(C.byref(plan._desc), C.byref(d))
        if need == C.c_size_t(-1).value:
            _check(ERR_INVALID_ARG)
        plan._prompts[key] = d, need
    d, need = plan._prompts[key]
    # from torch's allocator, so that calls on several streams or in several graphs have their own
    scratch = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    _check(lib.stepq_prompt(*plan._args, C.byref(d), qp, kp, vp, ap, bp, Sp, op,
                            C.c_void_p(scratch.data_ptr()) if need else None, need, _stream_ptr()))
    return out


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n: int | None = None):
    """The n (default: beams) best continuations of each group's beams
    (stepq_beam_select): logits [groups, beams, vocab] in float32, float16 or
    bfloat16, rows possibly strided; scores float32 [groups, beams].  Returns
    (scores float32, parents int32, tokens int32), each [groups, n], best
    first; score -inf, parent -1 and token -1 where no candidate is left."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _DTYPES or not logits.is_cuda:
        raise TypeError("logits must be a float32, float16 or bfloat16 CUDA tensor")
    if logits.dim() != 3:
        raise ValueError("logits must have shape [groups, beams, vocab]")
    G, B, V = logits.shape
    n = B if n is None else int(n)
    sp = _dev(scores, "scores", (G, B))
    if V > 0 and logits.stride(2) != 1:
        raise ValueError("logits: a row's tokens must be contiguous")
    stride = logits.stride(1) if B > 1 else (logits.stride(0) if G > 1 else V)
    if G > 1 and B > 1 and logits.stride(0) != B * stride:
        raise ValueError("logits: rows must be evenly spaced")
    dev = logits.device
    need = lib.stepq_beam_scratch_bytes(G, B, V, n)
    if need == 0:
        _check(ERR_INVALID_ARG)
    best, parents, tokens = torch.empty((3, G, n), dtype=torch.int32, device=dev).unbind(0)
    out = best.view(torch.float32), parents, tokens
    scratch = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib.stepq_beam_select(G, B, V, n, _DTYPES[logits.dtype], C.c_void_p(logits.data_ptr()), stride, sp,
                                 *(C.c_void_p(t.data_ptr()) for t in out), C.c_void_p(scratch.data_ptr()), need, _stream_ptr()))
    return out


def reorder_rows(rows: torch.Tensor, parents: torch.Tensor):
    """Reorder rows inside groups, in place (stepq_reorder_rows): with parents
    [groups, beams] (int32 CUDA), row g * beams + i of the contiguous CUDA
    tensor rows [groups * beams, ...] becomes what row g * beams + parents[g, i]
    was -- unquantised states, convolution windows, token histories."""
    if not isinstance(rows, torch.Tensor) or not rows.is_cuda or rows.dim() < 1:
        raise TypeError("rows must be a CUDA tensor")
    if not isinstance(parents, torch.Tensor) or parents.dim() != 2:
        raise ValueError("parents must have shape [groups, beams]")
    G, B = parents.shape
    if rows.shape[0] != G * B:
        raise ValueError(f"rows has {rows.shape[0]} rows, expected {G * B}")
    if not rows.is_contiguous():
        raise ValueError("rows must be contiguous")
    nbytes = rows.numel() // max(G * B, 1) * rows.element_size()
    _check(lib.stepq_reorder_rows(C.c_void_p(rows.data_ptr()), nbytes, G, B,
                                  _dev_any(parents, "parents", torch.int32, (G, B)), _stream_ptr()))
    return rows


# ---- calibration -------------------------------------------------------------

def _host(a, dtype):
    a = np.ascontiguousarray(a, dtype=dtype)
    return a, a.ctypes.data_as(C.c_void_p)


def calibrate(variant: int, S0: torch.Tensor, q, k, v, alpha, beta, widths, avg_bits: float,
              pivot_frac: float, sample_every: int, ls_iters: int = 1):
    """The library's calibration (stepq_calibrate): S0 [B, H, 128, 128] and the
    rollout's inputs q, k [T, B, H, 128], v [T, B, H, 128], alpha [T, B, H] or
    [T, B, H, 128], beta [T, B, H], all float32 CUDA tensors.  Returns
    (rho [H, 128] float32, bits [H, 128] uint8) as numpy arrays."""
    T, B, H = q.shape[0], q.shape[1], q.shape[2]
    w, wp = _host(widths, np.int32)
    cd = CalibDesc(variant, B, H, DK, DV, T, int(sample_every), int(ls_iters), int(w.size), wp,
                   float(avg_bits), float(pivot_frac))
    nbytes = lib.stepq_calib_scratch_bytes(C.byref(cd))
    if nbytes == 0:
        _check(ERR_INVALID_ARG)
    scratch = torch.empty(nbytes, dtype=torch.uint8, device=S0.device)
    rho = np.zeros((H, DK), np.float32); bits = np.zeros((H, DK), np.uint8)
    ash = (T, B, H, DK) if variant == KDA else (T, B, H)
    _check(lib.stepq_calibrate(C.byref(cd), _dev(S0, "S0", (B, H, DK, DV)), _dev(q, "q", (T, B, H, DK)),
                               _dev(k, "k", (T, B, H, DK)), _dev(v, "v", (T, B, H, DV)), _dev(alpha, "alpha", ash),
                               _dev(beta, "beta", (T, B, H)), C.c_void_p(scratch.data_ptr()), nbytes,
                               _stream_ptr(), rho.ctypes.data_as(C.c_void_p), bits.ctypes.data_as(C.c_void_p)))
    return rho, bits


def calib_accumulate(variant: int, q: torch.Tensor, alpha: torch.Tensor, acc_q2: torch.Tensor,
                     acc_loga: torch.Tensor):
    """One step's q [B, H, 128] and alpha into the float64 CUDA sums acc_q2
    [H, 128] and acc_loga ([H] or [H, 128])."""
    B, H = q.shape[0], q.shape[1]
    ash = (B, H, DK) if variant == KDA else (B, H)
    _check(lib.stepq_calib_accumulate(variant, B, H, _dev(q, "q", (B, H, DK)), _dev(alpha, "alpha", ash),
                                      _dev_any(acc_q2, "acc_q2", torch.float64, (H, DK)),
                                      _dev_any(acc_loga, "acc_loga", torch.float64, (H, DK) if variant == KDA else (H,)),
                                      _stream_ptr()))


def calib_row_error(S: torch.Tensor, rho: torch.Tensor, widths, ls_iters: int = 1):
    """Per-row squared errors of the states S [B, H, 128, 128] stored at each of
    `widths`: returns (err [B, H, nW, 128], rc [B, H, nW, 256]) float32 CUDA tensors."""
    B, H = S.shape[0], S.shape[1]
    w, wp = _host(widths, np.int32)
    err = torch.empty((B, H, w.size, DK), dtype=torch.float32, device=S.device)
    rc = torch.empty((B, H, w.size, DK + DV), dtype=torch.float32, device=S.device)
    _check(lib.stepq_calib_row_error(B, H, _dev(S, "S", (B, H, DK, DV)), _dev(rho, "rho", (H, DK)), int(w.size), wp,
                                     int(ls_iters), C.c_void_p(err.data_ptr()), C.c_void_p(rc.data_ptr()),
                                     _stream_ptr()))
    return err, rc


def calib_reduce(err: torch.Tensor, err_sum: torch.Tensor):
    """err_sum [H, nW, 128] (float64 CUDA) += err [B, H, nW, 128], request by request."""
    B, H, nW = err.shape[0], err.shape[1], err.shape[2]
    _check(lib.stepq_calib_reduce(B, H, nW, _dev(err, "err", (B, H, nW, DK)),
                                  _dev_any(err_sum, "err_sum", torch.float64, (H, nW, DK)), _stream_ptr()))


def calib_rho(acc_q2: np.ndarray, n_samples: float) -> np.ndarray:
    """Host: impact scores [H, 128] from the sums of q^2."""
    a, ap = _host(acc_q2, np.float64)
    H = a.shape[0]
    rho = np.zeros((H, DK), np.float32)
    _check(lib.stepq_calib_rho(H, float(n_samples), ap, rho.ctypes.data_as(C.c_void_p)))
    return rho


def calib_bits(variant: int, acc_loga, rho, err_sum, widths, avg_bits, pivot_frac, n_samples) -> np.ndarray:
    """Host: the row widths [H, 128] from the calibration sums (err_sum [H, nW, 128])."""
    la, lap = _host(acc_loga, np.float64)
    r, rp = _host(rho, np.float32)
    e, ep = _host(err_sum, np.float64)
    w, wp = _host(widths, np.int32)
    H = e.shape[0]
    bits = np.zeros((H, DK), np.uint8)
    _check(lib.stepq_calib_bits(variant, H, float(n_samples), lap, rp, ep, int(w.size), wp, float(avg_bits),
                                float(pivot_frac), bits.ctypes.data_as(C.c_void_p)))
    return bits
