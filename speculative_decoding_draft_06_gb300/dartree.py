"""Python binding of the DARTree C ABI (``include/dartree.h``).

Argument marshalling only: every step of a build runs in the CUDA library
``_build/libdartree.so``.  There is no fallback -- if the library has not been
built (``__graft_entry__.build()`` or ``python -m
speculative_decoding_draft_06_gb300.build``), :func:`load` raises.
Tensors are PyTorch CUDA tensors (PyTorch provides device memory and
streams); bf16 weights may be ``torch.bfloat16`` or 16-bit integer tensors
holding bf16 bit patterns.
"""
from __future__ import annotations

import ctypes
import os
import platform
import re

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", platform.machine(), "libdartree.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "dartree.h")

STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "DEVICE_CHECK",
          5: "TIMEOUT", 6: "OOM"}
W_F32, W_BF16 = 0, 1
WEIGHT_LAYOUTS = {"rows": 0, "blocks": 1}
HEAD_KINDS = {"recurrent": 0, "markov": 1}
CAND_KINDS = {"corrected": 0, "base": 1}
EXPANSIONS = {"depthwise": 0, "bestfirst": 1}

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("V", "H", "max_D", "max_W", "max_K", "max_B", "max_requests", "wdtype")]


class HeadWeights(ctypes.Structure):
    _fields_ = [("A", _vp), ("E", _vp), ("Wout", _vp)]


class Options(ctypes.Structure):
    _fields_ = [("head_kind", ctypes.c_int32), ("candidates", ctypes.c_int32),
                ("expansion", ctypes.c_int32)]


class Tree(ctypes.Structure):
    _fields_ = [("parent", _vp), ("token", _vp), ("depth", _vp), ("score", _vp),
                ("mask", _vp), ("n_out", _vp)]


class Cache(ctypes.Structure):
    _fields_ = [("pool", _vp), ("refs", _vp), ("layers", _i32), ("pages", _i32),
                ("page_tokens", _i32), ("Hkv", _i32), ("dh", _i32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class DartreeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"dartree {STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def declared_symbols() -> list[str]:
    """Function names declared by include/dartree.h."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"\b(dartree_[a-z_]+)\s*\(", txt)))


def load():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"DARTree CUDA library not built ({LIB_PATH} missing); "
                           "run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    st = ctypes.c_int
    sig = {
        "dartree_pool_size": (_i32, [_i32, _i32, _i32]),
        "dartree_create": (st, [ctypes.POINTER(Config), ctypes.POINTER(_vp)]),
        "dartree_destroy": (None, [_vp]),
        "dartree_build": (st, [_vp, _vp, _vp, ctypes.POINTER(HeadWeights), _i32, _i32, _i32,
                               _i32, _i32, ctypes.c_float, ctypes.POINTER(Tree), _vp]),
        "dartree_build_ex": (st, [_vp, _vp, _vp, ctypes.POINTER(HeadWeights), _i32, _i32,
                                  _i32, _i32, _i32, ctypes.c_float, ctypes.POINTER(Options),
                                  ctypes.POINTER(Tree), _vp]),
        "dartree_build_host": (st, [_vp, _vp, _vp, ctypes.POINTER(HeadWeights), _i32, _i32,
                                    _i32, _i32, _i32, ctypes.c_float, ctypes.POINTER(Tree), _vp]),
        "dartree_sync_status": (st, [_vp, _vp]),
        "dartree_head_calls": (ctypes.c_int64, [_vp]),
        "dartree_set_weight_layout": (st, [_vp, _i32]),
        "dartree_blocked_weight_bytes": (ctypes.c_size_t, [_i32, _i32]),
        "dartree_block_weights": (st, [_vp, _i32, _i32, _vp, _vp]),
        "dartree_last_error": (ctypes.c_char_p, [_vp]),
        "dartree_get_pool": (st, [_vp, _vp, _vp, _vp, _vp, _vp]),
        "dartree_get_rows": (st, [_vp, _i32, _vp, _vp, _vp, _vp]),
        "dartree_head_topk": (st, [_vp, _vp, _vp, ctypes.c_int64, _i32, _vp, _i32, _i32, _vp,
                                   _vp, _vp, _vp]),
        "dartree_state_step": (st, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp]),
        "dartree_prune": (st, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, ctypes.c_float,
                               ctypes.POINTER(Tree), _vp]),
        "dartree_set_timing": (st, [_vp, _i32]),
        "dartree_get_timing": (st, [_vp, _i32, ctypes.POINTER(ctypes.c_double),
                                    ctypes.POINTER(ctypes.c_int64)]),
        "dartree_reset_timing": (st, [_vp]),
        "dartree_state_step_noalloc": (st, [_vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp]),
        "dartree_get_states": (st, [_vp, _i32, _vp, _vp]),
        "dartree_tree_attention": (st, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                        ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp,
                                        _vp]),
        "dartree_tree_attention_workspace": (ctypes.c_size_t, [_i32, _i32, _i32, _i32, _i32]),
        "dartree_accept": (st, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    }
    cache, i64 = ctypes.POINTER(Cache), ctypes.c_int64
    sig.update({
        "dartree_cache_page_bytes": (ctypes.c_size_t, [_i32, _i32, _i32]),
        "dartree_cache_append": (st, [cache, _i32, _vp, _vp, i64, i64, _vp, _i32, _vp, _i32, _vp,
                                      _i32, _i32, _vp, _vp]),
        "dartree_cache_append_slots": (st, [cache, _i32, _vp, _vp, i64, _vp, _i32, _vp, _vp]),
        "dartree_cache_plan": (st, [cache, _vp, _i32, _vp, _vp] + [_i32] * 5 + [_vp] * 7),
        "dartree_cache_read": (st, [cache, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32,
                                    _vp, _vp]),
        "dartree_cache_read_ex": (st, [cache, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32,
                                       _i32, _vp, _vp]),
        "dartree_cache_attention": (st, [cache, _i32, _vp, i64, _vp, _vp, _vp, _i32, _vp, _i32,
                                         _i32, _i32, _i32, ctypes.c_float, _vp, _vp,
                                         ctypes.c_size_t, _vp, _vp]),
        "dartree_cache_attention_ex": (st, [cache, _i32, _vp, i64, _vp, _vp, _vp, _i32, _vp, _i32,
                                            _i32, _i32, _i32, ctypes.c_float, _i32, _vp, _vp,
                                            ctypes.c_size_t, _vp, _vp]),
        "dartree_cache_attention_workspace": (ctypes.c_size_t, [_i32] * 6),
        "dartree_cache_window_attention": (st, [cache, _i32, _vp, i64, i64, _vp, _vp, _vp, _vp, _i32,
                                                _vp] + [_i32] * 7 + [ctypes.c_float, _i32, _vp, _vp,
                                                                     ctypes.c_size_t, _vp, _vp]),
        "dartree_cache_window_attention_workspace": (ctypes.c_size_t, [_i32] * 9),
        "dartree_cache_reserve": (st, [cache, _vp, _i32, _vp, _vp, _i32, _vp, _vp]),
        "dartree_cache_reserve_ex": (st, [cache, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp]),
        "dartree_cache_fork": (st, [cache, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp]),
        "dartree_cache_fork_ex": (st, [cache, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp]),
        "dartree_cache_commit": (st, [cache, _vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp]),
        "dartree_cache_release": (st, [cache, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp]),
        "dartree_cache_copy_pages": (st, [cache, _vp, _vp, _i32, _vp, _vp]),
        "dartree_sample": (st, [_vp, _i32, i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                _vp, _vp]),
    })
    sig["dartree_verify"] = (st, [_vp, _vp, _vp, _vp, _i32, i64, i64, _vp, _i32, i64, i64] + [_i32] * 4
                             + [_vp] * 6 + [_i32] + [_vp] * 5)
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def pool_size(D: int, W: int, K: int) -> int:
    return int(load().dartree_pool_size(D, W, K))


def frontier_sizes(D: int, W: int, K: int) -> list[int]:
    f, out = 1, []
    for _ in range(D):
        f = min(W, K * f)
        out.append(f)
    return out


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor, name: str, dtypes) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


_W16 = (torch.bfloat16, torch.int16, torch.uint16)


class DARTree:
    """One library context: fixed V, H, capacities and weight dtype."""

    def __init__(self, V: int, H: int, *, max_D: int, max_W: int, max_K: int, max_B: int,
                 max_requests: int = 1, bf16: bool = True, device: int | None = None):
        lib = load()
        if device is not None:
            torch.cuda.set_device(device)
        torch.cuda.init()
        self.cfg = Config(V, H, max_D, max_W, max_K, max_B, max_requests,
                          W_BF16 if bf16 else W_F32)
        self.bf16 = bf16
        self.V, self.H = V, H
        h = ctypes.c_void_p()
        s = lib.dartree_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if s != 0:
            raise DartreeError(s, "dartree_create: " + lib.dartree_last_error(None).decode())
        self._h = h
        self._lib = lib

    # ------------------------------------------------------------ plumbing
    def close(self) -> None:
        if getattr(self, "_h", None):
            self._lib.dartree_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, s: int) -> None:
        if s != 0:
            raise DartreeError(s, self._lib.dartree_last_error(self._h).decode())

    def _wtypes(self):
        return _W16 if self.bf16 else (torch.float32,)

    def _head(self, A, E, Wout) -> HeadWeights:
        """A may be None (Markov head)."""
        wt = self._wtypes()
        _dev(E, "E", wt), _dev(Wout, "Wout", wt)
        if A is not None:
            _dev(A, "A", wt)
        return HeadWeights(None if A is None else A.data_ptr(), E.data_ptr(), Wout.data_ptr())

    def alloc_tree(self, R: int, B: int, *, device="cuda", pin: bool = False) -> dict:
        words = (B + 31) // 32
        kw = {"device": device} if device != "cpu" else {"pin_memory": pin}
        return {"parent": torch.empty(R, B, dtype=torch.int32, **kw),
                "token": torch.empty(R, B, dtype=torch.int32, **kw),
                "depth": torch.empty(R, B, dtype=torch.int32, **kw),
                "score": torch.empty(R, B, dtype=torch.float32, **kw),
                "mask": torch.empty(R, B, words, dtype=torch.int32, **kw),
                "n_out": torch.empty(R, dtype=torch.int32, **kw)}

    @staticmethod
    def _tree(out: dict) -> Tree:
        return Tree(*(out[k].data_ptr() for k in ("parent", "token", "depth", "score", "mask",
                                                  "n_out")))

    # ------------------------------------------------------------ the path
    def build(self, z, state0, A, E, Wout, *, D: int, W: int, K: int, B: int, beta: float,
              out: dict | None = None, stream=None, head: str = "recurrent",
              candidates: str = "corrected", expansion: str = "depthwise") -> dict:
        """Asynchronous supertree build; z [R,D,V] fp32, state0 [R,H] fp32.
        ``head`` / ``candidates`` / ``expansion`` select the build variant
        (dartree_build_ex); the defaults are dartree_build."""
        _dev(z, "z", (torch.float32,)), _dev(state0, "state0", (torch.float32,))
        R = state0.shape[0]
        if z.shape != (R, D, self.V) or state0.shape != (R, self.H):
            raise ValueError(f"z {tuple(z.shape)} / state0 {tuple(state0.shape)} do not match "
                             f"R={R}, D={D}, V={self.V}, H={self.H}")
        if out is None:
            out = self.alloc_tree(R, B, device=z.device)
        hw = self._head(A, E, Wout)
        t = self._tree(out)
        opt = (head, candidates, expansion)
        if opt == ("recurrent", "corrected", "depthwise"):
            self._check(self._lib.dartree_build(self._h, _ptr(z), _ptr(state0), ctypes.byref(hw),
                                                R, D, W, K, B, ctypes.c_float(beta),
                                                ctypes.byref(t), _stream(stream)))
        else:
            o = Options(HEAD_KINDS[head], CAND_KINDS[candidates], EXPANSIONS[expansion])
            self._check(self._lib.dartree_build_ex(
                self._h, _ptr(z), _ptr(state0), ctypes.byref(hw), R, D, W, K, B,
                ctypes.c_float(beta), ctypes.byref(o), ctypes.byref(t), _stream(stream)))
        return out

    def build_host(self, z_host, state0_host, A, E, Wout, *, D: int, W: int, K: int, B: int,
                   beta: float, out_host: dict, stream=None) -> dict:
        """Build from host inputs into host outputs (copies included, synchronous)."""
        for n, t in (("z", z_host), ("state0", state0_host)):
            if t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
                raise TypeError(f"{n} must be a contiguous fp32 host tensor")
        R = state0_host.shape[0]
        head = self._head(A, E, Wout)
        t = self._tree(out_host)
        self._check(self._lib.dartree_build_host(
            self._h, _ptr(z_host), _ptr(state0_host), ctypes.byref(head), R, D, W, K, B,
            ctypes.c_float(beta), ctypes.byref(t), _stream(stream)))
        return out_host

    def sync(self, stream=None) -> None:
        """Synchronise and raise on a device-side check."""
        self._check(self._lib.dartree_sync_status(self._h, _stream(stream)))

    def sync_status(self, stream=None) -> int:
        return int(self._lib.dartree_sync_status(self._h, _stream(stream)))

    KERNEL_KINDS = ("head", "state", "merge", "select", "prune", "root", "candidates",
                    "bestfirst")

    def set_timing(self, on: bool) -> None:
        self._check(self._lib.dartree_set_timing(self._h, 1 if on else 0))

    def reset_timing(self) -> None:
        self._check(self._lib.dartree_reset_timing(self._h))

    def timing(self) -> dict:
        """{kind: (total_ms, launches)} accumulated at each sync()."""
        out = {}
        for i, k in enumerate(self.KERNEL_KINDS):
            ms, n = ctypes.c_double(), ctypes.c_int64()
            self._check(self._lib.dartree_get_timing(self._h, i, ctypes.byref(ms),
                                                     ctypes.byref(n)))
            out[k] = (ms.value, n.value)
        return out

    def set_weight_layout(self, layout: str) -> None:
        """Layout of the Wout passed to later calls: "rows" ([V, H]
        row-major) or "blocks" (128 x 64 blocks, see block_weights;
        dartree_set_weight_layout)."""
        self._check(self._lib.dartree_set_weight_layout(self._h, WEIGHT_LAYOUTS[layout]))

    def head_calls(self) -> int:
        return int(self._lib.dartree_head_calls(self._h))

    def last_error(self) -> str:
        return self._lib.dartree_last_error(self._h).decode()

    def get_pool(self, R: int, P: int, stream=None) -> dict:
        o = {k: torch.empty(R, P, dtype=torch.int32) for k in ("parent", "token", "depth")}
        o["score"] = torch.empty(R, P, dtype=torch.float32)
        self._check(self._lib.dartree_get_pool(self._h, _ptr(o["parent"]), _ptr(o["token"]),
                                               _ptr(o["depth"]), _ptr(o["score"]),
                                               _stream(stream)))
        torch.cuda.synchronize()
        return o

    def get_rows(self, d: int, rows: int, K: int, stream=None) -> dict:
        o = {"lse": torch.empty(rows, dtype=torch.float64),
             "tok": torch.empty(rows, K, dtype=torch.int32),
             "logp": torch.empty(rows, K, dtype=torch.float32)}
        self._check(self._lib.dartree_get_rows(self._h, d, _ptr(o["lse"]), _ptr(o["tok"]),
                                               _ptr(o["logp"]), _stream(stream)))
        torch.cuda.synchronize()
        return o

    def get_states(self, d: int, rows: int, stream=None):
        """Head states of head call d as fp32 [rows, H] (bf16 values widened)."""
        dt = torch.int16 if self.bf16 else torch.float32
        o = torch.empty(rows, self.H, dtype=dt)
        self._check(self._lib.dartree_get_states(self._h, d, _ptr(o), _stream(stream)))
        torch.cuda.synchronize()
        if self.bf16:
            return (o.numpy().view(np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32)
        return o.numpy()

    # ------------------------------------------------ single-step entries
    def head_topk(self, S, z, Wout, *, K: int, rows_per_req: int | None = None,
                  z_req_stride: int = 0, stream=None) -> dict:
        """One batched head call: per row lse, top-K tokens and log-probs."""
        _dev(S, "S", self._wtypes()), _dev(z, "z", (torch.float32,))
        _dev(Wout, "Wout", self._wtypes())
        M = S.shape[0]
        dev = S.device
        o = {"lse": torch.empty(M, dtype=torch.float64, device=dev),
             "tok": torch.empty(M, K, dtype=torch.int32, device=dev),
             "logp": torch.empty(M, K, dtype=torch.float32, device=dev)}
        self._check(self._lib.dartree_head_topk(
            self._h, _ptr(S), _ptr(z), int(z_req_stride), rows_per_req or M, _ptr(Wout), M, K,
            _ptr(o["lse"]), _ptr(o["tok"]), _ptr(o["logp"]), _stream(stream)))
        return o

    def state_step(self, S_par, tok, A, E, stream=None):
        """S_out = q(tanh(A S_par + E[tok])) for every row."""
        wt = self._wtypes()
        _dev(S_par, "S_par", wt), _dev(tok, "tok", (torch.int32,))
        _dev(A, "A", wt), _dev(E, "E", wt)
        out = torch.empty_like(S_par)
        self._check(self._lib.dartree_state_step(self._h, _ptr(S_par), _ptr(tok), _ptr(A),
                                                 _ptr(E), S_par.shape[0], _ptr(out),
                                                 _stream(stream)))
        return out

    def prune(self, parent, token, depth, score, *, B: int, beta: float, stream=None) -> dict:
        """Deferred Top-B + compaction + mask over pools [R, P]."""
        for n, t in (("parent", parent), ("token", token), ("depth", depth)):
            _dev(t, n, (torch.int32,))
        _dev(score, "score", (torch.float32,))
        R, P = parent.shape
        out = self.alloc_tree(R, B, device=parent.device)
        t = self._tree(out)
        self._check(self._lib.dartree_prune(self._h, _ptr(parent), _ptr(token), _ptr(depth),
                                            _ptr(score), R, P, B, ctypes.c_float(beta),
                                            ctypes.byref(t), _stream(stream)))
        return out


def state_step_noalloc(S_par, tok, A, E, stream=None):
    """Context-free bf16 state step (dartree_state_step_noalloc): for callers
    that cannot allocate device memory.  The output tensor is allocated here
    by PyTorch only because this is the Python convenience wrapper; the C
    entry point itself allocates nothing.  Raises DartreeError on failure."""
    lib = load()
    for n, t in (("S_par", S_par), ("A", A), ("E", E)):
        _dev(t, n, _W16)
    _dev(tok, "tok", (torch.int32,))
    M, H = S_par.shape
    out = torch.empty_like(S_par)
    s = lib.dartree_state_step_noalloc(_ptr(S_par), _ptr(tok), _ptr(A), _ptr(E), H, M, _ptr(out),
                                       _stream(stream))
    if s != 0:
        raise DartreeError(s, lib.dartree_last_error(None).decode())
    return out


def weights_to_device(inp: dict, bf16: bool, device="cuda") -> dict:
    """Host input arrays (numpy) -> device tensors in the library's layout."""
    def w(a):
        t = torch.from_numpy(a)
        if bf16:
            t = t.view(torch.int16)
        return t.to(device)
    return {"A": w(inp["A"]), "E": w(inp["E"]), "Wout": w(inp["Wout"]),
            "z": torch.from_numpy(inp["z"]).to(device),
            "state0": torch.from_numpy(inp["state0"]).to(device)}


def _check_free(s: int) -> None:
    if s != 0:
        raise DartreeError(s, load().dartree_last_error(None).decode())


def tree_attention(Q, K, Vt, mask, *, Lp: int, scale: float | None = None,
                   want_bf16: bool = True, work=None, split: bool = True, err=None,
                   stream=None) -> dict:
    """Tree attention of the verification forward (dartree_tree_attention):
    Q [R,B+1,Hq,dh], key cache K [R,Hkv,Lp+B,dh] (prefix keys, then the tree
    nodes'), blocked transposed value cache Vt [R,Hkv,ceil(L/64),dh,64] (bf16
    CUDA tensors; see kv_cache),
    mask [R,B,words] int32 -> {"O": fp32, "O16": bf16 bits}.  ``work`` and
    ``split`` are kept for the interface: the key splits need no scratch."""
    for n, t in (("Q", Q), ("K", K), ("Vt", Vt)):
        _dev(t, n, _W16)
    _dev(mask, "mask", (torch.int32,))
    R, Bp1, Hq, dh = Q.shape
    Hkv = K.shape[1]
    O = torch.empty(R, Bp1, Hq, dh, dtype=torch.float32, device=Q.device)
    O16 = torch.empty(R, Bp1, Hq, dh, dtype=torch.int16, device=Q.device) if want_bf16 else None
    sc = float(scale) if scale is not None else dh ** -0.5
    wb = 0 if work is None else work.numel() * work.element_size()
    _check_free(load().dartree_tree_attention(
        _ptr(Q), _ptr(K), _ptr(Vt), _ptr(mask), R, Lp, Bp1 - 1, Hq, Hkv, dh,
        ctypes.c_float(sc), _ptr(O), _ptr(O16), _ptr(work), wb, _ptr(err), _stream(stream)))
    return {"O": O, "O16": O16}


def block_weights(W: torch.Tensor, stream=None) -> torch.Tensor:
    """The blocked layout (blocks of 128 rows x 64 columns, rows past V
    zero; dartree_block_weights) of a row-major bf16 CUDA matrix [V, H],
    as a [ceil(V/128) * 128, H] tensor of the same dtype."""
    _dev(W, "W", _W16)
    V, H = W.shape
    n = int(load().dartree_blocked_weight_bytes(V, H))
    if n == 0:
        raise ValueError("H must be a multiple of 64")
    out = torch.empty(n // (2 * H), H, dtype=W.dtype, device=W.device)
    _check_free(load().dartree_block_weights(_ptr(W), V, H, _ptr(out), _stream(stream)))
    return out


def kv_cache(Kp, Vp, Kt, Vt) -> tuple[torch.Tensor, torch.Tensor]:
    """Key cache [R, Hkv, Lp+B, dh] and blocked transposed value cache
    [R, Hkv, ceil(L/64), dh, 64] from prefix [R, Lp, Hkv, dh] and tree
    [R, B, Hkv, dh] keys / values (CUDA tensors; data movement only)."""
    K = torch.cat([Kp, Kt], dim=1).permute(0, 2, 1, 3).contiguous()   # [R, Hkv, L, dh]
    V = torch.cat([Vp, Vt], dim=1).permute(0, 2, 1, 3)                 # [R, Hkv, L, dh]
    R, Hkv, L, dh = V.shape
    nb = (L + 63) // 64
    Vb = torch.zeros(R, Hkv, nb * 64, dh, dtype=V.dtype, device=V.device)
    Vb[:, :, :L] = V
    VT = Vb.view(R, Hkv, nb, 64, dh).transpose(3, 4).contiguous()      # [R, Hkv, nb, dh, 64]
    return K, VT


def accept(parent, token, n_out, pred, *, max_len: int, stream=None) -> dict:
    """Longest accepted prefix per request (dartree_accept); CUDA int32
    tensors parent/token [R,B], n_out [R], pred [R,B+1]."""
    for n, t in (("parent", parent), ("token", token), ("n_out", n_out), ("pred", pred)):
        _dev(t, n, (torch.int32,))
    R, B = parent.shape
    dev = parent.device
    o = {"len": torch.empty(R, dtype=torch.int32, device=dev),
         "nodes": torch.empty(R, max(max_len, 1), dtype=torch.int32, device=dev),
         "bonus": torch.empty(R, dtype=torch.int32, device=dev)}
    _check_free(load().dartree_accept(_ptr(parent), _ptr(token), _ptr(n_out), _ptr(pred), R, B,
                                      max_len, _ptr(o["len"]), _ptr(o["nodes"]), _ptr(o["bonus"]),
                                      _stream(stream)))
    return o


# ------------------------------------------------------- paged 4-bit cache
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_I32 = torch.int32
_TOP = 1 << 31


def _ints(name: str, t: torch.Tensor, idx: int, n: int) -> int:
    """Address of a dense int32 tensor of n entries on CUDA device idx."""
    if t.dtype is _I32 and t.numel() == n and t.is_contiguous() and t.get_device() == idx:
        return t.data_ptr()
    if t.dtype is not _I32 or not t.is_contiguous() or t.get_device() != idx:
        raise TypeError(f"{name} must be a contiguous int32 tensor on cuda:{idx}")
    raise ValueError(f"{name} has {t.numel()} entries, expected {n}")


def _floats(name: str, t: torch.Tensor, idx: int, n: int) -> int:
    if t.dtype is not torch.float32 or not t.is_contiguous() or t.get_device() != idx:
        raise TypeError(f"{name} must be a contiguous fp32 tensor on cuda:{idx}")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} entries, expected {n}")
    return t.data_ptr()


def _alloc(stream, shape, dtype, dev) -> torch.Tensor:
    """A tensor whose memory belongs to the call's stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


# the current stream's handle without a Stream object (which costs as much as
# the rest of a call), where PyTorch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda idx: torch.cuda.current_stream(idx).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(fn, idx: int, stream, *args) -> None:
    """Calls fn(*args, stream) with the tensors' device current; raises on an
    error."""
    st = _raw_stream(idx) if stream is None else stream.cuda_stream
    if _device() == idx:
        s = fn(*args, st)
    else:
        with torch.cuda.device(idx):
            s = fn(*args, st)
    if s != 0:
        _check_free(s)


class KVCache:
    """A paged key/value cache in 4 bits (dartree_cache): the pool of pages
    and the pages' reference counts.  The sequences -- page tables [R,
    max_pages] int32 (-1: no page) and lengths [R] int32 -- are the caller's
    tensors.  ``pool`` (uint8 [layers, pages, page_bytes]) and ``refs`` (int32
    [pages]) may be given; otherwise they are allocated, all pages free.
    Bad indices found on the device gather in ``err`` until :meth:`check`."""

    def __init__(self, layers: int, pages: int, *, page_tokens: int = 64, Hkv: int, dh: int,
                 k_scale: float = 1.0, v_scale: float = 1.0, pool: torch.Tensor | None = None,
                 refs: torch.Tensor | None = None, device="cuda"):
        self._lib = load()
        self.page_bytes = int(self._lib.dartree_cache_page_bytes(page_tokens, Hkv, dh))
        if self.page_bytes == 0 or layers < 1 or pages < 1:
            raise ValueError("page_tokens must be 16, 32, 64 or 128, dh 64 or 128, layers, pages "
                             "and Hkv at least 1 (65535 at most)")
        for s in (k_scale, v_scale):
            if not (2.0 ** -64 <= s <= 2.0 ** 64 and np.frexp(s)[0] == 0.5):
                raise ValueError("k_scale and v_scale must be powers of two from 2^-64 to 2^64")
        if pool is None:
            pool = torch.zeros(layers, pages, self.page_bytes, dtype=torch.uint8, device=device)
        if not pool.is_cuda or pool.dtype is not torch.uint8 or not pool.is_contiguous():
            raise TypeError("pool must be a contiguous uint8 CUDA tensor")
        if pool.shape != (layers, pages, self.page_bytes):
            raise ValueError(f"pool has shape {tuple(pool.shape)}, expected "
                             f"{(layers, pages, self.page_bytes)}")
        if refs is None:
            refs = torch.zeros(pages, dtype=torch.int32, device=pool.device)
        self.dev, self._idx = pool.device, pool.get_device()
        _ints("refs", refs, self._idx, pages)
        self.pool, self.refs = pool, refs
        self.layers, self.pages, self.page_tokens, self.Hkv, self.dh = (layers, pages, page_tokens,
                                                                        Hkv, dh)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.dev)
        self._c = Cache(pool.data_ptr(), refs.data_ptr(), layers, pages, page_tokens, Hkv, dh,
                        k_scale, v_scale)
        self._ref = ctypes.byref(self._c)
        self._err = self.err.data_ptr()
        self._work_bytes: dict = {}  # workspace sizes by (R, B, max_len, Hq)

    def _seqs(self, table: torch.Tensor, lens: torch.Tensor):
        """Addresses and sizes of a page table and its lengths."""
        R, width = table.shape
        idx = self._idx
        return _ints("table", table, idx, R * width), width, _ints("lens", lens, idx, R), R

    def check(self) -> None:
        """Synchronises the device and raises if a call since the last check, on
        any stream, met a bad index (a token without a page, a row or page out
        of range)."""
        torch.cuda.synchronize(self.dev)
        e = int(self.err.item())
        if e:
            self.err.zero_()
            raise DartreeError(5 if e & 2 else 4, f"cache: device check {e}")

    def append(self, layer: int, K: torch.Tensor, V: torch.Tensor, table, lens, *, offset: int = 0,
               count: torch.Tensor | None = None, stream=None) -> None:
        """Quantise K, V [R, n, Hkv, dh] bf16 into positions lens[r] + offset
        + i (dartree_cache_append); request and token strides are multiples of
        8, the same in both."""
        t, width, ln, R = self._seqs(table, lens)
        idx, Hkv, dh = self._idx, self.Hkv, self.dh
        if K.dtype not in _BF16 or K.get_device() != idx:
            raise TypeError(f"K must be a bf16 tensor on {self.dev}")
        if V.dtype not in _BF16 or V.get_device() != idx:
            raise TypeError(f"V must be a bf16 tensor on {self.dev}")
        n, want = K.shape[1], (R, K.shape[1], Hkv, dh)
        if K.shape != want or V.shape != want:
            raise ValueError(f"K {tuple(K.shape)} / V {tuple(V.shape)} do not match R={R}, "
                             f"Hkv={Hkv}, dh={dh}")
        (sr, sn, sh, sd), (vr, vn, vh, vd) = K.stride(), V.stride()
        if R == 1:  # (a dimension of one has no stride)
            sr = vr = 0
        if n == 1:
            sn = vn = Hkv * dh
        if Hkv == 1:
            sh = vh = dh
        if (sr, sn, sh, sd) != (vr, vn, vh, vd) or sd != 1 or sh != dh:
            raise ValueError("K and V need equal strides, dense in heads and dims")
        _launch(self._lib.dartree_cache_append, idx, stream, self._ref, layer, K.data_ptr(),
                V.data_ptr(), sr, sn, t, width, ln, offset,
                None if count is None else _ints("count", count, idx, R), R, n, self._err)

    def append_slots(self, layer: int, K: torch.Tensor, V: torch.Tensor, slot: torch.Tensor, *,
                     stream=None) -> None:
        """Quantise packed K, V [T, Hkv, dh] bf16 into the slots [T] int32 of
        :meth:`plan` (dartree_cache_append_slots); the token stride is a multiple
        of 8, the same in both."""
        idx, Hkv, dh = self._idx, self.Hkv, self.dh
        if K.dtype not in _BF16 or K.get_device() != idx:
            raise TypeError(f"K must be a bf16 tensor on {self.dev}")
        if V.dtype not in _BF16 or V.get_device() != idx:
            raise TypeError(f"V must be a bf16 tensor on {self.dev}")
        n = K.shape[0]
        if K.shape != (n, Hkv, dh) or V.shape != K.shape or n < 1:
            raise ValueError(f"K {tuple(K.shape)} / V {tuple(V.shape)} are not [T, {Hkv}, {dh}]")
        (sn, sh, sd), (vn, vh, vd) = K.stride(), V.stride()
        if n == 1:  # (a dimension of one has no stride)
            sn = vn = Hkv * dh
        if Hkv == 1:
            sh = vh = dh
        if (sn, sh, sd) != (vn, vh, vd) or sd != 1 or sh != dh:
            raise ValueError("K and V need equal strides, dense in heads and dims")
        _launch(self._lib.dartree_cache_append_slots, idx, stream, self._ref, layer, K.data_ptr(),
                V.data_ptr(), sn, _ints("slot", slot, idx, n), n, self._err)

    def read(self, layer: int, table, lens, n: int, *, offset: int = 0,
             count: torch.Tensor | None = None, out: tuple | None = None, stream=None) -> tuple:
        """The values of the tokens lens[r] + offset + i, i < n, as bf16 (K,
        V) [R, n, Hkv, dh] (dartree_cache_read_ex).  Tokens behind count[r] and
        rows with lens[r] < 0 keep what ``out`` holds (zeros in a new one)."""
        t, width, ln, R = self._seqs(table, lens)
        shape = (R, n, self.Hkv, self.dh)
        new = out is None
        if new:
            # (two calls: halves of one tensor cost 10 us more)
            out = (_alloc(stream, shape, torch.bfloat16, self.dev),
                   _alloc(stream, shape, torch.bfloat16, self.dev))
        else:
            for x in out:
                if x.dtype not in _BF16 or x.get_device() != self._idx or not x.is_contiguous():
                    raise TypeError(f"out must be contiguous bf16 tensors on {self.dev}")
                if x.shape != shape:
                    raise ValueError(f"out has shape {tuple(x.shape)}, expected {shape}")
        _launch(self._lib.dartree_cache_read_ex, self._idx, stream, self._ref, layer,
                out[0].data_ptr(), out[1].data_ptr(), t, width, ln, offset,
                None if count is None else _ints("count", count, self._idx, R), R, n, new, self._err)
        return out

    def attention(self, layer: int, Q: torch.Tensor, table, lens, *, max_len: int,
                  mask: torch.Tensor | None = None, n_nodes: torch.Tensor | None = None,
                  scale: float | None = None, out: torch.Tensor | None = None,
                  work: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of Q [R, B+1, Hq, dh] bf16 (row 0 the root, then the tree
        nodes; B = 0: single tokens) over the cache (dartree_cache_attention_ex)
        -> O bf16 [R, B+1, Hq, dh].  ``max_len`` bounds lens[r] + n_nodes[r].
        Rows behind n_nodes[r] and requests with lens[r] < 0 keep what ``out``
        holds (zeros in a new one)."""
        t, width, ln, R = self._seqs(table, lens)
        idx, dh = self._idx, self.dh
        if Q.dtype not in _BF16 or Q.get_device() != idx:
            raise TypeError(f"Q must be a bf16 tensor on {self.dev}")
        r, rows, Hq, d = Q.shape
        if r != R or rows < 1 or d != dh:
            raise ValueError(f"Q {tuple(Q.shape)} does not match R={R}, dh={dh}")
        B, sq = rows - 1, Hq * dh
        if Hq % self.Hkv:
            raise ValueError(f"{Hq} query heads are not a multiple of {self.Hkv}")
        if not Q.is_contiguous():
            sr, s1, sh, sd = Q.stride()
            sq = s1 if B else max(sr, sq)
            if (sr != rows * sq and R > 1) or (sh != dh and Hq > 1) or sd != 1:
                raise ValueError("Q needs one stride between rows, dense in heads and dims")
        m = None
        if B > 0:
            if mask is None:
                raise ValueError("a tree needs its mask")
            m = _ints("mask", mask, idx, R * B * ((B + 31) // 32))
        nn = None if n_nodes is None else _ints("n_nodes", n_nodes, idx, R)
        new = out is None
        if new:
            out = _alloc(stream, (R, rows, Hq, dh), torch.bfloat16, self.dev)
        elif out.dtype not in _BF16 or out.get_device() != idx or not out.is_contiguous():
            raise TypeError(f"out must be a contiguous bf16 tensor on {self.dev}")
        elif out.shape != (R, rows, Hq, dh):
            raise ValueError(f"out has shape {tuple(out.shape)}")
        key = (R, B, max_len, Hq)
        need = self._work_bytes.get(key)
        if need is None:
            if len(self._work_bytes) > 4096:
                self._work_bytes.clear()
            need = self._work_bytes[key] = int(
                self._lib.dartree_cache_attention_workspace(R, B, max_len, Hq, self.Hkv, dh))
        wp, wb = None, 0
        if work is not None:
            if not work.is_contiguous() or work.get_device() != idx:
                raise TypeError(f"work must be a contiguous tensor on {self.dev}")
            wp, wb = work.data_ptr(), work.numel() * work.element_size()
        elif need:
            work = _alloc(stream, (need,), torch.uint8, self.dev)
            wp, wb = work.data_ptr(), need
        _launch(self._lib.dartree_cache_attention_ex, idx, stream, self._ref, layer, Q.data_ptr(), sq, m,
                nn, t, width, ln, R, B, max_len, Hq, dh ** -0.5 if scale is None else scale,
                new, out.data_ptr(), wp, wb, self._err)
        return out

    @staticmethod
    def _window(window, sinks, offset) -> tuple:
        """window (0: none) and sinks as the calls take them: no position passes
        2^31 - 2, so larger ones are as good as that."""
        if window is not None and window < 1:
            raise ValueError("window must be at least 1")
        if sinks < 0 or not -_TOP <= offset < _TOP:
            raise ValueError("sinks must not be negative, offset fit 32 bits")
        return 0 if window is None else min(window, _TOP - 1), min(sinks, _TOP - 1)

    def window_attention(self, layer: int, Q: torch.Tensor, table, lens, *, max_len: int,
                         window: int | None = None, sinks: int = 0, offset: int = -1,
                         mask: torch.Tensor | None = None, n_nodes: torch.Tensor | None = None,
                         start: torch.Tensor | None = None, max_rows: int | None = None,
                         scale: float | None = None, out: torch.Tensor | None = None,
                         work: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention over the cache in which a row at position q sees the tokens
        k < ``sinks`` and k > q - ``window`` (None: all) of those it sees otherwise
        (dartree_cache_window_attention) -> O bf16, shaped as Q.  Row i of request r
        is at place lens[r] + ``offset`` + i: a chain (single tokens, drafted chains,
        a prompt's tokens), or with ``mask`` a draft tree behind its root.  Q [R,
        B+1, Hq, dh] (n_nodes[r] + 1 rows of request r count), or packed [T, Hq, dh]
        with ``start`` [R+1] (:meth:`plan`'s) and ``max_rows``, a bound of a request's
        rows.  ``max_len`` bounds the place behind a request's last row.  Rows that
        belong to no request keep what ``out`` holds (zeros in a new one)."""
        t, width, ln, R = self._seqs(table, lens)
        idx, dh = self._idx, self.dh
        if Q.dtype not in _BF16 or Q.get_device() != idx:
            raise TypeError(f"Q must be a bf16 tensor on {self.dev}")
        shape = Q.shape
        if start is None:
            if len(shape) != 4:
                raise ValueError(f"Q {tuple(shape)} is not [R, B+1, Hq, {dh}]")
            r, rows, Hq, d = shape
            if r != R or rows < 1 or d != dh:
                raise ValueError(f"Q {tuple(shape)} does not match R={R}, dh={dh}")
            total, B, s = R * rows, rows - 1, None
        else:
            if max_rows is None or max_rows < 1:
                raise ValueError("packed rows need max_rows")
            if n_nodes is not None:
                raise ValueError("packed rows have their numbers in start")
            if len(shape) != 3 or shape[0] < 1 or shape[2] != dh:
                raise ValueError(f"Q {tuple(shape)} is not [T, Hq, {dh}]")
            total, Hq, d = shape
            rows, B, s = total, max_rows - 1, _ints("start", start, idx, R + 1)
        if Hq < 1 or Hq % self.Hkv:
            raise ValueError(f"{Hq} query heads are not a multiple of {self.Hkv}")
        w, sinks = self._window(window, sinks, offset)
        if not 0 <= max_len < _TOP or B >= _TOP:
            raise ValueError("max_len and max_rows must fit 31 bits")
        sq = Hq * dh
        if not Q.is_contiguous():
            *lead, sh, sd = Q.stride()
            if s is None and rows == 1:  # (a dimension of one has no stride)
                sq = lead[0] if R > 1 else sq
            else:
                sq = lead[-1] if rows > 1 else sq
                if s is None and R > 1 and lead[0] != rows * sq:
                    raise ValueError("Q needs one stride between rows")
            if (sh != dh and Hq > 1) or sd != 1:
                raise ValueError("Q must be dense in heads and dims")
        m = None
        if mask is not None and B > 0:
            m = _ints("mask", mask, idx, R * B * ((B + 31) // 32))
        nn = None if n_nodes is None else _ints("n_nodes", n_nodes, idx, R)
        new = out is None
        if new:
            out = _alloc(stream, shape, torch.bfloat16, self.dev)
        elif out.dtype not in _BF16 or out.get_device() != idx or not out.is_contiguous():
            raise TypeError(f"out must be a contiguous bf16 tensor on {self.dev}")
        elif out.shape != shape:
            raise ValueError(f"out has shape {tuple(out.shape)}")
        key = (R, B, max_len, w, sinks, m is None, Hq)
        need = self._work_bytes.get(key)
        if need is None:
            if len(self._work_bytes) > 4096:
                self._work_bytes.clear()
            need = self._work_bytes[key] = int(self._lib.dartree_cache_window_attention_workspace(
                R, B, max_len, w, sinks, m is None, Hq, self.Hkv, dh))
        wp, wb = None, 0
        if work is not None:
            if not work.is_contiguous() or work.get_device() != idx:
                raise TypeError(f"work must be a contiguous tensor on {self.dev}")
            wp, wb = work.data_ptr(), work.numel() * work.element_size()
        elif need:
            work = _alloc(stream, (need,), torch.uint8, self.dev)
            wp, wb = work.data_ptr(), need
        _launch(self._lib.dartree_cache_window_attention, idx, stream, self._ref, layer, Q.data_ptr(), sq,
                total, s, m, nn, t, width, ln, R, B, max_len, offset, w, sinks, Hq,
                dh ** -0.5 if scale is None else scale, new, out.data_ptr(), wp, wb, self._err)
        return out

    # ------------------------------------------------------ page operations
    def reserve(self, table, lens, want, *, pending: int = 0, stream=None) -> torch.Tensor:
        """Pages for want[r] more tokens per row -> ok [R] int32
        (dartree_cache_reserve_ex).  ``pending``: how many of the last tokens of
        lens are counted but not written yet (commit's ``extra``)."""
        t, width, ln, R = self._seqs(table, lens)
        ok = _alloc(stream, (R,), _I32, self.dev)
        _launch(self._lib.dartree_cache_reserve_ex, self._idx, stream, self._ref, t, width, ln,
                _ints("want", want, self._idx, R), R, pending, ok.data_ptr())
        return ok

    def plan(self, table, lens, count, *, max_tokens: int, offset: int = -1,
             window: int | None = None, sinks: int = 0, out: dict | None = None, stream=None) -> dict:
        """Pages for count[r] packed tokens per row from position lens[r] +
        ``offset`` on, and their maps (dartree_cache_plan) -> {"ok" [R], "start"
        [R+1], "row", "pos", "slot" [max_tokens]} int32 (``out``: an earlier call's, to
        be written again).  With ``window``, pages that it has left behind (but for
        the first ``sinks`` tokens') are let go."""
        t, width, ln, R = self._seqs(table, lens)
        w, sinks = self._window(window, sinks, offset)
        if not 0 <= max_tokens < _TOP:
            raise ValueError("max_tokens must not be negative, and fit 31 bits")
        c = _ints("count", count, self._idx, R)
        T = max_tokens
        if out is None:  # (an allocation each: views of one cost 4 to 7 us more)
            if stream is None:
                ok, start = torch.empty(R, dtype=_I32, device=self.dev), torch.empty(R + 1, dtype=_I32, device=self.dev)
                row, pos, slot = (torch.empty(T, dtype=_I32, device=self.dev), torch.empty(T, dtype=_I32, device=self.dev),
                                  torch.empty(T, dtype=_I32, device=self.dev))
            else:
                ok, start, row, pos, slot = (_alloc(stream, (n,), _I32, self.dev) for n in (R, R + 1, T, T, T))
            out = {"ok": ok, "start": start, "row": row, "pos": pos, "slot": slot}
            at = ok.data_ptr(), start.data_ptr(), row.data_ptr(), pos.data_ptr(), slot.data_ptr()
        else:
            at = [_ints(k, out[k], self._idx, n)
                  for k, n in (("ok", R), ("start", R + 1), ("row", T), ("pos", T), ("slot", T))]
        _launch(self._lib.dartree_cache_plan, self._idx, stream, self._ref, t, width, ln, c, R, offset,
                w, sinks, T, *at, self._err)
        return out

    def fork(self, table, lens, src, dst, *, pending: int = 0, stream=None) -> torch.Tensor:
        """Rows dst become copies of rows src -> ok [n] int32
        (dartree_cache_fork_ex).  ``pending``: how many of the last tokens of
        lens are counted but not written yet (commit's ``extra``): the pages
        they go to are not shared."""
        t, width, ln, R = self._seqs(table, lens)
        n = src.numel()
        ok = _alloc(stream, (n,), _I32, self.dev)
        _launch(self._lib.dartree_cache_fork_ex, self._idx, stream, self._ref, t, width, ln, R,
                _ints("src", src, self._idx, n), _ints("dst", dst, self._idx, n), n, pending,
                ok.data_ptr())
        return ok

    def commit(self, table, lens, nodes, length, *, extra: int = 0, stream=None) -> None:
        """Moves the accepted nodes' tokens to the prefixes' ends and adds
        length[r] + extra to lens (dartree_cache_commit); nodes [R, max_len]
        and length [R] as :func:`accept` returns them.  The ``extra`` tokens are
        pending (see :meth:`fork`, :meth:`reserve`) until they are appended."""
        t, width, ln, R = self._seqs(table, lens)
        r, most = nodes.shape
        _launch(self._lib.dartree_cache_commit, self._idx, stream, self._ref, t, width, ln,
                _ints("nodes", nodes, self._idx, R * most), _ints("length", length, self._idx, R), R,
                most, extra, self._err)

    def release(self, table, lens, rows, keep, *, stream=None) -> None:
        """Rows keep their first keep[i] tokens; pages behind them go back
        (dartree_cache_release)."""
        t, width, ln, R = self._seqs(table, lens)
        n = rows.numel()
        _launch(self._lib.dartree_cache_release, self._idx, stream, self._ref, t, width, ln, R,
                _ints("rows", rows, self._idx, n), _ints("keep", keep, self._idx, n), n, self._err)

    def copy_pages(self, src, dst, *, stream=None) -> None:
        """Copies pages src[i] to dst[i] in all layers
        (dartree_cache_copy_pages)."""
        n = src.numel()
        _launch(self._lib.dartree_cache_copy_pages, self._idx, stream, self._ref,
                _ints("src", src, self._idx, n), _ints("dst", dst, self._idx, n), n, self._err)


def sample(logits: torch.Tensor, u: torch.Tensor, *, temperature: torch.Tensor | None = None,
           top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
           min_p: torch.Tensor | None = None, rows_per_req: int = 1, stream=None) -> dict:
    """Tokens drawn from logits [rows, V] (fp32 or bf16) with the random
    numbers u [rows] in [0, 1) (dartree_sample) -> {"token": int32 [rows],
    "prob": fp32 [rows]}.  Row i uses entry i // rows_per_req of temperature,
    top_p, min_p (fp32) and top_k (int32).  With rows_per_req = B + 1 the
    tokens are :func:`accept`'s pred."""
    if not logits.is_cuda or logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be an fp32 or bf16 CUDA tensor")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [rows, V], dense in V")
    rows, V = logits.shape
    if rows < 1 or V < 1 or rows_per_req < 1:
        raise ValueError("logits and rows_per_req must not be empty")
    idx, n = logits.get_device(), -(-rows // rows_per_req)
    T = None if temperature is None else _floats("temperature", temperature, idx, n)
    k = None if top_k is None else _ints("top_k", top_k, idx, n)
    p = None if top_p is None else _floats("top_p", top_p, idx, n)
    m = None if min_p is None else _floats("min_p", min_p, idx, n)
    up = _floats("u", u, idx, rows)
    token = _alloc(stream, (rows,), _I32, logits.device)
    prob = _alloc(stream, (rows,), torch.float32, logits.device)
    _launch(load().dartree_sample, idx, stream, logits.data_ptr(),
            1 if logits.dtype is torch.bfloat16 else 0,
            logits.stride(0) if rows > 1 else max(V, logits.stride(0)), V, rows, rows_per_req, T, k,
            p, m, up, token.data_ptr(), prob.data_ptr())
    return {"token": token, "prob": prob}


def _logit_rows(name: str, x: torch.Tensor, R: int, rows, idx: int) -> tuple:
    """(address, is bf16, request stride, row stride, rows) of logits [R, rows,
    V], dense in V."""
    if x.get_device() != idx or x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be an fp32 or bf16 tensor on cuda:{idx}")
    if x.dim() != 3 or x.shape[0] != R or x.shape[1] not in rows or x.shape[2] < 1:
        raise ValueError(f"{name} {tuple(x.shape)} does not match R={R}, rows={rows}")
    n, V = x.shape[1:]
    if V > 1 and x.stride(2) != 1:
        raise ValueError(f"{name} must be dense in V")
    per = x.stride(1) if n > 1 else max(V, x.stride(1))  # (a dimension of one has no stride)
    return x.data_ptr(), int(x.dtype is torch.bfloat16), x.stride(0) if R > 1 else 0, per, n


def verify(parent: torch.Tensor | None, token: torch.Tensor, n_out: torch.Tensor, logits: torch.Tensor,
           draft: torch.Tensor, u: torch.Tensor, *, max_len: int,
           temperature: torch.Tensor | None = None, top_k: torch.Tensor | None = None,
           top_p: torch.Tensor | None = None, min_p: torch.Tensor | None = None,
           draft_temperature: torch.Tensor | None = None, stream=None) -> dict:
    """Which drafted tokens the target accepts, and its own token behind them
    (dartree_verify) -> {"len" [R], "nodes" [R, max_len], "bonus" [R], "prob" [R]},
    the first three as :func:`accept` gives them.  parent (None: chains), token [R, B],
    n_out [R]; the target's logits [R, B+1, V] and the drafter's, from which the
    tokens were drawn, draft [R, B or B+1, V] (fp32 or bf16, dense in V; -inf where
    the drafter's own cuts left a token out); u [R, B+1] in [0, 1): u[:, i+1] tests
    node i, u[:, 0] draws the last token.  :func:`sample` draws a chain's tokens; a
    tree's siblings one after the other, those before at -inf."""
    if not isinstance(token, torch.Tensor) or token.dim() != 2 or not token.is_cuda:
        raise TypeError("token must be a CUDA tensor [R, B]")
    R, B = token.shape
    if R < 1 or B < 1 or max_len < 1:
        raise ValueError("token and max_len must not be empty")
    idx, dev = token.get_device(), token.device
    par = None if parent is None else _ints("parent", parent, idx, R * B)
    tok, n = _ints("token", token, idx, R * B), _ints("n_out", n_out, idx, R)
    t = _logit_rows("logits", logits, R, (B + 1,), idx)
    d = _logit_rows("draft", draft, R, (B, B + 1), idx)
    V = logits.shape[2]
    if draft.shape[2] != V:
        raise ValueError(f"logits have {V} tokens, draft {draft.shape[2]}")
    T = None if temperature is None else _floats("temperature", temperature, idx, R)
    k = None if top_k is None else _ints("top_k", top_k, idx, R)
    p = None if top_p is None else _floats("top_p", top_p, idx, R)
    m = None if min_p is None else _floats("min_p", min_p, idx, R)
    dt = None if draft_temperature is None else _floats("draft_temperature", draft_temperature, idx, R)
    up = _floats("u", u, idx, R * (B + 1))
    o = {"len": _alloc(stream, (R,), _I32, dev), "nodes": _alloc(stream, (R, max_len), _I32, dev),
         "bonus": _alloc(stream, (R,), _I32, dev), "prob": _alloc(stream, (R,), torch.float32, dev)}
    _launch(load().dartree_verify, idx, stream, par, tok, n, *t[:4], *d, V, R, B, T, k, p, m, dt, up, max_len,
            *[o[x].data_ptr() for x in ("len", "nodes", "bonus", "prob")])
    return o
