"""KiviCache: a thin Python handle over the C ABI of libkivi.so.

PyTorch provides the device memory (the arena and the I/O tensors) and the
CUDA stream; every computation runs in the library's kernels.  The methods
only check shapes, dtypes and devices and marshal pointers.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, asdict

import torch

from . import _abi


@dataclass(frozen=True)
class KiviConfig:
    bits: int
    group: int
    residual: int
    sinks: int
    h_q: int
    h_kv: int
    head_dim: int
    batch: int
    max_tokens: int = 0
    window: int = 0
    outlier_permille: int = 0
    rope_base: float = 0.0

    def c(self) -> _abi.KiviParams:
        return _abi.KiviParams(self.bits, self.group, self.residual, self.sinks, self.h_q, self.h_kv,
                               self.head_dim, self.batch, self.max_tokens, self.window, self.outlier_permille, 0,
                               self.rope_base)

    @staticmethod
    def from_workload(w) -> "KiviConfig":
        return KiviConfig(bits=w.bits, group=w.group, residual=w.residual, sinks=w.sinks, h_q=w.h_q,
                          h_kv=w.h_kv, head_dim=w.head_dim, batch=w.batch, max_tokens=w.max_tokens,
                          window=w.window, outlier_permille=getattr(w, "outlier_permille", 0),
                          rope_base=getattr(w, "rope_base", 0.0))


@dataclass(frozen=True)
class RopeConfig:
    """Rotary positions with one to four axes: sections[x] pairs of channels
    turn by the position on axis x (time, height, width, ...), pair i of all
    by position * base^(-i / pairs); channels past the pairs stay.  order:
    "blocks" (axis 0's pairs first) or "interleaved" (pairs dealt in turn);
    pairing: "halves" (channels i, i + pairs) or "adjacent" (2i, 2i + 1)."""
    sections: tuple
    base: float = 10000.0
    order: str = "blocks"
    pairing: str = "halves"

    def __post_init__(self):
        object.__setattr__(self, "sections", tuple(self.sections))

    def c(self) -> _abi.KiviRopeParams:
        made = self.__dict__.get("_made")
        if made is None:
            made = self._make()
            object.__setattr__(self, "_made", made)
        return made

    def _make(self) -> _abi.KiviRopeParams:
        orders = {"blocks": _abi.KIVI_ROPE_BLOCKS, "interleaved": _abi.KIVI_ROPE_INTERLEAVED}
        pairings = {"halves": _abi.KIVI_ROPE_HALVES, "adjacent": _abi.KIVI_ROPE_ADJACENT}
        if self.order not in orders or self.pairing not in pairings:
            raise ValueError(f"order must be one of {sorted(orders)} and pairing one of {sorted(pairings)}")
        n = len(self.sections)
        if not 1 <= n <= _abi.KIVI_ROPE_AXES:
            raise ValueError(f"1 to {_abi.KIVI_ROPE_AXES} sections, got {n}")
        sections = (ctypes.c_int32 * _abi.KIVI_ROPE_AXES)(*[int(x) for x in self.sections])
        return _abi.KiviRopeParams(n, sections, orders[self.order], pairings[self.pairing], 0, self.base)


class DiffWeights:
    """The learned weights of differential attention (include/kivi.h):
    lambdas [4, d] float32 (λq1, λk1, λq2, λk2), the layer's lambda_init, and
    the norm's weight [2 d] float32 with its eps, or None for no norm.  All on
    the cache's device; each launch reads the tensors as they are then, changed
    in place or with other storage (tensor.data = ...)."""

    def __init__(self, lambdas: torch.Tensor, lambda_init: float, norm_weight: torch.Tensor | None = None,
                 eps: float = 1e-5):
        self._lambdas, self._norm_weight, self._lambda_init, self._eps = lambdas, norm_weight, lambda_init, eps
        self._check()

    def _check(self):
        """Refuses tensors that a launch cannot read."""
        lambdas, norm_weight = self._lambdas, self._norm_weight
        for t, what in ((lambdas, "lambdas"), (norm_weight, "norm_weight")):
            if t is None and what == "norm_weight":
                continue
            if t.dtype != torch.float32 or t.device.type != "cuda" or not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous float32 CUDA tensor")
        if lambdas.dim() != 2 or lambdas.shape[0] != 4:
            raise ValueError(f"lambdas must have shape (4, d), got {tuple(lambdas.shape)}")
        if norm_weight is not None and tuple(norm_weight.shape) != (2 * lambdas.shape[1],):
            raise ValueError(f"norm_weight must have shape {(2 * lambdas.shape[1],)}, got {tuple(norm_weight.shape)}")

    def _for(self, device: torch.device, d: int, flags: int = 0) -> _abi.KiviDiffParams:
        """What a launch of a cache on `device` with this head_dim takes.  The
        tensors are looked at in each call: their storage may have been exchanged."""
        lam, norm = self._lambdas, self._norm_weight
        f32 = torch.float32
        if (lam.device != device or lam.shape != (4, d) or lam.dtype is not f32 or not lam.is_contiguous() or
                (norm is not None and (norm.device != device or norm.shape != (2 * d,) or norm.dtype is not f32 or
                                       not norm.is_contiguous()))):
            self._check()
            raise ValueError(f"the weights must be on {device} and of head_dim {d}")
        return _abi.KiviDiffParams(lam.data_ptr(), None if norm is None else norm.data_ptr(), self._lambda_init,
                                   self._eps, flags)

    # read-only
    lambdas = property(lambda self: self._lambdas)
    norm_weight = property(lambda self: self._norm_weight)
    lambda_init = property(lambda self: self._lambda_init)
    eps = property(lambda self: self._eps)


_QKV_DTYPES = {torch.float16: _abi.KIVI_F16, torch.bfloat16: _abi.KIVI_BF16, torch.float32: _abi.KIVI_F32}


def cache_bytes(cfg: KiviConfig) -> int:
    """Arena bytes for these parameters (0 if they are invalid)."""
    p = cfg.c()
    return int(_abi.lib().kivi_cache_bytes(ctypes.byref(p)))


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


class KiviCache:
    """A quantized KV cache of one attention layer on one GPU."""

    def __init__(self, cfg: KiviConfig, device="cuda", stream=None, arena: torch.Tensor | None = None,
                 restore_tokens=None):
        """A new cache (the arena is zeroed), or with restore_tokens (one
        count per sequence) a handle over an `arena` that already holds a
        cache of this config (kivi_cache_restore)."""
        self.cfg = cfg
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("KiviCache lives on a CUDA device")
        L = _abi.lib()
        p = cfg.c()
        nbytes = int(L.kivi_cache_bytes(ctypes.byref(p)))
        if nbytes == 0:
            raise _abi.KiviError(_abi.KIVI_EINVAL, f"kivi_cache_bytes({cfg})")
        if arena is None:
            arena = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.arena = arena
        self._dev = arena.device
        self._lib = L
        self._scratch = None   # prefill scratch, grown on demand
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            if restore_tokens is None:
                _abi.check(L.kivi_cache_create(ctypes.byref(p), ctypes.c_void_p(arena.data_ptr()),
                                               arena.numel(), ctypes.c_void_p(_stream_ptr(stream)),
                                               ctypes.byref(h)), "kivi_cache_create")
            else:
                toks = (ctypes.c_int64 * cfg.batch)(*[int(t) for t in restore_tokens])
                _abi.check(L.kivi_cache_restore(ctypes.byref(p), ctypes.c_void_p(arena.data_ptr()),
                                                arena.numel(), toks, ctypes.c_void_p(_stream_ptr(stream)),
                                                ctypes.byref(h)), "kivi_cache_restore")
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            try:
                _abi.lib().kivi_cache_destroy(h)
            except Exception:
                pass
            self._h = None

    # ------------------------------------------------------------------ API
    def _check_io(self, t: torch.Tensor, shape, what: str):
        if t.dtype != torch.float16:
            raise TypeError(f"{what} must be float16, got {t.dtype}")
        if t.device != self.arena.device:
            raise ValueError(f"{what} must be on {self.arena.device}, got {t.device}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
        """k_new, v_new: [B, H_kv, n, d] float16 on the cache's device."""
        c = self.cfg
        n = k_new.shape[2] if k_new.dim() == 4 else -1
        shape = (c.batch, c.h_kv, n, c.head_dim)
        self._check_io(k_new, shape, "k_new")
        self._check_io(v_new, shape, "v_new")
        _abi.check(_abi.lib().kivi_append(self._h, ctypes.c_void_p(k_new.data_ptr()),
                                          ctypes.c_void_p(v_new.data_ptr()), n,
                                          ctypes.c_void_p(_stream_ptr(stream))), "kivi_append")

    def append_ragged(self, k_new: torch.Tensor, v_new: torch.Tensor, n_tokens, stream=None) -> None:
        """k_new, v_new: [B, H_kv, n_max, d] float16; sequence b takes the
        first n_tokens[b] tokens of its rows (kivi_append_ragged)."""
        c = self.cfg
        n_max = k_new.shape[2] if k_new.dim() == 4 else -1
        shape = (c.batch, c.h_kv, n_max, c.head_dim)
        self._check_io(k_new, shape, "k_new")
        self._check_io(v_new, shape, "v_new")
        counts = (ctypes.c_int64 * c.batch)(*[int(n) for n in n_tokens])
        _abi.check(_abi.lib().kivi_append_ragged(self._h, ctypes.c_void_p(k_new.data_ptr()),
                                                 ctypes.c_void_p(v_new.data_ptr()), counts, n_max,
                                                 ctypes.c_void_p(_stream_ptr(stream))), "kivi_append_ragged")

    def tokens_per_sequence(self) -> list:
        out = (ctypes.c_int64 * self.cfg.batch)()
        _abi.check(_abi.lib().kivi_cache_tokens(self._h, out), "kivi_cache_tokens")
        return list(out)

    def decode(self, q: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """q: [B, H_q, d] float16 -> out [B, H_q, d] float16."""
        c = self.cfg
        shape = (c.batch, c.h_q, c.head_dim)
        self._check_io(q, shape, "q")
        if out is None:
            out = torch.empty(shape, dtype=torch.float16, device=self.arena.device)
        self._check_io(out, shape, "out")
        _abi.check(_abi.lib().kivi_decode_attn(self._h, ctypes.c_void_p(q.data_ptr()),
                                               ctypes.c_void_p(out.data_ptr()),
                                               ctypes.c_void_p(_stream_ptr(stream))), "kivi_decode_attn")
        return out

    def append_decode(self, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """One decode step: append k_new, v_new ([B, H_kv, 1, d] float16) and
        return the attention of q ([B, H_q, d] float16) over the cache
        including them (kivi_append_decode_attn)."""
        c = self.cfg
        kv_shape = (c.batch, c.h_kv, 1, c.head_dim)
        self._check_io(k_new, kv_shape, "k_new")
        self._check_io(v_new, kv_shape, "v_new")
        shape = (c.batch, c.h_q, c.head_dim)
        self._check_io(q, shape, "q")
        if out is None:
            out = torch.empty(shape, dtype=torch.float16, device=self.arena.device)
        self._check_io(out, shape, "out")
        _abi.check(_abi.lib().kivi_append_decode_attn(
            self._h, ctypes.c_void_p(k_new.data_ptr()), ctypes.c_void_p(v_new.data_ptr()),
            ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(out.data_ptr()),
            ctypes.c_void_p(_stream_ptr(stream))), "kivi_append_decode_attn")
        return out

    def append_decode_host(self, k_host: torch.Tensor, v_host: torch.Tensor, q_host: torch.Tensor,
                           out_host: torch.Tensor, stream=None) -> torch.Tensor:
        """append_decode with host-resident tensors, queued on `stream`: pinned
        tensors are read and written by the step over the host mapping;
        pageable tensors are staged through the arena with copies."""
        c = self.cfg
        shapes = ((k_host, (c.batch, c.h_kv, 1, c.head_dim), "k_host"), (v_host, (c.batch, c.h_kv, 1, c.head_dim), "v_host"),
                  (q_host, (c.batch, c.h_q, c.head_dim), "q_host"), (out_host, (c.batch, c.h_q, c.head_dim), "out_host"))
        for t, shape, what in shapes:
            if t.device.type != "cpu" or t.dtype != torch.float16 or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous float16 CPU tensor of shape {shape}")
        _abi.check(_abi.lib().kivi_append_decode_attn_host(
            self._h, ctypes.c_void_p(k_host.data_ptr()), ctypes.c_void_p(v_host.data_ptr()),
            ctypes.c_void_p(q_host.data_ptr()), ctypes.c_void_p(out_host.data_ptr()),
            ctypes.c_void_p(_stream_ptr(stream))), "kivi_append_decode_attn_host")
        return out_host

    def decode_host(self, q_host: torch.Tensor, out_host: torch.Tensor, stream=None) -> torch.Tensor:
        """Host-resident q and out, queued on `stream`: pinned tensors are read
        and written by the decode over the host mapping; pageable tensors are
        staged with copies."""
        c = self.cfg
        shape = (c.batch, c.h_q, c.head_dim)
        for t, what in ((q_host, "q_host"), (out_host, "out_host")):
            if t.device.type != "cpu" or t.dtype != torch.float16 or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous float16 CPU tensor of shape {shape}")
        _abi.check(_abi.lib().kivi_decode_attn_host(self._h, ctypes.c_void_p(q_host.data_ptr()),
                                                    ctypes.c_void_p(out_host.data_ptr()),
                                                    ctypes.c_void_p(_stream_ptr(stream))),
                   "kivi_decode_attn_host")
        return out_host

    def prefill(self, q: torch.Tensor, out: torch.Tensor | None = None, scratch: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        """Causal attention of the M newest tokens (append the chunk first):
        q [B, M, H_q, d] float16 -> out [B, M, H_q, d] float16
        (kivi_prefill_attn).  `scratch` is a uint8 device tensor of at least
        prefill_scratch_bytes(M) bytes; by default the cache keeps one and
        grows it as needed."""
        c = self.cfg
        m = q.shape[1] if q.dim() == 4 else -1
        shape = (c.batch, m, c.h_q, c.head_dim)
        self._check_io(q, shape, "q")
        if out is None:
            out = torch.empty(shape, dtype=torch.float16, device=self.arena.device)
        self._check_io(out, shape, "out")
        need = self.prefill_scratch_bytes(m)
        if need == 0:
            raise _abi.KiviError(_abi.KIVI_EINVAL, "kivi_prefill_scratch_bytes")
        if scratch is None:
            if self._scratch is None or self._scratch.numel() < need:
                self._scratch = torch.empty(need, dtype=torch.uint8, device=self.arena.device)
            scratch = self._scratch
        _abi.check(_abi.lib().kivi_prefill_attn(self._h, ctypes.c_void_p(q.data_ptr()),
                                                ctypes.c_void_p(out.data_ptr()), m,
                                                ctypes.c_void_p(scratch.data_ptr()), scratch.numel(),
                                                ctypes.c_void_p(_stream_ptr(stream))), "kivi_prefill_attn")
        return out

    def prefill_ragged(self, q: torch.Tensor, n_queries, out: torch.Tensor | None = None,
                       scratch: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """q [B, m_max, H_q, d] float16; sequence b's n_queries[b] newest
        tokens attend (kivi_prefill_attn_ragged).  Rows past a sequence's
        count are left as they are in `out` (zeros when out is None)."""
        c = self.cfg
        m = q.shape[1] if q.dim() == 4 else -1
        shape = (c.batch, m, c.h_q, c.head_dim)
        self._check_io(q, shape, "q")
        if out is None:
            out = torch.zeros(shape, dtype=torch.float16, device=self.arena.device)
        self._check_io(out, shape, "out")
        need = self.prefill_scratch_bytes(m)
        if need == 0:
            raise _abi.KiviError(_abi.KIVI_EINVAL, "kivi_prefill_scratch_bytes")
        if scratch is None:
            if self._scratch is None or self._scratch.numel() < need:
                self._scratch = torch.empty(need, dtype=torch.uint8, device=self.arena.device)
            scratch = self._scratch
        counts = (ctypes.c_int64 * c.batch)(*[int(n) for n in n_queries])
        _abi.check(_abi.lib().kivi_prefill_attn_ragged(self._h, ctypes.c_void_p(q.data_ptr()),
                                                       ctypes.c_void_p(out.data_ptr()), counts, m,
                                                       ctypes.c_void_p(scratch.data_ptr()), scratch.numel(),
                                                       ctypes.c_void_p(_stream_ptr(stream))),
                   "kivi_prefill_attn_ragged")
        return out

    # The methods below are called once or more per layer and step, so their
    # checks are made cheap: shapes, device and function pointers are kept.
    def _on(self, t: torch.Tensor, shape: tuple, what: str):
        if t.dtype is not torch.float16 or t.shape != shape or t.device != self._dev or not t.is_contiguous():
            self._check_io(t, shape, what)   # says what is wrong

    def _here(self):
        """Makes the cache's device current for a call; the device to go back
        to, or None where it was."""
        now = torch.cuda.current_device()
        if now == self._dev.index:
            return None
        torch.cuda.set_device(self._dev)
        return now

    def _stream_here(self, stream) -> int:
        """The given stream, or the current one of the cache's device."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._dev.index)
        return stream.cuda_stream

    def _call(self, name: str, *args):
        back = self._here()
        try:
            status = getattr(self._lib, name)(self._h, *args)
        finally:
            if back is not None:
                torch.cuda.set_device(back)
        if status:
            raise _abi.KiviError(status, name)

    def rope_qkv(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, rope: RopeConfig,
                 n_tokens=None, out=None, stream=None):
        """Turns new tokens' q and k by their positions and lays q, k, v out
        for this cache (kivi_rope_qkv).

        q [B, n, H_q, d], k and v [B, n, H_kv, d]: float16, bfloat16 or
        float32, all alike; strided views (parts of one projection's output)
        whose heads follow one another.  positions [axes, B, n] int64.
        n_tokens: a count per sequence; later rows are neither read nor
        written (zeros when out is None).  Returns float16 (q [B, n, H_q, d],
        k [B, H_kv, n, d], v [B, H_kv, n, d]): prefill's q (q[:, 0] is
        decode's) and append's k and v."""
        c, dev = self.cfg, self._dev
        B, hq, hk, d = c.batch, c.h_q, c.h_kv, c.head_dim
        n = q.shape[1] if q.dim() == 4 else -1
        kind, kv_in, kv_shape, q_shape = q.dtype, (B, n, hk, d), (B, hk, n, d), (B, n, hq, d)
        if (kind not in _QKV_DTYPES or k.dtype is not kind or v.dtype is not kind or q.shape != q_shape or
                k.shape != kv_in or v.shape != kv_in or q.device != dev or k.device != dev or v.device != dev or
                positions.dtype is not torch.int64 or positions.shape != (len(rope.sections), B, n) or
                positions.device != dev or not positions.is_contiguous()):
            self._rope_refuse(q, k, v, positions, rope, n)
        sq, sk, sv = q.stride(), k.stride(), v.stride()
        if (sq[3] != 1 or sk[3] != 1 or sv[3] != 1 or (hq > 1 and sq[2] != d) or
                (hk > 1 and (sk[2] != d or sv[2] != d))):
            raise ValueError(f"the heads must follow one another (strides {sq}, {sk}, {sv})")
        if out is None:
            new = torch.empty if n_tokens is None else torch.zeros
            out = tuple(new(s, dtype=torch.float16, device=dev) for s in (q_shape, kv_shape, kv_shape))
            if stream is not None:
                self._made_here(out, stream)
        q_out, k_out, v_out = out
        self._on(q_out, q_shape, "out[0]")
        self._on(k_out, kv_shape, "out[1]")
        self._on(v_out, kv_shape, "out[2]")
        counts = None
        if n_tokens is not None:
            if len(n_tokens) != B:
                raise ValueError(f"n_tokens must have {B} entries")
            counts = (ctypes.c_int64 * B)(*[int(x) for x in n_tokens])
        # a stride of a dimension of one entry means nothing
        b0, t0 = int(B > 1), int(n > 1)
        io = _abi.KiviQkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), _QKV_DTYPES[kind], 0, sq[0] * b0, sq[1] * t0,
                          sk[0] * b0, sk[1] * t0, sv[0] * b0, sv[1] * t0)
        self._call("kivi_rope_qkv", rope.c(), io, positions.data_ptr(), counts, n, q_out.data_ptr(),
                   k_out.data_ptr(), v_out.data_ptr(), self._stream_here(stream))
        return q_out, k_out, v_out

    def _rope_refuse(self, q, k, v, positions, rope, n):
        """Says what is wrong with rope_qkv's inputs."""
        c, dev = self.cfg, self._dev
        if q.dtype not in _QKV_DTYPES:
            raise TypeError(f"q must be float16, bfloat16 or float32, got {q.dtype}")
        for t, heads, what in ((q, c.h_q, "q"), (k, c.h_kv, "k"), (v, c.h_kv, "v")):
            if t.dtype is not q.dtype:
                raise TypeError(f"{what} must be {q.dtype} as q is, got {t.dtype}")
            if t.device != dev:
                raise ValueError(f"{what} must be on {dev}, got {t.device}")
            if t.shape != (c.batch, n, heads, c.head_dim):
                raise ValueError(f"{what} must have shape {(c.batch, n, heads, c.head_dim)}, got {tuple(t.shape)}")
        if positions.dtype is not torch.int64 or positions.device != dev:
            raise ValueError(f"positions must be int64 on {dev}")
        raise ValueError(f"positions must be contiguous of shape {(len(rope.sections), c.batch, n)}, got "
                         f"{tuple(positions.shape)}")

    def reorder(self, src, stream=None) -> None:
        """In place: sequence b becomes what sequence src[b] was (src[b] = b
        keeps it, -1 frees it); forks, chains and cycles in any mix
        (kivi_cache_reorder)."""
        if len(src) != self.cfg.batch:
            raise ValueError(f"src must have {self.cfg.batch} entries, got {len(src)}")
        m = (ctypes.c_int32 * self.cfg.batch)(*[int(x) for x in src])
        self._call("kivi_cache_reorder", m, self._stream_here(stream))

    def free(self, sequences, stream=None) -> None:
        """Empties these sequences (their token counts become 0)."""
        gone = {int(b) for b in sequences}
        if not all(0 <= b < self.cfg.batch for b in gone):
            raise ValueError(f"sequences must lie in [0, {self.cfg.batch})")
        self.reorder([-1 if b in gone else b for b in range(self.cfg.batch)], stream)

    def compact(self, stream=None) -> list:
        """Moves the sequences that hold tokens to the front, in their order,
        and empties the rest; returns where each of them was."""
        live = [b for b, t in enumerate(self.tokens_per_sequence()) if t > 0]
        self.reorder(live + [-1] * (self.cfg.batch - len(live)), stream)
        return live

    def copy_from(self, other: "KiviCache", dst, src, stream=None) -> None:
        """Sequence dst[i] of this cache becomes sequence src[i] of `other`,
        a cache of the same parameters but for h_q, batch and max_tokens
        (kivi_cache_copy)."""
        if len(dst) != len(src):
            raise ValueError(f"dst and src must have as many entries, got {len(dst)} and {len(src)}")
        if other._dev != self._dev:
            raise ValueError(f"the caches must be on one device, got {self._dev} and {other._dev}")
        n = len(dst)
        to, fr = ((ctypes.c_int32 * n)(*[int(x) for x in y]) for y in (dst, src))
        self._call("kivi_cache_copy", other._h, to, fr, n, self._stream_here(stream))

    def _made_here(self, tensors, stream):
        """New tensors that another stream is about to use: their making
        (zeros) comes first, and their memory stays until it is through."""
        stream.wait_stream(torch.cuda.current_stream(self._dev))
        for t in tensors:
            t.record_stream(stream)

    def _diff_out(self, out, shape: tuple, stream, new=torch.empty) -> torch.Tensor:
        """The output tensor of a differential attention."""
        if out is None:
            out = new(shape, dtype=torch.float16, device=self._dev)
            if stream is not None:
                self._made_here((out,), stream)
            return out
        self._on(out, shape, "out")
        return out

    def diff_decode(self, q: torch.Tensor, weights: DiffWeights, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
        """Differential attention of one token (kivi_diff_decode_attn):
        q [B, H_q, d] float16 -> out [B, H_q / 2, 2 d] float16."""
        c = self.cfg
        self._on(q, (c.batch, c.h_q, c.head_dim), "q")
        params = weights._for(self._dev, c.head_dim)
        out = self._diff_out(out, (c.batch, c.h_q // 2, 2 * c.head_dim), stream)
        self._call("kivi_diff_decode_attn", params, q.data_ptr(), out.data_ptr(), self._stream_here(stream))
        return out

    def append_diff_decode(self, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor, weights: DiffWeights,
                           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """One step: append k_new, v_new ([B, H_kv, 1, d] float16) and return
        the differential attention of q over the cache including them
        (kivi_append_diff_decode_attn)."""
        c = self.cfg
        kv = (c.batch, c.h_kv, 1, c.head_dim)
        self._on(k_new, kv, "k_new")
        self._on(v_new, kv, "v_new")
        self._on(q, (c.batch, c.h_q, c.head_dim), "q")
        params = weights._for(self._dev, c.head_dim)
        out = self._diff_out(out, (c.batch, c.h_q // 2, 2 * c.head_dim), stream)
        self._call("kivi_append_diff_decode_attn", params, k_new.data_ptr(), v_new.data_ptr(), q.data_ptr(),
                   out.data_ptr(), self._stream_here(stream))
        return out

    def diff_prefill(self, q: torch.Tensor, weights: DiffWeights, out: torch.Tensor | None = None,
                     scratch: torch.Tensor | None = None, stream=None, exact: bool = False) -> torch.Tensor:
        """Causal differential attention of the M newest tokens (append the
        chunk first): q [B, M, H_q, d] float16 -> out [B, M, H_q / 2, 2 d]
        float16 (kivi_diff_prefill_attn).  scratch: a uint8 device tensor of
        diff_prefill_scratch_bytes(M) bytes; by default each call takes one
        of its own, so captured graphs and streams share none.  exact: keys
        and values of large chunks are not rounded to fp16 either, at up to ten
        times the time (KIVI_DIFF_EXACT_CODES)."""
        return self._diff_prefill(q, None, weights, out, scratch, stream, exact)

    def diff_prefill_ragged(self, q: torch.Tensor, n_queries, weights: DiffWeights, out: torch.Tensor | None = None,
                            scratch: torch.Tensor | None = None, stream=None, exact: bool = False) -> torch.Tensor:
        """diff_prefill of sequence b's n_queries[b] newest tokens; rows past a
        sequence's count are left as they are in `out` (zeros when out is
        None)."""
        return self._diff_prefill(q, n_queries, weights, out, scratch, stream, exact)

    def _diff_prefill(self, q, n_queries, weights, out, scratch, stream, exact):
        c = self.cfg
        m = q.shape[1] if q.dim() == 4 else -1
        self._on(q, (c.batch, m, c.h_q, c.head_dim), "q")
        counts = None
        if n_queries is not None:
            if len(n_queries) != c.batch:
                raise ValueError(f"n_queries must have {c.batch} entries")
            counts = (ctypes.c_int64 * c.batch)(*[int(x) for x in n_queries])
        params = weights._for(self._dev, c.head_dim, _abi.KIVI_DIFF_EXACT_CODES if exact else 0)
        out = self._diff_out(out, (c.batch, m, c.h_q // 2, 2 * c.head_dim), stream,
                             torch.empty if counts is None else torch.zeros)
        need = self.diff_prefill_scratch_bytes(m)
        if need == 0:
            raise _abi.KiviError(_abi.KIVI_EINVAL, "kivi_diff_prefill_scratch_bytes")
        if scratch is None:
            scratch = torch.empty(need, dtype=torch.uint8, device=self._dev)
            if stream is not None:
                self._made_here((scratch,), stream)
        elif scratch.dtype is not torch.uint8 or scratch.device != self._dev or not scratch.is_contiguous():
            raise ValueError(f"scratch must be a contiguous uint8 tensor on {self._dev}")
        self._call("kivi_diff_prefill_attn", params, q.data_ptr(), out.data_ptr(), counts, m,
                   scratch.data_ptr(), scratch.numel(), self._stream_here(stream))
        return out

    def diff_prefill_scratch_bytes(self, n_queries: int) -> int:
        return int(_abi.lib().kivi_diff_prefill_scratch_bytes(self._h, n_queries))

    def prefill_scratch_bytes(self, n_queries: int) -> int:
        return int(_abi.lib().kivi_prefill_scratch_bytes(self._h, n_queries))

    def prefill_bytes(self, n_queries: int) -> int:
        return int(_abi.lib().kivi_prefill_bytes(self._h, n_queries))

    def read_error(self, stream=None) -> int:
        """Reads and clears the device error word (synchronises the stream)."""
        flags = ctypes.c_uint32(0)
        _abi.check(_abi.lib().kivi_read_error(self._h, ctypes.byref(flags), ctypes.c_void_p(_stream_ptr(stream))),
                   "kivi_read_error")
        return int(flags.value)

    def set_num_splits(self, n: int) -> None:
        _abi.check(_abi.lib().kivi_set_num_splits(self._h, n), "kivi_set_num_splits")

    def layout(self) -> dict:
        L = _abi.KiviLayout()
        _abi.check(_abi.lib().kivi_cache_layout(self._h, ctypes.byref(L)), "kivi_cache_layout")
        return {n: getattr(L, n) for n, _ in _abi.KiviLayout._fields_}

    def decode_bytes(self) -> int:
        return int(_abi.lib().kivi_decode_bytes(self._h))

    @property
    def tokens(self) -> int:
        return self.layout()["tokens"]

    def cache_region(self) -> torch.Tensor:
        """A view of the cache bytes (without the workspace)."""
        return self.arena[: self.layout()["cache_bytes"]]

    def config_dict(self) -> dict:
        return asdict(self.cfg)
