"""Python binding of the iS-KV CUDA library (``libiskv.so``, C ABI in
``include/iskv.h``).

Argument marshalling only: tensors become raw pointers, the current CUDA
stream becomes the ``stream`` argument, status codes become exceptions.
Every step of the method runs in the library's kernels; there is no CPU or
PyTorch fallback, and importing this package fails loudly when the compiled
library is missing (build it with ``python online_rank_kv_b200/build.py``).
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

__all__ = ["Config", "Cache", "IskvError", "DecodeOperands", "QuantFormat", "quantize_rows",
           "lib_path", "LIB", "F32", "BF16", "WHICH_K", "WHICH_V", "ALL_LAYERS", "FOLD_DEFER_SYNC",
           "EXPORTED", "PAGE", "CODE_INT8", "CODE_E4M3", "PagePlan", "page_plan", "Q8Pages"]

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "libiskv.so")


if not os.path.exists(lib_path()):
    raise ImportError(
        f"{lib_path()} is missing: build the CUDA library first "
        "(python online_rank_kv_b200/build.py)")

LIB = ctypes.CDLL(lib_path())

OK = 0
F32, BF16 = 0, 1
WHICH_K, WHICH_V = 0, 1
ALL_LAYERS = -1
FOLD_DEFER_SYNC = 1
PAGE = 64
CODE_INT8, CODE_E4M3 = 0, 1

_ERRORS = {-1: "INVALID_ARG", -2: "CAPACITY", -3: "STATE", -4: "CUDA", -5: "NOCONVERGE",
           -6: "NOMEM", -7: "UNSUPPORTED", -8: "DEVICE_TIMEOUT", -9: "RANGE"}


class IskvError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        self.name = _ERRORS.get(code, str(code))
        msg = LIB.iskv_strerror(code).decode()
        super().__init__(f"{where}: ISKV_ERR_{self.name} ({msg})")


class QuantFormat(ctypes.Structure):
    """Mirror of ``iskv_quant_format``: latent-channel code groups."""
    _fields_ = [("groups", ctypes.c_int32), ("channels", ctypes.c_int32 * 4),
                ("bits", ctypes.c_int32 * 4)]

    @classmethod
    def of(cls, groups):
        """From a list of (channels, bits) pairs, first latent channel first."""
        q = cls()
        q.groups = len(groups)
        for i, (n, b) in enumerate(groups):
            q.channels[i] = int(n)
            q.bits[i] = int(b)
        return q


class _Cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "layers", "kv_heads", "q_heads", "head_dim", "rank_k", "rank_v", "window",
        "block", "max_tokens", "kv_dtype", "coef_dtype", "use_rope")] + [
        ("rope_theta", ctypes.c_double)] + [(n, ctypes.c_int32) for n in (
            "sync", "max_deferred", "jacobi_max_sweeps", "ring_extra", "protect",
            "coef_quant")] + [("quant_k", QuantFormat), ("quant_v", QuantFormat)] + [
        ("joint", ctypes.c_int32)]


class DecodeOperands(ctypes.Structure):
    """Mirror of ``iskv_decode_operands`` (allocation-free decode)."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "kv_heads", "q_heads", "head_dim", "rank_k", "rank_v", "kv_dtype",
        "coef_dtype")] + [(n, ctypes.c_int64) for n in ("T", "n_c", "coef_rows", "ring_rows")] + [
        (n, ctypes.c_void_p) for n in ("coef_k", "basis_k", "coef_v", "basis_v", "ring_k",
                                       "ring_v", "rope")]


class _PlanArgs(ctypes.Structure):
    """Mirror of ``iskv_page_plan_args``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "width", "pages", "tokens")] + [
        (n, ctypes.c_void_p) for n in ("lens", "add", "table", "free_pages", "n_free", "lens_out", "cu",
                                       "slots", "n_free_out", "status")]


class _Q8Pages(ctypes.Structure):
    """Mirror of ``iskv_q8_pages``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("pages", "kv_heads", "head_dim", "page", "code")] + [
        (n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]


class _Q8Attention(ctypes.Structure):
    """Mirror of ``iskv_q8_attention_args``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "width", "q_heads", "dtype", "max_new", "window")] + [
        (n, ctypes.c_float) for n in ("scale", "cap")] + [
        (n, ctypes.c_int64) for n in ("tokens", "q_stride")] + [
        (n, ctypes.c_void_p) for n in ("q", "out", "table", "lens", "cu", "prefix", "slopes", "workspace")] + [
        ("workspace_bytes", ctypes.c_int64), ("status", ctypes.c_void_p)]


_vp, _i, _i64p = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_int64)
_SIGS = {
    "iskv_config_default": ([ctypes.POINTER(_Cfg)], _i),
    "iskv_create": ([ctypes.POINTER(_Cfg), _vp, ctypes.POINTER(_vp)], _i),
    "iskv_destroy": ([_vp], _i),
    "iskv_append": ([_vp, _i, _vp, _vp, _i, _vp, ctypes.POINTER(_i)], _i),
    "iskv_compress_block": ([_vp, _i, _i, _vp], _i),
    "iskv_sync": ([_vp, _i, _vp], _i),
    "iskv_decode_attention": ([_vp, _i, _vp, _vp, _vp], _i),
    "iskv_reconstruct": ([_vp, _i, _i, _vp, _vp], _i),
    "iskv_get_factors": ([_vp, _i, _i, _vp, _vp, _vp, _vp], _i),
    "iskv_get_counts": ([_vp, _i, _i64p, _i64p], _i),
    "iskv_kv_bytes": ([_vp, _i64p, _i64p], _i),
    "iskv_decode_kernel": ([_vp, _i, ctypes.POINTER(_i)], _i),
    "iskv_compress_block_async": ([_vp, _i, _i, _vp, _vp], _i),
    "iskv_status": ([_vp], _i),
    "iskv_strerror": ([_i], ctypes.c_char_p),
    "iskv_decode_attention_noalloc": ([ctypes.POINTER(DecodeOperands), _vp, _vp, _vp], _i),
    "iskv_quantize_rows": ([ctypes.POINTER(QuantFormat), _i, _vp, ctypes.c_int64, _vp, _vp, _vp], _i),
    "iskv_quant_words": ([ctypes.POINTER(QuantFormat)], _i),
    "iskv_page_plan": ([ctypes.POINTER(_PlanArgs), _vp], _i),
    "iskv_q8_append": ([ctypes.POINTER(_Q8Pages), _vp, _vp, _i, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                        _vp, _vp, _vp], _i),
    "iskv_q8_attention": ([ctypes.POINTER(_Q8Pages), ctypes.POINTER(_Q8Attention), _vp], _i),
    "iskv_q8_workspace": ([ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32],
                          ctypes.c_int64),
}
for _name, (_args, _ret) in _SIGS.items():
    _fn = getattr(LIB, _name)
    _fn.argtypes = _args
    _fn.restype = _ret
EXPORTED = tuple(_SIGS)


def _check(code: int, where: str) -> None:
    if code != OK:
        raise IskvError(code, where)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t: torch.Tensor) -> ctypes.c_void_p:
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


_TORCH_DT = {F32: torch.float32, BF16: torch.bfloat16}


@dataclass
class Config:
    """Mirror of ``iskv_config``; defaults are the one-layer Qwen3-8B-shaped cache."""
    batch: int = 1
    layers: int = 1
    kv_heads: int = 8
    q_heads: int = 32
    head_dim: int = 128
    rank_k: int = 32
    rank_v: int = 64
    window: int = 1024
    block: int = 64
    max_tokens: int = 16384
    kv_dtype: int = BF16
    coef_dtype: int = F32
    use_rope: int = 1
    rope_theta: float = 1e6
    sync: int = 1
    max_deferred: int = 0
    jacobi_max_sweeps: int = 0
    ring_extra: int = 0
    protect: int = 0
    coef_quant: int = 0
    quant_k: tuple = ()        # ((channels, bits), ...) of the K factor's code groups
    quant_v: tuple = ()
    joint: int = 0             # 1: one factor per sequence over all KV heads (D = kv_heads*128)

    def _c(self) -> _Cfg:
        c = _Cfg()
        for f in _Cfg._fields_:
            if f[0] in ("quant_k", "quant_v"):
                groups = getattr(self, f[0])
                if groups:
                    setattr(c, f[0], QuantFormat.of(groups))
                continue
            setattr(c, f[0], getattr(self, f[0]))
        return c

    @property
    def kv_torch_dtype(self):
        return _TORCH_DT[self.kv_dtype]

    @property
    def coef_torch_dtype(self):
        return _TORCH_DT[self.coef_dtype]


class Cache:
    """One iS-KV cache (all layers of a batch).  Methods mirror the C ABI."""

    def __init__(self, cfg: Config, stream=None):
        self.cfg = cfg
        self._h = ctypes.c_void_p()
        self._cc = cfg._c()
        _check(LIB.iskv_create(ctypes.byref(self._cc), _stream(stream), ctypes.byref(self._h)),
               "iskv_create")

    def close(self) -> None:
        if getattr(self, "_h", None) and self._h.value:
            LIB.iskv_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> int:
        """k, v: [batch, kv_heads, t, d] pre-RoPE, device or host memory."""
        c = self.cfg
        if k.shape != v.shape or k.dim() != 4 or k.shape[:2] != (c.batch, c.kv_heads) \
                or k.shape[3] != c.head_dim:
            raise ValueError(f"k/v shape {tuple(k.shape)} does not match the cache")
        if k.dtype != c.kv_torch_dtype or v.dtype != c.kv_torch_dtype:
            raise TypeError("k/v dtype does not match kv_dtype")
        ready = ctypes.c_int(0)
        _check(LIB.iskv_append(self._h, layer, _ptr(k), _ptr(v), int(k.shape[2]), _stream(stream),
                               ctypes.byref(ready)), "iskv_append")
        return ready.value

    def compress_block(self, layer: int = ALL_LAYERS, defer: bool = False, stream=None) -> None:
        _check(LIB.iskv_compress_block(self._h, layer, FOLD_DEFER_SYNC if defer else 0,
                                       _stream(stream)), "iskv_compress_block")

    def compress_block_async(self, layer: int, stream, after=None, defer: bool = False) -> None:
        """The block update of `layer` on `stream` (a second stream), after the
        work enqueued so far on `after` (default: the current stream); later
        calls touching the layer are ordered after it by the library."""
        _check(LIB.iskv_compress_block_async(self._h, layer, FOLD_DEFER_SYNC if defer else 0,
                                             _stream(stream), _stream(after)),
               "iskv_compress_block_async")

    def sync(self, layer: int = ALL_LAYERS, stream=None) -> None:
        _check(LIB.iskv_sync(self._h, layer, _stream(stream)), "iskv_sync")

    def decode_attention(self, layer: int, q: torch.Tensor, out: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
        """q: [batch, q_heads, d] (rotated for position T-1); returns fp32 out."""
        c = self.cfg
        if tuple(q.shape) != (c.batch, c.q_heads, c.head_dim) or q.dtype != c.kv_torch_dtype:
            raise ValueError("q shape/dtype does not match the cache")
        if out is None:
            out = torch.empty(c.batch, c.q_heads, c.head_dim, dtype=torch.float32, device=q.device)
        _check(LIB.iskv_decode_attention(self._h, layer, _ptr(q), _ptr(out), _stream(stream)),
               "iskv_decode_attention")
        return out

    def reconstruct(self, layer: int, which: int, out: torch.Tensor | None = None,
                    stream=None, device="cuda") -> torch.Tensor:
        c = self.cfg
        n_c = self.counts(layer)[1]
        if out is None:
            out = torch.empty(c.batch, c.kv_heads, n_c, c.head_dim, dtype=torch.float32,
                              device=device)
        _check(LIB.iskv_reconstruct(self._h, layer, which, _ptr(out), _stream(stream)),
               "iskv_reconstruct")
        return out

    def factors(self, layer: int, which: int, stream=None, device="cuda"):
        """(basis [B,H,d,r] fp32, sigma [B,H,r] fp32, coef [B,H,n_c,r]); for a
        joint-head cache (basis [B,H*d,r], sigma [B,r], coef [B,n_c,r])."""
        c = self.cfg
        r = c.rank_k if which == WHICH_K else c.rank_v
        n_c = self.counts(layer)[1]
        cdt = torch.float32 if c.coef_quant else c.coef_torch_dtype   # coded: values code * scale
        if c.joint:
            basis = torch.empty(c.batch, c.kv_heads * c.head_dim, r, dtype=torch.float32, device=device)
            sigma = torch.empty(c.batch, r, dtype=torch.float32, device=device)
            coef = torch.empty(c.batch, n_c, r, dtype=cdt, device=device)
        else:
            basis = torch.empty(c.batch, c.kv_heads, c.head_dim, r, dtype=torch.float32, device=device)
            sigma = torch.empty(c.batch, c.kv_heads, r, dtype=torch.float32, device=device)
            coef = torch.empty(c.batch, c.kv_heads, n_c, r, dtype=cdt, device=device)
        _check(LIB.iskv_get_factors(self._h, layer, which, _ptr(basis), _ptr(sigma),
                                    _ptr(coef) if n_c else None, _stream(stream)),
               "iskv_get_factors")
        return basis, sigma, coef

    def counts(self, layer: int):
        T, n = ctypes.c_int64(), ctypes.c_int64()
        _check(LIB.iskv_get_counts(self._h, layer, ctypes.byref(T), ctypes.byref(n)),
               "iskv_get_counts")
        return T.value, n.value

    def kv_bytes(self):
        """(persistent bytes kept between decode steps, bytes of the uncompressed
        K/V cache at the same T), summed over every layer, sequence and KV head."""
        p, f = ctypes.c_int64(), ctypes.c_int64()
        _check(LIB.iskv_kv_bytes(self._h, ctypes.byref(p), ctypes.byref(f)), "iskv_kv_bytes")
        return p.value, f.value

    def decode_kernel(self, layer: int = 0) -> str:
        """The kernel the next decode_attention of `layer` runs: "cuda_core",
        "rotate" (tensor cores, keys rebuilt and rotated per tile) or
        "query_rope" (tensor cores, RoPE folded into the queries)."""
        k = _i()
        _check(LIB.iskv_decode_kernel(self._h, layer, ctypes.byref(k)), "iskv_decode_kernel")
        return {0: "cuda_core", 1: "rotate", 2: "query_rope"}[k.value]

    def status(self) -> int:
        return LIB.iskv_status(self._h)


def quantize_rows(groups, rows: torch.Tensor, stream=None):
    """Code fp32 rows [n, rank] (device) with the latent-channel format
    ``groups`` = ((channels, bits), ...): returns (codes [n, words] int32
    holding the uint32 words, scales [n, 4] fp32)."""
    fmt = QuantFormat.of(groups)
    words = LIB.iskv_quant_words(ctypes.byref(fmt))
    if words < 0:
        raise ValueError(f"invalid code format {groups}")
    if rows.dtype != torch.float32 or rows.dim() != 2:
        raise TypeError("rows must be a 2-d fp32 tensor")
    n, rank = rows.shape
    codes = torch.zeros(n, words, dtype=torch.int32, device=rows.device)
    scales = torch.zeros(n, 4, dtype=torch.float32, device=rows.device)
    _check(LIB.iskv_quantize_rows(ctypes.byref(fmt), rank, _ptr(rows), n, _ptr(codes), _ptr(scales),
                                  _stream(stream)), "iskv_quantize_rows")
    return codes, scales


# ---------------------------------------------------------------------------
# Paged 8-bit cache of exact tokens
# ---------------------------------------------------------------------------
_CODE_DT = {CODE_INT8: torch.int8, CODE_E4M3: torch.float8_e4m3fn}
_DT_CODE = {d: c for c, d in _CODE_DT.items()}
_DT_ELEM = {d: e for e, d in _TORCH_DT.items()}


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the same without building a stream object, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _launch(device: int, fn, where: str, *args, stream=None) -> None:
    """Call a library function that takes the stream last, on CUDA device `device`."""
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _launch(device, fn, where, *args, stream=stream)
    code = fn(*args, _raw_stream(device) if stream is None else stream.cuda_stream)
    if code != OK:
        raise IskvError(code, where)


def _new_on(stream, make, scratch=False):
    """make()'s tensors for a call on `stream` (None: the current one).  They
    come from that stream's pool, whose earlier work is done with the memory
    when the call runs, and go back to it only when the current stream, where
    the caller reads them, has passed them too (scratch: nobody does)."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        new = make()
    if not scratch:
        for t in new:
            t.record_stream(torch.cuda.current_stream(t.device))
    return new


def _hold(stream, *tensors) -> None:
    """Keep the memory of a call's tensors (None among them) until `stream` has
    passed the call, whatever the caller drops before."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _int32(device: int, shape, t: torch.Tensor, name: str) -> int:
    if t.dtype is not torch.int32 or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on cuda:{device}")
    return t.data_ptr()


def _all_int32(device: int, **tensors) -> None:
    """Say which of the (shape, tensor) pairs is not what it has to be."""
    for name, (shape, t) in tensors.items():
        _int32(device, shape, t, name)


_I31 = 2 ** 31


def _on_cuda(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t.get_device()


@dataclass
class PagePlan:
    """What one step of the page tables gives (int32, on the device): the
    lengths after the step [batch], cu [batch + 1] (exclusive sums of the added
    tokens), slots [tokens], n_free [1], status [1]."""
    lens: torch.Tensor
    cu: torch.Tensor
    slots: torch.Tensor
    n_free: torch.Tensor
    status: torch.Tensor

    @classmethod
    def empty(cls, batch: int, tokens: int, device="cuda") -> "PagePlan":
        def e(n):
            return torch.empty(n, dtype=torch.int32, device=device)
        return cls(e(batch), e(batch + 1), e(tokens), e(1), e(1))

    def _all(self):
        return self.lens, self.cu, self.slots, self.n_free, self.status


def page_plan(lens: torch.Tensor, add: torch.Tensor, table: torch.Tensor, free: torch.Tensor,
              n_free: torch.Tensor, tokens: int | None = None, out: PagePlan | None = None,
              stream=None) -> PagePlan:
    """One step of the page tables on the GPU (``iskv_page_plan``): request b
    holds lens[b] tokens and gets add[b] more, or has ended (-1).  `table`
    [batch, width] and the stack `free` [pages], of which `n_free` [1] entries
    are in use, are updated in place; the new lengths, slots and stack size go
    to `out` (or to new tensors for `tokens` slots).  To step in place, pass an
    `out` whose lens and n_free are the inputs.  ``status`` is 0, or the
    negative error code of a step that was refused as a whole."""
    dev = _on_cuda(lens, "lens")
    if lens.dim() != 1 or table.dim() != 2 or free.dim() != 1:
        raise ValueError("lens and free must be 1-d, table 2-d")
    batch, width = lens.shape[0], table.shape[1]
    if out is None:
        if tokens is None:
            raise ValueError("tokens (the number of slots) or out is needed")
        out = PagePlan(*_new_on(stream, lambda: PagePlan.empty(batch, tokens, lens.device)._all()))
    n, pages = out.slots.shape[0], free.shape[0]
    if max(n, width, pages) >= _I31:
        raise ValueError("slots, table columns and pages must be fewer than 2^31")
    every = (lens, add, table, free, n_free, out.lens, out.cu, out.slots, out.n_free, out.status)
    sizes = (batch, batch, batch * width, pages, 1, batch, batch + 1, n, 1, 1)
    i32 = torch.int32
    for t, size in zip(every, sizes):
        if t.dtype is not i32 or t.numel() != size or t.get_device() != dev or not t.is_contiguous():
            one = (1,)
            _all_int32(dev, lens=((batch,), lens), add=((batch,), add), table=((batch, width), table),
                       free=((pages,), free), n_free=(one, n_free), out_lens=((batch,), out.lens),
                       out_cu=((batch + 1,), out.cu), out_slots=((n,), out.slots), out_n_free=(one, out.n_free),
                       out_status=(one, out.status))
    args = _PlanArgs(batch, width, pages, n, *[t.data_ptr() for t in every])
    if stream is not None:
        _hold(stream, *every)
    _launch(dev, LIB.iskv_page_plan, "iskv_page_plan", ctypes.byref(args), stream=stream)
    return out


class Q8Pages:
    """The pages of one layer: K and V rows as 8-bit codes, 64 tokens a page,
    one scale per page and KV head.  ``k``, ``v`` [pages, kv_heads, 64, 128]
    (int8 or float8_e4m3fn) and ``k_scale``, ``v_scale`` [pages, kv_heads] are
    ordinary tensors; a stored row is codes * scale.  Requests take pages by
    ``page_plan``.  Forward only.  Calls given a `stream` run there, hold their
    tensors' memory until it has passed them, and leave it to the caller to order
    the streams.  Rows that a call reads may have any token stride of at least a
    row that is a multiple of 16 bytes."""

    def __init__(self, pages: int, kv_heads: int, code: int = CODE_INT8, device="cuda"):
        if code not in _CODE_DT:
            raise ValueError("code must be CODE_INT8 or CODE_E4M3")
        shape = (pages, kv_heads, PAGE, 128)
        bits = [torch.zeros(shape, dtype=torch.int8, device=device) for _ in range(2)]
        scale = [torch.zeros(pages, kv_heads, dtype=torch.float32, device=device) for _ in range(2)]
        self._take(bits[0].view(_CODE_DT[code]), bits[1].view(_CODE_DT[code]), *scale)

    @classmethod
    def of(cls, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor) -> "Q8Pages":
        """Pages in the caller's own tensors."""
        self = cls.__new__(cls)
        self._take(k, v, k_scale, v_scale)
        return self

    def _take(self, k, v, k_scale, v_scale):
        dev = _on_cuda(k, "k")
        if k.dtype not in _DT_CODE or v.dtype != k.dtype:
            raise TypeError("k and v must both be int8 or both float8_e4m3fn")
        if k.dim() != 4 or tuple(k.shape[2:]) != (PAGE, 128) or v.shape != k.shape:
            raise ValueError(f"k and v must be [pages, kv_heads, {PAGE}, 128]")
        for t, shape, dt in ((v, k.shape, k.dtype), (k_scale, k.shape[:2], torch.float32),
                             (v_scale, k.shape[:2], torch.float32)):
            if t.shape != shape or t.dtype != dt or t.get_device() != dev:
                raise ValueError("v, k_scale and v_scale must match k in shape, device and type")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.kv_heads, self._dev = k.device, k.shape[1], dev
        self._status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._need = {}   # workspace bytes by (q_heads, max_new, type)
        self._c = _Q8Pages(k.shape[0], k.shape[1], 128, PAGE, _DT_CODE[k.dtype], _ptr(k), _ptr(v), _ptr(k_scale),
                           _ptr(v_scale))
        self._ref, self._status_at = ctypes.byref(self._c), self._status.data_ptr()

    def _all(self):
        return self.k, self.v, self.k_scale, self.v_scale, self._status

    def _rows(self, t: torch.Tensor, heads: int | None, name: str) -> int:
        shape = t.shape
        if len(shape) != 3 or shape[2] != 128 or (heads is not None and shape[1] != heads) \
                or (shape[0] > 0 and (t.stride(2) != 1 or (shape[1] > 1 and t.stride(1) != 128))):
            raise ValueError(f"{name} must be [tokens, heads, 128] with contiguous tokens")
        if t.get_device() != self._dev:
            raise ValueError(f"{name} must be on {self.device}")
        code = _DT_ELEM.get(t.dtype)
        if code is None:
            raise TypeError(f"{name} must be bfloat16 or float32")
        return code

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """Store rows k, v [n, kv_heads, 128] in the slots [n] that
        ``page_plan`` gave; rows with slot -1 are skipped."""
        dt = self._rows(k, self.kv_heads, "k")
        if (k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
            raise ValueError("8-bit pages are forward only: detach k and v")
        if self._rows(v, self.kv_heads, "v") != dt or v.shape != k.shape:
            raise ValueError("k and v must agree in shape and type")
        n = k.shape[0]
        at = _int32(self._dev, (n,), slots, "slots")
        if stream is not None:
            _hold(stream, k, v, slots, *self._all())
        _launch(self._dev, LIB.iskv_q8_append, "iskv_q8_append", self._ref, k.data_ptr(), v.data_ptr(), dt, k.stride(0),
                v.stride(0), n, at, self._status_at, stream=stream)

    def attention(self, q: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor, max_new: int,
                  scale: float = 128 ** -0.5, cap: float = 0.0, slopes: torch.Tensor | None = None,
                  window: int = 0, prefix: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
        """Attention of q [tokens, q_heads, 128]: request b's queries are rows
        cu[b]:cu[b+1] and the last of its lens[b] stored tokens.  Causal;
        `window` > 0 limits how far back a query sees,
        prefix[b] tokens at the start are seen by all; `cap` caps scores by
        cap*tanh(x/cap); slopes[q_heads] (fp32) take slope * distance off.
        `max_new` is the largest number of queries of one request.  Returns
        out [tokens, q_heads, 128] in q's type; its rows from cu[batch] on are
        left as they were (of a new out: anything)."""
        dt = self._rows(q, None, "q")
        n, heads = q.shape[0], q.shape[1]
        dev = self._dev
        if q.requires_grad and torch.is_grad_enabled():
            raise ValueError("attention over 8-bit pages is forward only: detach q")
        if out is None:
            out, = _new_on(stream, lambda: (q.new_empty(q.shape),))
        elif out.shape != q.shape or out.dtype != q.dtype or out.get_device() != dev or not out.is_contiguous():
            raise ValueError("out must be contiguous and match q in shape, type and device")
        if lens.dim() != 1 or table.dim() != 2:
            raise ValueError("lens must be 1-d, table 2-d")
        batch, width = lens.shape[0], table.shape[1]
        if not (-_I31 <= window < _I31 and -_I31 <= max_new < _I31 and width < _I31):
            raise ValueError("window, max_new and the table's columns must be 32-bit numbers")
        if slopes is not None and (slopes.dtype != torch.float32 or tuple(slopes.shape) != (heads,)
                                   or slopes.get_device() != dev or not slopes.is_contiguous()):
            raise ValueError("slopes must be a contiguous fp32 tensor [q_heads] on the pages' device")
        need = self._need.get((heads, max_new, dt))
        if need is None:
            with torch.cuda.device(dev):
                need = LIB.iskv_q8_workspace(heads, self.kv_heads, n, max_new, dt)
            if len(self._need) < 64:
                self._need[(heads, max_new, dt)] = need
        ws, = _new_on(stream, lambda: (q.new_empty(max(need, 0), dtype=torch.uint8),), scratch=True)
        i32 = torch.int32
        if not (table.dtype is i32 and lens.dtype is i32 and cu.dtype is i32 and cu.numel() == batch + 1
                and table.get_device() == dev and lens.get_device() == dev and cu.get_device() == dev
                and table.shape[0] == batch and table.is_contiguous() and lens.is_contiguous() and cu.is_contiguous()):
            _all_int32(dev, table=((batch, width), table), lens=((batch,), lens), cu=((batch + 1,), cu))
        args = _Q8Attention(batch, width, heads, dt, max_new, window, scale, cap, n, q.stride(0), q.data_ptr(),
                            out.data_ptr(), table.data_ptr(), lens.data_ptr(), cu.data_ptr(),
                            None if prefix is None else _int32(dev, (batch,), prefix, "prefix"),
                            None if slopes is None else slopes.data_ptr(), ws.data_ptr(), need, self._status_at)
        if stream is not None:
            _hold(stream, q, out, table, lens, cu, prefix, slopes, *self._all())
        _launch(dev, LIB.iskv_q8_attention, "iskv_q8_attention", self._ref, ctypes.byref(args), stream=stream)
        return out

    def status(self) -> int:
        """Synchronize the device and return the sticky status of the calls on
        these pages, whichever streams they ran on:
        0, or the smallest code of non-finite rows (RANGE), a device-side wait
        that gave up (DEVICE_TIMEOUT) and slots outside the pool (INVALID_ARG)."""
        torch.cuda.synchronize(self._dev)
        return int(self._status.item())
