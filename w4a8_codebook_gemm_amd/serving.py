"""Python binding of libw4a8_serve.so: what a serving step does around the quantised products and
beside the int8 attention operators (include/w4a8_serve.h).

    batch = pages_assign(pages, new_tokens, tokens)               # pages, offsets, positions, slots
    seqs = Sequences(pages.page_table, batch.cu_tokens, batch.seq_lens)
    for each layer:
        p = add_norm_prepare(y, weight, h, h_out=h)               # residual, norm, the products' int8 input
        q, k, v = linear_multi(p.x_q, p.s_x, [wq, wk, wv])        # quantised projections
        q, k = qk_norm_rope(q, k, batch.positions, inv_freq, ...)
        kv4_append(k, v, cache, batch.slots)                      # into the cache in 4 bits
        o = kv4_attention(q, cache, seqs, workspace=ws)           # over the cache
        y = forward(o.view(m, -1), wo)
    pages_release(pages, keep_lens)                               # what ended or was refused

Argument marshalling only, as in the package itself: placement, dtype and layout are checked
here, the kernels run on the current stream of the tensors' device, and nothing falls back.
Every tensor begins at a multiple of 16 bytes (a slice such as slots[1:] does not) and a call
has at least one token; the library refuses others.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass, field
from typing import NamedTuple

import torch

from . import BF16, F32, STATUS, _dev
from .attention import Sequences, _current_device, _fits, _ptr, _raw_stream, _rows

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a8_serve.so")

COUNTER_BYTES = 8192     # W4A8_KV4_ATTENTION_COUNTER_BYTES
DEFAULT_UNIT = 2.0 ** -14
EXPORTS = ("w4a8_serve_status_string", "w4a8_add_norm_prepare", "w4a8_pages_assign", "w4a8_pages_release",
           "w4a8_kv4_append", "w4a8_kv4_attention_workspace_bytes", "w4a8_kv4_attention")
_FLOATS = (torch.float32, torch.bfloat16)


class ServingError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({lib().w4a8_serve_status_string(status).decode()})")


class CPages(C.Structure):
    """w4a8_pages."""
    _fields_ = [("page_table", C.c_void_p), ("seq_lens", C.c_void_p), ("free_pages", C.c_void_p), ("free_count", C.c_void_p),
                ("B", C.c_int64), ("table_width", C.c_int64), ("num_pages", C.c_int64), ("page_size", C.c_int)]


class CBatch(C.Structure):
    """w4a8_batch."""
    _fields_ = [("cu_tokens", C.c_void_p), ("seq_lens", C.c_void_p), ("positions", C.c_void_p), ("slots", C.c_void_p),
                ("free_count", C.c_void_p), ("missing", C.c_void_p)]


class CKV4Cache(C.Structure):
    """w4a8_kv4_cache."""
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p), ("k_unit", C.c_void_p),
                ("v_unit", C.c_void_p), ("num_pages", C.c_int64), ("kv_heads", C.c_int), ("page_size", C.c_int),
                ("head_dim", C.c_int)]


_lib = None


def lib():
    """The loaded C library (torch is imported first so HIP resolves to torch's runtime)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "or python w4a8_codebook_gemm_amd/build.py")
        L = C.CDLL(LIB_PATH)
        P, i64, i32, f32 = C.c_void_p, C.c_int64, C.c_int, C.c_float
        L.w4a8_serve_status_string.argtypes = [i32]
        L.w4a8_serve_status_string.restype = C.c_char_p
        L.w4a8_add_norm_prepare.argtypes = [P, i32, i64, P, i32, i64, P, f32, f32, i64, i64, P, P, i32, P, P, P]
        L.w4a8_add_norm_prepare.restype = i32
        L.w4a8_pages_assign.argtypes = [P, P, i64, P, P]
        L.w4a8_pages_assign.restype = i32
        L.w4a8_pages_release.argtypes = [P, P, P, P, P]
        L.w4a8_pages_release.restype = i32
        L.w4a8_kv4_append.argtypes = [P, i64, P, i64, i32, i64, P, P, P]
        L.w4a8_kv4_append.restype = i32
        L.w4a8_kv4_attention_workspace_bytes.argtypes = [i64, i64, i32, i32, i32]
        L.w4a8_kv4_attention_workspace_bytes.restype = i64
        L.w4a8_kv4_attention.argtypes = [P, i64, i32, i64, i32, P, P, f32, i32, i64, P, P, i64, P]
        L.w4a8_kv4_attention.restype = i32
        _lib = L
    return _lib


def _launch(dev: torch.device, what: str, f, *args):
    """f(*args, stream) with the tensors' device as the current one and its current stream."""
    i = dev.index
    if _current_device() == i:
        st = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            st = f(*args, _raw_stream(i))
    if st != 0:
        raise ServingError(st, what)


# ----------------------------------------------------------------------------- residual, norm, int8

class Prepared(NamedTuple):
    """What add_norm_prepare gives; None where it was not asked for."""
    h: torch.Tensor | None        # [M, K] the residual stream, of the residual's type
    x_q: torch.Tensor | None      # int8 [M, K], for linear and linear_multi
    s_x: torch.Tensor | None      # float32 [M]
    normed: torch.Tensor | None   # [M, K]


def _matrix(t, name: str, shape, dev):
    """Pointer, dtype code and row stride of [M, K] rows of consecutive values."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    dt = t.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError(f"{name} has dtype {dt}, expected one of {_FLOATS}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st, sk = t.stride()
    if sk != 1 and shape[1] != 1:
        raise ValueError(f"{name}: the values of a row must be consecutive, strides are {t.stride()}")
    return t.data_ptr(), BF16 if dt is torch.bfloat16 else F32, st if shape[0] > 1 else shape[1]


def add_norm_prepare(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
                     weight_offset: float = 0.0, quantise: bool = True, normed_dtype=None, h_out: torch.Tensor | None = None,
                     out=None) -> Prepared:
    """h = x + residual (of the residual's type), its RMS norm, and that rotated and quantised as
    prepare_activation does, in one launch.

    x, residual [M, K] (rows may be strided); weight float32 [K].  Without a residual x is normed and no
    h is kept.  normed_dtype: also return the norm itself; quantise=False: only that.  h_out [M, K]
    contiguous, of the residual's type: may be the residual.  out: (x_q, s_x) to write into."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    shape = x.shape
    m, k = shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError(f"x must be on a GPU device, got {dev}")
    # (torch makes a tensor like another one sooner than one from keywords)
    dense = x.is_contiguous()
    xp, xdt, xs = _matrix(x, "x", shape, dev)
    wp = _ptr(weight, "weight", torch.float32, (k,), dev)
    rp, rdt, rs, hp = 0, 0, 0, 0
    if residual is not None:
        rp, rdt, rs = _matrix(residual, "residual", shape, dev)
        if h_out is None:
            h_out = torch.empty_like(residual) if residual.is_contiguous() else residual.new_empty(m, k)
            hp = h_out.data_ptr()
        else:
            hp = _ptr(h_out, "h_out", residual.dtype, shape, dev)
    elif h_out is not None:
        raise ValueError("h_out without a residual")
    normed, np_, ndt = None, 0, 0
    if normed_dtype is not None:
        if normed_dtype not in _FLOATS:
            raise TypeError(f"normed_dtype {normed_dtype}, expected one of {_FLOATS}")
        normed = torch.empty_like(x, dtype=normed_dtype) if dense else x.new_empty((m, k), dtype=normed_dtype)
        np_, ndt = normed.data_ptr(), BF16 if normed_dtype is torch.bfloat16 else F32
    elif not quantise:
        raise ValueError("neither the quantised norm nor the norm itself is wanted")
    x_q = s_x = None
    qp = sp = 0
    if quantise:
        if out is None:
            x_q = torch.empty_like(x, dtype=torch.int8) if dense else x.new_empty((m, k), dtype=torch.int8)
            s_x = weight.new_empty(m)
            qp, sp = x_q.data_ptr(), s_x.data_ptr()
        else:
            x_q, s_x = out
            qp, sp = _ptr(x_q, "x_q", torch.int8, shape, dev), _ptr(s_x, "s_x", torch.float32, (m,), dev)
    elif out is not None:
        raise ValueError("out without quantise")
    _launch(dev, "w4a8_add_norm_prepare", lib().w4a8_add_norm_prepare, xp, xdt, xs, rp, rdt, rs, wp, weight_offset, eps, m, k,
            hp, np_, ndt, qp, sp)
    return Prepared(h_out, x_q, s_x, normed)


# ----------------------------------------------------------------------------- pages

@dataclass(frozen=True)
class Pages:
    """The pages of B sequences and the free ones, as int32 device tensors: page_table [B, width],
    seq_lens [B], free_pages [num_pages] (the last of the first free_count is handed out first), free_count [1].
    The tensors are checked here, once; their contents change with every call."""
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    free_pages: torch.Tensor
    free_count: torch.Tensor
    page_size: int
    c: CPages = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if not isinstance(self.page_table, torch.Tensor) or self.page_table.dim() != 2:
            raise ValueError("page_table must be 2-D [sequences, width]")
        if not isinstance(self.free_pages, torch.Tensor) or self.free_pages.dim() != 1:
            raise ValueError("free_pages must be 1-D [pages]")
        b, w = self.page_table.shape
        dev, i32 = self.page_table.device, (torch.int32,)
        _fits(32, page_size=self.page_size)
        object.__setattr__(self, "c", CPages(
            _dev(self.page_table, "page_table", i32), _dev(self.seq_lens, "seq_lens", i32, (b,), dev),
            _dev(self.free_pages, "free_pages", i32, None, dev), _dev(self.free_count, "free_count", i32, (1,), dev), b, w,
            self.free_pages.numel(), self.page_size))

    @staticmethod
    def empty(sequences: int, width: int, pages: int, page_size: int, device="cuda") -> "Pages":
        """Sequences without a token, and all pages free; page 0 is handed out first."""
        i32 = dict(dtype=torch.int32, device=device)
        return Pages(torch.full((sequences, width), -1, **i32), torch.zeros(sequences, **i32),
                     torch.arange(pages - 1, -1, -1, **i32), torch.full((1,), pages, **i32), page_size)


@dataclass(frozen=True)
class Batch:
    """What pages_assign says of a step's new tokens: cu_tokens [B + 1], seq_lens [B], positions [M],
    free_count [1] and missing [1] int32, slots [M] int64."""
    cu_tokens: torch.Tensor
    seq_lens: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    free_count: torch.Tensor
    missing: torch.Tensor
    c: CBatch = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if not isinstance(self.seq_lens, torch.Tensor) or self.seq_lens.dim() != 1:
            raise ValueError("seq_lens must be 1-D [sequences]")
        if not isinstance(self.positions, torch.Tensor) or self.positions.dim() != 1:
            raise ValueError("positions must be 1-D [tokens]")
        b, m = self.seq_lens.shape[0], self.positions.shape[0]
        dev, i32 = self.seq_lens.device, (torch.int32,)
        object.__setattr__(self, "c", CBatch(
            _dev(self.cu_tokens, "cu_tokens", i32, (b + 1,), dev), _dev(self.seq_lens, "seq_lens", i32),
            _dev(self.positions, "positions", i32, None, dev), _dev(self.slots, "slots", (torch.int64,), (m,), dev),
            _dev(self.free_count, "free_count", i32, (1,), dev), _dev(self.missing, "missing", i32, (1,), dev)))

    @staticmethod
    def empty(sequences: int, tokens: int, device="cuda", seq_lens: torch.Tensor | None = None,
              free_count: torch.Tensor | None = None) -> "Batch":
        """Outputs for up to `tokens` rows; seq_lens and free_count: the pages' own, to be updated in place."""
        i32 = dict(dtype=torch.int32, device=device)
        return Batch(torch.empty(sequences + 1, **i32), torch.empty(sequences, **i32) if seq_lens is None else seq_lens,
                     torch.empty(tokens, **i32), torch.empty(tokens, dtype=torch.int64, device=device),
                     torch.empty(1, **i32) if free_count is None else free_count, torch.empty(1, **i32))


def pages_assign(pages: Pages, new_tokens: torch.Tensor, tokens: int, *, out: Batch | None = None) -> Batch:
    """Room for new_tokens [B] (int32, on the device) more tokens of each sequence, `tokens` rows in all (or
    fewer, see w4a8_pages_assign): the page table's new entries, and what the other operators of the step need.

    Without out, the pages' own lengths and count are updated.  out: a Batch of `tokens` rows; where its seq_lens and
    free_count are not the pages' own, those stay as they were."""
    pc = pages.c
    dev = pages.page_table.device
    np_ = _ptr(new_tokens, "new_tokens", torch.int32, (pc.B,), dev)
    if out is None:
        out = Batch.empty(pc.B, tokens, dev, pages.seq_lens, pages.free_count)
    elif out.seq_lens.device != dev or out.seq_lens.shape[0] != pc.B or out.positions.shape[0] != tokens:
        raise ValueError(f"out is for {out.seq_lens.shape[0]} sequences and {out.positions.shape[0]} tokens on {out.seq_lens.device}, "
                         f"the call has {pc.B} and {tokens} on {dev}")
    _launch(dev, "w4a8_pages_assign", lib().w4a8_pages_assign, C.addressof(pc), np_, tokens, C.addressof(out.c))
    return out


def pages_release(pages: Pages, keep_lens: torch.Tensor, *, in_place: bool = True) -> tuple[torch.Tensor, torch.Tensor]:
    """Sequences cut to their first keep_lens [B] tokens (int32, on the device; 0: ended), the pages behind back on the
    free list.  Returns (seq_lens, free_count): the pages' own, or new ones (in_place False: the list's pages
    are written, its count and the lengths stay as they were)."""
    pc = pages.c
    dev = pages.page_table.device
    kp = _ptr(keep_lens, "keep_lens", torch.int32, (pc.B,), dev)
    lens, count = (pages.seq_lens, pages.free_count) if in_place else (torch.empty_like(pages.seq_lens), torch.empty_like(pages.free_count))
    _launch(dev, "w4a8_pages_release", lib().w4a8_pages_release, C.addressof(pc), kp, lens.data_ptr(), count.data_ptr())
    return lens, count


# ----------------------------------------------------------------------------- the cache in 4 bits

@dataclass(frozen=True)
class KV4Cache:
    """A cache in 4 bits, in pages: codes uint8 [pages, kv_heads, page_size, head_dim / 2], scale bytes uint8 of
    keys [pages, kv_heads, page_size, head_dim / 16] and of values [pages, kv_heads, head_dim / 16, page_size], a
    unit float32 for each head of keys and of values (w4a8_kv4_cache has the format).  The tensors are checked
    here, once."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_unit: torch.Tensor
    v_unit: torch.Tensor
    c: CKV4Cache = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if not isinstance(self.k, torch.Tensor) or self.k.dim() != 4:
            raise ValueError("k must be 4-D [pages, kv_heads, page_size, head_dim / 2]")
        n, h, p, half = self.k.shape
        dev, u8, f32, g = self.k.device, (torch.uint8,), (torch.float32,), half // 8
        object.__setattr__(self, "c", CKV4Cache(
            _dev(self.k, "k", u8), _dev(self.v, "v", u8, (n, h, p, half), dev),
            _dev(self.k_scale, "k_scale", u8, (n, h, p, g), dev), _dev(self.v_scale, "v_scale", u8, (n, h, g, p), dev),
            _dev(self.k_unit, "k_unit", f32, (h,), dev), _dev(self.v_unit, "v_unit", f32, (h,), dev), n, h, p, 2 * half))

    @staticmethod
    def empty(pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda", k_unit: float = DEFAULT_UNIT,
              v_unit: float = DEFAULT_UNIT) -> "KV4Cache":
        """A cache of zero-filled pages, one unit for all heads."""
        z = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=device)  # noqa: E731
        n, h, p, d = pages, kv_heads, page_size, head_dim
        return KV4Cache(z(n, h, p, d // 2), z(n, h, p, d // 2), z(n, h, p, d // 16), z(n, h, d // 16, p),
                        torch.full((h,), float(k_unit), device=device), torch.full((h,), float(v_unit), device=device))


def kv4_append(k: torch.Tensor, v: torch.Tensor, cache: KV4Cache, slots: torch.Tensor) -> None:
    """k, v [M, kv_heads, head_dim] (rows may be strided) into their slots [M] (int64, page * page_size + place; those
    outside the cache, -1 among them, are dropped).  No slot twice in a call."""
    cc = cache.c
    kp, ks = _rows(k, "k", _FLOATS, cc.kv_heads, cc.head_dim)
    dev = k.device
    vp, vs = _rows(v, "v", (k.dtype,), cc.kv_heads, cc.head_dim, dev)
    m = k.shape[0]
    if v.shape[0] != m:
        raise ValueError(f"k has {m} tokens, v {v.shape[0]}")
    if cache.k.device != dev:
        raise ValueError(f"tokens on {dev}, cache on {cache.k.device}")
    _launch(dev, "w4a8_kv4_append", lib().w4a8_kv4_append, kp, ks, vp, vs, BF16 if k.dtype is torch.bfloat16 else F32, m,
            C.addressof(cc), _ptr(slots, "slots", torch.int64, (m,), dev))


def kv4_attention_workspace_bytes(tokens: int, sequences: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Workspace bytes kv4_attention needs for up to `tokens` rows and `sequences` sequences."""
    _fits(64, tokens=tokens, sequences=sequences)
    _fits(32, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim)
    n = lib().w4a8_kv4_attention_workspace_bytes(tokens, sequences, q_heads, kv_heads, head_dim)
    if n < 0:
        raise ServingError(-n, "w4a8_kv4_attention_workspace_bytes")
    return n


def kv4_attention_workspace(tokens: int, sequences: int, q_heads: int, kv_heads: int, head_dim: int,
                            device="cuda") -> torch.Tensor:
    """A workspace for kv4_attention, its counters zero: one for each call that may run at a time."""
    with torch.cuda.device(device):
        n = kv4_attention_workspace_bytes(tokens, sequences, q_heads, kv_heads, head_dim)
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        ws[:COUNTER_BYTES].zero_()
        return ws


def kv4_attention(q: torch.Tensor, cache: KV4Cache, seqs: Sequences, *, scale: float | None = None, causal: bool = True,
                  window: int = 0, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the new tokens' queries q [M, Hq, D] (rows may be strided) over a cache in 4 bits.

    Arguments as for attention.kv_attention; workspace: from kv4_attention_workspace, a new one is made where it is
    None.  Rows that belong to no sequence are left as they were (in an out made here: not set)."""
    cc, sc = cache.c, seqs.c
    if window:
        _fits(64, window=window)
    qp, qs = _rows(q, "q", _FLOATS, None, cc.head_dim)
    m, hq, d = q.shape
    dev, dtype = q.device, q.dtype
    if cache.k.device != dev or seqs.page_table.device != dev:
        raise ValueError(f"tokens on {dev}, cache on {cache.k.device}, sequences on {seqs.page_table.device}")
    if workspace is None:
        workspace = kv4_attention_workspace(max(m, 1), sc.B, hq, cc.kv_heads, d, dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of q")
    if out is None:
        out = q.new_empty(m, hq, d)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", dtype, (m, hq, d), dev)
    _launch(dev, "w4a8_kv4_attention", lib().w4a8_kv4_attention, qp, qs, BF16 if dtype is torch.bfloat16 else F32, m, hq,
            C.addressof(cc), C.addressof(sc), d ** -0.5 if scale is None else scale, 1 if causal else 0, window, op,
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out
