"""Python binding of libw4a8_attn.so: the attention operators between the quantised
projections (include/w4a8_attn.h).

    q, k, v = forward_multi(x, [wq, wk, wv])                      # quantised projections
    q, k = qk_norm_rope(q, k, positions, inv_freq, ...)           # head norm, rotary positions
    kv_append(k, v, cache, seqs)                                  # into the int8 paged cache
    o = kv_attention(q, cache, seqs, workspace=ws)                # over the cache
    y = forward(o.view(m, -1), wo)                                # output projection

Argument marshalling only, as in the package itself: placement, dtype and layout are checked
here, the kernels run on the current stream of the tensors' device, and nothing falls back.
Every tensor begins at a multiple of 16 bytes (a slice such as positions[3:] does not) and a call
has at least one token; the library refuses others.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass, field

import torch

from . import BF16, F32, STATUS, _dev

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a8_attn.so")

COUNTER_BYTES = 8192  # W4A8_KV_ATTENTION_COUNTER_BYTES
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = 0, 1, 2, 3
_SCALINGS = {"plain": ROPE_PLAIN, "linear": ROPE_LINEAR, "ntk": ROPE_NTK, "yarn": ROPE_YARN}
EXPORTS = ("w4a8_attn_status_string", "w4a8_rope_frequencies", "w4a8_qk_norm_rope", "w4a8_kv_append",
           "w4a8_kv_attention_workspace_bytes", "w4a8_kv_attention")
_FLOATS = (torch.float32, torch.bfloat16)


class AttentionError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({lib().w4a8_attn_status_string(status).decode()})")


class CHeads(C.Structure):
    """w4a8_heads."""
    _fields_ = [("x", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64), ("heads", C.c_int),
                ("weight", C.c_void_p), ("out", C.c_void_p)]


class CCache(C.Structure):
    """w4a8_kv_cache."""
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("num_pages", C.c_int64), ("kv_heads", C.c_int), ("page_size", C.c_int), ("head_dim", C.c_int)]


class CSequences(C.Structure):
    """w4a8_sequences."""
    _fields_ = [("page_table", C.c_void_p), ("cu_tokens", C.c_void_p), ("seq_lens", C.c_void_p), ("B", C.c_int64),
                ("table_width", C.c_int64)]


_lib = None


def lib():
    """The loaded C library (torch is imported first so HIP resolves to torch's runtime)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "or python w4a8_codebook_gemm_amd/build.py")
        L = C.CDLL(LIB_PATH)
        P, i64, i32, f32, f64 = C.c_void_p, C.c_int64, C.c_int, C.c_float, C.c_double
        L.w4a8_attn_status_string.argtypes = [i32]
        L.w4a8_attn_status_string.restype = C.c_char_p
        L.w4a8_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, P, P]
        L.w4a8_rope_frequencies.restype = i32
        L.w4a8_qk_norm_rope.argtypes = [P, P, i64, i32, i32, i32, P, P, i32, i32, f32, f32, f32, P]
        L.w4a8_qk_norm_rope.restype = i32
        L.w4a8_kv_append.argtypes = [P, i64, P, i64, i32, i64, P, P, P]
        L.w4a8_kv_append.restype = i32
        L.w4a8_kv_attention_workspace_bytes.argtypes = [i64, i64, i32, i32, i32]
        L.w4a8_kv_attention_workspace_bytes.restype = i64
        L.w4a8_kv_attention.argtypes = [P, i64, i32, i64, i32, P, P, f32, i32, i64, P, P, i64, P]
        L.w4a8_kv_attention.restype = i32
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        raise AttentionError(status, what)


def _public_raw_stream(i: int) -> int:
    return torch.cuda.current_stream(i).cuda_stream


# the accessors under torch's public ones take less time; a build of torch may lack them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(dev: torch.device, what: str, f, *args):
    """f(*args, stream) with the tensors' device as the current one and its current stream."""
    i = dev.index
    if _current_device() == i:
        st = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            st = f(*args, _raw_stream(i))
    if st != 0:
        raise AttentionError(st, what)


def _ptr(t, name: str, dtype, shape, dev) -> int:
    """_dev for one dtype, its tests in the order of a good call: the message is made only for a bad one."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    return _dev(t, name, (dtype,), shape, dev)


def _fits(bits: int, **numbers):
    """Refuses integers that the library would see as others: ctypes takes their low bits without a word."""
    for name, x in numbers.items():
        if not -(1 << bits - 1) <= x < 1 << bits - 1:
            raise ValueError(f"{name} {x} does not fit {bits} bits")


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original_context: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device="cuda") -> tuple[torch.Tensor, float]:
    """(inv_freq fp64 [rotary_dim / 2], attn_factor) for qk_norm_rope; computed on the host.

    scaling: "plain", "linear", "ntk" or "yarn" (see w4a8_rope_scaling)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {tuple(_SCALINGS)}, got {scaling!r}")
    _fits(32, rotary_dim=rotary_dim)
    out = torch.empty(max(int(rotary_dim), 0) // 2 + 1, dtype=torch.float64)
    attn = C.c_float(0.0)
    _check(lib().w4a8_rope_frequencies(rotary_dim, base, _SCALINGS[scaling], factor, original_context, beta_fast,
                                       beta_slow, out.data_ptr(), C.addressof(attn)), "w4a8_rope_frequencies")
    return out[:rotary_dim // 2].to(device), attn.value


def _rows(t: torch.Tensor, name: str, dtypes, heads=None, dim=None, device=None):
    """Pointer and token stride of [M, heads, dim] rows whose last two axes are dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other operands on {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or (dim is not None and t.shape[2] != dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [tokens, {heads or 'heads'}, {dim or 'head_dim'}]")
    m, h, d = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 and d != 1) or (sh != d and h != 1):
        raise ValueError(f"{name}: the values of a token must be consecutive, strides are {t.stride()}")
    return t.data_ptr(), st if m > 1 else h * d


def _heads(t, name, weight, out_dtype, out, m, d, dev, dtype):
    """w4a8_heads of one operand, and its output."""
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[0] != m or shape[2] != d:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [{m}, heads, {d}]")
    h = shape[1]
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the values of a head must be consecutive, strides are {t.stride()}")
    if m == 1:
        st = 0
    elif st < d and st != 0:
        raise ValueError(f"{name}: tokens overlap, strides are {t.stride()}")
    if out is None:
        out = t.new_empty(m, h, d) if out_dtype is dtype else t.new_empty((m, h, d), dtype=out_dtype)
        op = out.data_ptr()
    else:
        op = _ptr(out, name + "'s output", out_dtype, (m, h, d), dev)
    wp = 0 if weight is None else _ptr(weight, name + "_weight", torch.float32, (d,), dev)
    return CHeads(t.data_ptr(), st, sh if h > 1 else d, h, wp, op), out


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor, *,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 weight_offset: float = 0.0, interleaved: bool = False, attn_factor: float = 1.0, out_dtype=None,
                 out=None):
    """Head norm and rotary positions of q [M, Hq, D] and k [M, Hkv, D] (or None) in one launch.

    q and k may be views with any token and head strides (multiples of 8 elements); the outputs
    are contiguous.  Without a weight that operand is rotated only.  inv_freq fp64 [R / 2] turns
    the first R values of a head (rope_frequencies makes it); positions int32 [M].
    out: (q_out, k_out) to write into.  Returns (q_out, k_out)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be 3-D [tokens, heads, head_dim]")
    m, _, d = q.shape
    dev, dtype = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError(f"q must be on a GPU device, got {dev}")
    if dtype not in _FLOATS:
        raise TypeError(f"q has dtype {dtype}, expected one of {_FLOATS}")
    if out_dtype is None:
        out_dtype = dtype
    elif out_dtype not in _FLOATS:
        raise TypeError(f"out_dtype {out_dtype}, expected one of {_FLOATS}")
    q_out, k_out = out if out is not None else (None, None)
    ch, q_out = _heads(q, "q", q_weight, out_dtype, q_out, m, d, dev, dtype)
    kp = 0
    if k is not None:
        ck, k_out = _heads(k, "k", k_weight, out_dtype, k_out, m, d, dev, dtype)
        kp = C.addressof(ck)
    else:
        k_out = None
    half = inv_freq.numel()
    _launch(dev, "w4a8_qk_norm_rope", lib().w4a8_qk_norm_rope, C.addressof(ch), kp, m, d, BF16 if dtype is torch.bfloat16 else F32,
            BF16 if out_dtype is torch.bfloat16 else F32, _ptr(positions, "positions", torch.int32, (m,), dev),
            _ptr(inv_freq, "inv_freq", torch.float64, (half,), dev), 2 * half, 1 if interleaved else 0, attn_factor, eps,
            weight_offset)
    return q_out, k_out


@dataclass(frozen=True)
class KVCache:
    """An int8 cache in pages: codes [pages, kv_heads, page_size, head_dim], a scale for each
    page and head, finite and not negative.  The tensors are checked here, once."""
    k: torch.Tensor         # int8
    v: torch.Tensor         # int8
    k_scale: torch.Tensor   # float32 [pages, kv_heads]
    v_scale: torch.Tensor   # float32 [pages, kv_heads]
    c: CCache = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if not isinstance(self.k, torch.Tensor) or self.k.dim() != 4:
            raise ValueError("k must be 4-D [pages, kv_heads, page_size, head_dim]")
        n, h, p, d = self.k.shape
        dev = self.k.device
        object.__setattr__(self, "c", CCache(
            _dev(self.k, "k", (torch.int8,)), _dev(self.v, "v", (torch.int8,), (n, h, p, d), dev),
            _dev(self.k_scale, "k_scale", (torch.float32,), (n, h), dev),
            _dev(self.v_scale, "v_scale", (torch.float32,), (n, h), dev), n, h, p, d))

    @staticmethod
    def empty(pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> "KVCache":
        """A cache of zero-filled pages."""
        shape = (pages, kv_heads, page_size, head_dim)
        return KVCache(torch.zeros(shape, dtype=torch.int8, device=device), torch.zeros(shape, dtype=torch.int8, device=device),
                       torch.zeros(shape[:2], device=device), torch.zeros(shape[:2], device=device))


@dataclass(frozen=True)
class Sequences:
    """The sequences of a call, as int32 device tensors: page_table [B, width], cu_tokens [B + 1]
    (offsets of the new tokens' rows), seq_lens [B] (new tokens included).  The tensors are
    checked here, once; their contents may change between calls."""
    page_table: torch.Tensor
    cu_tokens: torch.Tensor
    seq_lens: torch.Tensor
    c: CSequences = field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if not isinstance(self.page_table, torch.Tensor) or self.page_table.dim() != 2:
            raise ValueError("page_table must be 2-D [sequences, width]")
        b, w = self.page_table.shape
        dev = self.page_table.device
        object.__setattr__(self, "c", CSequences(
            _dev(self.page_table, "page_table", (torch.int32,)), _dev(self.cu_tokens, "cu_tokens", (torch.int32,), (b + 1,), dev),
            _dev(self.seq_lens, "seq_lens", (torch.int32,), (b,), dev), b, w))


def _same_device(dev: torch.device, cache: KVCache, seqs: Sequences):
    if cache.k.device != dev or seqs.page_table.device != dev:
        raise ValueError(f"tokens on {dev}, cache on {cache.k.device}, sequences on {seqs.page_table.device}")


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, seqs: Sequences) -> None:
    """Append k, v [M, kv_heads, head_dim] (rows may be strided) to the pages of their sequences
    (see w4a8_kv_append for the scales).  Sequences of one call must not share a page they
    append to."""
    cc = cache.c
    kp, ks = _rows(k, "k", _FLOATS, cc.kv_heads, cc.head_dim)
    dev = k.device
    vp, vs = _rows(v, "v", (k.dtype,), cc.kv_heads, cc.head_dim, dev)
    m = k.shape[0]
    if v.shape[0] != m:
        raise ValueError(f"k has {m} tokens, v {v.shape[0]}")
    _same_device(dev, cache, seqs)
    _launch(dev, "w4a8_kv_append", lib().w4a8_kv_append, kp, ks, vp, vs, BF16 if k.dtype is torch.bfloat16 else F32, m,
            C.addressof(cc), C.addressof(seqs.c))


def kv_attention_workspace_bytes(tokens: int, sequences: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Workspace bytes kv_attention needs for up to `tokens` rows and `sequences` sequences."""
    _fits(64, tokens=tokens, sequences=sequences)
    _fits(32, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim)
    n = lib().w4a8_kv_attention_workspace_bytes(tokens, sequences, q_heads, kv_heads, head_dim)
    if n < 0:
        _check(-n, "w4a8_kv_attention_workspace_bytes")
    return n


def kv_attention_workspace(tokens: int, sequences: int, q_heads: int, kv_heads: int, head_dim: int,
                           device="cuda") -> torch.Tensor:
    """A workspace for kv_attention, its counters zero: one for each call that may run at a time."""
    with torch.cuda.device(device):
        n = kv_attention_workspace_bytes(tokens, sequences, q_heads, kv_heads, head_dim)
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        ws[:COUNTER_BYTES].zero_()
        return ws


def kv_attention(q: torch.Tensor, cache: KVCache, seqs: Sequences, *, scale: float | None = None, causal: bool = True,
                 window: int = 0, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the new tokens' queries q [M, Hq, D] (rows may be strided) over the cache.

    scale: of the scores, 1 / sqrt(D) by default.  window: positions a query sees, its own
    included (0: all before it; causal only).  workspace: from kv_attention_workspace; a new one
    is made where it is None.  out [M, Hq, D] contiguous, of q's type, apart from the other operands;
    rows that belong to no sequence are left as they were (in an out made here: not set).  Single tokens
    beside long prompts are faster as a call of their own (see w4a8_kv_attention)."""
    cc, sc = cache.c, seqs.c
    if window:
        _fits(64, window=window)
    qp, qs = _rows(q, "q", _FLOATS, None, cc.head_dim)
    m, hq, d = q.shape
    dev, dtype = q.device, q.dtype
    _same_device(dev, cache, seqs)
    if workspace is None:
        workspace = kv_attention_workspace(max(m, 1), sc.B, hq, cc.kv_heads, d, dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of q")
    if out is None:
        out = q.new_empty(m, hq, d)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", dtype, (m, hq, d), dev)
    _launch(dev, "w4a8_kv_attention", lib().w4a8_kv_attention, qp, qs, BF16 if dtype is torch.bfloat16 else F32, m, hq,
            C.addressof(cc), C.addressof(sc), d ** -0.5 if scale is None else scale, 1 if causal else 0, window, op,
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out
