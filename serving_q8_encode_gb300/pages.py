"""Private tokens in pages: the torch-facing side of the polykv_pages_* calls.

The checks of the tensors, the allocation of results and the workspaces are in the extension ``_pages`` (built
from csrc/pages_torch.cpp with the library): for the small calls of a decode step the same steps in Python took
longer than the kernels.
"""
from __future__ import annotations

import math

import torch

from . import (POLYKV_BF16, POLYKV_CODE_E4M3, POLYKV_CODE_INT8, POLYKV_F16, PagesDesc, PolyKVError, load_library,
               polykv_pages_create, polykv_pages_create_coded, polykv_pages_free)

load_library()
try:
    from . import _pages as _ext
except ImportError as e:
    raise ImportError("the extension _pages is not built; run `python -c \"import __graft_entry__ as g; g.build()\"` "
                      "(needs nvcc and g++)") from e
_ext.init(PolyKVError)


def _bad(t, name, shape, dtype, device):
    """The error for a tensor that is not a contiguous one of this shape, type and device."""
    if tuple(t.shape) != tuple(shape):
        return ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        return ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        return ValueError(f"{name} is on {t.device}, the cache on {device}")
    return ValueError(f"{name} must be contiguous")


def _pi(bits):
    """pi * 2^bits, by Machin's formula 16 atan(1/5) - 4 atan(1/239)."""
    def atan_of_inverse(n):
        term = (1 << (bits + 32)) // n
        total, k = term, 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total
    return (16 * atan_of_inverse(5) - 4 * atan_of_inverse(239)) >> 32


_PI_BITS = 1200   # a double's 1,024 before the point, 64 behind it
_PI = _pi(_PI_BITS)


def _turns(f):
    """f / (2 pi) modulo 1, in units of 2^-64, to the nearest."""
    num, den = f.as_integer_ratio()
    return (((num << (_PI_BITS + 64)) // (den * _PI) + 1) >> 1) % (1 << 64)


class Rope:
    """The position rotation of a model's heads, as PageCache.append takes it: pair j turns by
    position * inv_freq[j] radians.

    inv_freq: rotary_dim / 2 frequencies (float64 on the host: a sequence, array or tensor), with whatever
    scaling scheme the model uses already applied. interleaved: pairs (2j, 2j + 1), else (j, j + rotary_dim / 2).
    mscale: factor of the cosines and sines. Kept in turns as 64-bit fixed point, the nearest to the
    frequencies as given, so that a position's angle is off by at most position * 2^-65 turns."""

    def __init__(self, inv_freq, interleaved: bool = False, mscale: float = 1.0, device="cuda"):
        freq = inv_freq.tolist() if hasattr(inv_freq, "tolist") else [float(f) for f in inv_freq]
        if not freq or not all(math.isfinite(f) for f in freq):
            raise ValueError("inv_freq must hold finite frequencies")
        if len(freq) % 8 != 0:
            raise ValueError(f"rotary_dim {2 * len(freq)} must be a multiple of 16")
        bits = [_turns(f) for f in freq]
        self.turns = torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device=device)
        self.rotary_dim = 2 * len(freq)
        self.interleaved = bool(interleaved)
        self.mscale = float(mscale)

    @classmethod
    def from_theta(cls, rotary_dim: int, theta: float = 10000.0, **kw):
        """inv_freq[j] = theta^(-2j / rotary_dim)."""
        if rotary_dim < 16 or rotary_dim % 16 != 0:
            raise ValueError(f"rotary_dim {rotary_dim} must be a multiple of 16")
        return cls([theta ** (-2.0 * j / rotary_dim) for j in range(rotary_dim // 2)], **kw)


class PageCache:
    """Each sequence's own keys and values in pages of buffers that the caller owns, uncompressed or in 8 bits.

    k_pages, v_pages: device, fp16 or bf16, [L][n_pages][H][page_tokens][d], contiguous; or codes, int8 or
    float8_e4m3fn, with ``scales`` (fp32, [L][n_pages][H][2]: a factor per page and kv head for the keys and one for the
    values) and ``row_dtype`` (fp16 or bf16: the type of q, k, v and 16-bit results). append gives a page's values the
    smallest power of two under which they fit 127 or 448, rewrites its earlier codes when that rises, and begins anew
    with the page's first slot; a page that gets a value that is not finite reads as NaN.
    key_bounds: [L][n_pages][H][2][d] of the same type, or None: per page and kv head the lowest and highest key,
    kept by append and read by select (16-bit caches).

    Every call takes block_table (device int32 [A][max_pages]: each sequence's page ids in order) and lens (device
    int32 [A]: its tokens; negative for an idle slot), so the caller's allocator decides which pages a sequence
    has, and a captured graph follows the tensors' contents. ``layer`` is the cache layer that the call's tensors
    begin with. Work goes to ``stream``, or to the current stream of the cache's device; what a call allocates
    belongs to that stream. The calls have no backward pass: where gradients are recorded, a tensor that requires
    one is refused."""

    def __init__(self, k_pages, v_pages, key_bounds=None, scales=None, row_dtype=None):
        self.handle = None
        if k_pages.dim() != 5:
            raise ValueError(f"k_pages must be [L][n_pages][H][page_tokens][d], got shape {tuple(k_pages.shape)}")
        if k_pages.dtype not in (torch.bfloat16, torch.float16, torch.int8, torch.float8_e4m3fn):
            raise ValueError(f"k_pages must be bf16 or fp16, or int8 or float8_e4m3fn codes, got {k_pages.dtype}")
        coded = k_pages.element_size() == 1
        if coded and row_dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"row_dtype must be bf16 or fp16 for a cache of codes, got {row_dtype}")
        if not coded and row_dtype not in (None, k_pages.dtype):
            raise ValueError(f"row_dtype of a 16-bit cache is its pages' type, {k_pages.dtype}, got {row_dtype}")
        if coded != (scales is not None):
            raise ValueError("a cache of codes needs scales" if coded else "scales belong to a cache of codes")
        if coded and key_bounds is not None:
            raise ValueError("key_bounds are kept for 16-bit caches only")
        L, P, H, page, d = k_pages.shape
        dev, dt = k_pages.device, k_pages.dtype
        if not k_pages.is_contiguous():
            raise ValueError("k_pages must be contiguous")
        if v_pages.shape != k_pages.shape or v_pages.dtype != dt or v_pages.device != dev or not v_pages.is_contiguous():
            raise _bad(v_pages, "v_pages", k_pages.shape, dt, dev)
        if key_bounds is not None and (tuple(key_bounds.shape) != (L, P, H, 2, d) or key_bounds.dtype != dt or
                                       key_bounds.device != dev or not key_bounds.is_contiguous()):
            raise _bad(key_bounds, "key_bounds", (L, P, H, 2, d), dt, dev)
        if scales is not None and (tuple(scales.shape) != (L, P, H, 2) or scales.dtype != torch.float32 or
                                   scales.device != dev or not scales.is_contiguous()):
            raise _bad(scales, "scales", (L, P, H, 2), torch.float32, dev)
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (k_pages, v_pages, key_bounds, scales)):
            raise ValueError("a buffer of the cache requires a gradient, which the cache's calls do not give")
        self.k_pages, self.v_pages, self.key_bounds, self.scales = k_pages, v_pages, key_bounds, scales
        self.n_layers, self.n_pages, self.n_kv_heads, self.page_tokens, self.head_dim = L, P, H, page, d
        self.device, self.dtype = dev, row_dtype if coded else dt
        self._status = torch.zeros(1, dtype=torch.int32, device=dev)
        bf16 = self.dtype == torch.bfloat16
        desc = PagesDesc(L, H, d, page, P, POLYKV_BF16 if bf16 else POLYKV_F16, k_pages.data_ptr(), v_pages.data_ptr(),
                         key_bounds.data_ptr() if key_bounds is not None else None, self._status.data_ptr())
        self.handle = polykv_pages_create_coded(
            desc, POLYKV_CODE_INT8 if dt == torch.int8 else POLYKV_CODE_E4M3, scales.data_ptr()) if coded else \
            polykv_pages_create(desc)
        self._c = _ext.cache(self.handle, k_pages, int(bf16))

    @classmethod
    def empty(cls, n_layers: int, n_kv_heads: int, head_dim: int, n_pages: int, page_tokens: int = 32,
              dtype: str = "bf16", bounds: bool = False, device="cuda", codes: str | None = None):
        """A cache in buffers of its own; codes: None, "int8" or "e4m3"."""
        dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        shape = (n_layers, n_pages, n_kv_heads, page_tokens, head_dim)
        if codes is not None:
            if codes not in ("int8", "e4m3"):
                raise ValueError(f'codes must be None, "int8" or "e4m3", got {codes!r}')
            if bounds:
                raise ValueError("key_bounds are kept for 16-bit caches only")
            kind = torch.int8 if codes == "int8" else torch.float8_e4m3fn
            scales = torch.zeros((n_layers, n_pages, n_kv_heads, 2), dtype=torch.float32, device=device)
            return cls(torch.empty(shape, dtype=kind, device=device), torch.empty(shape, dtype=kind, device=device),
                       scales=scales, row_dtype=dt)
        b = torch.empty((n_layers, n_pages, n_kv_heads, 2, head_dim), dtype=dt, device=device) if bounds else None
        return cls(torch.empty(shape, dtype=dt, device=device), torch.empty(shape, dtype=dt, device=device), b)

    def close(self):
        """Releases the handle; the cache's calls refuse from then on."""
        if getattr(self, "handle", None):
            self._c = None
            polykv_pages_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _on(self, stream):
        if stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the cache on {self.device}")
        return torch.cuda.stream(stream)

    def status(self, stream=None) -> int:
        """Raises PolyKVError if a kernel met a bad page, length or choice (E_STATE) or gave up on a wait (E_TIMEOUT)
        since the last call (synchronises)."""
        if stream is not None:
            with self._on(stream):
                return _ext.status(self._c)
        return _ext.status(self._c)

    def append(self, k, v, block_table, lens, starts=None, q=None, q_out=None, rope: Rope | None = None,
               positions=None, pos_offset: int = 0, layer: int = 0, stream=None):
        """Writes k and v to the sequences' next slots, rotating k (and q) by their positions with ``rope``.

        k, v: [L][n][H][d], q: [L][n][Hq][d], the cache's dtype, last dimension contiguous (slices of a fused
        projection will do). Row i of sequence s becomes its token lens[s] + i, lens being the lengths before
        the call, which does not change them. starts: device int32 [A + 1], sequence s owns rows [starts[s],
        starts[s + 1]), rows behind the last belong to nobody; None: n = A, one row each. A row's position is
        its place in its sequence + pos_offset, or positions[row] (device int64 [n]). Returns the rotated q
        (q_out if given, which may be q itself and whose rows must not overlap), or None without q. Rows that no
        sequence appends, behind the last or of an idle slot, are left as they are: in a q that the call allocates,
        not initialised."""
        if stream is not None:
            with self._on(stream):
                return self.append(k, v, block_table, lens, starts, q, q_out, rope, positions, pos_offset, layer)
        if rope is None:
            return _ext.append(self._c, k, v, block_table, lens, starts, q, q_out, None, 0, False, 1.0, positions,
                               pos_offset, layer)
        return _ext.append(self._c, k, v, block_table, lens, starts, q, q_out, rope.turns, rope.rotary_dim,
                           rope.interleaved, rope.mscale, positions, pos_offset, layer)

    def attend(self, q, block_table, lens, selected=None, out=None, out_dtype=None, softmax_scale: float = 0.0,
               layer: int = 0, workspace=None, stream=None, window: int = 0, sinks: int = 0):
        """Attention of one new token per sequence over its tokens t < lens[s] (lens counts the new token once it
        is appended), or over those of its selected pages (from select). q: [L][A][Hq][d], last dimension
        contiguous. Returns [L][A][Hq][d] in out_dtype: fp32 (the default) or the cache's dtype. Zeros for a
        sequence without tokens. window: sees the last `window` tokens and the first `sinks` only (0: all); pages that lie
        wholly between are not looked up. workspace: polykv_pages_attend_workspace_size bytes, the first 4 KiB zero
        before its first use, for one stream at a time; by default the cache keeps one per stream."""
        if stream is not None:
            with self._on(stream):
                return self.attend(q, block_table, lens, selected, out, out_dtype, softmax_scale, layer, workspace,
                                   window=window, sinks=sinks)
        if out_dtype is None:
            kind = 0 if out is None else -1
        elif out_dtype is torch.float32:
            kind = 0
        elif out_dtype is self.dtype:
            kind = 1
        else:
            raise ValueError(f"out must be fp32 or {self.dtype}, got {out_dtype}")
        return _ext.attend(self._c, q, block_table, lens, selected, out, kind, softmax_scale, layer, workspace, window, sinks)

    def attend_rows(self, q, block_table, lens, starts, window: int = 0, sinks: int = 0, out=None,
                    softmax_scale: float = 0.0, layer: int = 0, workspace=None, stream=None):
        """Causal attention of runs of rows over the pages that hold them already: prompts, chunks of them, drafted tokens.

        q: [L][n][Hq][d], the cache's dtype, last dimension contiguous. Sequence s owns rows [starts[s], starts[s + 1])
        (device int32 [A + 1]), its last tokens: lens counts them (a plan's `after`), and row i of its n is token
        lens[s] - n + i. It sees the tokens up to itself, or with a window the last `window` of those and the first `sinks`.
        Returns [L][n][Hq][d] in the cache's dtype (``out`` if given, which must not overlap q), into whose precision probabilities are rounded where
        they meet the values; codes are taken as gather gives them, from copies in the workspace. Rows that no sequence owns,
        behind the last or of an idle slot, are left as they are: in a result that the call allocates, not initialised.
        workspace: polykv_pages_attend_rows_workspace_size bytes, the first 4 KiB zero before its first use, for one stream
        at a time; by default the cache keeps one per stream."""
        if stream is not None:
            with self._on(stream):
                return self.attend_rows(q, block_table, lens, starts, window, sinks, out, softmax_scale, layer, workspace)
        return _ext.attend_rows(self._c, q, block_table, lens, starts, window, sinks, out, softmax_scale, layer, workspace)

    def gather(self, block_table, lens, starts, n_rows: int, k=None, v=None, layer: int = 0, n_layers: int | None = None,
               stream=None):
        """(k, v) of the sequences' last tokens as rows [n_layers][n_rows][H][d] in the cache's dtype: those of sequence s
        are rows [starts[s], starts[s + 1]), the last of them token lens[s] - 1. Codes come as their values. For what reads
        16-bit tokens, such as Pool.encode (after a transpose). n_layers: from ``layer`` on; all by default. Rows that no
        sequence owns are left as they are (not initialised in results that the call allocates)."""
        if stream is not None:
            with self._on(stream):
                return self.gather(block_table, lens, starts, n_rows, k, v, layer, n_layers)
        if n_layers is None:
            n_layers = self.n_layers - layer
        return _ext.gather(self._c, block_table, lens, starts, n_rows, n_layers, k, v, layer)

    def select(self, q, block_table, lens, n_selected: int, keep_first: int = 0, keep_last: int = 1, out=None,
               layer: int = 0, workspace=None, stream=None):
        """The pages that a sparse attention reads: per (layer, sequence, kv head) the n_selected pages with the
        highest upper bound max over the group's heads of sum_d max(q_d lowest_d, q_d highest_d), ascending, -1
        behind them; the first keep_first and last keep_last pages always. Returns int32 [L][A][H][n_selected].
        workspace: as for attend, of polykv_pages_select_workspace_size bytes."""
        if stream is not None:
            with self._on(stream):
                return self.select(q, block_table, lens, n_selected, keep_first, keep_last, out, layer, workspace)
        return _ext.select(self._c, q, block_table, lens, n_selected, keep_first, keep_last, out, layer, workspace)

    def _attend_with_pool(self, pool, q, n_ctx, block_table, lens, selected, out, softmax_scale, workspace, stream):
        """Pool.attend_with_pages."""
        if stream is not None:
            with self._on(stream):
                return self._attend_with_pool(pool, q, n_ctx, block_table, lens, selected, out, softmax_scale, workspace, None)
        return _ext.attend_with_pool(self._c, pool.handle, pool.buf, pool.desc.n_layers, pool.desc.head_dim, q, n_ctx,
                                     block_table, lens, selected, out, softmax_scale, workspace)
