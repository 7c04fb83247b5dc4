"""Private tokens in pages: the torch-facing side of the polykv_pages_* calls.

Small calls are bound by what the host does, so the checks read each tensor's attributes once, the structures
that cross the ABI are built in one go, and attention's workspace is kept per stream.
"""
from __future__ import annotations

import math

import torch

from . import (POLYKV_BF16, POLYKV_F16, PagesAppendArgs, PagesDesc, PagesSeqs, RowStrides,
               polykv_attend_pages, polykv_attend_pages_workspace_size, polykv_pages_append, polykv_pages_attend,
               polykv_pages_attend_workspace_size, polykv_pages_create, polykv_pages_free, polykv_pages_select,
               polykv_pages_select_workspace_size, polykv_pages_status)

_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
_f32, _i32, _i64 = torch.float32, torch.int32, torch.int64


def _bad(t, name, shape, dtype, device):
    """The error for a tensor that is not a contiguous one of this shape, type and device."""
    if tuple(t.shape) != tuple(shape):
        return ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        return ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        return ValueError(f"{name} is on {t.device}, the cache on {device}")
    return ValueError(f"{name} must be contiguous")


class Rope:
    """The position rotation of a model's heads, as PageCache.append takes it: pair j turns by
    position * inv_freq[j] radians.

    inv_freq: rotary_dim / 2 frequencies (float64 on the host: a sequence, array or tensor), with whatever
    scaling scheme the model uses already applied. interleaved: pairs (2j, 2j + 1), else (j, j + rotary_dim / 2).
    mscale: factor of the cosines and sines. Kept in turns as 64-bit fixed point, so angles stay exact at
    far positions."""

    def __init__(self, inv_freq, interleaved: bool = False, mscale: float = 1.0, device="cuda"):
        freq = inv_freq.tolist() if hasattr(inv_freq, "tolist") else [float(f) for f in inv_freq]
        if not freq or not all(math.isfinite(f) for f in freq):
            raise ValueError("inv_freq must hold finite frequencies")
        if len(freq) % 8 != 0:
            raise ValueError(f"rotary_dim {2 * len(freq)} must be a multiple of 16")
        bits = [int(f / (2.0 * math.pi) * 2.0 ** 64) % (1 << 64) for f in freq]
        self.turns = torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=_i64, device=device)
        self.rotary_dim = 2 * len(freq)
        self.interleaved = bool(interleaved)
        self.mscale = float(mscale)

    @classmethod
    def from_theta(cls, rotary_dim: int, theta: float = 10000.0, **kw):
        """inv_freq[j] = theta^(-2j / rotary_dim)."""
        return cls([theta ** (-2.0 * j / rotary_dim) for j in range(rotary_dim // 2)], **kw)


class PageCache:
    """Each sequence's own keys and values, uncompressed, in pages of buffers that the caller owns.

    k_pages, v_pages: device, fp16 or bf16, [L][n_pages][H][page_tokens][d], contiguous.
    key_bounds: [L][n_pages][H][2][d] of the same type, or None: per page and kv head the lowest and highest key,
    kept by append and read by select.

    Every call takes block_table (device int32 [A][max_pages]: each sequence's page ids in order) and lens (device
    int32 [A]: its tokens; negative for an idle slot), so the caller's allocator decides which pages a sequence
    has, and a captured graph follows the tensors' contents. ``layer`` is the cache layer that the call's tensors
    begin with. Work goes to ``stream``, or to the current stream of the cache's device; what a call allocates
    belongs to that stream."""

    def __init__(self, k_pages, v_pages, key_bounds=None):
        self.handle = None
        if k_pages.dim() != 5:
            raise ValueError(f"k_pages must be [L][n_pages][H][page_tokens][d], got shape {tuple(k_pages.shape)}")
        if k_pages.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"k_pages must be bf16 or fp16, got {k_pages.dtype}")
        L, P, H, page, d = k_pages.shape
        dev, dt = k_pages.device, k_pages.dtype
        if not k_pages.is_contiguous():
            raise ValueError("k_pages must be contiguous")
        if v_pages.shape != k_pages.shape or v_pages.dtype != dt or v_pages.device != dev or not v_pages.is_contiguous():
            raise _bad(v_pages, "v_pages", k_pages.shape, dt, dev)
        if key_bounds is not None and (tuple(key_bounds.shape) != (L, P, H, 2, d) or key_bounds.dtype != dt or
                                       key_bounds.device != dev or not key_bounds.is_contiguous()):
            raise _bad(key_bounds, "key_bounds", (L, P, H, 2, d), dt, dev)
        self.k_pages, self.v_pages, self.key_bounds = k_pages, v_pages, key_bounds
        self.n_layers, self.n_pages, self.n_kv_heads, self.page_tokens, self.head_dim = L, P, H, page, d
        self.device, self.dtype = dev, dt
        self._index = dev.index if dev.type == "cuda" else -1   # -1: calls refuse
        self._status = torch.zeros(1, dtype=_i32, device=dev)
        self._attend_ws = {}   # (stream, query heads): workspace of attend
        self._select_ws = {}   # stream: workspace of select
        self._joint_ws = {}    # stream: workspace of attention together with a pool
        self.handle = polykv_pages_create(PagesDesc(
            L, H, d, page, P, POLYKV_BF16 if dt == torch.bfloat16 else POLYKV_F16, k_pages.data_ptr(),
            v_pages.data_ptr(), key_bounds.data_ptr() if key_bounds is not None else None, self._status.data_ptr()))

    @classmethod
    def empty(cls, n_layers: int, n_kv_heads: int, head_dim: int, n_pages: int, page_tokens: int = 32,
              dtype: str = "bf16", bounds: bool = False, device="cuda"):
        """A cache in buffers of its own."""
        dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        shape = (n_layers, n_pages, n_kv_heads, page_tokens, head_dim)
        b = torch.empty((n_layers, n_pages, n_kv_heads, 2, head_dim), dtype=dt, device=device) if bounds else None
        return cls(torch.empty(shape, dtype=dt, device=device), torch.empty(shape, dtype=dt, device=device), b)

    def close(self):
        if getattr(self, "handle", None):
            polykv_pages_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- what every call does first
    def _elsewhere(self, stream) -> bool:
        """Whether the call has to be made again with another device or stream current. Refuses host memory."""
        if self._index < 0:
            raise ValueError(f"the cache is on {self.device}, not on a CUDA device")
        return stream is not None or _current_device() != self._index

    def _there(self, stream):
        if stream is not None and stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the cache on {self.device}")
        return torch.cuda.device(self._index) if stream is None else torch.cuda.stream(stream)

    def _seqs(self, block_table, lens, A: int, layer: int, n_layers: int) -> PagesSeqs:
        shape = block_table.shape
        if len(shape) != 2:
            raise ValueError(f"block_table must be [A][max_pages], got shape {tuple(shape)}")
        if (shape[0] != A or block_table.dtype is not _i32 or block_table.device != self.device or
                not block_table.is_contiguous()):
            raise _bad(block_table, "block_table", (A, shape[1]), _i32, self.device)
        if lens.shape != (A,) or lens.dtype is not _i32 or lens.device != self.device or not lens.is_contiguous():
            raise _bad(lens, "lens", (A,), _i32, self.device)
        return PagesSeqs(block_table.data_ptr(), lens.data_ptr(), shape[1], A, layer, n_layers)

    def _rows(self, t, name, shape):
        """Strides (layer, row, head) of a [layers][rows][heads][d] tensor whose last dimension is contiguous."""
        if t.shape != shape or t.dtype is not self.dtype or t.device != self.device:
            raise _bad(t, name, shape, self.dtype, self.device)
        layer, row, head, last = t.stride()
        if last != 1:
            raise ValueError(f"{name}'s last dimension must be contiguous")
        # the stride of a dimension of one element says nothing
        return (layer if shape[0] > 1 else 0, row if shape[1] > 1 else 0, head if shape[2] > 1 else 0)

    def _selected(self, selected, L: int, A: int):
        if selected is None:
            return None, -1
        if selected.dim() != 4:
            raise ValueError(f"selected must be [L][A][H][n], got shape {tuple(selected.shape)}")
        n = selected.shape[3]
        if (selected.shape != (L, A, self.n_kv_heads, n) or selected.dtype is not _i32 or
                selected.device != self.device or not selected.is_contiguous()):
            raise _bad(selected, "selected", (L, A, self.n_kv_heads, n), _i32, self.device)
        return selected.data_ptr(), n

    def _workspace(self, kept: dict, key, need: int):
        """A workspace whose arrival counts are zero. Calls on one stream are ordered and share one; a graph under
        capture gets its own, which it clears itself."""
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(need, dtype=torch.uint8, device=self.device)
        ws = kept.get(key)
        if ws is None or ws.numel() < need:
            ws = kept[key] = torch.zeros(need, dtype=torch.uint8, device=self.device)
        return ws

    def status(self, stream=None) -> int:
        """Raises PolyKVError(E_STATE) if a kernel met a bad page, length or choice since the last call (synchronises)."""
        if self._elsewhere(stream):
            with self._there(stream):
                return self.status()
        return polykv_pages_status(self.handle, _raw_stream(self._index))

    # -- the operators
    def append(self, k, v, block_table, lens, starts=None, q=None, q_out=None, rope: Rope | None = None,
               positions=None, pos_offset: int = 0, layer: int = 0, stream=None):
        """Writes k and v to the sequences' next slots, rotating k (and q) by their positions with ``rope``.

        k, v: [L][n][H][d], q: [L][n][Hq][d], the cache's dtype, last dimension contiguous (slices of a fused
        projection will do). Row i of sequence s becomes its token lens[s] + i, lens being the lengths before
        the call, which does not change them. starts: device int32 [A + 1], sequence s owns rows [starts[s],
        starts[s + 1]), rows behind the last belong to nobody; None: n = A, one row each. A row's position is
        its place in its sequence + pos_offset, or positions[row] (device int64 [n]). Returns the rotated q
        (q_out if given, which may be q itself; rows behind the last are left as they are), or None without q."""
        shape = k.shape
        if len(shape) != 4:
            raise ValueError(f"k must be [L][n][H][d], got shape {tuple(shape)}")
        L, n = shape[0], shape[1]
        A, dev = lens.shape[0], self.device
        want = (L, n, self.n_kv_heads, self.head_dim)
        ks, vs = self._rows(k, "k", want), self._rows(v, "v", want)
        seqs = self._seqs(block_table, lens, A, layer, L)
        at = where = turns = None
        rot, inter, mscale = 0, 0, 1.0
        if starts is not None:
            if starts.shape != (A + 1,) or starts.dtype is not _i32 or starts.device != dev or not starts.is_contiguous():
                raise _bad(starts, "starts", (A + 1,), _i32, dev)
            at = starts.data_ptr()
        if positions is not None:
            if positions.shape != (n,) or positions.dtype is not _i64 or positions.device != dev or not positions.is_contiguous():
                raise _bad(positions, "positions", (n,), _i64, dev)
            where = positions.data_ptr()
        if rope is not None:
            if rope.turns.device != dev:
                raise ValueError(f"rope is on {rope.turns.device}, the cache on {dev}")
            turns, rot, inter, mscale = rope.turns.data_ptr(), rope.rotary_dim, rope.interleaved, rope.mscale
        if q is not None:
            if q.dim() != 4:
                raise ValueError(f"q must be [L][n][Hq][d], got shape {tuple(q.shape)}")
            heads = q.shape[2]
            q_want = (L, n, heads, self.head_dim)
            qs = self._rows(q, "q", q_want)
            if q_out is not None:
                qos = self._rows(q_out, "q_out", q_want)
        elif q_out is not None:
            raise ValueError("q_out without q")
        if self._elsewhere(stream):
            with self._there(stream):
                return self.append(k, v, block_table, lens, starts, q, q_out, rope, positions, pos_offset, layer)
        if q is not None:
            if q_out is None:
                q_out = torch.empty(q_want, dtype=self.dtype, device=dev)
                qos = (n * heads * self.head_dim, heads * self.head_dim, self.head_dim)
            args = PagesAppendArgs(k.data_ptr(), v.data_ptr(), q.data_ptr(), q_out.data_ptr(), ks, vs, qs, qos, heads, n,
                                   at, where, pos_offset, turns, rot, inter, mscale)
        else:
            args = PagesAppendArgs(k.data_ptr(), v.data_ptr(), None, None, ks, vs, (0, 0, 0), (0, 0, 0), 0, n, at, where,
                                   pos_offset, turns, rot, inter, mscale)
        polykv_pages_append(self.handle, seqs, args, _raw_stream(self._index))
        return q_out

    def attend(self, q, block_table, lens, selected=None, out=None, out_dtype=None, softmax_scale: float = 0.0,
               layer: int = 0, workspace=None, stream=None):
        """Attention of one new token per sequence over its tokens t < lens[s] (lens counts the new token once it
        is appended), or over those of its selected pages (from select). q: [L][A][Hq][d], last dimension
        contiguous. Returns [L][A][Hq][d] in out_dtype: fp32 (the default) or the cache's dtype. Zeros for a
        sequence without tokens. workspace: polykv_pages_attend_workspace_size bytes, the first 4 KiB zero before
        its first use, for one stream at a time; by default the cache keeps one per stream."""
        shape = q.shape
        if len(shape) != 4:
            raise ValueError(f"q must be [L][A][Hq][d], got shape {tuple(shape)}")
        L, A, Hq, _ = shape
        want = (L, A, Hq, self.head_dim)
        qs = self._rows(q, "q", want)
        seqs = self._seqs(block_table, lens, A, layer, L)
        sel, n_sel = self._selected(selected, L, A)
        if out is None:
            if out_dtype is None:
                out_dtype = _f32
        elif (out.shape != want or (out_dtype is not None and out.dtype != out_dtype) or out.device != self.device or
                not out.is_contiguous()):
            raise _bad(out, "out", want, out_dtype or out.dtype, self.device)
        else:
            out_dtype = out.dtype
        if out_dtype is not _f32 and out_dtype is not self.dtype:
            raise ValueError(f"out must be fp32 or {self.dtype}, got {out_dtype}")
        if self._elsewhere(stream):
            with self._there(stream):
                return self.attend(q, block_table, lens, selected, out, out_dtype, softmax_scale, layer, workspace)
        st = _raw_stream(self._index)
        if out is None:
            out = torch.empty(want, dtype=out_dtype, device=self.device)
        if workspace is None:
            workspace = self._attend_ws.get((st, Hq))
            if workspace is None or torch.cuda.is_current_stream_capturing():
                workspace = self._workspace(self._attend_ws, (st, Hq), polykv_pages_attend_workspace_size(self.handle, Hq))
        elif workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {self.device}")
        polykv_pages_attend(self.handle, seqs, q.data_ptr(), RowStrides(*qs), Hq, sel, n_sel, softmax_scale,
                            out.data_ptr(), out_dtype is _f32, workspace.data_ptr(), workspace.nbytes, st)
        return out

    def select(self, q, block_table, lens, n_selected: int, keep_first: int = 0, keep_last: int = 1, out=None,
               layer: int = 0, workspace=None, stream=None):
        """The pages that a sparse attention reads: per (layer, sequence, kv head) the n_selected pages with the
        highest upper bound max over the group's heads of sum_d max(q_d lowest_d, q_d highest_d), ascending, -1
        behind them; the first keep_first and last keep_last pages always. Returns int32 [L][A][H][n_selected]."""
        shape = q.shape
        if len(shape) != 4:
            raise ValueError(f"q must be [L][A][Hq][d], got shape {tuple(shape)}")
        L, A, Hq, _ = shape
        qs = self._rows(q, "q", (L, A, Hq, self.head_dim))
        seqs = self._seqs(block_table, lens, A, layer, L)
        want = (L, A, self.n_kv_heads, n_selected)
        if out is not None and (out.shape != want or out.dtype is not _i32 or out.device != self.device or
                                not out.is_contiguous()):
            raise _bad(out, "out", want, _i32, self.device)
        if workspace is not None and (workspace.device != self.device or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous and on {self.device}")
        if self._elsewhere(stream):
            with self._there(stream):
                return self.select(q, block_table, lens, n_selected, keep_first, keep_last, out, layer, workspace)
        st = _raw_stream(self._index)
        if workspace is None:
            need = polykv_pages_select_workspace_size(self.handle, seqs)
            if need:
                workspace = self._workspace(self._select_ws, st, need)
        if out is None:
            out = torch.empty(want, dtype=_i32, device=self.device)
        polykv_pages_select(self.handle, seqs, q.data_ptr(), RowStrides(*qs), Hq, n_selected, keep_first, keep_last,
                            out.data_ptr(), workspace.data_ptr() if workspace is not None else None,
                            workspace.nbytes if workspace is not None else 0, st)
        return out

    def _attend_with_pool(self, pool, q, n_ctx, block_table, lens, selected, out, softmax_scale, workspace, stream):
        """Pool.attend_with_pages."""
        if q.dim() != 4:
            raise ValueError(f"q must be [L][A][Hq][d], got shape {tuple(q.shape)}")
        L, A, Hq, _ = q.shape
        want = (pool.desc.n_layers, A, Hq, pool.desc.head_dim)
        if tuple(q.shape) != want or q.element_size() != 2 or q.device != self.device or not q.is_contiguous():
            raise _bad(q, "q", want, q.dtype if q.element_size() == 2 else self.dtype, self.device)
        if pool.buf.device != self.device:
            raise ValueError(f"the pool is on {pool.buf.device}, the cache on {self.device}")
        seqs = self._seqs(block_table, lens, A, 0, L)
        sel, n_sel = self._selected(selected, L, A)
        if out is not None and (tuple(out.shape) != want or out.dtype != _f32 or out.device != self.device or
                                not out.is_contiguous()):
            raise _bad(out, "out", want, _f32, self.device)
        if workspace is not None and (workspace.device != self.device or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous and on {self.device}")
        if self._elsewhere(stream):
            with self._there(stream):
                return self._attend_with_pool(pool, q, n_ctx, block_table, lens, selected, out, softmax_scale,
                                              workspace, None)
        st = _raw_stream(self._index)
        if out is None:
            out = torch.empty(want, dtype=_f32, device=self.device)
        if workspace is None:
            need = polykv_attend_pages_workspace_size(pool.handle, self.handle, seqs, Hq, n_ctx)
            workspace = self._workspace(self._joint_ws, st, need)
        polykv_attend_pages(pool.handle, self.handle, seqs, q.data_ptr(), out.data_ptr(), Hq, n_ctx, softmax_scale,
                            sel, n_sel, workspace.data_ptr(), workspace.nbytes, st)
        return out
