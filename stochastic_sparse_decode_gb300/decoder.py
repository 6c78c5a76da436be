"""A convenience wrapper: owns the problem description and the workspaces.

    dec = Decoder(batch=1, num_q_heads=32, num_kv_heads=8, head_dim=128,
                  total_tokens=32768, max_len=32768, tile=256, S=128, dtype="bf16")
    out = dec("prop", q, k, v, kv_indptr, U)

Workspaces are allocated once per mode with torch (device memory only); each
call is one C-ABI call on the current stream.  Debug buffers can be requested
to inspect tile records, budgets and sampled indices.
"""

from __future__ import annotations

import ctypes

import torch

from . import (BF16, MODES, Debug, Pages, Rope, Window, _check, _stream, decode, k_feature_blocked_size, kv4_size, lib,
               make_pages, make_problem, santa_decode_prop_bernoulli, santa_decode_prop_paged, santa_k_feature_blocked,
               santa_prop_pass1, santa_prop_pass2, split_workspace_size, workspace_size)

_F32, _I32, _I64, _U8 = (frozenset((t,)) for t in (torch.float32, torch.int32, torch.int64, torch.uint8))

# torch's own shortcuts to the current device and its current stream's handle, where it has them
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _fits(t, dtypes, shape, dev) -> bool:
    return t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == dev


def rope_table(max_pos, rot_dim, theta=10000.0, device="cuda") -> torch.Tensor:
    """cos_sin of santa_norm_rope, [max_pos][rot_dim] float32: angles n * theta^(-2i / rot_dim),
    formed in double precision (in single, the angle of position 100000 is off by 0.004)."""
    half = rot_dim // 2
    freq = float(theta) ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    ang = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)


class Decoder:
    def __init__(self, batch, num_q_heads, num_kv_heads, head_dim, total_tokens, max_len, tile, S, dtype,
                 device=None):
        self.problem = make_problem(batch, num_q_heads, num_kv_heads, head_dim, total_tokens, max_len, tile, S,
                                    dtype)
        self.device = torch.device(device if device is not None else "cuda")
        self.Tmax = -(-max_len // tile) if max_len > 0 else 0
        self._ws = {}
        self._prepare()

    def __getstate__(self):
        # references into the C structures stay behind: a copy makes its own
        return {k: v for k, v in self.__dict__.items() if k not in ("_pref", "_windows")}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._prepare()

    def workspace(self, mode: str) -> torch.Tensor:
        if mode not in self._ws:
            n = workspace_size(self.problem, MODES[mode])
            # zero-filled: a prop workspace must start zero (santa_workspace_init)
            self._ws[mode] = torch.zeros(n, dtype=torch.uint8, device=self.device)
        return self._ws[mode]

    def debug_buffers(self, mode: str, sample_stride: int = 0):
        """(Debug struct, dict of the tensors it points to)."""
        p = self.problem
        B, Hq, T = p.batch, p.num_q_heads, max(self.Tmax, 1)
        dev = self.device
        bufs = {
            "tile_m": torch.full((B, Hq, T), float("nan"), device=dev),
            "tile_z": torch.full((B, Hq, T), float("nan"), device=dev),
            "tile_count": torch.full((B, Hq, T), -1, dtype=torch.int32, device=dev),
            "error_flags": torch.zeros(1, dtype=torch.int32, device=dev),
        }
        if mode in ("prop", "prop_fused", "strat", "iid", "prop_bernoulli"):
            bufs["sample_idx"] = torch.full((B, Hq, p.S), -1, dtype=torch.int32, device=dev)
        if mode == "prop_bernoulli":
            bufs["features_read"] = torch.full((B, p.num_kv_heads), -1, dtype=torch.int32, device=dev)
        elif mode == "flash":
            bufs["sample_idx"] = torch.full((B, Hq, T, max(sample_stride, 1)), -1, dtype=torch.int32, device=dev)
        dbg = Debug()
        dbg.tile_m = bufs["tile_m"].data_ptr()
        dbg.tile_z = bufs["tile_z"].data_ptr()
        dbg.tile_count = bufs["tile_count"].data_ptr()
        dbg.sample_idx = bufs["sample_idx"].data_ptr() if "sample_idx" in bufs else None
        dbg.sample_stride = int(sample_stride) if mode == "flash" else 0
        dbg.error_flags = bufs["error_flags"].data_ptr()
        if "features_read" in bufs:
            dbg.features_read = bufs["features_read"].data_ptr()
        return dbg, bufs

    def __call__(self, mode, q, k, v, kv_indptr, U=None, out=None, debug=None, stream=None) -> torch.Tensor:
        p = self.problem
        if out is None:
            out = torch.empty((p.batch, p.num_q_heads, p.head_dim), dtype=torch.float32, device=self.device)
        decode(mode, p, q, k, v, kv_indptr, U, out, self.workspace(mode), debug, stream)
        return out

    def pass1(self, q, k, kv_indptr, debug=None, stream=None) -> None:
        """Pass 1 of prop alone, into the prop workspace (santa_prop_pass1)."""
        santa_prop_pass1(self.problem, q, k, kv_indptr, self.workspace("prop"), debug, stream)

    def pass2(self, v, kv_indptr, U, out=None, debug=None, stream=None) -> torch.Tensor:
        """Pass 2 of prop alone, on the prop workspace pass 1 filled (santa_prop_pass2)."""
        p = self.problem
        if out is None:
            out = torch.empty((p.batch, p.num_q_heads, p.head_dim), dtype=torch.float32, device=self.device)
        santa_prop_pass2(self.problem, v, kv_indptr, U, out, self.workspace("prop"), debug, stream)
        return out

    def prop_paged(self, q, k_pool, v_pool, page_table, kv_lens, page_size, U, out=None, debug=None,
                   stream=None) -> torch.Tensor:
        """S2ANTA-prop on a paged cache (santa_decode_prop_paged); the problem's
        total_tokens must be the pools' rows, num_pages * page_size."""
        p = self.problem
        if out is None:
            out = torch.empty((p.batch, p.num_q_heads, p.head_dim), dtype=torch.float32, device=self.device)
        pages = make_pages(page_table, kv_lens, page_size, p.total_tokens // page_size)
        santa_decode_prop_paged(p, pages, q, k_pool, v_pool, U, out, self.workspace("prop"), debug, stream)
        return out

    def feature_blocked(self, k, stream=None) -> torch.Tensor:
        """The feature-blocked copy of the token-major K cache k (santa_k_feature_blocked)."""
        p = self.problem
        esz = 2 if k.dtype in (torch.bfloat16, torch.int16, torch.uint16) else 4
        n = k_feature_blocked_size(p)
        kfb = torch.empty(n // esz, dtype=k.dtype, device=self.device)
        santa_k_feature_blocked(p, k, kfb, stream)
        return kfb

    def prop_bernoulli(self, q, k_fb, v, kv_indptr, U, bern_u, draws, group_mean, out=None, debug=None,
                       stream=None) -> torch.Tensor:
        """S2ANTA-prop with the Bernoulli score stage (santa_decode_prop_bernoulli)."""
        p = self.problem
        if out is None:
            out = torch.empty((p.batch, p.num_q_heads, p.head_dim), dtype=torch.float32, device=self.device)
        santa_decode_prop_bernoulli(p, q, k_fb, v, kv_indptr, U, bern_u, draws, group_mean, out,
                                    self.workspace("prop"), debug, stream)
        return out

    # ---- the operators around the attention
    #
    # These calls are a few microseconds of GPU time, so the host's share is kept small: every
    # tensor is checked by one expression (_fits), and only a refusal looks for the reason.

    def _prepare(self):
        p = self.problem
        # bf16 may come as its bit pattern, as for the other modes
        self._dt = frozenset((torch.bfloat16, torch.int16, torch.uint16) if p.dtype == BF16 else (torch.float32,))
        self._q_shape = (p.batch, p.num_q_heads, p.head_dim)
        self._kv_shape = (p.total_tokens, p.num_kv_heads, p.head_dim)
        self._kv4_shape = (p.total_tokens, p.num_kv_heads, p.head_dim + p.head_dim // 8)
        self._pref = ctypes.byref(p)
        self._windows = {}

    def _refuse(self, name, t, dtypes, shape, dev, how=""):
        """Says why a tensor that the C call would misread is refused: dtype, shape (None: any size), device,
        layout."""
        if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
            raise ValueError(f"{name}: a tensor of {' or '.join(sorted(map(str, dtypes)))} is needed")
        if len(t.shape) != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, needed {shape}")
        if t.get_device() != dev:
            raise ValueError(f"{name}: on {t.device}, not with the other tensors")
        raise ValueError(f"{name}: not contiguous {how}".rstrip())

    def _stream(self, dev, stream):
        """The raw stream of a call whose tensors are on device `dev`, which must be the current one."""
        if dev < 0 or dev != _current_device():
            raise ValueError(f"the tensors are on {'the CPU' if dev < 0 else f'CUDA device {dev}'}, "
                             "not on the current CUDA device")
        return _raw_stream(dev) if stream is None else _stream(stream)

    def _out(self, out, dev):
        if out is None:
            return torch.empty(self._q_shape, dtype=torch.float32, device=dev)
        if not _fits(out, _F32, self._q_shape, dev):
            self._refuse("out", out, _F32, self._q_shape, dev)
        return out

    def split_workspace(self) -> torch.Tensor:
        """The workspace of window and kv4 calls (kept; calls that overlap need a Decoder each).  The first use
        prepares it, which a stream capture would only record: call this before capturing."""
        if "split" not in self._ws:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the workspace must exist before a capture: call split_workspace() first")
            # zero-filled: what santa_split_workspace_init does; complete before a call on any stream
            self._ws["split"] = torch.zeros(split_workspace_size(self.problem), dtype=torch.uint8, device=self.device)
            torch.cuda.current_stream(self._ws["split"].device).synchronize()
        return self._ws["split"]

    def _window(self, window, sinks):
        if not (0 <= window < 1 << 31 and 0 <= sinks < 1 << 31):
            raise ValueError(f"window {window}, sinks {sinks}: whole numbers from 0 to 2^31 - 1 are needed")
        if len(self._windows) >= 64:
            self._windows.clear()
        return self._windows.setdefault((window, sinks), ctypes.byref(Window(window, sinks)))

    def _attend(self, kind, q, k, v, kv_indptr, pages, window, sinks, out, debug, stream):
        dev = q.get_device()
        if not _fits(q, self._dt, self._q_shape, dev):
            self._refuse("q", q, self._dt, self._q_shape, dev)
        if kind == "window":
            for name, t in (("k", k), ("v", v)):
                if not _fits(t, self._dt, self._kv_shape, dev):
                    self._refuse(name, t, self._dt, self._kv_shape, dev)
        elif not _fits(k, _U8, self._kv4_shape, dev):
            self._refuse("kv4", k, _U8, self._kv4_shape, dev)
        p = self.problem
        indptr = pref = None
        if pages is None:
            if not _fits(kv_indptr, _I64, (p.batch + 1,), dev):
                self._refuse("kv_indptr", kv_indptr, _I64, (p.batch + 1,), dev)
            indptr = kv_indptr.data_ptr()
        else:
            table, lens, size = pages
            if table.dim() != 2 or not _fits(table, _I32, (p.batch, table.shape[1]), dev):
                self._refuse("page_table", table, _I32, (p.batch, None), dev)
            if not _fits(lens, _I32, (p.batch,), dev):
                self._refuse("kv_lens", lens, _I32, (p.batch,), dev)
            if size < 1 or p.total_tokens % size:
                raise ValueError(f"page_size {size} does not divide total_tokens {p.total_tokens}")
            pref = ctypes.byref(Pages(table.data_ptr(), lens.data_ptr(), size, table.shape[1], p.total_tokens // size))
        out = self._out(out, dev)
        w = self._windows.get((window, sinks))
        if w is None:
            w = self._window(window, sinks)
        ws = self._ws.get("split")
        if ws is None:
            ws = self.split_workspace()
        if ws.get_device() != dev:
            raise ValueError(f"the tensors are on CUDA device {dev}, this Decoder's workspace on {ws.device}")
        st = self._stream(dev, stream)
        dbg = None if debug is None else ctypes.byref(debug)
        L = lib()
        if kind == "window":
            _check("santa_decode_window", L.santa_decode_window(
                self._pref, w, pref, q.data_ptr(), k.data_ptr(), v.data_ptr(), indptr, out.data_ptr(), ws.data_ptr(),
                ws.numel(), dbg, st))
        else:
            _check("santa_decode_kv4", L.santa_decode_kv4(
                self._pref, w, pref, q.data_ptr(), k.data_ptr(), indptr, out.data_ptr(), ws.data_ptr(), ws.numel(), dbg, st))
        return out

    def window(self, q, k, v, kv_indptr, window, sinks=0, out=None, debug=None, stream=None) -> torch.Tensor:
        """Exact decode over the last `window` keys and the first `sinks` (santa_decode_window); window 0: all."""
        return self._attend("window", q, k, v, kv_indptr, None, window, sinks, out, debug, stream)

    def window_paged(self, q, k_pool, v_pool, page_table, kv_lens, page_size, window, sinks=0, out=None, debug=None,
                     stream=None) -> torch.Tensor:
        """The same on a paged cache; total_tokens must be the pools' rows, num_pages * page_size."""
        return self._attend("window", q, k_pool, v_pool, None, (page_table, kv_lens, page_size), window, sinks, out, debug,
                            stream)

    def kv4(self, q, kv4, kv_indptr, window=0, sinks=0, out=None, debug=None, stream=None) -> torch.Tensor:
        """Exact decode over the 4-bit cache (santa_decode_kv4)."""
        return self._attend("kv4", q, kv4, None, kv_indptr, None, window, sinks, out, debug, stream)

    def kv4_paged(self, q, kv4, page_table, kv_lens, page_size, window=0, sinks=0, out=None, debug=None,
                  stream=None) -> torch.Tensor:
        """The same on a paged 4-bit cache."""
        return self._attend("kv4", q, kv4, None, None, (page_table, kv_lens, page_size), window, sinks, out, debug, stream)

    def kv4_cache(self) -> torch.Tensor:
        """An empty 4-bit cache for the problem's total_tokens: [rows][Hkv][d + d / 8] bytes."""
        kv4_size(self.problem)  # checks the problem
        return torch.zeros(self._kv4_shape, dtype=torch.uint8, device=self.device)

    def _slots(self, slot_map, n, dev):
        if slot_map is None:
            return None
        if not _fits(slot_map, _I64, (n,), dev):
            self._refuse("slot_map", slot_map, _I64, (n,), dev)
        return slot_map.data_ptr()

    def _rows(self, name, t, n, heads, dev):
        """(address, elements from token to token) of [tokens][heads][d], whose tokens may lie apart."""
        d = self.problem.head_dim
        if t.dtype in self._dt and t.shape == (n, heads, d) and t.get_device() == dev:
            if t.is_contiguous():
                return t.data_ptr(), heads * d
            s = t.stride()
            if s[2] == 1 and (s[1] == d or heads == 1) and (n == 1 or s[0] >= heads * d):
                return t.data_ptr(), s[0] if n > 1 else heads * d
        self._refuse(name, t, self._dt, (n, heads, d), dev, "row by row ")

    def _token_rows(self, name, t, slot_map, n, dev):
        """Refuses what is not a buffer of a row per token in the place of a cache."""
        rows = self.problem.total_tokens
        if slot_map is not None or n > rows:  # the call writes no row beyond the cache's
            self._refuse(name, t, self._dt, self._kv_shape, dev)
        shape = (n, *self._kv_shape[1:])
        if not _fits(t, self._dt, shape, dev):
            self._refuse(name, t, self._dt, shape, dev)

    def kv4_append(self, k, v, slot_map, kv4, debug=None, stream=None) -> torch.Tensor:
        """Stores tokens k, v [tokens][Hkv][d] into rows slot_map of the 4-bit cache (santa_kv4_append)."""
        h, n, dev = self.problem.num_kv_heads, k.shape[0], k.get_device()
        kp, ks = self._rows("k", k, n, h, dev)
        vp, vs = self._rows("v", v, n, h, dev)
        slots = self._slots(slot_map, n, dev)
        if not _fits(kv4, _U8, self._kv4_shape, dev):
            self._refuse("kv4", kv4, _U8, self._kv4_shape, dev)
        _check("santa_kv4_append", lib().santa_kv4_append(
            self._pref, n, kp, ks, vp, vs, slots, kv4.data_ptr(),
            None if debug is None else ctypes.byref(debug), self._stream(dev, stream)))
        return kv4

    def kv4_read(self, kv4, slot_map, k_out=None, v_out=None, debug=None, stream=None):
        """Rows slot_map of the 4-bit cache as (k, v) [tokens][Hkv][d] (santa_kv4_read)."""
        p, n, dev = self.problem, slot_map.shape[0], kv4.get_device()
        shape = (n, p.num_kv_heads, p.head_dim)
        if not _fits(kv4, _U8, self._kv4_shape, dev):
            self._refuse("kv4", kv4, _U8, self._kv4_shape, dev)
        if k_out is None:
            k_out = torch.empty(shape, dtype=torch.bfloat16 if p.dtype == BF16 else torch.float32, device=dev)
        elif not _fits(k_out, self._dt, shape, dev):
            self._refuse("k_out", k_out, self._dt, shape, dev)
        if v_out is None:
            v_out = torch.empty(shape, dtype=torch.bfloat16 if p.dtype == BF16 else torch.float32, device=dev)
        elif not _fits(v_out, self._dt, shape, dev):
            self._refuse("v_out", v_out, self._dt, shape, dev)
        _check("santa_kv4_read", lib().santa_kv4_read(
            self._pref, n, kv4.data_ptr(), self._slots(slot_map, n, dev), k_out.data_ptr(), v_out.data_ptr(),
            None if debug is None else ctypes.byref(debug), self._stream(dev, stream)))
        return k_out, v_out

    def norm_rope(self, q, k, v, positions, slot_map, cos_sin, k_cache, v_cache, q_weight=None, k_weight=None,
                  eps=1e-6, interleaved=False, out=None, debug=None, stream=None):
        """Norms and rotation of the step's q [tokens][Hq][d] and k [tokens][Hkv][d]; k and v go to rows slot_map
        of the caches (santa_norm_rope).  cos_sin: rope_table.  Returns the rotated queries.  q, or k with
        k_cache, or v with v_cache may be None.  Without a slot map token t goes to row t, and k_cache and v_cache
        may also be [tokens][Hkv][d], with at most total_tokens tokens: the rotated keys by themselves, as
        kv4_append takes them."""
        p, dev = self.problem, positions.get_device()
        n, d = positions.shape[0], p.head_dim
        if not _fits(positions, _I32, (n,), dev):
            self._refuse("positions", positions, _I32, (None,), dev)
        if cos_sin.dim() != 2 or not _fits(cos_sin, _F32, cos_sin.shape, dev):
            self._refuse("cos_sin", cos_sin, _F32, (None, None), dev)
        qp = kp = vp = op = kc = vc = qw = kw = None
        qs = ks = vs = 0
        if q is not None:
            qp, qs = self._rows("q", q, n, p.num_q_heads, dev)
            shape = (n, p.num_q_heads, d)
            if out is None:
                out = torch.empty(shape, dtype=q.dtype, device=dev)
            elif not _fits(out, self._dt, shape, dev):
                self._refuse("out", out, self._dt, shape, dev)
            op = out.data_ptr()
        if k is not None:
            kp, ks = self._rows("k", k, n, p.num_kv_heads, dev)
        if v is not None:
            vp, vs = self._rows("v", v, n, p.num_kv_heads, dev)
        if k_cache is not None:
            if not _fits(k_cache, self._dt, self._kv_shape, dev):
                self._token_rows("k_cache", k_cache, slot_map, n, dev)
            kc = k_cache.data_ptr()
        if v_cache is not None:
            if not _fits(v_cache, self._dt, self._kv_shape, dev):
                self._token_rows("v_cache", v_cache, slot_map, n, dev)
            vc = v_cache.data_ptr()
        if q_weight is not None:
            if not _fits(q_weight, self._dt, (d,), dev):
                self._refuse("q_weight", q_weight, self._dt, (d,), dev)
            qw = q_weight.data_ptr()
        if k_weight is not None:
            if not _fits(k_weight, self._dt, (d,), dev):
                self._refuse("k_weight", k_weight, self._dt, (d,), dev)
            kw = k_weight.data_ptr()
        r = Rope(qw, kw, eps, cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], bool(interleaved))
        _check("santa_norm_rope", lib().santa_norm_rope(
            self._pref, ctypes.byref(r), n, qp, qs, kp, ks, vp, vs, positions.data_ptr(), self._slots(slot_map, n, dev), op,
            kc, vc, None if debug is None else ctypes.byref(debug), self._stream(dev, stream)))
        return out

    def page_plan(self, kv_lens, new_lens, page_table, free_pages, page_size, slot_map, positions, lens_out, counts,
                  debug=None, stream=None) -> None:
        """Pages, cache rows and positions for the step's new tokens (santa_page_plan); page_table is
        updated in place, slot_map, positions, lens_out and counts are written."""
        rows, dev = self.problem.total_tokens, kv_lens.get_device()
        n, tokens, free = kv_lens.numel(), slot_map.numel(), free_pages.numel()
        if page_size < 1 or rows % page_size:
            raise ValueError(f"page_size {page_size} does not divide total_tokens {rows}")
        pages = page_table.shape[-1]
        for name, t, dtypes, shape in (
                ("kv_lens", kv_lens, _I32, (n,)), ("new_lens", new_lens, _I32, (n,)),
                ("page_table", page_table, _I32, (n, pages)), ("free_pages", free_pages, _I32, (free,)),
                ("slot_map", slot_map, _I64, (tokens,)), ("positions", positions, _I32, (tokens,)),
                ("lens_out", lens_out, _I32, (n,)), ("counts", counts, _I32, (2,))):
            if not _fits(t, dtypes, shape, dev):
                self._refuse(name, t, dtypes, shape, dev)
        _check("santa_page_plan", lib().santa_page_plan(
            n, page_size, pages, rows // page_size, kv_lens.data_ptr(), new_lens.data_ptr(), page_table.data_ptr(),
            free_pages.data_ptr(), free, slot_map.data_ptr(), positions.data_ptr(), tokens, lens_out.data_ptr(),
            counts.data_ptr(), None if debug is None else ctypes.byref(debug), self._stream(dev, stream)))
