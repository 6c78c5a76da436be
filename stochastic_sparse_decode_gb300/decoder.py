"""A convenience wrapper: owns the problem description and the workspaces.

    dec = Decoder(batch=1, num_q_heads=32, num_kv_heads=8, head_dim=128,
                  total_tokens=32768, max_len=32768, tile=256, S=128, dtype="bf16")
    out = dec("prop", q, k, v, kv_indptr, U)

Workspaces are allocated once per mode with torch (device memory only); each
call is one C-ABI call on the current stream.  Debug buffers can be requested
to inspect tile records, budgets and sampled indices.
"""

from __future__ import annotations

import torch

from . import (BF16, MODES, Debug, Rope, Window, decode, k_feature_blocked_size, kv4_size, make_pages, make_problem,
               santa_decode_kv4, santa_decode_prop_bernoulli, santa_decode_prop_paged, santa_decode_window,
               santa_k_feature_blocked, santa_kv4_append, santa_kv4_read, santa_norm_rope, santa_page_plan,
               santa_prop_pass1, santa_prop_pass2, split_workspace_size, workspace_size)


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

    def _dtypes(self):
        # bf16 may come as its bit pattern, as for the other modes
        return (torch.bfloat16, torch.int16, torch.uint16) if self.problem.dtype == BF16 else (torch.float32,)

    def _tensor(self, name, t, dtypes, *shape, rows=False, like=None):
        """Refuses a tensor that the C call would misread: dtype, shape (None: any size), layout
        (`rows`: [tokens][heads][d] whose tokens may lie apart), device."""
        if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
            raise ValueError(f"{name}: a tensor of {' or '.join(map(str, dtypes))} is needed")
        if len(t.shape) != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, needed {shape}")
        if not (t.is_contiguous() or (rows and (t.shape[0] == 0 or t[0].is_contiguous()))):
            raise ValueError(f"{name}: not contiguous")
        if t.device.type != "cuda" or t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name}: on {t.device}, not on the current CUDA device")
        return t

    def _out(self, out):
        p = self.problem
        if out is None:
            return torch.empty((p.batch, p.num_q_heads, p.head_dim), dtype=torch.float32,
                               device=torch.device("cuda", torch.cuda.current_device()))
        return self._tensor("out", out, (torch.float32,), p.batch, p.num_q_heads, p.head_dim)

    def split_workspace(self) -> torch.Tensor:
        """The workspace of window and kv4 calls (kept; calls that overlap need a Decoder each)."""
        if "split" not in self._ws:
            # zero-filled: what santa_split_workspace_init does
            self._ws["split"] = torch.zeros(split_workspace_size(self.problem), dtype=torch.uint8, device=self.device)
        return self._ws["split"]

    def _cache(self, name, t):
        p = self.problem
        return self._tensor(name, t, self._dtypes(), p.total_tokens, p.num_kv_heads, p.head_dim)

    def _kv4_cache(self, t):
        p = self.problem
        return self._tensor("kv4", t, (torch.uint8,), p.total_tokens, p.num_kv_heads, p.head_dim + p.head_dim // 8)

    def _query(self, q):
        p = self.problem
        return self._tensor("q", q, self._dtypes(), p.batch, p.num_q_heads, p.head_dim)

    def _indptr(self, t):
        return self._tensor("kv_indptr", t, (torch.int64,), self.problem.batch + 1)

    def _pages(self, page_table, kv_lens, page_size):
        p = self.problem
        self._tensor("page_table", page_table, (torch.int32,), p.batch, None)
        self._tensor("kv_lens", kv_lens, (torch.int32,), p.batch)
        if page_size < 1 or p.total_tokens % page_size:
            raise ValueError(f"page_size {page_size} does not divide total_tokens {p.total_tokens}")
        return make_pages(page_table, kv_lens, page_size, p.total_tokens // page_size)

    def window(self, q, k, v, kv_indptr, window, sinks=0, out=None, debug=None, stream=None) -> torch.Tensor:
        """Exact decode over the last `window` keys and the first `sinks` (santa_decode_window); window 0: all."""
        out = self._out(out)
        santa_decode_window(self.problem, Window(window, sinks), self._query(q), self._cache("k", k),
                            self._cache("v", v), self._indptr(kv_indptr), out, self.split_workspace(), None, debug,
                            stream)
        return out

    def window_paged(self, q, k_pool, v_pool, page_table, kv_lens, page_size, window, sinks=0, out=None, debug=None,
                     stream=None) -> torch.Tensor:
        """The same on a paged cache; total_tokens must be the pools' rows, num_pages * page_size."""
        out = self._out(out)
        santa_decode_window(self.problem, Window(window, sinks), self._query(q), self._cache("k_pool", k_pool),
                            self._cache("v_pool", v_pool), None, out, self.split_workspace(),
                            self._pages(page_table, kv_lens, page_size), debug, stream)
        return out

    def kv4_cache(self) -> torch.Tensor:
        """An empty 4-bit cache for the problem's total_tokens: [rows][Hkv][d + d / 8] bytes."""
        p = self.problem
        kv4_size(p)  # checks the problem
        return torch.zeros((p.total_tokens, p.num_kv_heads, p.head_dim + p.head_dim // 8), dtype=torch.uint8,
                           device=self.device)

    def _slots(self, slot_map, n):
        return None if slot_map is None else self._tensor("slot_map", slot_map, (torch.int64,), n)

    def kv4_append(self, k, v, slot_map, kv4, debug=None, stream=None) -> torch.Tensor:
        """Stores tokens k, v [tokens][Hkv][d] into rows slot_map of the 4-bit cache (santa_kv4_append)."""
        p = self.problem
        self._tensor("k", k, self._dtypes(), None, p.num_kv_heads, p.head_dim, rows=True)
        self._tensor("v", v, self._dtypes(), k.shape[0], p.num_kv_heads, p.head_dim, rows=True)
        santa_kv4_append(p, k, v, self._slots(slot_map, k.shape[0]), self._kv4_cache(kv4), debug, stream)
        return kv4

    def kv4_read(self, kv4, slot_map, k_out=None, v_out=None, debug=None, stream=None):
        """Rows slot_map of the 4-bit cache as (k, v) [tokens][Hkv][d] (santa_kv4_read)."""
        p, n = self.problem, slot_map.shape[0]
        self._kv4_cache(kv4)
        k_out, v_out = (torch.empty((n, p.num_kv_heads, p.head_dim), dtype=self._dtypes()[0], device=kv4.device)
                        if t is None else self._tensor(name, t, self._dtypes(), n, p.num_kv_heads, p.head_dim)
                        for name, t in (("k_out", k_out), ("v_out", v_out)))
        santa_kv4_read(p, n, kv4, self._slots(slot_map, n), k_out, v_out, debug, stream)
        return k_out, v_out

    def kv4(self, q, kv4, kv_indptr, window=0, sinks=0, out=None, debug=None, stream=None) -> torch.Tensor:
        """Exact decode over the 4-bit cache (santa_decode_kv4)."""
        out = self._out(out)
        santa_decode_kv4(self.problem, Window(window, sinks), self._query(q), self._kv4_cache(kv4),
                         self._indptr(kv_indptr), out, self.split_workspace(), None, debug, stream)
        return out

    def kv4_paged(self, q, kv4, page_table, kv_lens, page_size, window=0, sinks=0, out=None, debug=None,
                  stream=None) -> torch.Tensor:
        """The same on a paged 4-bit cache."""
        out = self._out(out)
        santa_decode_kv4(self.problem, Window(window, sinks), self._query(q), self._kv4_cache(kv4), None, out,
                         self.split_workspace(), self._pages(page_table, kv_lens, page_size), debug, stream)
        return out

    def norm_rope(self, q, k, v, positions, slot_map, cos_sin, k_cache, v_cache, q_weight=None, k_weight=None,
                  eps=1e-6, interleaved=False, out=None, debug=None, stream=None):
        """Norms and rotation of the step's q [tokens][Hq][d] and k [tokens][Hkv][d]; k and v go to rows slot_map
        of the caches (santa_norm_rope).  cos_sin: rope_table.  Returns the rotated queries.  q, or k with
        k_cache, or v with v_cache may be None."""
        p, dt = self.problem, self._dtypes()
        n = next((t.shape[0] for t in (q, k, v) if t is not None), 0)
        for name, t, heads in (("q", q, p.num_q_heads), ("k", k, p.num_kv_heads), ("v", v, p.num_kv_heads)):
            if t is not None:
                self._tensor(name, t, dt, n, heads, p.head_dim, rows=True)
        for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
            if t is not None:
                self._tensor(name, t, dt, p.head_dim)
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t is not None:
                self._cache(name, t)
        self._tensor("positions", positions, (torch.int32,), n)
        self._tensor("cos_sin", cos_sin, (torch.float32,), None, None)
        if q is not None:
            if out is None:
                out = torch.empty((n, p.num_q_heads, p.head_dim), dtype=q.dtype, device=q.device)
            self._tensor("out", out, dt, n, p.num_q_heads, p.head_dim)
        r = Rope(None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
                 eps, cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], int(interleaved))
        santa_norm_rope(p, r, q, k, v, positions, self._slots(slot_map, n), out if q is not None else None, k_cache,
                        v_cache, debug, stream)
        return out

    def page_plan(self, kv_lens, new_lens, page_table, free_pages, page_size, slot_map, positions, lens_out, counts,
                  debug=None, stream=None) -> None:
        """Pages, cache rows and positions for the step's new tokens (santa_page_plan); page_table is
        updated in place, slot_map, positions, lens_out and counts are written."""
        p, i32 = self.problem, (torch.int32,)
        self._tensor("kv_lens", kv_lens, i32, None)
        n = kv_lens.shape[0]
        self._tensor("new_lens", new_lens, i32, n)
        self._tensor("page_table", page_table, i32, n, None)
        self._tensor("free_pages", free_pages, i32, None)
        self._tensor("slot_map", slot_map, (torch.int64,), None)
        self._tensor("positions", positions, i32, slot_map.shape[0])
        self._tensor("lens_out", lens_out, i32, n)
        self._tensor("counts", counts, i32, 2)
        if page_size < 1 or p.total_tokens % page_size:
            raise ValueError(f"page_size {page_size} does not divide total_tokens {p.total_tokens}")
        santa_page_plan(page_size, p.total_tokens // page_size, kv_lens, new_lens, page_table, free_pages, slot_map,
                        positions, lens_out, counts, debug, stream)
