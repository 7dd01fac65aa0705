"""B200-native (sm_100a) Gated DeltaNet token mixer.

The compute runs in ``libgdn.so`` (hand-written CUDA, C ABI in ``include/gdn.h``); this
package marshals torch tensors into it. The library is loaded on first use and a missing
library raises -- there is no fallback.

Entry points (same names as the C ABI): ``gdn_conv1d_silu``, ``gdn_chunk_prefill`` (states at
block boundaries on request), ``gdn_chunk_prefill_workspace_size``,
``gdn_chunk_prefill_noalloc``, ``gdn_decode_step`` and ``gdn_decode_tokens`` (fp32 or bf16
states, taken from the state tensor); ``prefill_layer`` chains the conv and the chunked
prefill over one packed batch without copies.

For servers that keep states in pages of a pool: ``gdn_decode_paged`` reads and writes pages,
``gdn_pages_copy`` / ``_fork`` / ``_compact`` move them, ``gdn_pages_take`` / ``_ref`` /
``_plan`` keep their counts. Around the block: ``gdn_gated_norm`` (the norm and gate of the
mixer's output) and ``gdn_add_norm`` (residual add and norm), each with its ``_bwd``.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._lib import (GDNError, LIB_PATH, gdn_chunk_prefill, gdn_chunk_prefill_noalloc,
                   gdn_chunk_prefill_path, gdn_chunk_prefill_launches, gdn_chunk_prefill_workspace_size, gdn_conv1d_silu, gdn_decode_step,
                   gdn_decode_tokens, gdn_prefill_noalloc_status, gdn_prefill_status, lib,
                   gdn_decode_paged, gdn_pages_copy, gdn_pages_take, gdn_pages_ref, gdn_pages_fork,
                   gdn_pages_plan, gdn_pages_compact, gdn_gated_norm, gdn_gated_norm_bwd, gdn_add_norm,
                   gdn_add_norm_bwd, gdn_norm_bwd_workspace_size, _check_gate)

__all__ = ["GDNError", "LIB_PATH", "lib", "gdn_conv1d_silu", "gdn_chunk_prefill",
           "gdn_chunk_prefill_workspace_size", "gdn_chunk_prefill_noalloc", "gdn_chunk_prefill_path", "gdn_chunk_prefill_launches", "gdn_decode_step",
           "gdn_decode_tokens", "gdn_prefill_status", "gdn_prefill_noalloc_status",
           "gdn_decode_paged", "gdn_pages_copy", "gdn_pages_take", "gdn_pages_ref", "gdn_pages_fork",
           "gdn_pages_plan", "gdn_pages_compact", "gdn_gated_norm", "gdn_gated_norm_bwd", "gdn_add_norm",
           "gdn_add_norm_bwd", "gdn_norm_bwd_workspace_size", "prefill_layer", "qkv_views"]


def qkv_views(y: torch.Tensor, Hk: int, Hv: int, d: int):
    """q, k, v as strided views of a conv output y [T, Cc] in channel order
    [q: Hk*d | k: Hk*d | v: Hv*d] (no copy)."""
    T, Cc = y.shape
    q = y.as_strided((T, Hk, d), (Cc, d, 1), y.storage_offset())
    k = y.as_strided((T, Hk, d), (Cc, d, 1), y.storage_offset() + Hk * d)
    v = y.as_strided((T, Hv, d), (Cc, d, 1), y.storage_offset() + 2 * Hk * d)
    return q, k, v


def prefill_layer(x: torch.Tensor, conv_w: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  Hk: int, Hv: int, d: int, cu_seqlens: Optional[torch.Tensor] = None,
                  initial_state: Optional[torch.Tensor] = None,
                  conv_state_in: Optional[torch.Tensor] = None,
                  final_state: Optional[torch.Tensor] = None,
                  conv_state_out: Optional[torch.Tensor] = None, scale: float = 1.0,
                  y: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                  norm_w: Optional[torch.Tensor] = None, eps: float = 1e-6) -> torch.Tensor:
    """The mixer core over one packed batch: conv + SiLU, then the chunked gated delta
    rule with q/k L2 norm. Returns o [T, Hv, d]; fills final_state / conv_state_out when
    given. With the gate z [T, Hv, d] and norm_w [d], o is normalised and gated in place
    (``gdn_gated_norm``), as ``gdn_decode_paged`` does for single tokens."""
    if (z is None) != (norm_w is None):
        raise ValueError("z and norm_w come together")
    if z is not None:                # before the states and taps advance
        if o is None:
            o = torch.empty((x.shape[0], Hv, d), dtype=x.dtype, device=x.device)
        _check_gate(o, z, norm_w, eps)
    y = gdn_conv1d_silu(x, conv_w, cu_seqlens, conv_state_in, conv_state_out, y)
    q, k, v = qkv_views(y, Hk, Hv, d)
    o = gdn_chunk_prefill(q, k, v, g, beta, cu_seqlens, initial_state, final_state, scale,
                          True, o, workspace)
    return o if z is None else gdn_gated_norm(o, z, norm_w, eps, y=o)
