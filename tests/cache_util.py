"""Helpers of the cache operators' GPU tests."""
from __future__ import annotations

import numpy as np
import torch

from paged_fp8_kv_04_gb300 import binding as B


def dev(a, device="cuda"):
    """A numpy array on the device; uint16 arrays are bf16 bits."""
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(a).to(device)


def host(t):
    """Back to numpy; bf16 tensors as their bits."""
    t = t.detach().cpu()
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()


def same(a, b) -> bool:
    """Equal shapes and bytes (NaN payloads and signs of zero included)."""
    x, y = (np.ascontiguousarray(v).view(np.uint8) for v in (a, b))
    return a.dtype == b.dtype and x.shape == y.shape and bool((x == y).all())


def word(device="cuda"):
    return torch.zeros(1, dtype=torch.int32, device=device)


def run_mass(p, lse, mass, decay=1.0, *, out=None, max_q_len=None, status=None, **kw):
    """attn_mass over a synth.Problem; mass a device tensor."""
    scal = {"k_scale_scalar": p.k_scale_scalar} if p.scale_mode == "scalar" else {}
    return B.attn_mass(dev(p.q), dev(p.k_cache), dev(p.block_table), dev(p.context_lens), dev(p.cu_seqlens_q),
                       dev(lse), mass, max_q_len=max_q_len or max(p.max_q_len, 1), sm_scale=p.sm_scale,
                       decay=decay, out=out, k_scale=dev(p.k_scale), status=status, **scal, **kw)
