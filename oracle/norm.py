"""Residual addition, RMS norm and 8-bit quantization of rows (oracle).

    h     = x, or x + residual rounded to their type
    z     = h * weight                         (one float32 rounding)
    s0    = f32(max |z|) / 127 or 448          (float32; per row or 128 channels)
    codes = clamp(rint_half_even(z / s0)), or z / s0 rounded to e4m3; 0 if s0 = 0
    scale = s0 / sqrt(mean(h^2) + eps)         (float64 here)
"""

from __future__ import annotations

import numpy as np

from .rounding import e4m3 as e4m3_grid


def rms_norm_quant(h, weight, eps=1e-6, group=0, e4m3=False):
    """h, weight: float32 values (exact values of the stored type).  Returns
    (codes as float64 values, scales float64 [rows][groups])."""
    h = np.asarray(h, np.float32)
    rows, d = h.shape
    z = np.multiply(h, np.asarray(weight, np.float32), dtype=np.float32)
    z = z.reshape(rows, -1, group or d)
    top = np.float32(448 if e4m3 else 127)
    s0 = np.divide(np.abs(z).max(axis=-1), top, dtype=np.float32)[..., None]
    u = np.divide(z, np.where(s0 == 0, np.float32(1), s0), dtype=np.float32)
    u = np.where(s0 == 0, np.float32(0), u)
    c = e4m3_grid(u) if e4m3 else np.clip(np.rint(u), -127, 127)
    rms = np.sqrt((h.astype(np.float64) ** 2).mean(axis=1) + eps)
    return (np.asarray(c, np.float64).reshape(rows, d),
            s0[..., 0].astype(np.float64) / rms[:, None])
