"""Plain forms of the 8-bit operators for the tests: float32 where an output is compared bit for bit,
float64 where it is compared with a tolerance. CPU, NumPy and torch's number formats only."""
from __future__ import annotations

import numpy as np
import torch

GROUP = 128
FLOOR = np.float32(2.0 ** -100)


def groups_amax(x: np.ndarray, rows: int) -> np.ndarray:
    """Largest magnitude of each rows x 128 block of float32 x (NaN if one is in it)."""
    M, K = x.shape
    R = -(-M // rows)
    pad = np.zeros((R * rows, K), x.dtype)
    pad[:M] = np.abs(x)
    return pad.reshape(R, rows, K // GROUP, GROUP).max(axis=(1, 3))


def quantize(x: np.ndarray, rows: int = 1):
    """(codes as uint8, scales) of float32 x, step by step in float32 as the contract states."""
    with np.errstate(all="ignore"):
        a = np.maximum(groups_amax(x, rows), FLOOR).astype(np.float32)
        inv = np.float32(448.0) / a
        scale = a * (np.float32(1.0) / np.float32(448.0))
        at = np.arange(x.shape[0]) // rows
        y = x * np.repeat(inv[at], GROUP, axis=1)
    return torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), scale


def values(codes: torch.Tensor, scales: torch.Tensor, rows: int) -> np.ndarray:
    """What codes and scales stand for, in float64."""
    c = codes.cpu().to(torch.float32).double().numpy()
    s = scales.cpu().double().numpy()
    at = np.arange(c.shape[0]) // rows
    return c * np.repeat(s[at], GROUP, axis=1)


def rmsnorm(x: np.ndarray, r, w: np.ndarray, eps: float):
    """(h, n) in float64."""
    h = x.astype(np.float64) + (0.0 if r is None else r.astype(np.float64))
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w.astype(np.float64)
