"""Plain reference of rotary_and_cache: rotation and cache rows from the
definitions, each product, sum and quotient the exact one (64 bits) rounded to
32 bits, codes by a search of the format's values or by rounding."""
import numpy as np
import torch

QMAX = {"int8_per_token_head": 127.0, "fp8_per_token_head": 448.0, "fp8_e5m2_per_token_head": 57344.0}


def r32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def cos_sin_table(positions: int, rotary: int, base: float = 10000.0):
    half = rotary // 2
    a = np.arange(positions, dtype=np.float64)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(a), np.sin(a)], -1).astype(np.float32)


def rotate(x, table, positions, interleaved):
    """x float64 [T, H, D] (fp32 values) -> float64 (fp32 values)."""
    rotary = table.shape[1]
    half = rotary // 2
    row = table[positions].astype(np.float64)[:, None, :]
    c, s = row[..., :half], row[..., half:]
    out = np.array(x, np.float64)
    a, b = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, half), slice(half, rotary))
    out[..., a] = r32(r32(x[..., a] * c) - r32(x[..., b] * s))
    out[..., b] = r32(r32(x[..., b] * c) + r32(x[..., a] * s))
    return out


def _fp8(y, e5m2):
    """Codes of y (float64 holding fp32 values): the OCP formats through
    torch's CPU cast (round to nearest even), saturating."""
    top = 57344.0 if e5m2 else 448.0
    t = torch.from_numpy(np.clip(y, -top, top).astype(np.float32))
    return t.to(torch.float8_e5m2 if e5m2 else torch.float8_e4m3fn).view(torch.uint8).numpy()


def bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy()


def rows(dtype, x, scale):
    """x float64 [..., D] (fp32 values) -> uint8 cache rows."""
    D = x.shape[-1]
    if dtype == "auto":
        return bf16_bits(x).view(np.uint8).reshape(*x.shape[:-1], 2 * D)
    if dtype in ("fp8_e4m3", "fp8_e5m2"):
        return _fp8(r32(x / np.float64(np.float32(scale))), dtype == "fp8_e5m2")
    amax = np.abs(x).max(-1, keepdims=True)
    pad = np.zeros((*x.shape[:-1], 12), np.uint8)
    with np.errstate(divide="ignore", invalid="ignore"):
        if dtype in QMAX:
            s = r32(amax / QMAX[dtype])
            y = np.where(s > 0, r32(x / s), 0.0)
            if dtype == "int8_per_token_head":
                codes = np.clip(np.rint(y), -128, 127).astype(np.int8).view(np.uint8)
            else:
                codes = _fp8(y, "e5m2" in dtype)
                codes = np.where(s > 0, codes, 0).astype(np.uint8)
            return np.concatenate([codes, s.astype(np.float32).view(np.uint8).reshape(*x.shape[:-1], 4), pad], -1)
        s = r32(amax / 889.0)
        g = x.reshape(*x.shape[:-1], 8, D // 8)
        m = np.where(s > 0, np.minimum(127.0, np.ceil(r32(r32(np.abs(g).max(-1) / s) / 7.0))), 0.0)
        step = r32(s * m)[..., None]
        code = np.where(step > 0, np.clip(np.rint(r32(g / step)), -7, 7), 0.0) + 8
    n = code.astype(np.uint32).reshape(*x.shape[:-1], D // 8, 8)
    w = np.zeros(n.shape[:-1], np.uint32)
    for i in range(8):  # dim 2 j in nibble j, dim 2 j + 1 in nibble j + 4
        w |= n[..., i] << np.uint32(4 * (i // 2 + 4 * (i % 2)))
    return np.concatenate([w.view(np.uint8).reshape(*x.shape[:-1], D // 2),
                           s.astype(np.float32).view(np.uint8).reshape(*x.shape[:-1], 4),
                           m.astype(np.uint8), pad[..., :4]], -1)
