"""Plain 64-bit forms of the 4-bit cache and of the norm and rotation step."""
import numpy as np
import torch


def kv4_values(codes, params):
    """float64 [..., d] values of code rows [..., d / 2] uint8 and parameters [..., d / 32, 2]:
    channel c has nibble c % 4 of 16-bit word (c % 32) // 4 * (d // 32) + c // 32."""
    codes, params = codes.cpu().numpy(), params.cpu().double().numpy()
    d = 2 * codes.shape[-1]
    words = codes[..., 0::2].astype(np.int64) | codes[..., 1::2].astype(np.int64) << 8
    out = np.empty((*codes.shape[:-1], d))
    for c in range(d):
        n = words[..., c % 32 // 4 * (d // 32) + c // 32] >> 4 * (c % 4) & 15
        out[..., c] = params[..., c // 32, 1] + params[..., c // 32, 0] * n
    return out


def kv4_quantised(x):
    """float64 values that rows x [..., d] are stored as (NaN for a group with a NaN)."""
    x = x.cpu().double().numpy()
    out = np.empty_like(x)
    with np.errstate(all="ignore"):
        for c in range(0, x.shape[-1], 32):
            g = x[..., c:c + 32]
            lo, hi = (np.clip(f(g, -1, keepdims=True), -60000, 60000) for f in (np.min, np.max))
            m = lo.astype(np.float16).astype(np.float64)
            s = ((hi - m) / 15).astype(np.float32).astype(np.float16).astype(np.float64)
            n = np.where(s > 0, np.clip(np.rint((g - m) / s), 0, 15), np.where(np.isnan(m), np.nan, 0))
            out[..., c:c + 32] = m + s * n
    return out


def rope_forward(x, w, cos, sin, pos, axes, interleaved, eps):
    """float64 rows [B, N, H, d] normed (w not None) and rotated; differentiable."""
    half = cos.shape[1]
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w
    pos = pos.long().view(*pos.shape[:2], -1)
    i = torch.arange(half)
    at = pos[..., torch.tensor(axes, dtype=torch.long)] if half else pos[..., :0]
    c, s = cos.double()[at, i][:, :, None], sin.double()[at, i][:, :, None]
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
    a, b = x[..., a_at], x[..., b_at]
    z = x.clone()
    z[..., a_at], z[..., b_at] = a * c - b * s, b * c + a * s
    return z
