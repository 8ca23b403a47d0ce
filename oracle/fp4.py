"""Microscaled 4-bit floating point by its definition: e2m1 codes (OCP
Microscaling Formats, table of FP4), NVFP4 blocks of 16 with e4m3 scales under an
fp32 one, MXFP4 blocks of 32 with e8m0 scales.  numpy fp32, step by step, so codes
and scales can be compared bit for bit."""
import numpy as np

from .moe_oracle import e4m3_decode, e4m3_encode

__all__ = ["E2M1", "FP4_BLOCKS", "e2m1_encode", "fp4_quantize", "fp4_decode", "fp4_scale_values"]

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)
FP4_BLOCKS = {"nvfp4": 16, "mxfp4": 32}


def e2m1_encode(v: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even one, beyond 6 to 6 (NaN as well)."""
    a = np.abs(np.asarray(v, np.float64))
    a = np.where(np.isnan(a), 6.0, np.minimum(a, 6.0))
    d = np.abs(a[..., None] - E2M1.astype(np.float64))
    best = d.min(axis=-1, keepdims=True)
    even = np.where(d == best, np.arange(8) % 2, 2)   # among the nearest, even before odd
    code = np.argmin(even, axis=-1).astype(np.uint8)
    return code | (np.signbit(v).astype(np.uint8) << 3)


def fp4_quantize(x: np.ndarray, fmt: str, g=None):
    """fp32 [rows, H] to (codes [rows, H / 2], scales [rows, H / block]) uint8; g: a number
    or [rows] fp32."""
    x = np.asarray(x, np.float32)
    n = FP4_BLOCKS[fmt]
    b = x.reshape(x.shape[0], -1, n)
    with np.errstate(all="ignore"):
        amax = np.max(np.abs(b), axis=2)
        amax = np.where(np.isnan(b).any(axis=2), np.float32(np.nan), amax)
        bad = ~np.isfinite(amax)
        if fmt == "nvfp4":
            g = np.broadcast_to(np.float32(1.0) if g is None else np.asarray(g, np.float32), (x.shape[0],))[:, None]
            some = ~bad & (amax != 0)   # a block of zeros has scale 0, whatever g is
            t = np.where(some, amax, np.float32(0)) / np.where(some, np.float32(6.0) * g, np.float32(1))
            scale = e4m3_encode(np.minimum(t, np.float32(448.0)))
            s = e4m3_decode(scale).astype(np.float32)
            r = np.where(s > 0, np.float32(1.0) / (s * g), np.float32(0))
            scale = np.where(bad, 0x7F, scale).astype(np.uint8)
        else:
            e = (np.where(bad, np.float32(0), amax).view(np.uint32) >> 23).astype(np.int64) - 2
            e = np.maximum(e, 0)
            r = np.ldexp(np.float32(1.0), (127 - e).astype(np.int32)).astype(np.float32)
            scale = np.where(bad, 0xFF, e).astype(np.uint8)
        r = np.where(bad, np.float32(0), r).astype(np.float32)
        c = e2m1_encode(b * r[..., None]).reshape(x.shape)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), scale


def fp4_scale_values(scales: np.ndarray, fmt: str) -> np.ndarray:
    """Block scales as float64."""
    if fmt == "nvfp4":
        return e4m3_decode(scales).astype(np.float64)
    return np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))


def fp4_decode(codes: np.ndarray, scales: np.ndarray, fmt: str) -> np.ndarray:
    """Codes [..., H / 2] and scales [..., H / block] to float64 values [..., H]."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * E2M1.astype(np.float64)[c & 7]
    return v * np.repeat(fp4_scale_values(scales, fmt), FP4_BLOCKS[fmt], axis=-1)
