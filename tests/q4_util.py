"""The 4-bit cache record in numpy, and error bounds, for the tests.

Quantising follows the definition in fp32 IEEE arithmetic (numpy), reading back
is done in float64; nothing here calls the library.
"""
from __future__ import annotations

import numpy as np
import torch

GROUP = 32
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half a step of the type, relative
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}


def record_bytes(D):
    return 16 * (1 + -(-D // GROUP))


def bits_of(x, dtype):
    """float32 values rounded to the 16-bit type, as uint16 patterns."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[dtype]).view(
        torch.int16).numpy().view(np.uint16)


def values_of(bits, dtype):
    """float64 values of uint16 patterns."""
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(
        TORCH[dtype]).double().numpy()


def quantise(bits, dtype):
    """Records uint8 [..., R] of 16-bit rows (uint16 patterns [..., D])."""
    x = values_of(bits, dtype).astype(np.float32)
    D = x.shape[-1]
    G = -(-D // GROUP)
    rec = np.zeros(x.shape[:-1] + (record_bytes(D),), np.uint8)
    for g in range(G):
        xs = x[..., g * GROUP:(g + 1) * GROUP]
        with np.errstate(all="ignore"):
            lo, hi = xs.min(-1), xs.max(-1)  # a NaN propagates
            spread = hi - lo
            ok = np.isfinite(spread)
            s16 = bits_of(np.where(ok, spread / np.float32(15), 0), dtype)
            s = values_of(s16, dtype).astype(np.float32)
            step = np.where(s > 0, s, np.float32(1))
            c = np.minimum(np.rint((xs - lo[..., None]) / step[..., None]), 15)
        c = np.where((ok & (s > 0))[..., None], c, 0).astype(np.uint8)
        c = np.concatenate([c, np.zeros(c.shape[:-1] + (GROUP - c.shape[-1],), np.uint8)], -1)
        rec[..., 16 + 16 * g:32 + 16 * g] = c[..., 0::2] | (c[..., 1::2] << 4)
        m16 = bits_of(np.where(ok, lo, 0), dtype)
        s16 = np.where(ok, s16, 0x7FFF).astype(np.uint16)
        m16 = np.where(ok, m16, 0x7FFF).astype(np.uint16)
        par = np.stack([s16, m16], -1)
        rec[..., 4 * g:4 * g + 4] = par.view(np.uint8).reshape(par.shape[:-1] + (4,))
    return rec


def parts(rec, D, dtype):
    """(scale, minimum [..., G], codes [..., G, 32]) of records, in float64."""
    G = -(-D // GROUP)
    par = np.ascontiguousarray(rec[..., :4 * G]).view(np.uint16)
    par = values_of(par, dtype).reshape(rec.shape[:-1] + (G, 2))
    body = rec[..., 16:16 + 16 * G].astype(np.float64)
    c = np.empty(rec.shape[:-1] + (G * GROUP,))
    c[..., 0::2], c[..., 1::2] = body % 16, body // 16
    return par[..., 0], par[..., 1], c.reshape(rec.shape[:-1] + (G, GROUP))


def dequantise(rec, D, dtype):
    """float64 values [..., D] that records stand for."""
    s, m, c = parts(rec, D, dtype)
    x = c * s[..., None] + m[..., None]
    return x.reshape(rec.shape[:-1] + (-1,))[..., :D]


def half_spans(rec, D, dtype):
    """8 * scale of each value's group, [..., D]: how far a value is from the
    middle of its group's range, at most."""
    s, _, _ = parts(rec, D, dtype)
    return np.repeat(8.0 * s, GROUP, -1)[..., :D]


def random_rows(rng, shape, dtype, keys=False):
    """uint16 patterns of normal rows [B, H, S, D]; keys get channel offsets."""
    x = rng.standard_normal(shape).astype(np.float32)
    if keys:
        x += rng.standard_normal((1, shape[1], 1, shape[3])).astype(np.float32)
    return bits_of(x, dtype)


def dev16(bits, dtype):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(TORCH[dtype]).cuda()


def to64(t):
    return t.double().cpu().numpy()


def paged(rec, page_size, rng, spare=2, fill=0xFF):
    """(pool, block table) of records [B, H, S, R]; unused rows and pages hold
    ``fill`` (0xFF: NaN scales)."""
    B, H, S, R = rec.shape
    per = -(-S // page_size)
    pool = np.full((B * per + spare, H, page_size, R), fill, np.uint8)
    table = rng.permutation(B * per + spare)[:B * per].reshape(B, per).astype(np.int32)
    for b in range(B):
        for i in range(per):
            part = rec[b, :, i * page_size:(i + 1) * page_size]
            pool[table[b, i], :, :part.shape[1]] = part
    return pool, table
