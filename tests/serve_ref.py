"""64-bit references of the serving operators (numpy / torch on the CPU),
written from the formulas in include/dsa_index.h."""

from __future__ import annotations

import numpy as np
import torch

LAT, ROPE, ENTRY = 512, 64, 416
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_table() -> np.ndarray:
    """Value of each E4M3 code from its definition: sign, 4 exponent bits
    (bias 7, subnormal steps of 2^-9), 3 mantissa bits; 0x7F and 0xFF NaN."""
    c = np.arange(256)
    ex, man = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (1 + man / 8.0) * 2.0 ** (ex.astype(float) - 7))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


E4M3 = e4m3_table()


def nearest_even(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the grid value nearest to x >= 0 (ties to the even index, saturating)."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def kv4_encode(latent: np.ndarray, rope_bits: np.ndarray) -> np.ndarray:
    """Cache entries (T, 416) uint8 of fp64 latent rows and rotary bf16 bits."""
    T = latent.shape[0]
    x = latent.reshape(T, 32, 16)
    sc = nearest_even(np.abs(x).max(-1) / 6.0, E4M3[:127])
    sv = E4M3[sc][..., None]
    y = np.divide(x, sv, out=np.zeros_like(x), where=sv > 0)
    code = nearest_even(np.abs(y), E2M1) + 8 * (np.signbit(y))
    code = code.reshape(T, 256, 2)
    packed = (code[..., 0] | (code[..., 1] << 4)).astype(np.uint8)
    return np.concatenate([packed, sc.astype(np.uint8), rope_bits.astype(np.uint16).view(np.uint8).reshape(T, 128)], 1)


def kv4_decode(entries: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """fp64 (latent, rope) of entries (..., 416) uint8."""
    by = entries[..., :256]
    code = np.stack([by & 15, by >> 4], -1).reshape(*entries.shape[:-1], LAT)
    val = E2M1[code & 7] * np.where(code >= 8, -1.0, 1.0)
    val = (val.reshape(*entries.shape[:-1], 32, 16) * E4M3[entries[..., 256:288]][..., None]).reshape(code.shape)
    bits = np.ascontiguousarray(entries[..., 288:]).view(np.uint16).astype(np.uint32) << 16
    return val, bits.view(np.float32).astype(np.float64)


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """bf16 bit patterns (RNE) of fp64/fp32 numbers."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


def bf16_f64(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def attend(q, entries, table, page, row_seq, idx, scale):
    """fp64 attention: q (T,H,576), entries (n_slots, 416) uint8.  Returns
    (out, lse, weighted |latent| (T,H,512), bound on |q||k| per (T,H), sum of
    |latent| over the list (T,512))."""
    T, H, _ = q.shape
    out = np.zeros((T, H, LAT))
    lse = np.full((T, H), -np.inf)
    wabs = np.zeros((T, H, LAT))
    mag = np.zeros((T, H))
    vsum = np.zeros((T, LAT))
    for t in range(T):
        if row_seq[t] < 0:
            continue
        pos = idx[t][idx[t] >= 0].astype(np.int64)
        pos = pos[pos // page < table.shape[1]]
        if len(pos) == 0:
            continue
        pages = table[row_seq[t]][pos // page].astype(np.int64)
        ok = (pages >= 0) & (pages * page < entries.shape[0])
        slots = (pages * page + pos % page)[ok]
        if len(slots) == 0:
            continue
        lat, rope = kv4_decode(entries[slots])
        key = np.concatenate([lat, rope], 1)
        z = scale * (q[t] @ key.T)
        mag[t] = abs(scale) * (np.abs(q[t]) @ np.abs(key).T).max(-1)
        m = z.max(-1, keepdims=True)
        p = np.exp(z - m)
        s = p.sum(-1, keepdims=True)
        out[t] = (p / s) @ lat
        wabs[t] = (p / s) @ np.abs(lat)
        vsum[t] = np.abs(lat).sum(0)
        lse[t] = (m + np.log(s))[:, 0]
    return out, lse, wabs, mag, vsum


def check_attend(got_out, got_lse, ref, label=""):
    """out and lse against the fp64 reference.

    A score is a sum of 576 products (exact in fp32: 8 x 6 or 8 x 8 significant
    bits), accumulated in fp32: its error is at most dz = 2^-14 * scale *
    sum|q||k| (576 + 36 roundings of at most 2^-23 each).  exp(z) is then off
    by a factor exp(+-dz), the weights by a factor within 2 dz (numerator and
    sum), plus their own rounding to 16 bits (2^-11 in fp16, once in the
    product with the latents) and 2^-11 for exp2, fp32 sums and the quotient
    together; all weigh |latent|.  Weights that small end in fp16's subnormals:
    below 2^-14 of the reference that they are taken to, a weight is off by up
    to half a subnormal step, 2^-25, of a sum that is at least 1 (the largest
    entry's weight, the reference being at most the maximum), so the output by
    at most 2^-25 sum_j |latent_j|.  The output rounds once to bf16: 2^-8, or
    half a subnormal step, 2^-134.
    """
    out, lse, wabs, mag, vsum = ref
    dz = 2.0 ** -14 * mag
    tol = 2.0 ** -8 * np.abs(out) + (wabs * (2.0 ** -10 + 2 * dz)[..., None] + 2.0 ** -25 * vsum[:, None]) * (1 + 2.0 ** -8)
    tol += 2.0 ** -134
    err = np.abs(got_out - out)
    assert np.isfinite(got_out).all(), label
    assert (err <= tol).all(), f"{label}: out off by {(err - tol).max()} beyond its bound"
    fin = np.isfinite(lse)
    assert (np.isfinite(got_lse) == fin).all() and (got_lse[~fin] == -np.inf).all(), label
    err = np.abs(got_lse[fin] - lse[fin])
    assert (err <= dz[fin] + 2.0 ** -20 * np.maximum(1, np.abs(lse[fin]))).all(), f"{label}: lse off by {err.max()}"


def norm_rotate(x, position, inv_freq, norm, weight, bias, eps, interleaved):
    """fp64 rows (T, heads, 128) of the index preparation."""
    x = x.astype(np.float64)
    if norm == "layer":
        x = x - x.mean(-1, keepdims=True)
    if norm != "none":
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        x = x * (1.0 if weight is None else weight.astype(np.float64)) + (0.0 if bias is None else bias.astype(np.float64))
    rot = 2 * len(inv_freq)
    ang = position.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y = x.copy()
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i0] * s + x[..., i1] * c
    return y


def block_tables(cached, new, table, free, begin, n_pages, page, T_cap):
    """The layout by a loop over requests; returns (slot, pos, owner, start,
    seq, end, table, status bit 1)."""
    B, max_blocks = table.shape
    table = table.copy()
    slot, pos, owner = (np.full(T_cap, -1, np.int32) for _ in range(3))
    cached, new = cached.astype(np.int64), new.astype(np.int64)
    bad = (cached < 0).any() or (new < 0).any() or (cached + new > max_blocks * page).any() or begin < 0
    if not bad:
        need = (-(-(cached + new) // page) - -(-cached // page)).sum()
        bad = new.sum() > T_cap or begin + need > len(free)
    if bad:
        return slot, pos, owner, np.zeros(B + 1, np.int32), cached.astype(np.int32), begin, table, True
    start, r, flag = [0], 0, False
    for b in range(B):
        c, m = int(cached[b]), int(new[b])
        for blk in range(-(-c // page), -(-(c + m) // page)):
            table[b, blk] = free[begin]
            begin += 1
        for i in range(c, c + m):
            pg = int(table[b, i // page])
            pos[r], owner[r] = i, b
            if 0 <= pg < n_pages:
                slot[r] = pg * page + i % page
            else:
                flag = True
            r += 1
        start.append(r)
    return slot, pos, owner, np.array(start, np.int32), (cached + new).astype(np.int32), begin, table, flag
