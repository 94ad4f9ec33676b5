"""Float64 CPU reference of the serving operators: rotary positions, the 4-bit cache's
definition and attention over it.  Plain numpy, written from the formulas; it shares nothing
with the CUDA path.  Test infrastructure only."""
import numpy as np

GROUP, BLOCK = 64, 16


def frequencies(r, base, alpha=None, scaling="none", factor=1.0, orig_len=0.0, slow=1.0,
                fast=32.0, fixed_bands=0):
    M = r // 2
    t = base ** (-2.0 * np.arange(M) / r)
    if scaling == "linear":
        t = t / factor
    elif scaling == "parts":
        g = np.clip((orig_len * t / (2 * np.pi) - slow) / (fast - slow), 0.0, 1.0)
        t = (1 - g) * t / factor + g * t
    if alpha is not None:
        t = t * np.exp(np.asarray(alpha, np.float64))
    if fixed_bands:
        t[M - fixed_bands:] = 0.0
    return t


def pairs(r, layout):
    """Channel numbers (first, second) of every band."""
    m = np.arange(r // 2)
    return (2 * m, 2 * m + 1) if layout == "interleaved" else (m, m + r // 2)


def rotate(x, pos, theta, layout, amplitude=1.0, sign=1.0):
    """x [..., d] float64; pos broadcasts against x[..., 0]."""
    x = np.array(x, np.float64)
    a, b = pairs(2 * len(theta), layout)
    phi = sign * np.asarray(pos, np.float64)[..., None] * theta
    c, s = amplitude * np.cos(phi), amplitude * np.sin(phi)
    y = x.copy()
    y[..., a] = c * x[..., a] - s * x[..., b]
    y[..., b] = s * x[..., a] + c * x[..., b]
    return y


def rotary_dalpha(x, dy, pos, theta, layout, amplitude=1.0):
    """theta_m sum p <dx_m, J x_m> and the same sum of absolute values (for tolerances)."""
    dx = rotate(dy, pos, theta, layout, amplitude, -1.0)
    a, b = pairs(2 * len(theta), layout)
    w = dx[..., b] * x[..., a] - dx[..., a] * x[..., b]
    size = (abs(dx[..., b]) + abs(dx[..., a])) * (abs(x[..., a]) + abs(x[..., b]))
    p = np.broadcast_to(np.asarray(pos, np.float64)[..., None], w.shape)
    ax = tuple(range(w.ndim - 1))
    return theta * (p * w).sum(ax), abs(theta) * (abs(p) * size).sum(ax)


def quantise(x):
    """codes [..., d] uint8, step and lo [..., d/64] float16 of x (float32), as defined: fp32
    arithmetic, every operation rounded."""
    x = np.asarray(x, np.float32)
    y = x.reshape(x.shape[:-1] + (-1, GROUP))
    lo = y.min(-1).astype(np.float16)
    lo32 = lo.astype(np.float32)
    step = np.maximum((y.max(-1) - lo32) * np.float32(1.0 / 15.0), np.float32(0)).astype(np.float16)
    s32 = step.astype(np.float32)
    inv = np.where(s32 > 0, np.float32(1) / np.where(s32 > 0, s32, np.float32(1)), np.float32(0))
    code = np.rint((y - lo32[..., None]) * inv[..., None].astype(np.float32))
    return np.clip(code, 0, 15).astype(np.uint8).reshape(x.shape), step, lo


def block_bytes(d):
    return 2 * BLOCK * (d // 2 + 4 * (d // GROUP))


def pack_block(part, row, codes, step, lo, d):
    """Write one token's codes and pairs into `part` (K or V half of a block, uint8, in place)."""
    part[row * (d // 2):(row + 1) * (d // 2)] = codes[0::2] | (codes[1::2] << 4)
    n = 4 * (d // GROUP)
    at = BLOCK * d // 2 + row * n
    part[at:at + n] = np.stack([step, lo], -1).astype(np.float16).reshape(-1).view(np.uint8)


def unpack_cache(cache, d):
    """cache uint8 [pages, H, blocks, bytes] -> k, v float64 [pages, H, blocks * 16, d]."""
    out = []
    half = block_bytes(d) // 2
    for part in (cache[..., :half], cache[..., half:]):
        c = part[..., :BLOCK * d // 2].reshape(part.shape[:-1] + (BLOCK, d // 2))
        codes = np.stack([c & 15, c >> 4], -1).reshape(part.shape[:-1] + (BLOCK, d // GROUP, GROUP))
        p = np.ascontiguousarray(part[..., BLOCK * d // 2:]).view(np.float16)
        p = p.reshape(part.shape[:-1] + (BLOCK, d // GROUP, 2)).astype(np.float64)
        v = p[..., 1:] + p[..., :1] * codes
        out.append(v.reshape(part.shape[0], part.shape[1], -1, d))
    return out


def sequence_rows(values, table_row, L, page_size):
    """[H, L, d] of one sequence from unpacked pages; rows of pages outside are NaN."""
    H, d = values.shape[1], values.shape[-1]
    out = np.full((H, L, d), np.nan)
    for p0 in range(0, L, page_size):
        page = int(table_row[p0 // page_size])
        n = min(page_size, L - p0)
        if 0 <= page < values.shape[0]:
            out[:, p0:p0 + n] = values[page, :, :n]
    return out


def attention(q, k, v, scale, causal=True, window=0):
    """q [n, Hq, d], k, v [Hkv, L, d] of one sequence (its last n tokens' queries); keys that are
    NaN count as masked.  Returns o [n, Hq, d], lse [n, Hq] and sum_j p_j |v_j| [n, Hq, d]."""
    n, Hq, d = q.shape
    Hkv, L, _ = k.shape
    G = Hq // Hkv
    o, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    mag = np.zeros((n, Hq, d))
    for h in range(Hq):
        kh, vh = k[h // G], v[h // G]
        good = ~np.isnan(kh[:, 0]) if L else np.zeros(0, bool)
        for i in range(n):
            pos = L - n + i
            see = good.copy()
            if causal:
                see &= np.arange(L) <= pos
                if window:
                    see &= np.arange(L) > pos - window
            if not see.any():
                continue
            s = kh[see] @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            o[i, h] = p @ vh[see] / l
            mag[i, h] = p @ abs(vh[see]) / l
            lse[i, h] = m + np.log(l)
    return o, lse, mag
