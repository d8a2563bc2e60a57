"""fp64 NumPy definitions of the paged-cache operators (TEST INFRASTRUCTURE ONLY):
position rotation, appending tokens to the pages, dense decode.  They share no
code with the CUDA path and are written token by token, as the operators are defined.
"""
import numpy as np

B = 64


def rotate_row(x, pos, inv_freq, interleaved=False, inverse=False):
    """x [..., d] fp64 at one position: pair f turned by pos * inv_freq[f]."""
    x = np.array(x, dtype=np.float64)
    ang = float(pos) * np.asarray(inv_freq, dtype=np.float64)
    if inverse:
        ang = -ang
    r = 2 * len(inv_freq)
    out = x.copy()
    for f in range(r // 2):
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + r // 2)
        c, s = np.cos(ang[f]), np.sin(ang[f])
        out[..., i] = x[..., i] * c - x[..., j] * s
        out[..., j] = x[..., j] * c + x[..., i] * s
    return out


def rotate(x, inv_freq, positions=None, interleaved=False, inverse=False):
    """x [b, heads, n, d]; positions None, [n] or [b, n]."""
    x = np.asarray(x, dtype=np.float64)
    b, _, n, _ = x.shape
    out = np.empty_like(x)
    for bi in range(b):
        for i in range(n):
            p = i if positions is None else positions[i] if np.ndim(positions) == 1 else positions[bi][i]
            out[bi, :, i] = rotate_row(x[bi, :, i], p, inv_freq, interleaved, inverse)
    return out


def append(tokens, k_pages, v_pages, block_table, seq_lens, counts, inv_freq=None, interleaved=False, starts=None):
    """tokens[b](i) -> (q or None, k, v) of sequence b's i-th new token, each [heads, d].
    Writes fp64 copies of the pages; returns (q rows by (b, i), k_pages, v_pages, filled):
    filled[b] lists the pages sequence b filled, in order."""
    kp, vp = np.array(k_pages, dtype=np.float64), np.array(v_pages, dtype=np.float64)
    q_rows, filled = {}, []
    turn = (lambda x, p: np.array(x, np.float64)) if inv_freq is None else \
        (lambda x, p: rotate_row(x, p, inv_freq, interleaved))
    for b, n in enumerate(counts):
        filled.append([])
        for i in range(n):
            pos = int(seq_lens[b]) - n + i
            q, k, v = tokens(b, i)
            if pos < 0:
                continue
            if q is not None:
                q_rows[b, i] = turn(q, pos)
            c = pos // B
            page = int(block_table[b][c]) if c < len(block_table[b]) else -1
            if 0 <= page < len(kp):
                kp[page, :, pos % B] = turn(k, pos)
                vp[page, :, pos % B] = v
                if pos % B == B - 1:
                    filled[b].append(page)
    return q_rows, kp, vp, filled


def decode_dense(q, k_pages, v_pages, block_table, seq_lens, scale, window=0):
    """q [b, h, d] -> out [b, h, d], lse [b, h], and what error bounds need: the weighted
    magnitude sum_j p_j |v_j| and the largest scale * sum |q||k|."""
    q = np.asarray(q, np.float64)
    b, h, d = q.shape
    g = k_pages.shape[1]
    out, mag = np.zeros((b, h, d)), np.zeros((b, h, d))
    lse, size = np.full((b, h), -np.inf), np.zeros((b, h))
    for bi in range(b):
        n = int(seq_lens[bi])
        if n <= 0:
            continue
        first = max(0, ((n - 1) // B + 1 - window // B) * B) if window else 0
        keys = [(int(block_table[bi][j // B]), j % B) for j in range(first, min(n, B * len(block_table[bi])))]
        keys = [(p, r) for p, r in keys if 0 <= p < len(k_pages)]
        if not keys:
            continue
        pg, rw = np.array(keys).T
        for hi in range(h):
            k = np.asarray(k_pages[pg, hi // (h // g), rw], np.float64)
            v = np.asarray(v_pages[pg, hi // (h // g), rw], np.float64)
            s = k @ q[bi, hi] * scale
            m = s.max()
            e = np.exp(s - m)
            lse[bi, hi] = m + np.log(e.sum())
            p = e / e.sum()
            out[bi, hi], mag[bi, hi] = p @ v, p @ np.abs(v)
            size[bi, hi] = (np.abs(k) @ np.abs(q[bi, hi])).max() * abs(scale)
    return out, lse, mag, size
