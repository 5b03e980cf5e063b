"""Plain float64 / integer definitions of the operators around attention.

TEST INFRASTRUCTURE ONLY (see the package docstring): the page plan of a
serving step, the RMS norm of head rows with the position rotation and its
gradients, and the 4-bit cache's quantisation and block layout.
"""

from __future__ import annotations

import numpy as np

PAGE = 64
BAD_PAGE, BAD_LENGTH, NO_PAGES = 1, 4, 16


def page_plan(cached, new, table, free, num_rows, num_pages, head=0):
    """One step's plan, request by request.  Returns a dict with the updated
    table, seq_lens, cu_seqlens, slots, positions, used and the error bits."""
    table = np.array(table, dtype=np.int64)
    B, width = table.shape
    cu = [0]
    for n in new:
        cu.append(cu[-1] + max(0, int(n)))
    seq, slots, positions = [0] * B, [-1] * num_rows, [-1] * num_rows
    err, used, want_total = 0, 0, 0
    if not 0 <= head <= len(free):
        err |= NO_PAGES
        head = len(free)
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        if c < 0 or n < 0 or c + n > width * PAGE:
            err |= BAD_LENGTH
            continue
        have, want = -(-c // PAGE), -(-(c + n) // PAGE)
        first, want_total = want_total, want_total + want - have
        if n > 0 and cu[b + 1] > num_rows:
            err |= BAD_LENGTH
            continue
        if want > have and want_total > len(free) - head:
            err |= NO_PAGES
            continue
        seq[b] = c + n
        pages = {}
        for i in range(have, want):
            page = int(free[head + first + i - have])
            if not 0 <= page < num_pages:
                err |= BAD_PAGE
                page = -1
            pages[i] = table[b, i] = page
        used = max(used, want_total if want > have else 0)
        for i in range(n):
            pos = c + i
            page = int(table[b, pos // PAGE])
            positions[cu[b] + i] = pos
            if 0 <= page < num_pages:
                slots[cu[b] + i] = page * PAGE + pos % PAGE
            else:
                err |= BAD_PAGE
    return dict(table=table, seq_lens=np.array(seq), cu_seqlens=np.minimum(cu, num_rows), slots=np.array(slots),
                positions=np.array(positions), used=used, error=err)


def rotation(cos, sin, positions, d, interleaved):
    """R of every position, [N, d, d]: y = R n."""
    cos, sin = np.asarray(cos, np.float64)[positions], np.asarray(sin, np.float64)[positions]
    half = cos.shape[-1]
    R = np.tile(np.eye(d), (len(positions), 1, 1))
    for f in range(half):
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
        R[:, i, i] = R[:, j, j] = cos[:, f]
        R[:, i, j], R[:, j, i] = -sin[:, f], sin[:, f]
    return R


def norm_rope(x, w, R, eps, norm=True):
    """y [N, H, d] of rows x [N, H, d]; R [N, d, d] or None; w [d] or None."""
    x = np.asarray(x, np.float64)
    n = x
    if norm:
        n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * (1.0 if w is None else np.asarray(w, np.float64))
    return n if R is None else np.einsum("nij,nhj->nhi", R, n)


def norm_rope_grad(x, dy, w, R, eps, norm=True):
    """(dx, dw) of sum(dy * norm_rope(x, w)): the formula, row by row."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    dn = dy if R is None else np.einsum("nji,nhj->nhi", R, dy)
    if not norm:
        return dn, None
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    unit, g = x * r, dn * w
    return r * (g - unit * np.mean(g * unit, -1, keepdims=True)), (dn * unit).sum((0, 1))


def _bf16(x):
    """Nearest bfloat16 (ties to even) of float32 values, as float32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return r.astype(np.uint32).view(np.float32)


def q4_quantise(x):
    """Codes, scales and minima of rows x [..., d] (bfloat16 values): one group
    per 64 columns, float32 arithmetic as the format defines it."""
    x = np.asarray(x, np.float32)
    g = x.reshape(x.shape[:-1] + (-1, 64))
    with np.errstate(all="ignore"):
        low, high = g.min(-1), g.max(-1)
        span = high - low
        bad = ~np.isfinite(g).all(-1) | ~np.isfinite(span)
        scale = _bf16(span / np.float32(15))
        q = np.where(scale[..., None] > 0, (g - low[..., None]) / scale[..., None], np.float32(0))
        code = np.clip(np.rint(q), 0, 15)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    return code.reshape(x.shape), np.where(bad, np.float32(0), scale), np.where(bad, np.float32(np.nan), low)


def q4_values(code, scale, low):
    """What the codes stand for, float64."""
    c = np.asarray(code, np.float64).reshape(code.shape[:-1] + (-1, 64))
    out = c * np.asarray(scale, np.float64)[..., None] + np.asarray(low, np.float64)[..., None]
    return out.reshape(code.shape)


def _places(d):
    """Byte and shift in the block of every (token, column) code, for K and V."""
    tok, col = np.arange(PAGE)[:, None], np.arange(d)[None]
    j = col // 32
    kbit = 16 * (col % 2) + 4 * (col % 8 // 2)
    kbyte = tok * (d // 2) + 4 * ((d // 32) * (col % 32 // 8) + j) + kbit // 8
    vbit = 16 * (tok % 2) + 4 * (col % 4)
    vbyte = 32 * d + (tok // 2) * d + 4 * ((d // 32) * (col % 32 // 4) + j) + vbit // 8
    return (kbyte, np.broadcast_to(kbit % 8, (PAGE, d))), (vbyte, vbit % 8)


def q4_blocks(k, v):
    """Blocks [..., 72 d] of keys and values [..., 64, d]."""
    lead, d = k.shape[:-2], k.shape[-1]
    out = np.zeros(lead + (72 * d,), np.uint8)
    params = []
    for x, (byte, shift) in zip((k, v), _places(d)):
        code, scale, low = q4_quantise(x)
        for t in range(PAGE):
            for c in range(d):
                out[..., byte[t, c]] |= code[..., t, c] << np.uint8(shift[t, c])
        p = np.stack([scale, low], -1).astype(np.float32).view(np.uint32) >> 16
        params.append(p.astype(np.uint16).reshape(lead + (-1,)))
    out[..., 64 * d:] = np.concatenate(params, -1).view(np.uint8)
    return out


def q4_unblock(block, d):
    """Keys and values [..., 64, d], float64, that blocks [..., 72 d] stand for."""
    block = np.ascontiguousarray(block)
    lead = block.shape[:-1]
    p = np.ascontiguousarray(block[..., 64 * d:]).view(np.uint16).astype(np.uint32) << 16
    p = p.view(np.float32).reshape(lead + (2, PAGE, d // 64, 2))
    (kb, ks), (vb, vs) = _places(d)
    k = q4_values((block[..., kb] >> ks.astype(np.uint8)) & 15, p[..., 0, :, :, 0], p[..., 0, :, :, 1])
    v = q4_values((block[..., vb] >> vs.astype(np.uint8)) & 15, p[..., 1, :, :, 0], p[..., 1, :, :, 1])
    return k, v
