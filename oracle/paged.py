"""Oracle: norm and rotation of heads, the paged cache's append, and the decode
attention that reads it, in fp64.

Test infrastructure only (see the package docstring for who may import it).

Definitions (none of them is in the method's sources; the public ones of the
operations are used):

* norm and rotation of a row x of d elements at position p:
  y = x / sqrt(mean(x^2) + eps) * w, then for each pair (a, b) of the first
  2 * cos.shape[1] elements, (a cos - b sin, b cos + a sin) with the table row
  of p; pairs (j, j + half) or, interleaved, (2j, 2j + 1);
* append: token i of the n new ones of sequence b goes to position
  len_b - n + i.  An E4M3 page keeps one scale per kv head, the smallest power
  of two s >= 2^-126 with absmax <= 448 s; appending behind tokens that the
  page holds takes the larger of the old and the new one and re-encodes the
  old codes' values;
* attention: every row is a three-pass softmax over the values that the cache
  stands for;
* masks: the row at position p reads the keys at positions up to p, with a window
  of W only those less than W before it and the first S (sinks); a node of a tree
  of drafted tokens reads the tokens before the nodes and its line of parents.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64, three_pass_row
from .fp8_quant_gemm import E4M3_MAX, e4m3_decode, e4m3_encode


def norm_rope(x, pos, cos=None, sin=None, interleaved=False, weight=None, eps=1e-6) -> np.ndarray:
    """x [T, H, d], pos [T]; returns fp64 of the same shape."""
    y = _f64(x).copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * _f64(weight)
    if cos is None:
        return y
    c, s = _f64(cos)[np.asarray(pos)], _f64(sin)[np.asarray(pos)]
    half = c.shape[1]
    out = y.copy()
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        out[..., a] = y[..., a] * c[:, None, j] - y[..., b] * s[:, None, j]
        out[..., b] = y[..., b] * c[:, None, j] + y[..., a] * s[:, None, j]
    return out


def pow2_scale(a: float) -> float:
    """The smallest power of two s >= 2^-126 with a <= 448 s."""
    s = 2.0 ** -126
    while a > E4M3_MAX * s:
        s *= 2.0
    return s


def append_e4m3(codes, scale, x, off: int):
    """One page of one kv head: codes [page_size, d] and its scale, new values
    x [n, d] to slots off .. off + n - 1.  Returns the new (codes, scale)."""
    codes = np.array(codes, dtype=np.uint8)
    x = _f64(x)
    finite = np.abs(x[np.isfinite(x)])
    s = pow2_scale(float(finite.max()) if finite.size else 0.0)
    if off > 0:
        old = float(scale)
        s = max(s, old)
        if s != old:
            codes[:off] = e4m3_encode(e4m3_decode(codes[:off]) * (old / s))
    codes[off:off + len(x)] = e4m3_encode(x / s)
    return codes, s


def append(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, new, k, v):
    """The whole append.  Pages uint8 (scales given) or float; new [B] tokens of
    each sequence, k (already normed and rotated) and v [total, Hkv, d].
    Returns the four arrays after it (pages of a float cache unrounded)."""
    e4m3 = k_scale is not None
    pages = [np.array(k_pages), np.array(v_pages)]
    scales = [np.array(k_scale), np.array(v_scale)] if e4m3 else [None, None]
    ps = pages[0].shape[2]
    at = 0
    for b, n in enumerate(new):
        length = int(seq_lens[b])
        rows = [_f64(k)[at:at + n], _f64(v)[at:at + n]]
        at += n
        if length == 0 or n == 0:
            continue
        start = length - n
        for page in range(start // ps, (length - 1) // ps + 1):
            lo, hi = max(page * ps, start), min((page + 1) * ps, length)
            phys, off = int(block_table[b][page]), lo - page * ps
            for w in range(2):
                for h in range(pages[w].shape[1]):
                    x = rows[w][lo - start:hi - start, h]
                    if e4m3:
                        pages[w][phys, h], scales[w][phys, h] = append_e4m3(
                            pages[w][phys, h], scales[w][phys, h], x, off)
                    else:
                        pages[w][phys, h, off:off + hi - lo] = x
    return pages[0], pages[1], scales[0], scales[1]


def values(pages, scale) -> np.ndarray:
    """What the cache stands for, fp64 [pages, Hkv, page_size, d]."""
    if scale is None:
        return _f64(pages)
    return e4m3_decode(np.asarray(pages)) * np.asarray(scale, np.float64)[:, :, None, None]


def decode(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, scale: float,
           row=three_pass_row) -> np.ndarray:
    """q [B, Tq, Hq, d]; returns o fp64 of the same shape.  ``row`` computes one
    query row from its q [d], keys, values and scale."""
    q = _f64(q)
    B, Tq, Hq, d = q.shape
    K, V = values(k_pages, k_scale), values(v_pages, v_scale)
    Hkv, ps = K.shape[1], K.shape[2]
    o = np.zeros_like(q)
    for b in range(B):
        n = int(seq_lens[b])
        pages = [int(x) for x in np.asarray(block_table)[b][:-(-n // ps)]]
        for h in range(Hkv if n else 0):
            kb = np.concatenate([K[x, h] for x in pages])[:n]
            vb = np.concatenate([V[x, h] for x in pages])[:n]
            for t in range(Tq):
                seen = max(0, n - Tq + t + 1)
                for g in range(Hq // Hkv):
                    hq = h * (Hq // Hkv) + g
                    o[b, t, hq] = row(q[b, t, hq], kb[:seen], vb[:seen], scale)
    return o


def line_of(parents, t: int):
    """Node t of a tree and those it descends from, up to the root; None where an
    entry is neither -1 nor that of an earlier node."""
    line = [t]
    while True:
        up = int(parents[t])
        if up == -1:
            return line
        if not 0 <= up < t:
            return None
        line.append(up)
        t = up


def seen_keys(n: int, Tq: int, t: int, window: int = 0, sinks: int = 0, parents=None):
    """The keys that query token t of the last Tq of a sequence of n tokens reads,
    ascending.  A chain's token is at its own place; a tree's node at the place of
    its depth behind the n - Tq tokens before the nodes."""
    first = n - Tq
    if parents is None:
        places = {j: j for j in range(max(0, first + t + 1))}          # key -> position
        pos = first + t
    else:
        line = line_of(parents, t)
        if line is None or first < 0:
            return []
        pos = first + len(line) - 1
        places = {j: j for j in range(first)}
        places.update({first + u: pos - i for i, u in enumerate(line)})
    return sorted(j for j, at in places.items() if window == 0 or pos - at < window or at < sinks)


def decode_masked(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, scale: float,
                  window: int = 0, sinks: int = 0, parents=None, row=three_pass_row) -> np.ndarray:
    """``decode`` over the keys of ``seen_keys``; parents [B, Tq] or None."""
    q = _f64(q)
    B, Tq, Hq, d = q.shape
    K, V = values(k_pages, k_scale), values(v_pages, v_scale)
    Hkv, ps = K.shape[1], K.shape[2]
    o = np.zeros_like(q)
    for b in range(B):
        n = int(seq_lens[b])
        for t in range(Tq if n else 0):
            keys = seen_keys(n, Tq, t, window, sinks, None if parents is None else parents[b])
            at = [(int(block_table[b][j // ps]), j % ps) for j in keys]
            for hq in range(Hq):
                h = hq // (Hq // Hkv)
                kb = np.array([K[x, h, i] for x, i in at]).reshape(-1, d)
                vb = np.array([V[x, h, i] for x, i in at]).reshape(-1, d)
                o[b, t, hq] = row(q[b, t, hq], kb, vb, scale)
    return o


def window_prompt(q, k, v, new, keys, scale: float, window: int = 0, sinks: int = 0,
                  row=three_pass_row) -> np.ndarray:
    """Prompts: q [sum(new), Hq, d], k and v [sum(keys), Hkv, d]; the new tokens of
    a sequence are the last of its keys'.  Returns o fp64 of q's shape."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    o = np.zeros_like(q)
    q0 = k0 = 0
    for n, nk in zip(new, keys):
        for t in range(n):
            seen = [k0 + j for j in seen_keys(nk, n, t, window, sinks)]
            for hq in range(q.shape[1]):
                h = hq // (q.shape[1] // k.shape[1])
                o[q0 + t, hq] = row(q[q0 + t, hq], k[seen, h], v[seen, h], scale)
        q0, k0 = q0 + n, k0 + nk
    return o
