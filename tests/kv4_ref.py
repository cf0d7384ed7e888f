"""Plain 64-bit definitions of the 4-bit cache, its attention and beam selection (include/talker_kv4.h)."""
import numpy as np

PAGE = 64


def q4_quantize(x):
    """x [..., n] (f32 or bf16 values) -> codes uint8 [..., n], scales fp16 [..., n / 32] by the definition. f64 holds
    every border 16 x = (17 - 2 k) m of 32-bit inputs exactly (24 + 5 bits)."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    b = np.where(np.isfinite(b), b, 0.0)
    at = np.argmax(np.abs(b), -1)[..., None]                   # the first on ties
    m = np.clip(np.take_along_axis(b, at, -1), -524032.0, 524032.0)
    codes = np.zeros(b.shape, np.int64)
    for k in range(1, 16):                                     # code >= k  <=>  8.5 - 8 x / m >= k
        codes += np.where(m > 0, -16.0 * b >= (2 * k - 17) * m, -16.0 * b <= (2 * k - 17) * m)
    codes = np.where((m == 0) | bad[..., None], 8, codes)
    d = (m[..., 0] / -8.0).astype(np.float32).astype(np.float16)
    d = np.where(bad, np.float16(np.nan), d)
    return codes.astype(np.uint8).reshape(x.shape), d


def q4_values(codes, d):
    c = np.asarray(codes, np.float64)
    b = c.reshape(c.shape[:-1] + (-1, 32))
    return ((b - 8.0) * np.asarray(d, np.float64)[..., None]).reshape(c.shape)


def q4_roundtrip(x):
    return q4_values(*q4_quantize(x))


def tile_bytes(codes, d, is_v):
    """One tile from codes [64, hd] and scales [64, hd / 32], byte by byte."""
    hd = codes.shape[1]
    nb = hd // 32
    out = np.zeros(36 * hd, np.uint8)
    rows = out[:32 * hd].reshape(64, hd // 2)
    for b in range(nb):
        for r in range(0, 32, 2):
            p = (r // 4) * 2 * nb + 2 * b + (r % 4) // 2 if is_v else (r // 8) * 4 * nb + 4 * b + (r % 8) // 2
            rows[:, p] = codes[:, 32 * b + r] | (codes[:, 32 * b + r + 1] << 4)
    out[32 * hd:] = np.ascontiguousarray(d.astype(np.float16)).view(np.uint8).reshape(-1)
    return out


def attend(q, k, v, scale):
    """q [n_q, hd], k and v [n, n_kv, hd] -> [n_q, hd]; zeros without rows."""
    n_q, hd = q.shape
    n, n_kv = k.shape[:2]
    if n == 0:
        return np.zeros((n_q, hd))
    g = n_q // n_kv
    w = np.einsum("hgd,nhd->hgn", q.reshape(n_kv, g, hd), k) * scale
    w = np.exp(w - w.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return np.einsum("hgn,nhd->hgd", w, v).reshape(n_q, hd)


def beam_select(logits, scores, ended, eos):
    """One sequence: logits [W, V], scores [W] -> tokens, beams, scores, ended, by sorting every candidate."""
    def unmask(x):
        x = np.asarray(x, np.float64)
        return np.where(x > -1e30, x, -np.inf)
    x, s = unmask(logits), unmask(scores)
    s = np.where(s == np.inf, -np.inf, s)
    W, V = x.shape
    c = np.full((W, V), -np.inf)
    for w in range(W):
        if ended is not None and ended[w]:
            c[w, eos] = s[w]
        elif np.isfinite(x[w].max()):
            m = x[w].max()
            c[w] = (x[w] - (m + np.log(np.exp(x[w] - m).sum()))) + s[w]
    order = np.argsort(-c.reshape(-1), kind="stable")[:W]
    tok, par = order % V, order // V
    done = (tok == eos) | (np.zeros(W, bool) if ended is None else np.asarray(ended, bool)[par])
    return tok, par, c.reshape(-1)[order], done
