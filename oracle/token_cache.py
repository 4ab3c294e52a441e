"""Float64 CPU implementations of the token-cache operators: rotary positions with
several axes, the 8-bit rolling cache, and the decode steps with a position per
sequence.  Used only by the tests; shares no code with the CUDA path."""
import numpy as np

E8_MIN, E8_MAX = -40, 40


def rope_nd(x, pos, pairs, theta=10000.0, inverse=False):
    """x [N, H, D] turned by pos [N, axes]; angles in extended precision."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    i = 0
    for a, n in enumerate(pairs):
        for j in range(n):
            ang = pos[:, a].astype(np.longdouble) * np.longdouble(theta) ** (np.longdouble(-j) / n)
            c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
            if inverse:
                s = -s
            u, w = x[:, :, 2 * i], x[:, :, 2 * i + 1]
            y[:, :, 2 * i], y[:, :, 2 * i + 1] = u * c - w * s, u * s + w * c
            i += 1
    return y


def e4m3_round(y):
    """Nearest e4m3 value, ties to even; beyond 448 becomes 448, NaN stays."""
    y = np.asarray(y, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        mag = np.minimum(np.abs(y), 448.0)
        exp = np.floor(np.log2(np.maximum(mag, 2.0 ** -6)))
        step = 2.0 ** (exp - 3)
        return np.copysign(np.minimum(np.rint(mag / step) * step, 448.0), y)


def quantise8(x):
    """(stored values, exponents) of rows x[..., D]: the least e with max|x| <= 448 * 2^e."""
    x = np.asarray(x, dtype=np.float64)
    top = np.max(np.where(np.isnan(x), 0.0, np.abs(x)), axis=-1)
    e = np.full(top.shape, E8_MIN)
    for k in range(E8_MIN, E8_MAX):
        e = np.where(top > 448.0 * 2.0 ** k, k + 1, e)
    return e4m3_round(x / 2.0 ** e[..., None]), e


def softmax_sum(q, k, v):
    """softmax(q k^T / sqrt(D)) v, and the weights times |v| (what a rounding of the weights can move)."""
    s = q @ k.T / np.sqrt(q.shape[-1])
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    return p @ v, p @ np.abs(v)


def decode_step(q, k_new, v_new, k_cache, v_cache, pos, prefix=None, chosen=None, block=0):
    """One step with a position per sequence: q [B, Hq, D], caches [B, W, Hkv, D].
    ``chosen[b][h]``: the blocks that (b, h) attends to.  Returns out, its weight scale
    (softmax_sum), and the updated caches."""
    q = np.asarray(q, np.float64)
    k_cache, v_cache = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    B, Hq, D = q.shape
    W, Hkv = k_cache.shape[1:3]
    G = Hq // Hkv
    out, scale = np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        if pos[b] < 0:
            continue
        k_cache[b, pos[b] % W], v_cache[b, pos[b] % W] = k_new[b], v_new[b]
        n = min(int(pos[b]) + 1, W)
        for h in range(Hkv):
            rows = np.arange(n)
            if chosen is not None:
                rows = np.concatenate([np.arange(j * block, min((j + 1) * block, n)) for j in chosen[b][h]])
            k, v = k_cache[b, rows, h], v_cache[b, rows, h]
            if prefix is not None:
                k, v = np.concatenate([prefix[0][:, h], k]), np.concatenate([prefix[1][:, h], v])
            g = slice(h * G, (h + 1) * G)
            out[b, g], scale[b, g] = softmax_sum(q[b, g], k, v)
    return out, scale, k_cache, v_cache


def block_bounds(k_cache, pos, block):
    """[B, Hkv, blocks, 2, D] lowest and highest valid key of each block (zeros where there is none)."""
    B, W, Hkv, D = k_cache.shape
    n = -(-W // block)
    out = np.zeros((B, Hkv, n, 2, D))
    for b in range(B):
        valid = min(int(pos[b]) + 1, W)
        for j in range(n):
            rows = k_cache[b, j * block:min((j + 1) * block, valid)]
            if len(rows):
                out[b, :, j, 0], out[b, :, j, 1] = np.fmin.reduce(rows, 0), np.fmax.reduce(rows, 0)
    return out


def select_blocks(q, bounds, pos, W, block, n_select, n_first, n_last):
    """The chosen blocks of every (b, KV head), ascending."""
    B, Hkv = bounds.shape[:2]
    G = q.shape[1] // Hkv
    chosen = []
    for b in range(B):
        n = min(int(pos[b]) + 1, W)
        used = -(-n // block) if n > 0 else 0
        rows = []
        for h in range(Hkv):
            score = np.zeros(used)
            for g in range(G):
                x = np.asarray(q[b, h * G + g], np.float64)
                score += np.maximum(x * bounds[b, h, :used, 0], x * bounds[b, h, :used, 1]).sum(-1)
            newest = int(pos[b]) % W // block
            forced = [j < n_first or (newest - j) % used < n_last for j in range(used)]
            order = sorted(range(used), key=lambda j: (not forced[j], -score[j] if not forced[j] else 0, j))
            rows.append(sorted(order[:n_select]))
        chosen.append(rows)
    return chosen
