"""Plain 64-bit implementations of the balance loss and of MXFP4 rounding and
products, and the inputs that reach their edges (tests only)."""
import numpy as np
import torch

from oracle import layer as olayer

U32 = 2.0 ** -24                       # half a step of fp32, relative
HALF_STEP = {torch.float32: U32, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


# --- balance loss -----------------------------------------------------------
def balance64(scores, idx, offsets=None, mask=None, dloss=None):
    """(loss, counts, tokens, dscores, scale of the gradient's terms) in float64
    NumPy, written from the definition token by token."""
    T, n = scores.shape
    k = idx.shape[1]
    s = np.asarray(scores, np.float64)
    off = np.array([0, T]) if offsets is None else np.asarray(offsets)
    S = len(off) - 1
    loss, counts = np.zeros(S), np.zeros((S, n), np.int64)
    tokens = np.zeros(S, np.int64)
    grad, size = np.zeros((T, n)), np.zeros((T, n))
    for q in range(S):
        rows = [t for t in range(off[q], off[q + 1]) if mask is None or mask[t]]
        tokens[q] = N = len(rows)
        for t in rows:
            for e in idx[t]:
                if 0 <= e < n:
                    counts[q, e] += 1
        if N == 0:
            continue
        w = n / (k * N * N)
        for t in rows:
            total = s[t].sum()
            if total == 0:
                continue
            inner = (counts[q] * s[t]).sum() / total
            loss[q] += w * inner
            g = w * (1.0 if dloss is None else float(dloss[q])) / total
            grad[t] = g * (counts[q] - inner)
            size[t] = abs(g) * (counts[q] + inner)
    return loss, counts, tokens, grad, size


# --- MXFP4 ------------------------------------------------------------------
def pad32(v):
    rows, K = v.shape
    out = np.zeros((rows, -(-K // 32) * 32))
    out[:, :K] = v
    return out


def mx_encode64(v):
    """Rows of float64 -> (codes one per byte, scale bytes) of the padded rows; a
    block with an infinity or NaN is scale 255, codes 0."""
    p = pad32(np.asarray(v, np.float64))
    fine = np.isfinite(p).reshape(p.shape[0], -1, 32).all(axis=2)
    clean = np.where(np.repeat(fine, 32, axis=1), p, 0.0)
    codes, sb = olayer.mxfp4_act_quantize(clean)
    return np.where(np.repeat(fine, 32, axis=1), codes, 0).astype(np.uint8), \
        np.where(fine, sb, 255).astype(np.uint8)


def mx_decode64(codes, sb):
    mag = np.array([0, .5, 1, 1.5, 2, 3, 4, 6.0])[codes & 7]
    val = np.where(codes & 8, -mag, mag)
    scale = np.ldexp(1.0, sb.astype(np.int64) - 127)
    scale = np.where(sb == 255, np.nan, scale)
    return val * np.repeat(scale, 32, axis=1)


def mx_round64(v):
    return mx_decode64(*mx_encode64(v))[:, :np.shape(v)[1]]


def nibbles(packed):
    """Codes, one per byte, of packed bytes."""
    p = packed.cpu().numpy()
    out = np.empty(p.shape[:-1] + (2 * p.shape[-1],), np.uint8)
    out[..., 0::2] = p & 15
    out[..., 1::2] = p >> 4
    return out


def edge_rows(rows, K, dtype, seed):
    """Rows whose blocks hit every branch of the rounding: ordinary values over
    many magnitudes, ties, neighbours of ties, zeros and signs, saturation, the
    smallest and largest values of the type, infinities and NaN."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-12, 12, (rows, 1)).astype(float))
    t = torch.from_numpy(v).to(dtype)
    n = min(K, 32)
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 6.0, 7.5, 0.0])
    lo, hi = {torch.float32: (-120, 120), torch.bfloat16: (-120, 120),
              torch.float16: (-10, 10)}[dtype]
    for r in range(0, rows, 3):
        kind = (r // 3) % 8
        e = int(rng.integers(lo, hi))
        if kind == 0:      # ties under a maximum of 4 or 7.5
            b = rng.choice(grid[:10], n) * 2.0 ** e
            b[0] = 4.0 * 2.0 ** e
            x = torch.from_numpy(b * rng.choice([-1.0, 1.0], n)).to(dtype)
        elif kind == 1:    # the neighbours of ties in the type
            b = torch.from_numpy(rng.choice(grid[:7], n) * 2.0 ** e).to(dtype)
            x = torch.nextafter(b, torch.full_like(b, 100.0 if r % 2 else 0.0))
            x[0] = 7.0 * 2.0 ** e
        elif kind == 2:
            x = torch.zeros(n, dtype=dtype)
            x[::2] = -0.0
        elif kind == 3:    # the smallest values of the type
            x = (torch.arange(n) % 5).to(dtype) * torch.finfo(dtype).smallest_normal / 4
        elif kind == 4:
            x = torch.full((n,), torch.finfo(dtype).max, dtype=dtype)
            x[1::2] *= -0.3
        elif kind == 5:
            x = t[r, :n].clone()
            x[n // 2] = float("inf") if r % 2 else float("-inf")
        elif kind == 6:
            x = t[r, :n].clone()
            x[-1] = float("nan")
        else:              # one large value over small ones
            x = t[r, :n] * 2.0 ** -8
            x[n // 3] = 2.0 ** min(e, 12)
        at = int(rng.integers(0, max(1, K // 32))) * 32
        m = min(n, K - at)
        t[r, at:at + m] = x[:m]
    return t


def as64(t):
    return t.to(torch.float64).cpu().numpy()


def product_bound(a, b, out_dtype, K):
    """How far an fp32 MFMA sum of K exact products a b^T may be off, rounding or
    truncating each addition (2^-23 of the partial sums' size, which the sum of
    magnitudes bounds), plus the rounding of the output."""
    size = np.abs(a) @ np.abs(b).T
    ref = a @ b.T
    acc = (K + 8) * 2.0 ** -23 * size
    return ref, acc + HALF_STEP[out_dtype] * (np.abs(ref) + acc) + 2.0 ** -140
