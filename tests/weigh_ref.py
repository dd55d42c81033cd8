"""Attention weights that keys receive, in 64 bits on the CPU (test infrastructure only)."""
import torch

F64 = torch.float64


def received(q, k, lse, at, n_keys, scale, window):
    """One sequence: q [r, hq, D] at positions `at`, k [n, hkv, D], lse [r, hq], all float64.
    Returns [n, hkv] sums of exp(scale q.k - lse), and what bounds their error: sums of p (2^-19 Z + 2^-21 (1 + |a|)) with
    a = scale q.k - lse and Z = scale sum |q k|: products of codes or 16-bit values are exact, the matrix unit and the sums
    over blocks cut off at most 2^-20 Z, the factor's and the argument's roundings count 2^-23 |a| and 2^-24 Z, the exponential
    2^-22."""
    r, hq, _ = q.shape
    n, hkv, _ = k.shape
    g = hq // hkv
    out, tol = torch.zeros(n, hkv, dtype=F64), torch.zeros(n, hkv, dtype=F64)
    for i in range(r):
        p = int(at[i])
        lo, hi = (max(0, p - window + 1) if window else 0), min(p + 1, n_keys)
        if hi <= lo:
            continue
        kk = k[lo:hi].repeat_interleave(g, 1)
        a = torch.einsum("hd,nhd->nh", q[i], kk) * scale - lse[i]
        z = torch.einsum("hd,nhd->nh", q[i].abs(), kk.abs()) * scale
        w = a.exp()
        out[lo:hi] += w.unflatten(1, (hkv, g)).sum(2)
        # (what is below the normal numbers is 0: at most 2^-126 each)
        off = torch.where(w > 0, w * (2.0 ** -19 * z + 2.0 ** -21 * (1 + a.abs())), 0.0) + 2.0 ** -126
        tol[lo:hi] += off.unflatten(1, (hkv, g)).sum(2)
    return out, tol + 2.0 ** -21 * out


def seen_lse(q, k, at, n_keys, scale, window):
    """What attention gives beside its result: [r, hq] float64, -inf where nothing is seen."""
    r, hq, _ = q.shape
    g = hq // k.shape[1]
    out = torch.full((r, hq), -float("inf"), dtype=F64)
    for i in range(r):
        p = int(at[i])
        lo, hi = (max(0, p - window + 1) if window else 0), min(p + 1, n_keys)
        if hi > lo:
            out[i] = torch.logsumexp(torch.einsum("hd,nhd->nh", q[i], k[lo:hi].repeat_interleave(g, 1)) * scale, 0)
    return out
