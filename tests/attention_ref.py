"""Plain 64-bit statements of the attention operators, on the CPU (test infrastructure only)."""
import numpy as np
import torch

F64 = torch.float64
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a rounding step


def rotate(x, pos, cos, sin, interleaved, dtype=F64):
    """x [T, h, D], pos [T]; every operation rounded in `dtype`."""
    x, half = x.to(dtype), cos.shape[1]
    c, s = cos[pos].to(dtype)[:, None], sin[pos].to(dtype)[:, None]
    y = x.clone()
    a = x[..., 0:2 * half:2] if interleaved else x[..., :half]
    b = x[..., 1:2 * half:2] if interleaved else x[..., half:2 * half]
    ya, yb = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ya, yb
    else:
        y[..., :half], y[..., half:2 * half] = ya, yb
    return y


def quantise(x):
    """fp32 [..., D] -> codes int [..., D] (0..15) and fp16 scales [..., D/32]."""
    x = x.float().unflatten(-1, (-1, 32))
    codes = torch.zeros(x.shape, dtype=torch.int64)
    flat, out = x.reshape(-1, 32), codes.view(-1, 32)
    scales = torch.zeros(flat.shape[0], dtype=torch.float16)
    xs = flat.numpy()
    for i in range(flat.shape[0]):
        b = xs[i]
        if not np.isfinite(b).all():
            scales[i] = float("nan")
            continue
        top = np.abs(b).max()
        m = top if (b == top).any() else -top
        d = np.float32(m) / np.float32(-8)
        if d == 0:
            out[i] = 8
        else:
            out[i] = torch.from_numpy(np.minimum(15, np.trunc(b / d + np.float32(8.5))).astype(np.int64))
        scales[i] = float(np.clip(d, -65504, 65504))
    return codes.flatten(-2), scales.reshape(x.shape[:-1])


def values(codes, scales):
    return (codes.double() - 8) * scales.double().repeat_interleave(32, -1)


class Cache:
    """The pages as the header describes them, byte by byte."""

    def __init__(self, n_pages, hkv, d, page_size):
        self.hkv, self.d, self.ps = hkv, d, page_size
        self.pages = torch.zeros(n_pages, hkv * (page_size // 32) * 36 * d, dtype=torch.uint8)

    def _at(self, page, head, tok):
        return page, (head * (self.ps // 32) + tok // 32) * 36 * self.d, tok % 32

    def put(self, page, tok, head, value, codes, scales):
        p, base, r = self._at(page, head, tok)
        base += 18 * self.d * value
        for b in range(self.d // 32):
            q = codes[32 * b:32 * b + 32]
            at = base + (b * 32 + r) * 16
            self.pages[p, at:at + 16] = (q[:16] | (q[16:] << 4)).to(torch.uint8)
        at = base + 16 * self.d + r * (self.d // 16)
        self.pages[p, at:at + self.d // 16] = scales.view(torch.uint8)

    def get(self, page, tok, head, value):
        p, base, r = self._at(page, head, tok)
        base += 18 * self.d * value
        codes = []
        for b in range(self.d // 32):
            at = base + (b * 32 + r) * 16
            q = self.pages[p, at:at + 16].long()
            codes += [q & 15, q >> 4]
        at = base + 16 * self.d + r * (self.d // 16)
        return values(torch.cat(codes), self.pages[p, at:at + self.d // 16].view(torch.float16))


def sequence(pages, row, n, page_size, hkv, d):
    """All cached keys and values of a sequence, vectorised: [n, hkv, d] each, float64 (pages on the CPU)."""
    held = pages[row[:-(-n // page_size)].long()].unflatten(1, (hkv, page_size // 32, 36 * d))
    out = []
    for off in (0, 18 * d):
        t = held[..., off:off + 18 * d]
        codes = t[..., :16 * d].unflatten(-1, (d // 32, 32, 16)).transpose(-2, -3).long()
        sc = t[..., 16 * d:].contiguous().view(torch.float16).unflatten(-1, (32, d // 32)).double()
        v = (torch.cat([codes & 15, codes >> 4], -1).double() - 8) * sc[..., None]
        out.append(v.flatten(-2).permute(0, 2, 3, 1, 4).flatten(0, 2)[:n])
    return out


def attend(q, k, v, at, n_keys, scale, window):
    """One sequence: q [r, hq, D] at positions `at`, k, v [n, hkv, D], all float64.
    Returns o, lse [r, hq], and per row sum p |v| / sum p and max_j scale sum_d |q k| (for tolerances)."""
    r, hq, d = q.shape
    g = hq // k.shape[1]
    o, mag = torch.zeros(r, hq, d, dtype=F64), torch.zeros(r, hq, d, dtype=F64)
    lse, size = torch.full((r, hq), -float("inf"), dtype=F64), torch.zeros(r, hq, dtype=F64)
    for i in range(r):
        p = int(at[i])
        lo = max(0, p - window + 1) if window else 0
        hi = min(p + 1, n_keys)
        if hi <= lo:
            continue
        kk, vv = k[lo:hi].repeat_interleave(g, 1), v[lo:hi].repeat_interleave(g, 1)
        s = torch.einsum("hd,nhd->hn", q[i], kk) * scale
        size[i] = (torch.einsum("hd,nhd->hn", q[i].abs(), kk.abs()) * abs(scale)).amax(1)
        w = torch.softmax(s, -1)
        lse[i] = torch.logsumexp(s, -1)
        o[i] = torch.einsum("hn,nhd->hd", w, vv)
        mag[i] = torch.einsum("hn,nhd->hd", w, vv.abs())
    return o, lse, mag, size
