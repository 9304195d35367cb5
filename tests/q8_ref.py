"""Plain 64-bit forms of the 8-bit paged store's operators, for the tests (CPU, numpy / torch)."""
import math

import numpy as np
import torch

PAGE = 16
KINDS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def e4m3_nearest(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value of |y| <= 448, ties to even: steps of 2^(e-3), e = max(floor(log2|y|), -6)."""
    _, e = np.frexp(y)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(y / step) * step


def quantise(x: torch.Tensor, kind: str):
    """Values [..., D] and scales [...] of bf16 rows, in float64 (scales as rounded to fp32)."""
    x = x.double().numpy()
    a = np.abs(x).max(-1, keepdims=True)
    bad, empty = ~np.isfinite(a), a < 2.0 ** -100
    safe = np.where(bad | empty, 1.0, a)
    xs = np.where(bad | empty, 0.0, x)
    if kind == "int8":
        v, s = np.rint(127.0 * xs / safe), safe / 127.0
    else:
        e = np.ceil(np.log2(safe / 448.0))  # exact at powers of two: safe has 8 significant bits, 448 = 7 * 64
        s = np.exp2(e)
        v = e4m3_nearest(xs / s)
    s = np.where(bad, np.nan, np.where(empty, 1.0, s)).astype(np.float32).astype(np.float64)
    return v, s[..., 0]


def stored(cache: torch.Tensor) -> np.ndarray:
    """The values of an 8-bit cache in float64."""
    return cache.cpu().float().double().numpy()


class Store:
    """A device store with stale junk (random bytes, NaN scales, and NaN bytes for e4m3) everywhere."""

    def __init__(self, kind, num_pages, Hkv, D, page_table, seed=0, device="cuda:0"):
        g = torch.Generator().manual_seed(seed)
        raw = torch.randint(-128, 128, (2, num_pages, Hkv, PAGE, D), generator=g, dtype=torch.int8)
        if kind == "e4m3":
            raw[..., ::3] = 0x7F  # e4m3 NaN
        self.kind = kind
        self.k = raw[0].contiguous().to(device).view(KINDS[kind])
        self.v = raw[1].contiguous().to(device).view(KINDS[kind])
        self.ks = torch.full((num_pages, Hkv, PAGE), float("nan"), device=device)
        self.vs = self.ks.clone()
        self.pt = page_table.to(torch.int32).to(device).contiguous()

    @property
    def args(self):
        return self.k, self.v, self.ks, self.vs, self.pt

    def value_scales(self, pages, n):
        """float64 [Hkv, n] scales of the first n value rows of a sequence."""
        idx = torch.as_tensor(pages, dtype=torch.long, device=self.vs.device)
        s = self.vs[idx].cpu().double().numpy()
        return s.transpose(1, 0, 2).reshape(s.shape[1], -1)[:, :n]

    def values(self, side, pages, n):
        """float64 [Hkv, n, D] of the first n tokens of a sequence whose pages are `pages`."""
        cache, scale = (self.k, self.ks) if side == "k" else (self.v, self.vs)
        idx = torch.as_tensor(pages, dtype=torch.long, device=cache.device)
        raw = cache.view(torch.int8)[idx].cpu().view(cache.dtype)
        x = raw.float().double().numpy() * scale[idx].cpu().double().numpy()[..., None]  # [P, Hkv, 16, D]
        return x.transpose(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def page_table(lens, max_pages, seed=0, spare=3):
    """[B, max_pages] table over a shuffled pool (-1 past each end) and the pool's size."""
    counts = [-(-n // PAGE) for n in lens]
    total = sum(counts) + spare
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed))
    pt = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        pt[b, :c] = perm[at:at + c].to(torch.int32)
        at += c
    return pt, total


def attend(q, k, v, scale, sv=None):
    """Row softmax(scale q.k) v in float64: q [Hq, D], k, v [Hkv, n, D] -> (out, sum p |v|), [Hq, D] each.

    With sv [Hkv, n], the value rows' scales, the second result has 2^-22 max_t(p_t sv_t) sum_t |v_t / sv_t|
    added: 2^-10 of that (the factor of assert_attention_close) is what f16's least step can take. A
    weight is held as 2^7 p_t sv_t / r with r <= max(p sv) (r follows the maximum from below). Below f16's
    normal numbers that is rounded to a multiple of 2^-24, so it is off by 2^-25 at most, which is
    2^-32 r <= 2^-32 max(p sv) of p_t sv_t, once for each stored value v_t / sv_t."""
    Hkv, n, D = k.shape
    if n == 0:
        z = np.zeros((q.shape[0], D))
        return z, z
    qg = q.reshape(Hkv, -1, D)
    s = np.einsum("hgd,hnd->hgn", qg, k) * scale
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    mag = np.einsum("hgn,hnd->hgd", p, np.abs(v))
    if sv is not None:
        top = (p * sv[:, None, :]).max(-1, keepdims=True)                       # [Hkv, G, 1]
        mag = mag + 2.0 ** -22 * top * np.abs(v / sv[..., None]).sum(1)[:, None, :]
    return np.einsum("hgn,hnd->hgd", p, v).reshape(q.shape), mag.reshape(q.shape)


def assert_attention_close(got: torch.Tensor, ref: np.ndarray, mag: np.ndarray):
    """|got - ref| <= 2^-8 |ref| (the bf16 output's half step) + 2^-10 sum p |v|: a weight is
    rounded to f16 (half a step 2^-11 relative), and the fp32 scores (|z| < 64 here, a few
    rounding steps of 2^-24 each) move a weight by less than 64 * 8 * 2^-24 = 2^-15; twice that
    for numerator and denominator stays below the other 2^-11."""
    err = np.abs(got.cpu().double().numpy() - ref)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag + 1e-30
    bad = err > tol
    assert not bad.any(), (float((err / tol).max()), int(bad.sum()), err.size)


def norm_rope(x, w, cos_sin, pos, eps):
    """float64 qk_norm_rope of x [T, H, D] with the fp32 table."""
    x = x.double().numpy()
    D = x.shape[-1]
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w.double().numpy()
    cs = cos_sin.double().numpy()[pos.numpy()]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = n[..., : D // 2], n[..., D // 2:]
    mag = np.concatenate([np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)], -1)
    return np.concatenate([a * c - b * s, b * c + a * s], -1), mag


def default_scale(D):
    return 1.0 / math.sqrt(D)
