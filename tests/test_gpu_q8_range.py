"""Attention over the 8-bit store where value rows differ widely in size: the softmax's
denominator keeps every token that carries weight, whatever its value scale, and each form of
the calls (decode, wide tiles, few rows, clusters) gives the same bits."""
import numpy as np
import pytest
import torch

import invariant_deterministic_04_b200 as bi
import q8_ref
import synth
from gpu_util import dev, same_bits
from test_gpu_q8 import fill

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3"]


def attend(q, k, v, sv, scale):
    """float64 softmax(scale q.k) v of q [Hq, D], k, v [Hkv, n, D] and the error it may have, [Hq, D] each.

    A weight enters the products as w = 2^7 p sv / r in f16, r the largest p sv of value rows that are
    not zero, or less. Half a step of that is 2^-11 of w for f16's normal numbers (finfo.eps / 2, counted
    for w) and 2^-25 below them, 2^-32 r of p sv; the sum over tokens of |v / sv| times 2^-32 r bounds the
    latter. The fp32 scores are off by less than 2^-24 * 8 of |z| (below 128 here: 2^-14 of w), once for
    the numerator and once for the denominator: 2^-13, and the f16 step of the one weight that the others
    are measured by, 2^-11 more: 2^-10 sum p |v| covers the three. The output is rounded to bf16: 2^-8
    of it, and 2^-134 below the normal numbers."""
    Hkv, n, D = k.shape
    s = np.einsum("hgd,hnd->hgn", q.reshape(Hkv, -1, D), k) * scale
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    out = np.einsum("hgn,hnd->hgd", p, v)
    loud = np.where(np.abs(v).max(-1) > 0, sv, 0.0)
    r = (p * loud[:, None, :]).max(-1, keepdims=True)
    tol = (2.0 ** -8 * np.abs(out) + 2.0 ** -10 * np.einsum("hgn,hnd->hgd", p, np.abs(v))
           + 2.0 ** -32 * r * np.abs(v / sv[..., None]).sum(1)[:, None, :] + 2.0 ** -134)
    return out.reshape(q.shape), tol.reshape(q.shape)


def check_all_forms(kind, k, v, q, scale):
    """One sequence of k, v [n, Hkv, D] and queries q [Hq, D] at its end: decode against 64 bits; a
    wide tile, few rows alone, and few rows with a long page table (clusters) against decode."""
    n, Hkv, D = k.shape
    S, pt = fill(kind, [n], Hkv, D, -(-n // 16) + 70, seed=900, k=k.bfloat16(), v=v.bfloat16())
    lens = torch.tensor([n], dtype=torch.int32, device=dev())
    dec = bi.attention_decode_q8(q[None].to(dev()), *S.args, lens, scale=scale)
    pages = pt[0, : -(-n // 16)].tolist()
    ref, tol = attend(q.double().numpy(), S.values("k", pages, n), S.values("v", pages, n), S.value_scales(pages, n), scale)
    err = np.abs(dec[0].cpu().double().numpy() - ref)
    assert (err <= tol).all(), (float((err / tol).max()), float(np.linalg.norm(err) / np.linalg.norm(ref)))
    short = S.pt[:, : max(1, -(-n // 16))].contiguous()
    for T, table in ((1, S.pt), (3, S.pt), (40, S.pt), (40, short), (1, short)):
        pre = bi.attention_prefill_q8(q.repeat(T, 1, 1).to(dev()), torch.zeros(T, dtype=torch.int32, device=dev()),
                                      torch.full((T,), n - 1, dtype=torch.int32, device=dev()), *S.args[:4], table, scale=scale)
        assert same_bits(pre, dec.expand_as(pre).contiguous()), T
    assert bi.get_device_error() == 0


def scored(scores, Hkv, D):
    """Keys [n, Hkv, D] whose product with the query (1, 0, 0, ...) of every head is `scores` [n]."""
    k = torch.zeros(len(scores), Hkv, D)
    k[:, :, 0] = torch.as_tensor(scores, dtype=torch.float32)[:, None]
    return k


def first_axis(Hq, D):
    q = torch.zeros(Hq, D, dtype=torch.bfloat16)
    q[:, 0] = 1.0
    return q


LN2 = float(np.log(2.0))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,faint,loud", [(2, 0, 1), (2, 1, 0), (40, 5, 30), (40, 30, 5), (256, 250, 3), (700, 3, 600),
                                          (700, 600, 3)])
def test_a_faint_value_row_with_the_weight_beside_a_loud_one(kind, n, faint, loud):
    """Nearly all of the weight on a value row near 2^-54, 2^-8 of it on one near 2^97: the denominator is
    the faint token's, in one page, one split or another split."""
    D = 128
    z = torch.full((n,), -40.0)
    z[faint], z[loud] = 0.0, -8.0
    v = synth.normal_bf16((n, 1, D), 800).float()
    v *= torch.where(torch.arange(n) == loud, 2.0 ** 97, 2.0 ** -54)[:, None, None]
    check_all_forms(kind, scored(z, 1, D), v, first_axis(4, D), LN2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size,one", [(2.0 ** 118, 2.0 ** -8), (2.0 ** 125, 1.0), (2.0 ** -90, 1.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_many_small_weights_beside_a_large_one(kind, size, one, D):
    """32768 weights of 2^-20.5 beside one of 1: together 1/46 of the softmax, at either end of the
    values' range, with values of one size or the large weight's smaller."""
    n = 32769
    z = torch.full((n,), -20.5)
    z[17] = 0.0
    v = synth.normal_bf16((n, 1, D), 801).float().abs().clamp(0.5, 2.0) * size
    v[17] *= -one
    check_all_forms(kind, scored(z, 1, D), v, first_axis(8, D), LN2)


@pytest.mark.parametrize("kind", KINDS)
def test_scores_and_sizes_that_rise_and_fall_together(kind):
    """Scores that climb by 3 a page and values that fall by 4 (base 2), and the other way round: both
    references move on most pages."""
    n, D = 512, 64
    page = torch.arange(n) // 16
    for up in (1, -1):
        z = up * 3.0 * page.float() - 48.0
        v = synth.normal_bf16((n, 2, D), 802).float() * torch.exp2(-up * 4.0 * (page.float() - 16))[:, None, None]
        check_all_forms(kind, scored(z, 2, D), v, first_axis(6, D), LN2)
