"""Attention over the 8-bit store where value rows differ widely in size, or are zeros: the
softmax's denominator keeps every token that carries weight, whatever its value scale, the other
rows' weights keep their bits, and each form of the calls (decode, wide tiles, few rows,
clusters) gives the same bits."""
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


def zero_score(p, n):
    """The base-2 score at which one token holds the share p beside n - 1 tokens of score 0."""
    return float(np.log2(p / (1 - p) * (n - 1)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [0.1, 0.02, 1e-4, 2.0 ** -60, 2.0 ** 60])
@pytest.mark.parametrize("p", [0.5, 0.99, 0.9999])
@pytest.mark.parametrize("at,D", [([0], 128), ([1023], 64), ([300, 301, 777], 128), (list(range(512, 528)), 64)])
def test_zero_value_rows_with_most_of_the_weight(kind, size, p, at, D):
    """A null token or a sink: rows of zeros take p of the softmax from the first, a middle and the last
    place, and as a page of their own; what the other rows give must not lose bits to them."""
    n = 1024
    z = torch.linspace(-2, 2, n)
    z[at] = zero_score(p, n) - float(np.log2(len(at)))
    v = synth.normal_bf16((n, 2, D), 810).float() * size
    v[at] = 0
    check_all_forms(kind, scored(z, 2, D), v, first_axis(8, D), LN2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1e-7, 1e-8, 2.0 ** -97])
def test_small_values_beside_zero_rows_of_equal_weight(kind, size):
    n, D = 256, 128
    v = synth.normal_bf16((n, 1, D), 811).float().clamp(-4, 4) * size
    v[100] = 0
    check_all_forms(kind, scored(torch.zeros(n), 1, D), v, first_axis(3, D), LN2)


@pytest.mark.parametrize("kind", KINDS)
def test_nothing_but_zero_value_rows(kind):
    n, D = 300, 64
    S, _ = fill(kind, [n], 2, D, 20, seed=901, v=torch.zeros(n, 2, D, dtype=torch.bfloat16))
    q = synth.normal_bf16((1, 6, D), 812).to(dev())
    dec = bi.attention_decode_q8(q, *S.args, torch.tensor([n], dtype=torch.int32, device=dev()))
    assert bool((dec == 0).all())
    pre = bi.attention_prefill_q8(q.repeat(40, 1, 1), torch.zeros(40, dtype=torch.int32, device=dev()),
                                  torch.arange(n - 40, n, dtype=torch.int32, device=dev()), *S.args)
    assert bool((pre == 0).all()) and bi.get_device_error() == 0


@pytest.mark.parametrize("kind,one", [("int8", 127.0), ("e4m3", 448.0), ("e4m3", 225.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_whose_scale_is_one_are_not_taken_for_zero_rows(kind, one, D):
    """A row with the scale of an empty one, 1, and a single value that is not zero, in each eighth of the
    row; beside rows of zeros, with the weight spread evenly."""
    n = 40
    v = torch.zeros(n, 2, D)
    for i, d in enumerate(range(0, D, D // 8)):
        v[3 + 2 * i, 0, d + i % (D // 8)] = -one if i % 2 else one
        v[4 + 2 * i, 1, D - 1 - d] = one
    v[30:, :, :] = 1e-3 * synth.normal_bf16((10, 2, D), 813).float()
    check_all_forms(kind, scored(torch.linspace(-1, 1, n), 2, D), v, first_axis(4, D), LN2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1.0, 2.0 ** 118, 2.0 ** -92])
def test_the_least_row_that_is_kept_beside_others(kind, size):
    """A row whose largest value is 2^-100 is no zero row; it holds most of the weight here."""
    n, D = 200, 64
    z = torch.zeros(n)
    z[33] = zero_score(0.999, n)
    v = synth.normal_bf16((n, 1, D), 814).float().clamp(-4, 4) * size
    v[33] = 2.0 ** -100
    check_all_forms(kind, scored(z, 1, D), v, first_axis(4, D), LN2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_small_weights_beside_a_zero_row(kind, D):
    """32768 weights of 2^-20.5 on rows near 2^-96 beside one of 1 on a row below 2^-100, which is empty."""
    n = 32769
    z = torch.full((n,), -20.5)
    z[17] = 0.0
    v = synth.normal_bf16((n, 1, D), 801).float().abs().clamp(0.5, 2.0) * 2.0 ** -96
    v[17] *= -(2.0 ** -8)
    check_all_forms(kind, scored(z, 1, D), v, first_axis(8, D), LN2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (8, 1, 64), (16, 1, 128)])
def test_prompts_over_mixed_value_rows_have_the_decode_bits(kind, Hq, Hkv, D):
    """Value rows of 2^-40 to 2^40, every fifth one zeros, and one with a NaN that later rows see: a
    whole prompt, whose tiles mix rows that see such tokens with rows that do not, against decode."""
    n = 700
    g = torch.Generator().manual_seed(820)
    v = synth.normal_bf16((n, Hkv, D), 821).float() * torch.exp2(torch.randint(-40, 41, (n, Hkv, 1), generator=g).float())
    v[torch.rand(n, Hkv, generator=g) < 0.2] = 0
    v[649, 0, 3] = float("nan")
    S, pt = fill(kind, [n], Hkv, D, 60, seed=902, v=v.bfloat16())
    q = synth.normal_bf16((n, Hq, D), 822).to(dev())
    seq, pos = torch.zeros(n, dtype=torch.int32, device=dev()), torch.arange(n, dtype=torch.int32, device=dev())
    pre = bi.attention_prefill_q8(q, seq, pos, *S.args)
    dec = bi.attention_decode_q8(q, *S.args[:4], S.pt.expand(n, -1).contiguous(), pos + 1)
    assert same_bits(pre, dec) and bi.get_device_error() == 0
    assert bool(torch.isnan(dec[649:, : Hq // Hkv]).all()) and not bool(torch.isnan(dec[:649]).any())
    pages = pt[0, : -(-n // 16)].tolist()
    k64, v64, sv = S.values("k", pages, n), S.values("v", pages, n), S.value_scales(pages, n)
    for t in (0, 16, 255, 256, 600, 648):
        ref, tol = attend(q[t].cpu().double().numpy(), k64[:, : t + 1], v64[:, : t + 1], sv[:, : t + 1], D ** -0.5)
        err = np.abs(dec[t].cpu().double().numpy() - ref)
        assert (err <= tol).all(), (t, float((err / tol).max()))


@pytest.mark.parametrize("kind", KINDS)
def test_slots_without_a_value_scale_have_no_weight(kind):
    """Slots of a store that was cleared to zeros and not written (no contract covers them): a value
    scale of 0 takes the token out of the softmax, in decode and in prefill alike."""
    n, D, Hkv = 300, 128, 2
    S, pt = fill(kind, [n], Hkv, D, 20, seed=903)
    hole = [0, 5, 17, 256, 290]
    for i in hole:
        for t in (S.k.view(torch.int8), S.v.view(torch.int8), S.ks, S.vs):
            t[pt[0, i // 16], :, i % 16] = 0
    q = synth.normal_bf16((n, 8, D), 830).to(dev())
    seq, pos = torch.zeros(n, dtype=torch.int32, device=dev()), torch.arange(n, dtype=torch.int32, device=dev())
    pre = bi.attention_prefill_q8(q, seq, pos, *S.args)
    dec = bi.attention_decode_q8(q, *S.args[:4], S.pt.expand(n, -1).contiguous(), pos + 1)
    assert same_bits(pre, dec) and bool((dec[0] == 0).all()) and bi.get_device_error() == 0
    keep = [i for i in range(n) if i not in hole]
    pages = pt[0, : -(-n // 16)].tolist()
    ref, tol = attend(q[-1].cpu().double().numpy(), S.values("k", pages, n)[:, keep], S.values("v", pages, n)[:, keep],
                      S.value_scales(pages, n)[:, keep], D ** -0.5)
    assert (np.abs(dec[-1].cpu().double().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_non_finite_queries_over_pages_that_are_not_there(kind, D):
    """A query with a NaN or an infinity that sees no page of the store reads zeros, one that sees some
    reads NaN, in a wide tile as in decode."""
    n, T = 300, 40
    S, pt = fill(kind, [n], 2, D, 20, seed=904)
    q = synth.normal_bf16((T, 8, D), 840)
    q[::2, 0, 3], q[1::2, 5, D - 1] = float("nan"), float("inf")
    q = q.to(dev())
    pos = torch.arange(n - T, n, dtype=torch.int32, device=dev())
    for gone in (range(20), range(0, 20, 2)):
        S.pt[0] = pt[0].to(dev())
        for i in gone:
            S.pt[0, i] = S.k.shape[0] + i if i % 3 else -1
        pre = bi.attention_prefill_q8(q, torch.zeros_like(pos), pos, *S.args)
        assert bi.get_device_error() == 8
        dec = bi.attention_decode_q8(q, *S.args[:4], S.pt.expand(T, -1).contiguous(), pos + 1)
        assert bi.get_device_error() == 8 and same_bits(pre, dec)
        bad = ~torch.isfinite(q.float()).all(-1)
        assert torch.equal(torch.isnan(dec).all(-1), bad & (len(gone) < 20)) and (len(gone) < 20 or bool((dec == 0).all()))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing_but_non_finite_tokens(kind, D):
    """NaN keys, then NaN values, in all of the first 17 tokens: rows 0 to 16 see nothing else, and all
    rows read NaN, with NaN and finite queries, in a wide tile as in decode."""
    n = 60
    for side in (0, 1):
        kv = [synth.normal_bf16((n, 2, D), 850), synth.normal_bf16((n, 2, D), 851)]
        kv[side][:17, :, 1] = float("nan")
        S, _ = fill(kind, [n], 2, D, 8, seed=905, k=kv[0], v=kv[1])
        q = synth.normal_bf16((n, 8, D), 852)
        q[::3, 2, 0] = float("inf")
        q, pos = q.to(dev()), torch.arange(n, dtype=torch.int32, device=dev())
        pre = bi.attention_prefill_q8(q, torch.zeros_like(pos), pos, *S.args)
        dec = bi.attention_decode_q8(q, *S.args[:4], S.pt.expand(n, -1).contiguous(), pos + 1)
        assert same_bits(pre, dec) and bool(torch.isnan(dec).all()) and bi.get_device_error() == 0
