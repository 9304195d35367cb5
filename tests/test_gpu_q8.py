"""The 8-bit paged KV store on the GPU: quantising append and read back bit for bit, per-head
norm with rotation, and decode / prefill attention against plain 64-bit forms, with stale
slots poisoned, rows that see nothing, odd lengths and head groups, extreme scales, non-finite
rows, bad ids, captured graphs and other streams; and the bits of a row across batches."""
import numpy as np
import pytest
import torch

import invariant_deterministic_04_b200 as bi
import q8_ref
import synth
from gpu_util import dev, same_bits
from invariant_deterministic_04_b200.llama import rope_cos_sin

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3"]


def raw(t):
    return t.view(torch.int8) if t.element_size() == 1 else t.view(torch.int32)


def special_rows(D, seed):
    """bf16 rows [n, D] where a quantiser goes wrong."""
    x = synth.normal_bf16((24, D), seed).float()
    x[1] = 0
    x[2] = -0.0
    x[3] = 0
    x[3, 5] = 2.0 ** -101                      # below the smallest stored maximum
    x[4] = 0
    x[4, 7] = -(2.0 ** -100)
    x[5, 3] = float("nan")
    x[6, D - 1] = float("inf")
    x[7, 0] = float("-inf")
    x[8] *= 2.0 ** 120
    x[9] *= 2.0 ** -90
    x[10] = 129 / 128                          # 127 x / a with a = 129/128: 63.5 is a tie
    x[10, ::2] = 129 / 256
    x[11] = torch.arange(D) % 128 * 2 - 127    # a = 127: halves and integers
    x[11, 1::2] /= 2
    x[12] = 448.0                              # e4m3's largest: the scale is 1
    x[12, ::3] = 17.0                          # ties between e4m3 neighbours 16 and 18
    x[12, 1::3] = 2.0 ** -10                   # half of e4m3's least subnormal
    x[13] = 450.0
    x[13, ::2] = 3.0
    x[14] = torch.finfo(torch.bfloat16).max
    x[14, ::2] = 1.0
    x[15, ::2] *= 2.0 ** -12
    return x.bfloat16()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,Hkv,T", [(128, 8, 1), (128, 3, 45), (64, 8, 77), (64, 1, 2)])
def test_append_writes_the_documented_bits_and_nothing_else(kind, D, Hkv, T):
    lens = [40, 7, 64]
    pt, total = q8_ref.page_table(lens, 5, seed=3)
    S = q8_ref.Store(kind, total, Hkv, D, pt, seed=4)
    before = [raw(t).clone() for t in (S.k, S.v, S.ks, S.vs)]
    slots = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    order = synth.permutation(len(slots), 5)[:T].tolist()
    seq = torch.tensor([slots[i][0] for i in order], dtype=torch.int32)
    pos = torch.tensor([slots[i][1] for i in order], dtype=torch.int32)
    sp = special_rows(D, 6)
    fused = synth.normal_bf16((T, 3 * Hkv * D + 8), 7)  # k and v as parts of wider rows
    k, v = fused[:, : Hkv * D].view(T, Hkv, D), fused[:, 2 * Hkv * D: 3 * Hkv * D].view(T, Hkv, D)
    for i in range(T * Hkv):
        k[i // Hkv, i % Hkv] = sp[i % 24]
        v[i // Hkv, i % Hkv] = sp[(i + 11) % 24]
    fd = fused.to(dev())
    kd, vd = fd[:, : Hkv * D].view(T, Hkv, D), fd[:, 2 * Hkv * D: 3 * Hkv * D].view(T, Hkv, D)
    bi.kv_append_q8(kd, vd, seq.to(dev()), pos.to(dev()), *S.args)
    assert bi.get_device_error() == 0
    page, at = pt[seq.long(), pos.long() // 16].long(), pos.long() % 16
    for x, cache, scale, b0, b1 in ((k, S.k, S.ks, before[0], before[2]), (v, S.v, S.vs, before[1], before[3])):
        val, sc = q8_ref.quantise(x, kind)
        got = raw(cache).cpu()[page, :, at].view(cache.dtype).float().double().numpy()
        gs = scale.cpu()[page, :, at].double().numpy()
        assert np.array_equal(got, val)
        assert np.array_equal(gs, sc, equal_nan=True)
        keep = torch.ones(total, 16, dtype=torch.bool)
        keep[page, at] = False
        keep = keep[:, None, :].expand(total, Hkv, 16)
        assert torch.equal(raw(cache).cpu()[keep], b0.cpu()[keep])
        assert torch.equal(raw(scale).cpu()[keep], b1.cpu()[keep])
    ko, vo = bi.kv_read_q8(seq.to(dev()), pos.to(dev()), *S.args)
    for out, x in ((ko, k), (vo, v)):
        val, sc = q8_ref.quantise(x, kind)
        ref = torch.from_numpy(val * sc[..., None])  # fp32 exact: at most 8 + 24 bits, rounded once to fp32 ...
        ref = ref.float().bfloat16()                 # ... and then to bf16, as the call documents
        assert torch.equal(torch.isnan(ref), torch.isnan(out.cpu()))
        fine = ~torch.isnan(ref)
        assert torch.equal(out.cpu()[fine], ref[fine])


@pytest.mark.parametrize("kind", KINDS)
def test_rows_do_not_depend_on_their_batch(kind):
    pt, total = q8_ref.page_table([64] * 3, 4, seed=8)
    k, v = synth.normal_bf16((50, 4, 128), 9).to(dev()), synth.normal_bf16((50, 4, 128), 10).to(dev())
    seq = torch.arange(50, dtype=torch.int32) % 3
    pos = torch.arange(50, dtype=torch.int32)
    A = q8_ref.Store(kind, total, 4, 128, pt, seed=11)
    B = q8_ref.Store(kind, total, 4, 128, pt, seed=11)
    bi.kv_append_q8(k, v, seq.to(dev()), pos.to(dev()), *A.args)
    for t in synth.permutation(50, 12).tolist():
        bi.kv_append_q8(k[t:t + 1], v[t:t + 1], seq[t:t + 1].to(dev()), pos[t:t + 1].to(dev()), *B.args)
    for x, y in zip(A.args, B.args):
        assert torch.equal(raw(x), raw(y))


@pytest.mark.parametrize("kind", KINDS)
def test_append_and_read_flag_bad_ids(kind):
    pt, total = q8_ref.page_table([64, 64], 4, seed=13)
    pt[1, 2] = total + 5
    pt[1, 1] = -1
    S = q8_ref.Store(kind, total, 2, 64, pt, seed=14)
    seq = torch.tensor([0, 2, -1, 0, 0, 1, 1], dtype=torch.int32, device=dev())
    pos = torch.tensor([3, 3, 3, 64, -1, 17, 40], dtype=torch.int32, device=dev())
    k, v = synth.normal_bf16((7, 2, 64), 15).to(dev()), synth.normal_bf16((7, 2, 64), 16).to(dev())
    for t in range(7):
        before = [raw(x).clone() for x in S.args]
        bi.kv_append_q8(k[t:t + 1], v[t:t + 1], seq[t:t + 1], pos[t:t + 1], *S.args)
        assert bi.get_device_error() == (0 if t == 0 else 8)
        if t:
            assert all(torch.equal(a, raw(b)) for a, b in zip(before, S.args))
    ko, vo = bi.kv_read_q8(seq, pos, *S.args)
    assert bi.get_device_error() == 8
    assert bool((ko[1:] == 0).all()) and bool((vo[1:] == 0).all()) and bool((ko[0] != 0).any())
    again = bi.kv_read_q8(seq[:1].repeat(5), pos[:1].repeat(5), *S.args)  # rows may repeat
    assert bi.get_device_error() == 0
    assert all(same_bits(again[0][i], ko[0]) and same_bits(again[1][i], vo[0]) for i in range(5))
    # empty calls
    e = torch.empty(0, dtype=torch.int32, device=dev())
    bi.kv_append_q8(k[:0], v[:0], e, e, *S.args)
    assert bi.kv_read_q8(e, e, *S.args)[0].shape == (0, 2, 64)


# ---------------------------------------------------------------------------


@pytest.mark.parametrize("Hq,Hkv,D,T", [(32, 8, 128, 1), (32, 8, 64, 37), (7, 1, 256, 5), (3, 3, 64, 1), (28, 4, 128, 130)])
def test_qk_norm_rope_matches_64_bits_in_place_and_out(Hq, Hkv, D, T):
    W = (Hq + 2 * Hkv) * D
    fused = synth.normal_bf16((T, W), 20)
    fused[0, :D] = 0                       # a zero head: eps keeps it finite
    fused[T // 2, D: 2 * D] *= 2.0 ** 40   # loud and faint heads
    fused[T // 2, 2 * D: 3 * D] *= 2.0 ** -10
    qw, kw = synth.normal_bf16((D,), 21, 0.1, 1.0), synth.normal_bf16((D,), 22, 0.1, 1.0)
    pos = torch.randint(0, 384, (T,), generator=synth.generator(23), dtype=torch.int32)
    table = rope_cos_sin(384, D, 10000.0, dev())
    fd = fused.to(dev())
    q, k = fd[:, : Hq * D].view(T, Hq, D), fd[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
    qo, ko = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev()), torch.empty_like(k.contiguous())
    r = bi.qk_norm_rope(q, k, qw.to(dev()), kw.to(dev()), pos.to(dev()), table, 1e-6, q_out=qo, k_out=ko)
    assert r[0] is qo and r[1] is ko
    assert torch.equal(fd.cpu().view(torch.int16), fused.view(torch.int16))  # inputs untouched
    for out, x, w in ((qo, fused[:, : Hq * D].view(T, Hq, D), qw), (ko, fused[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D), kw)):
        ref, mag = q8_ref.norm_rope(x, w, table.cpu(), pos, 1e-6)
        # half a bf16 step of the result, and fp32 steps (a handful, the norm's sum of D squares
        # D/16 + 5 more at most, halved by the root) of the two products it is the sum of
        err = np.abs(out.cpu().double().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 32 * 2.0 ** -24 * mag + 1e-38).all()
    tail = fd[:, (Hq + Hkv) * D:].clone()
    bi.qk_norm_rope(q, k, qw.to(dev()), kw.to(dev()), pos.to(dev()), table, 1e-6)   # in place
    assert same_bits(q, qo) and same_bits(k, ko) and same_bits(fd[:, (Hq + Hkv) * D:], tail)
    t = T - 1                              # a row alone has the same bits
    one = fused[t:t + 1].to(dev())
    q1, k1 = one[:, : Hq * D].view(1, Hq, D), one[:, Hq * D: (Hq + Hkv) * D].view(1, Hkv, D)
    bi.qk_norm_rope(q1, k1, qw.to(dev()), kw.to(dev()), pos[t:].to(dev()), table, 1e-6)
    assert same_bits(q1[0], qo[t]) and same_bits(k1[0], ko[t])
    assert bi.get_device_error() == 0


def test_qk_norm_rope_flags_bad_positions_and_leaves_their_rows():
    q, k = synth.normal_bf16((4, 8, 64), 24).to(dev()), synth.normal_bf16((4, 2, 64), 25).to(dev())
    w = torch.ones(64, dtype=torch.bfloat16, device=dev())
    table = rope_cos_sin(10, 64, 10000.0, dev())
    pos = torch.tensor([9, 10, -1, 0], dtype=torch.int32, device=dev())
    q0, k0 = q.clone(), k.clone()
    bi.qk_norm_rope(q, k, w, w, pos, table)
    assert bi.get_device_error() == 8
    assert same_bits(q[1:3], q0[1:3]) and same_bits(k[1:3], k0[1:3])
    assert not same_bits(q[0], q0[0]) and not same_bits(k[3], k0[3])
    bi.qk_norm_rope(q[:0], k[:0], w, w, pos[:0], table)
    assert bi.get_device_error() == 0


# ---------------------------------------------------------------------------


def fill(kind, lens, Hkv, D, max_pages, seed, k=None, v=None):
    """A store holding sequences of these lengths (every other slot stale), and its page table."""
    pt, total = q8_ref.page_table(lens, max_pages, seed=seed)
    S = q8_ref.Store(kind, total, Hkv, D, pt, seed=seed + 1)
    T = sum(lens)
    if T:
        seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(lens)]).to(dev())
        pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).to(dev())
        k = synth.normal_bf16((T, Hkv, D), seed + 2) if k is None else k
        v = synth.normal_bf16((T, Hkv, D), seed + 3) if v is None else v
        bi.kv_append_q8(k.to(dev()), v.to(dev()), seq, pos, *S.args)
    return S, pt


def reference(S, pt, q, b, n, scale=None):
    pages = pt[b, : -(-n // 16)].tolist()
    D = q.shape[-1]
    return q8_ref.attend(q.double().numpy(), S.values("k", pages, n), S.values("v", pages, n),
                         q8_ref.default_scale(D) if scale is None else scale, S.value_scales(pages, n))


LENS = [0, 1, 15, 16, 17, 255, 256, 257, 700, 513, 31]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (32, 8, 64), (4, 4, 128), (14, 2, 64), (8, 1, 128), (9, 1, 128),
                                      (32, 2, 64), (10, 2, 128), (3, 1, 64)])
def test_decode_matches_64_bits(kind, Hq, Hkv, D):
    S, pt = fill(kind, LENS, Hkv, D, 45, seed=Hq + D)
    q = synth.normal_bf16((len(LENS), Hq, D), 31)
    lens = torch.tensor(LENS, dtype=torch.int32, device=dev())
    out = bi.attention_decode_q8(q.to(dev()), *S.args, lens)
    assert bi.get_device_error() == 0
    assert bool((out[0].view(torch.int16) == 0).all())  # no key: +0 in every bit
    for b, n in enumerate(LENS):
        q8_ref.assert_attention_close(out[b], *reference(S, pt, q[b], b, n))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (32, 8, 64), (5, 1, 128), (16, 1, 64), (4, 4, 128)])
def test_prefill_rows_are_the_decode_rows_bit_for_bit(kind, Hq, Hkv, D):
    """Whole prompts, chunks, shuffled rows and mixed batches all give a row the decode bits."""
    lens = [300, 1, 530, 64]
    S, pt = fill(kind, lens, Hkv, D, 40, seed=Hq + 2 * D)
    rows = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    T = len(rows)
    seq = torch.tensor([r[0] for r in rows], dtype=torch.int32, device=dev())
    pos = torch.tensor([r[1] for r in rows], dtype=torch.int32, device=dev())
    wide = synth.normal_bf16((T, Hq * D + 64), 32).to(dev())
    q = wide[:, : Hq * D].view(T, Hq, D)                       # strided rows
    whole = bi.attention_prefill_q8(q, seq, pos, *S.args)
    # every row by decode: the page-table row of its sequence, its own length
    table = S.pt[seq.long()].contiguous()
    dec = bi.attention_decode_q8(q.contiguous(), *S.args[:4], table, pos + 1)
    assert bi.get_device_error() == 0
    assert same_bits(whole, dec)
    for n in (1, 7, 64, 513):                                   # chunks that cut anywhere
        parts = [bi.attention_prefill_q8(q[a:a + n], seq[a:a + n], pos[a:a + n], *S.args) for a in range(0, T, n)]
        assert same_bits(torch.cat(parts), whole)
    perm = synth.permutation(T, 33).to(dev())                   # rows in any order
    assert same_bits(bi.attention_prefill_q8(q[perm].contiguous(), seq[perm], pos[perm], *S.args), whole[perm])
    some = torch.cat([torch.arange(290, 300), torch.tensor([300, T - 1]), torch.arange(301, 420)]).to(dev())
    assert same_bits(bi.attention_prefill_q8(q[some].contiguous(), seq[some], pos[some], *S.args), whole[some])
    for t in (0, 15, 16, 255, 256, 299, 300, T - 1):
        b, p = rows[t]
        q8_ref.assert_attention_close(whole[t], *reference(S, pt, q[t].cpu(), b, p + 1))


@pytest.mark.parametrize("kind", KINDS)
def test_decode_rows_do_not_depend_on_batch_order_or_stale_slots(kind):
    S, pt = fill(kind, LENS, 8, 128, 45, seed=40)
    B = len(LENS)
    q = synth.normal_bf16((B, 32, 128), 41).to(dev())
    lens = torch.tensor(LENS, dtype=torch.int32, device=dev())
    out = bi.attention_decode_q8(q, *S.args, lens)
    perm = synth.permutation(B, 42).to(dev())
    again = bi.attention_decode_q8(q[perm].contiguous(), *S.args[:4], S.pt[perm].contiguous(), lens[perm].contiguous())
    assert same_bits(again, out[perm])
    for b in (1, 8, 9):
        one = bi.attention_decode_q8(q[b:b + 1], *S.args[:4], S.pt[b:b + 1], lens[b:b + 1])
        assert same_bits(one[0], out[b])
    # other junk in every slot that no sequence sees
    live = torch.zeros(S.k.shape[0], 16, dtype=torch.bool)
    for b, n in enumerate(LENS):
        for p in range(n):
            live[pt[b, p // 16], p % 16] = True
    dead = ~live.to(dev())[:, None, :].expand(-1, 8, -1)
    for t in (S.k, S.v):
        raw(t)[dead] = 0x7E if kind == "e4m3" else -128
    for t in (S.ks, S.vs):
        t[dead] = float("inf")
    assert same_bits(bi.attention_decode_q8(q, *S.args, lens), out)


@pytest.mark.parametrize("kind", KINDS)
def test_non_finite_rows_reach_the_rows_that_see_them_and_no_others(kind):
    lens = [40, 40, 40, 40]
    k, v = synth.normal_bf16((160, 2, 64), 50), synth.normal_bf16((160, 2, 64), 51)
    k[40 + 20, 1, 3] = float("nan")        # sequence 1, token 20, kv-head 1
    v[80 + 33, 0, 0] = float("inf")        # sequence 2, token 33, kv-head 0
    S, pt = fill(kind, lens, 2, 64, 4, seed=52, k=k, v=v)
    q = synth.normal_bf16((4, 6, 64), 53)
    q[3, 0, 5] = float("nan")
    q[3, 1, 5] = float("-inf")
    for n in (40, 21, 20, 34, 33):
        out = bi.attention_decode_q8(q.to(dev()), *S.args, torch.full((4,), n, dtype=torch.int32, device=dev())).cpu()
        nan = torch.isnan(out).all(-1)
        assert torch.equal(nan, torch.isnan(out).any(-1))
        want = torch.zeros(4, 6, dtype=torch.bool)
        want[1, 3:] = n > 20
        want[2, :3] = n > 33
        want[3, :2] = True
        assert torch.equal(nan, want)
        seq = torch.arange(4, dtype=torch.int32, device=dev())
        pre = bi.attention_prefill_q8(q.to(dev()), seq, torch.full_like(seq, n - 1), *S.args).cpu()
        assert torch.equal(torch.isnan(pre).all(-1), want)


@pytest.mark.parametrize("kind", KINDS)
def test_scales_far_apart(kind):
    """Loud and faint tokens, zero keys and zero values: a faint value row with most of the weight
    must not be lost to a loud one with little, nor the other way round."""
    n, Hkv, D = 300, 2, 128
    k, v = synth.normal_bf16((n, Hkv, D), 60).float(), synth.normal_bf16((n, Hkv, D), 61).float()
    v[::7] = 0
    k[::11] = 0
    v[5] *= 2.0 ** -30
    v[6] *= 2.0 ** 20
    k[8] *= 8
    v[200:] *= 2.0 ** 40
    S, pt = fill(kind, [n], Hkv, D, 20, seed=62, k=k.bfloat16(), v=v.bfloat16())
    for loud in (1.0, 2.0 ** -60, 4.0):
        q = (synth.normal_bf16((1, 8, D), 63).float() * loud).bfloat16()
        for L in (n, 199, 16):
            out = bi.attention_decode_q8(q.to(dev()), *S.args, torch.tensor([L], dtype=torch.int32, device=dev()))
            q8_ref.assert_attention_close(out[0], *reference(S, pt, q[0], 0, L))
    # huge queries against tiny keys: the product is ordinary
    S, pt = fill(kind, [n], Hkv, D, 20, seed=64, k=(synth.normal_bf16((n, Hkv, D), 65).float() * 2.0 ** -70).bfloat16())
    q = (synth.normal_bf16((1, 8, D), 66).float() * 2.0 ** 70).bfloat16()
    out = bi.attention_decode_q8(q.to(dev()), *S.args, torch.tensor([n], dtype=torch.int32, device=dev()))
    q8_ref.assert_attention_close(out[0], *reference(S, pt, q[0], 0, n))


def test_closed_forms_and_other_scales():
    S, pt = fill("int8", [1, 300], 2, 64, 20, seed=70, k=torch.ones(301, 2, 64, dtype=torch.bfloat16))
    q = synth.normal_bf16((2, 4, 64), 71).to(dev())
    out = bi.attention_decode_q8(q, *S.args, torch.tensor([1, 300], dtype=torch.int32, device=dev()))
    ko, vo = bi.kv_read_q8(torch.zeros(1, dtype=torch.int32, device=dev()), torch.zeros(1, dtype=torch.int32, device=dev()),
                           *S.args)
    assert same_bits(out[0], vo[0].repeat_interleave(2, 0))     # one key: its value
    mean = S.values("v", pt[1, :19].tolist(), 300).mean(1).repeat(2, axis=0)  # equal keys: the mean
    mag = np.abs(S.values("v", pt[1, :19].tolist(), 300)).mean(1).repeat(2, axis=0)
    q8_ref.assert_attention_close(out[1], mean, mag)
    zero = bi.attention_decode_q8(q, *S.args, torch.tensor([1, 300], dtype=torch.int32, device=dev()), scale=0.0)
    q8_ref.assert_attention_close(zero[1], mean, mag)
    S, pt = fill("e4m3", [77], 2, 64, 20, seed=72)
    neg = bi.attention_decode_q8(q[:1], *S.args, torch.tensor([77], dtype=torch.int32, device=dev()), scale=-0.3)
    q8_ref.assert_attention_close(neg[0], *reference(S, pt, q[0].cpu(), 0, 77, scale=-0.3))


@pytest.mark.parametrize("kind", KINDS)
def test_attention_flags_bad_pages_and_lengths(kind):
    lens = [64, 64, 64]
    S, pt = fill(kind, lens, 2, 128, 4, seed=80)
    S.pt[1, 1] = S.k.shape[0]          # tokens 16..31 of sequence 1 are not seen
    S.pt[2, :] = -1                    # sequence 2 has no page at all
    q = synth.normal_bf16((3, 8, 128), 81).to(dev())
    out = bi.attention_decode_q8(q, *S.args, torch.tensor(lens, dtype=torch.int32, device=dev()))
    assert bi.get_device_error() == 8
    q8_ref.assert_attention_close(out[0], *reference(S, pt, q[0].cpu(), 0, 64))
    pages = [int(pt[1, i]) for i in (0, 2, 3)]
    q8_ref.assert_attention_close(out[1], *q8_ref.attend(q[1].cpu().double().numpy(), S.values("k", pages, 48),
                                                         S.values("v", pages, 48), 128 ** -0.5))
    assert bool((out[2] == 0).all())
    seq = torch.arange(3, dtype=torch.int32, device=dev())
    pre = bi.attention_prefill_q8(q, seq, torch.full_like(seq, 63), *S.args)
    assert bi.get_device_error() == 8 and same_bits(pre, out)
    # lengths beyond the table, bad sequence ids, positions below -1; -1 sees nothing without an error
    bad = bi.attention_decode_q8(q, *S.args, torch.tensor([65, -1, 0], dtype=torch.int32, device=dev()))
    assert bi.get_device_error() == 8 and bool((bad == 0).all())
    for s, p, code in ((3, 5, 8), (-1, 5, 8), (0, 64, 8), (0, -2, 8), (0, -1, 0)):
        r = bi.attention_prefill_q8(q[:1], torch.tensor([s], dtype=torch.int32, device=dev()),
                                    torch.tensor([p], dtype=torch.int32, device=dev()), *S.args)
        assert bi.get_device_error() == code and bool((r == 0).all())


def test_empty_batches_and_given_outputs():
    S, _ = fill("int8", [64], 2, 64, 4, seed=85)
    e = torch.empty(0, dtype=torch.int32, device=dev())
    q0 = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=dev())
    assert bi.attention_decode_q8(q0, *S.args, e).shape == (0, 4, 64)
    assert bi.attention_prefill_q8(q0, e, e, *S.args).shape == (0, 4, 64)
    q = synth.normal_bf16((3, 4, 64), 86).to(dev())
    seq, pos = torch.zeros(3, dtype=torch.int32, device=dev()), torch.arange(3, dtype=torch.int32, device=dev())
    pool = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device=dev())
    ws = torch.empty(bi.attention_prefill_q8_workspace_size(3), dtype=torch.uint8, device=dev())
    r = bi.attention_prefill_q8(q, seq, pos, *S.args, out=pool[1:4], workspace=ws)
    assert r.data_ptr() == pool[1:4].data_ptr()
    assert bool((pool[0] == 7).all()) and bool((pool[4] == 7).all())
    assert same_bits(r, bi.attention_prefill_q8(q, seq, pos, *S.args))
    with pytest.raises(bi.BIError, match="WORKSPACE"):
        bi.attention_prefill_q8(q, seq, pos, *S.args, workspace=ws[:256])
    with pytest.raises(bi.BIError, match="SHAPE"):              # out over q
        bi.attention_prefill_q8(q, seq, pos, *S.args, out=q)


@pytest.mark.parametrize("kind", KINDS)
def test_a_store_beyond_32_bit_offsets(kind):
    """Pages past 4 GiB of cache bytes are found (num_pages * Hkv * 16 * D > 2^32)."""
    Hkv, D = 8, 128
    total = (1 << 32) // (Hkv * 16 * D) + 40
    pt = torch.tensor([[total - 1, total - 9, 5], [total - 2, total - 30, total - 31]], dtype=torch.int32)
    S = q8_ref.Store.__new__(q8_ref.Store)
    S.kind = kind
    S.k = torch.empty((total, Hkv, 16, D), dtype=torch.int8, device=dev()).view(q8_ref.KINDS[kind])
    S.v = torch.empty((total, Hkv, 16, D), dtype=torch.int8, device=dev()).view(q8_ref.KINDS[kind])
    S.ks = torch.empty((total, Hkv, 16), device=dev())
    S.vs = torch.empty((total, Hkv, 16), device=dev())
    S.pt = pt.to(dev())
    k, v = synth.normal_bf16((96, Hkv, D), 90).to(dev()), synth.normal_bf16((96, Hkv, D), 91).to(dev())
    seq = (torch.arange(96, dtype=torch.int32) // 48).to(dev())
    pos = (torch.arange(96, dtype=torch.int32) % 48).to(dev())
    bi.kv_append_q8(k, v, seq, pos, *S.args)
    ko, _ = bi.kv_read_q8(seq, pos, *S.args)
    val, sc = q8_ref.quantise(k.cpu(), kind)
    assert torch.equal(ko.cpu(), torch.from_numpy(val * sc[..., None]).float().bfloat16())
    q = synth.normal_bf16((2, 32, D), 92)
    out = bi.attention_decode_q8(q.to(dev()), *S.args, torch.tensor([48, 41], dtype=torch.int32, device=dev()))
    pre = bi.attention_prefill_q8(q.to(dev()), torch.tensor([0, 1], dtype=torch.int32, device=dev()),
                                  torch.tensor([47, 40], dtype=torch.int32, device=dev()), *S.args)
    assert bi.get_device_error() == 0 and same_bits(out, pre)
    for b, n in ((0, 48), (1, 41)):
        q8_ref.assert_attention_close(out[b], *reference(S, pt, q[b], b, n))


def test_streams_and_captured_graphs():
    """Two captured graphs (append, norm, decode, prefill) with their own workspaces, replayed on two
    streams in turn on changed inputs, and eager calls on a side stream, give the eager bits."""
    Hq, Hkv, D, B = 8, 2, 128, 5
    lens = [300, 20, 1, 257, 64]
    table = rope_cos_sin(512, D, 10000.0, dev())
    w = synth.normal_bf16((D,), 95, 0.1, 1.0).to(dev())

    class Side:
        def __init__(self, seed):
            self.S, _ = fill("int8", lens, Hkv, D, 30, seed=seed)
            self.q = synth.normal_bf16((B, Hq, D), seed + 5).to(dev())
            self.k, self.v = (synth.normal_bf16((B, Hkv, D), seed + i).to(dev()) for i in (6, 7))
            self.seq = torch.arange(B, dtype=torch.int32, device=dev())
            self.pos = torch.tensor(lens, dtype=torch.int32, device=dev()) - 1
            self.qn, self.kn = torch.empty_like(self.q), torch.empty_like(self.k)
            self.wsd = torch.empty(bi.attention_workspace_size(B, Hq, D, 30), dtype=torch.uint8, device=dev())
            self.wsp = torch.empty(bi.attention_prefill_q8_workspace_size(B), dtype=torch.uint8, device=dev())
            self.od, self.op = torch.empty_like(self.q), torch.empty_like(self.q)

        def step(self, **kw):
            bi.qk_norm_rope(self.q, self.k, w, w, self.pos, table, q_out=self.qn, k_out=self.kn, **kw)
            bi.kv_append_q8(self.kn, self.v, self.seq, self.pos, *self.S.args, **kw)
            bi.attention_decode_q8(self.qn, *self.S.args, self.pos + 1 if not kw else self.lens, out=self.od,
                                   workspace=self.wsd, **kw)
            bi.attention_prefill_q8(self.qn, self.seq, self.pos, *self.S.args, out=self.op, workspace=self.wsp, **kw)

    sides = [Side(100), Side(200)]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in sides:
        s.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step()
        graphs.append(g)
    for rnd in range(3):
        for i, s in enumerate(sides):
            s.q.copy_(synth.normal_bf16((B, Hq, D), 300 + 10 * rnd + i).to(dev()))
            s.k.copy_(synth.normal_bf16((B, Hkv, D), 400 + 10 * rnd + i).to(dev()))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        got = [(s.od.clone(), s.op.clone(), raw(s.S.k).clone()) for s in sides]
        for s, (od, op, k) in zip(sides, got):
            assert same_bits(od, op)
            s.lens = s.pos + 1
            torch.cuda.synchronize()
            s.step(stream=streams[0])
            streams[0].synchronize()
            assert same_bits(s.od, od) and same_bits(s.op, op) and torch.equal(raw(s.S.k), k)
    assert bi.get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [2.0 ** -97, 2.0 ** 120])
def test_value_rows_at_both_ends_of_the_range(kind, size):
    """Sums over 8192 tokens whose value rows are all near the least or the largest stored size. The
    first page of every 256 tokens scores 0 and all others 7.89 (base 2): just under the step that
    moves the softmax's reference, so the sums are as large as they get. |z| < 128 here: the fp32
    scores move a weight by less than 128 * 8 * 2^-24 = 2^-14, and the reciprocal of a value scale
    keeps 12 bits (2^-13); together, for numerator and denominator, under the 2^-11 of the tolerance."""
    n, Hq, D = 8192, 4, 64
    k = torch.zeros(n, 1, D)
    k[torch.arange(n) % 256 >= 16, :, 0] = 1
    v = (synth.normal_bf16((n, 1, D), 70).float().abs().clamp(0.25, 2.0) * size).bfloat16()
    S, pt = fill(kind, [n], 1, D, n // 16, seed=71, k=k.bfloat16(), v=v)
    q = torch.zeros(1, Hq, D, dtype=torch.bfloat16)
    q[..., 0] = 5.46875
    ref, mag = reference(S, pt, q[0], 0, n, scale=1.0)
    out = bi.attention_decode_q8(q.to(dev()), *S.args, torch.tensor([n], dtype=torch.int32, device=dev()), scale=1.0)
    q8_ref.assert_attention_close(out[0].double() / size, ref / size, mag / size)
    T = 40                                            # rows enough for a wide tile and its last rows
    pre = bi.attention_prefill_q8(q.repeat(T, 1, 1).to(dev()), torch.zeros(T, dtype=torch.int32, device=dev()),
                                  torch.full((T,), n - 1, dtype=torch.int32, device=dev()), *S.args, scale=1.0)
    assert bi.get_device_error() == 0 and same_bits(pre, out.expand_as(pre).contiguous())


def test_a_captured_chunk_replays_with_the_eager_bits():
    """A prompt chunk, its last rows and a decode row of another sequence in one captured prefill
    call: the work list and its ticket are rebuilt by every replay, on one stream after the other."""
    Hq, Hkv, D, n = 8, 8, 128, 700
    S, _ = fill("e4m3", [n, 90], Hkv, D, 50, seed=310)
    rows = list(range(n - 401, n)) + [89]
    seq = torch.tensor([0] * 401 + [1], dtype=torch.int32, device=dev())
    pos = torch.tensor(rows, dtype=torch.int32, device=dev())
    q = synth.normal_bf16((402, Hq, D), 311).to(dev())
    ws = torch.empty(bi.attention_prefill_q8_workspace_size(402), dtype=torch.uint8, device=dev())
    out = torch.empty_like(q)
    bi.attention_prefill_q8(q, seq, pos, *S.args, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bi.attention_prefill_q8(q, seq, pos, *S.args, out=out, workspace=ws)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rnd in range(4):
        q.copy_(synth.normal_bf16((402, Hq, D), 320 + rnd).to(dev()))
        pos[:401] -= 60 * rnd                         # other lengths, and in the end rows that see nothing
        torch.cuda.synchronize()
        want = bi.attention_prefill_q8(q, seq, pos.clamp(min=-1), *S.args)
        out.fill_(float("nan"))
        pos.clamp_(min=-1)
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[rnd % 2]):
            g.replay()
            g.replay()
        torch.cuda.synchronize()
        assert same_bits(out, want)
    assert int((pos == -1).sum()) > 0 and bi.get_device_error() == 0


@pytest.mark.parametrize("kind,Hq,Hkv,D", [("int8", 16, 2, 128), ("e4m3", 14, 2, 64), ("int8", 16, 1, 64),
                                           ("e4m3", 32, 8, 128)])
def test_few_rows_of_long_contexts_have_the_decode_bits(kind, Hq, Hkv, D):
    """Short chunks and decode rows over up to 37 splits (more than a cluster's warps take at a time),
    alone and beside a chunk of many rows or many decode rows, and rows that see nothing."""
    lens = [9300, 1024, 1025, 8193, 40, 0]
    S, _ = fill(kind, lens, Hkv, D, 600, seed=330)
    chunks = [(0, range(9290, 9300)), (5, [-1]), (1, [1023]), (2, range(1020, 1025)), (3, [8192, 8191, 3]), (4, range(30, 40))]
    wide = chunks + [(0, range(9000, 9280))]
    many = [(b, [n - 1]) for b, n in enumerate(lens)] * 30
    for parts in (chunks, wide, many):
        seq = torch.tensor([b for b, r in parts for _ in r], dtype=torch.int32, device=dev())
        pos = torch.tensor([x for _, r in parts for x in r], dtype=torch.int32, device=dev())
        q = synth.normal_bf16((len(seq), Hq, D), 331).to(dev())
        pre = bi.attention_prefill_q8(q, seq, pos, *S.args)
        dec = bi.attention_decode_q8(q, *S.args[:4], S.pt[seq.long()].contiguous(), pos + 1)
        assert bi.get_device_error() == 0 and same_bits(pre, dec)
