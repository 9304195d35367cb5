"""The forms that the 8-bit store's calls take by size: each is run here, against decode rows bit
for bit, against the 64-bit form, or against the same rows alone."""
import numpy as np
import pytest
import torch

import invariant_deterministic_04_b200 as bi
import q8_ref
import synth
from gpu_util import dev, same_bits
from invariant_deterministic_04_b200.llama import rope_cos_sin
from test_gpu_q8 import fill, reference

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3"]


@pytest.mark.parametrize("Hq,Hkv,period", [(16, 2, 2), (8, 2, 4), (8, 2, 2), (4, 4, 16), (16, 1, 1)])
def test_rows_of_sequences_in_turn_are_few_row_tiles(Hq, Hkv, period):
    """Runs of one row: none of them may take a wide tile. The first two numbers of the workspace are the
    counts of wide and of few-row tiles. A run of one row more than a few-row tile holds is wide."""
    D, few = 64, 16 // (Hq // Hkv)
    lens = [40 + i for i in range(period + 1)]
    S, _ = fill("int8", lens, Hkv, D, 8, seed=500)
    T = 20 * (period + 1)
    seq = torch.arange(T, dtype=torch.int32, device=dev()) % (period if period > 1 else 2)
    seq[T - few - 1:] = period  # one run of few + 1 rows
    pos = torch.arange(T, dtype=torch.int32, device=dev()) % 40
    q = synth.normal_bf16((T, Hq, D), 501).to(dev())
    ws = torch.zeros(bi.attention_prefill_q8_workspace_size(T), dtype=torch.uint8, device=dev())
    pre = bi.attention_prefill_q8(q, seq, pos, *S.args, workspace=ws)
    dec = bi.attention_decode_q8(q, *S.args[:4], S.pt[seq.long()].contiguous(), pos + 1)
    assert same_bits(pre, dec) and bi.get_device_error() == 0
    assert ws[:8].view(torch.int32).tolist() == [1, T - few - 1]


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def close(S, pt, out, q, b, n):
    """Row out [Hq, D] of sequence b at length n against 64 bits."""
    q8_ref.assert_attention_close(out, *reference(S, pt, q.cpu(), b, n))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,T", [(32, 32, 700), (32, 8, 600), (32, 8, 730), (64, 4, 380), (28, 4, 830)])
def test_wide_tiles_of_more_than_128_query_rows(kind, Hq, Hkv, T):
    """Prompts cut into tiles of 129 to 192 query rows of 128 dims, three tiles of 8 to some or all folding
    warps (the workspace's first number is the count of wide tiles), after 90 cached tokens."""
    D, n = 128, T + 90
    S, pt = fill(kind, [n], Hkv, D, 64, seed=510)
    q = synth.normal_bf16((T, Hq, D), 511).to(dev())
    seq = torch.zeros(T, dtype=torch.int32, device=dev())
    pos = torch.arange(90, n, dtype=torch.int32, device=dev())
    ws = torch.zeros(bi.attention_prefill_q8_workspace_size(T), dtype=torch.uint8, device=dev())
    pre = bi.attention_prefill_q8(q, seq, pos, *S.args, workspace=ws)
    tiles = int(ws[:4].view(torch.int32))
    if sms() == 148:  # the tile follows the SM count
        assert tiles > 0 and T // tiles * (Hq // Hkv) > 128
    dec = bi.attention_decode_q8(q, *S.args[:4], S.pt.expand(T, -1).contiguous(), pos + 1)
    assert same_bits(pre, dec) and bi.get_device_error() == 0
    for t in (0, 1, T // 2, T - 1):
        close(S, pt, pre[t], q[t], 0, 91 + t)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 1, 128), (11, 1, 128), (16, 1, 64), (10, 1, 64), (32, 4, 128)])
def test_decode_of_more_than_two_rounds_of_splits(kind, Hq, Hkv, D):
    """One CTA an SM (12 or 16 warps), by the rule on rows x splits x kv-heads, with ragged lengths,
    rows that see nothing and one of the longest; each row has the bits that it has alone, where CTAs have
    four warps, and in a prefill call."""
    G = Hq // Hkv
    warps = 12 if D * (1 if G <= 8 else 2) == 256 else 16
    B, max_pages = 37, max(16 * (2 * warps * sms() // (37 * Hkv) + 1), 563)  # (563 pages: the longest row)
    g = torch.Generator().manual_seed(520)
    lens = torch.randint(1, 1500, (B,), generator=g).tolist()
    lens[3], lens[20], lens[36] = 0, 9000, 1
    S, pt = fill(kind, lens, Hkv, D, max_pages, seed=521)
    q = synth.normal_bf16((B, Hq, D), 522).to(dev())
    n = torch.tensor(lens, dtype=torch.int32, device=dev())
    out = bi.attention_decode_q8(q, *S.args, n)
    for b in range(B):
        pages = max(1, -(-lens[b] // 16))
        one = bi.attention_decode_q8(q[b:b + 1], *S.args[:4], S.pt[b:b + 1, :pages].contiguous(), n[b:b + 1])
        assert same_bits(one[0], out[b]), b
    seq = torch.arange(B, dtype=torch.int32, device=dev())
    assert same_bits(bi.attention_prefill_q8(q, seq, n - 1, *S.args), out)
    assert bi.get_device_error() == 0 and bool((out[3] == 0).all())
    for b in (0, 20, 36):
        close(S, pt, out[b], q[b], b, lens[b])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(16, 1), (11, 1), (20, 2)])
def test_prefill_of_more_than_eight_heads_a_group(kind, Hq, Hkv):
    """9 to 16 query heads of 128 dims to a kv-head: a prompt, chunks of it, and few rows of a long
    context alone (clusters) and beside a chunk."""
    D, lens = 128, [330, 9100, 40]
    S, pt = fill(kind, lens, Hkv, D, 600, seed=530)
    whole = [(0, t) for t in range(330)]
    few = [(1, t) for t in range(9093, 9100)] + [(2, 39)]
    for rows in (whole, few, whole + few, [(1, 9099)]):
        seq = torch.tensor([r[0] for r in rows], dtype=torch.int32, device=dev())
        pos = torch.tensor([r[1] for r in rows], dtype=torch.int32, device=dev())
        q = synth.normal_bf16((len(rows), Hq, D), 531).to(dev())
        pre = bi.attention_prefill_q8(q, seq, pos, *S.args)
        dec = bi.attention_decode_q8(q, *S.args[:4], S.pt[seq.long()].contiguous(), pos + 1)
        assert same_bits(pre, dec)
        parts = [bi.attention_prefill_q8(q[a:a + 21], seq[a:a + 21], pos[a:a + 21], *S.args) for a in range(0, len(rows), 21)]
        assert same_bits(torch.cat(parts), pre)
        for t in (0, len(rows) - 1):
            close(S, pt, pre[t], q[t], rows[t][0], rows[t][1] + 1)
    assert bi.get_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(28, 2, 128), (28, 4, 128), (5, 2, 64), (12, 1, 256), (1, 1, 128)])
@pytest.mark.parametrize("in_place", [True, False])
def test_qk_norm_rope_of_many_rows(Hq, Hkv, D, in_place):
    """Four heads a group of lanes (head counts that are and are not multiples of four): each row has
    the bits that it has in a small call, which takes one head a group, and is right in 64 bits."""
    T = sms() * 4096 * 16 // ((Hq + Hkv) * D) + 37
    table = rope_cos_sin(300, D, 10000.0, dev())
    qw, kw = (synth.normal_bf16((D,), s, 0.2, 1.0).to(dev()) for s in (541, 542))
    wide = synth.normal_bf16((T, (Hq + Hkv) * D + 8), 543).to(dev())   # fused rows with a gap
    q, k = (wide[:, a * D: b * D].view(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + Hkv)))
    pos = (torch.arange(T, dtype=torch.int32) * 7 % 300).to(dev())
    q0, k0, gap = q.clone(), k.clone(), wide[:, -8:].clone()
    outs = {} if in_place else dict(q_out=torch.empty_like(q0), k_out=torch.empty_like(k0))
    qn, kn = bi.qk_norm_rope(q, k, qw, kw, pos, table, **outs)
    if not in_place:
        assert same_bits(q, q0) and same_bits(k, k0)
    assert same_bits(wide[:, -8:], gap)
    step = T // 4 + 1                                                   # below the rule's limit
    for a in range(0, T, step):
        qs, ks = bi.qk_norm_rope(q0[a:a + step], k0[a:a + step], qw, kw, pos[a:a + step], table,
                                 q_out=torch.empty_like(q0[a:a + step]), k_out=torch.empty_like(k0[a:a + step]))
        assert same_bits(qn[a:a + step], qs) and same_bits(kn[a:a + step], ks)
    one = torch.tensor([0, 1, T // 3, T - 1])
    assert bi.get_device_error() == 0
    for x, w, got in ((q0, qw, qn), (k0, kw, kn)):
        y, mag = q8_ref.norm_rope(x[one].cpu(), w.cpu(), table.cpu(), pos[one].cpu(), 1e-6)
        # one rounding to bf16 (2^-8 of y), fp32 before it: 16 + 4 sums and 5 products, 2^-19 of the terms
        err = np.abs(got[one].cpu().double().numpy() - y)
        assert (err <= 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * mag).all()


def test_captured_clusters_and_large_decode_replay_with_the_eager_bits():
    """Few rows of long contexts (clusters of CTAs) and a decode of more than two rounds of splits in one
    captured graph, replayed on changed queries and lengths, beside a second graph on another stream."""
    Hq, Hkv, D, B, max_pages = 16, 2, 128, 40, 1600
    lens = [9000, 1, 0, 4000] + [300 + 7 * i for i in range(B - 4)]

    class Side:
        def __init__(self, seed, kind):
            self.S, _ = fill(kind, lens, Hkv, D, max_pages, seed=seed)
            self.n = torch.tensor(lens, dtype=torch.int32, device=dev())
            self.q = synth.normal_bf16((B, Hq, D), seed).to(dev())
            self.few = synth.normal_bf16((6, Hq, D), seed + 1).to(dev())
            self.seq = torch.tensor([0, 0, 0, 3, 1, 2], dtype=torch.int32, device=dev())
            self.pos = torch.tensor([8997, 8998, 8999, 3999, 0, -1], dtype=torch.int32, device=dev())

        def step(self):
            return (bi.attention_decode_q8(self.q, *self.S.args, self.n),
                    bi.attention_prefill_q8(self.few, self.seq, self.pos, *self.S.args))

    sides, streams = [Side(550, "int8"), Side(560, "e4m3")], [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for s in sides:
        s.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.out = s.step()
        graphs.append(g)
    for rnd in range(3):
        for i, s in enumerate(sides):
            s.q.copy_(synth.normal_bf16((B, Hq, D), 570 + 2 * rnd + i).to(dev()))
            s.few.copy_(synth.normal_bf16((6, Hq, D), 580 + 2 * rnd + i).to(dev()))
            s.n[4:] -= 40
            s.pos[:4] -= 300 * rnd
            for t in s.out:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for s in sides:
            dec, pre = s.step()
            assert same_bits(s.out[0], dec) and same_bits(s.out[1], pre)
    assert bi.get_device_error() == 0
    for g in graphs:
        g.reset()
