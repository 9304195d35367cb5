"""Cases of the 8-bit paged KV store's operators, in plain torch and through the library.

Operators (see include/bi.h for the contracts):
  qk_norm_rope                  per-head RMSNorm of queries and keys with the rotation in the same pass
  kv_append_q8, kv_read_q8      quantise rows as they are written into the store, and read them back
  attention_decode_q8           one new token per sequence over the store
  attention_prefill_q8          prompt rows (and decode rows among them) over the store

`run` computes an operator in plain torch operations, or with `own` set through the
library. The store: k_cache, v_cache [num_pages, Hkv, 16, D] in int8 or e4m3, k_scale,
v_scale [num_pages, Hkv, 16] fp32; a page table row lists a sequence's pages, -1 past its end.
"""
import math
import random

import torch

own = False

PAGE = 16
DTYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # one decode token of a 32/8-head model: the launch itself is the cost
        dict(name="norm_rope 1 row", op="norm", T=1, Hq=32, Hkv=8, D=128, max_pos=32768),
        # a mixed step of the small decoder's layout (32/8 heads of 64), an odd row count
        dict(name="norm_rope 577 rows d64", op="norm", T=577, Hq=32, Hkv=8, D=64, max_pos=384),
        # a long prompt's rows
        dict(name="norm_rope 32768 rows", op="norm", T=32768, Hq=32, Hkv=8, D=128, max_pos=32768),
        # the new tokens of a decode batch of 64
        dict(name="append 64 rows e4m3", op="append", kind="e4m3", T=64, Hkv=8, D=128, seqs=64, max_len=4096),
        # many prompts written at once
        dict(name="append 65536 rows int8", op="append", kind="int8", T=65536, Hkv=8, D=128, seqs=16, max_len=4096),
        # one user's long context
        dict(name="decode B1 L16921 int8", op="decode", kind="int8", B=1, Hq=32, Hkv=8, D=128, min_len=16921,
             max_len=16921, lens_seed=1),
        # the small decoder's full batch near its end (prompts of 128, up to 256 generated)
        dict(name="decode B64 L384 d64 e4m3", op="decode", kind="e4m3", B=64, Hq=32, Hkv=8, D=64, min_len=128,
             max_len=384, lens_seed=2),
        # a middling batch with eight query heads to a kv-head
        dict(name="decode B16 G8 e4m3", op="decode", kind="e4m3", B=16, Hq=64, Hkv=8, D=128, min_len=1,
             max_len=32768, lens_seed=3),
        # the long-context batch: lengths uniform in 1..32768
        dict(name="decode B64 L32768 int8", op="decode", kind="int8", B=64, Hq=32, Hkv=8, D=128, min_len=1,
             max_len=32768, lens_seed=4),
        # a 4096-token prompt in one piece
        dict(name="prefill S4096 int8", op="prefill", kind="int8", chunks="1x4096+0", decodes=0, Hq=32, Hkv=8, D=128,
             max_len=4096, lens_seed=5),
        # its last 512-token chunk, after 3584 cached tokens
        dict(name="prefill chunk 512 e4m3", op="prefill", kind="e4m3", chunks="1x512+3584", decodes=0, Hq=32, Hkv=8,
             D=128, max_len=4096, lens_seed=6),
        # a mixed step of the small decoder: odd prompt chunks and 48 decode tokens
        dict(name="prefill mixed d64 int8", op="prefill", kind="int8", chunks="15x77+40", decodes=48, Hq=32, Hkv=8,
             D=64, max_len=384, lens_seed=7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


HEADS = [(32, 8), (32, 8), (64, 8), (32, 32), (16, 2), (28, 4), (40, 8), (16, 1), (12, 12)]


def draw(rng):
    op = rng.choice(["norm", "append", "decode", "decode", "prefill", "prefill"])
    kind = rng.choice(["int8", "e4m3"])
    Hq, Hkv = rng.choice(HEADS)
    seed = rng.randrange(1 << 20)
    if op == "norm":
        D = rng.choice([64, 128, 128, 256])
        top = 32768 * 40 * 128 // ((Hq + Hkv) * D)
        return dict(op=op, T=_log_int(rng, 1, min(32768, top)), Hq=Hq, Hkv=Hkv, D=D, max_pos=rng.choice([4096, 32768]))
    D = rng.choice([64, 128])
    if op == "append":
        top = 65536 * 8 * 128 // (Hkv * D)
        T = _log_int(rng, 1, min(65536, top))
        seqs = rng.randint(1, 64)
        return dict(op=op, kind=kind, T=T, Hkv=Hkv, D=D, seqs=seqs, max_len=max(64, -(-T // seqs) + rng.randint(0, 999)))
    if op == "decode":
        B = _log_int(rng, 1, 256)
        top = 64 * 32768 * 8 * 128 // (B * Hkv * D)
        return dict(op=op, kind=kind, B=B, Hq=Hq, Hkv=Hkv, D=D, min_len=1, max_len=_log_int(rng, 1, min(32768, top)),
                    lens_seed=seed)
    shape = rng.choice(["whole", "chunk", "mixed"])
    if shape == "whole":
        chunks, decodes, max_len = "1x%d+0" % _log_int(rng, 1, 2048), 0, 4096
    elif shape == "chunk":
        n = _log_int(rng, 1, 512)
        chunks, decodes, max_len = "1x%d+%d" % (n, rng.randint(0, 4096 - n)), 0, 4096
    else:
        n = rng.randint(1, 128)
        chunks, decodes, max_len = "%dx%d+%d" % (rng.randint(1, 8), n, rng.randint(0, 384 - n)), rng.randint(1, 32), 384
    return dict(op=op, kind=kind, chunks=chunks, decodes=decodes, Hq=Hq, Hkv=Hkv, D=D, max_len=max_len, lens_seed=seed)


def _lens(case):
    r = random.Random(case["lens_seed"])
    return [r.randint(case["min_len"], case["max_len"]) for _ in range(case["B"])]


def _rows(case):
    """(sequence, position) of a prefill case's rows: chunks of consecutive positions, and
    between them decode tokens of further sequences."""
    n, rest = case["chunks"].split("x")
    size, first = rest.split("+")
    n, size, first = int(n), int(size), int(first)
    r = random.Random(case["lens_seed"])
    parts = [[(s, first + i) for i in range(size)] for s in range(n)]
    parts += [[(n + d, r.randrange(case["max_len"]))] for d in range(case["decodes"])]
    r.shuffle(parts)
    return n + case["decodes"], [x for p in parts for x in p]


def work(case):
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "norm":
        T, H = case["T"], case["Hq"] + Hkv
        return {"bytes": 4 * T * H * D + 4 * T + 4 * D + 4 * D * min(T, case["max_pos"]), "flops": 9 * T * H * D}
    if case["op"] == "append":
        n = case["T"] * Hkv
        return {"bytes": n * (4 * D + 2 * (2 * D + 8) + 4 * D) + 16 * case["T"], "flops": 6 * n * D}
    Hq = case["Hq"]
    if case["op"] == "decode":
        lens = _lens(case)
        n, rows = sum(lens), case["B"]
        return {"bytes": n * Hkv * (2 * D + 8) + 4 * rows * Hq * D + sum(-(-x // PAGE) for x in lens) * 4,
                "flops": 4 * n * Hq * D}
    seqs, rows = _rows(case)
    top = {}
    for s, p in rows:
        top[s] = max(top.get(s, 0), p + 1)
    n = sum(top.values())
    return {"bytes": n * Hkv * (2 * D + 8) + 4 * len(rows) * Hq * D + 8 * len(rows),
            "flops": 4 * Hq * D * sum(p + 1 for _, p in rows)}


# ---------------------------------------------------------------------------
# Inputs


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rope_table(max_pos, D, theta=10000.0):
    inv = theta ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.stack([ang.cos(), ang.sin()], -1).float().cuda()


def _pages(lens, max_pages, g):
    """Page table (-1 past each sequence's end) over a shuffled pool with three spare pages."""
    counts = torch.tensor([-(-n // PAGE) for n in lens], device="cuda")
    total = int(counts.sum()) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(counts, 0) - counts
    i = torch.arange(max_pages, device="cuda")
    at = (first[:, None] + i).clamp(max=total - 1)
    return torch.where(i < counts[:, None], perm[at], -1).to(torch.int32).contiguous(), total


def _store(lens, max_len, Hkv, D, kind, g):
    """A store that holds sequences of these lengths: keys with some louder channels, values
    of lognormal loudness, and in slots that no sequence owns stale bytes with NaN scales."""
    max_pages = -(-max_len // PAGE)
    table, total = _pages(lens, max_pages, g)
    k = torch.empty((total, Hkv, PAGE, D), dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    ks = torch.empty((total, Hkv, PAGE), dtype=torch.float32, device="cuda")
    vs = torch.empty_like(ks)
    gain = 1.0 + 3.0 * (_randn(g, Hkv, 1, D) > 1.8)
    step = max(1, (1 << 26) // (Hkv * PAGE * D))
    for a in range(0, total, step):
        b = min(total, a + step)
        x = (_randn(g, b - a, Hkv, PAGE, D) * gain).bfloat16()
        k[a:b], ks[a:b] = _quantise(x, kind)
        x = (_randn(g, b - a, Hkv, PAGE, D) * (0.5 * _randn(g, b - a, Hkv, PAGE, 1)).exp()).bfloat16()
        v[a:b], vs[a:b] = _quantise(x, kind)
    owned = torch.zeros((total, PAGE), dtype=torch.bool, device="cuda")
    at = torch.arange(max_pages * PAGE, device="cuda")
    live = at < torch.tensor(lens, device="cuda")[:, None]
    slot = table.long().clamp(min=0).repeat_interleave(PAGE, 1) * PAGE + at % PAGE
    owned.view(-1)[slot[live]] = True
    stale = ~owned[:, None, :].expand(total, Hkv, PAGE)
    ks.masked_fill_(stale, float("nan"))
    vs.masked_fill_(stale, float("nan"))
    return dict(k_cache=k.view(DTYPES[kind]), v_cache=v.view(DTYPES[kind]), k_scale=ks, v_scale=vs, page_table=table)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    Hkv, D = case["Hkv"], case["D"]
    s = dict(case)
    if case["op"] == "norm":
        # q and k are parts of the rows of a fused projection's output
        T, Hq = case["T"], case["Hq"]
        qkv = _randn(g, T, (Hq + 2 * Hkv) * D).bfloat16()
        s["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        s["qw"] = (1 + 0.1 * _randn(g, D)).bfloat16()
        s["kw"] = (1 + 0.1 * _randn(g, D)).bfloat16()
        s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda").to(torch.int32)
        s["cos_sin"] = _rope_table(case["max_pos"], D)
        return s
    if case["op"] == "append":
        T, n = case["T"], case["seqs"]
        s |= _store([case["max_len"]] * n, case["max_len"], Hkv, D, case["kind"], g)
        at = torch.randperm(n * case["max_len"], generator=g, device="cuda")[:T]
        s["q_seq"] = (at // case["max_len"]).to(torch.int32)
        s["q_pos"] = (at % case["max_len"]).to(torch.int32)
        kv = _randn(g, T, 2 * Hkv * D).bfloat16()
        s["k_new"] = kv[:, : Hkv * D].view(T, Hkv, D)
        s["v_new"] = kv[:, Hkv * D:].view(T, Hkv, D)
        return s
    if case["op"] == "decode":
        lens = _lens(case)
        s |= _store(lens, case["max_len"], Hkv, D, case["kind"], g)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _randn(g, case["B"], case["Hq"], D).bfloat16()
        return s
    n, rows = _rows(case)
    top = [0] * n
    for a, p in rows:
        top[a] = max(top[a], p + 1)
    s |= _store(top, case["max_len"], Hkv, D, case["kind"], g)
    s["q_seq"] = torch.tensor([a for a, _ in rows], dtype=torch.int32, device="cuda")
    s["q_pos"] = torch.tensor([p for _, p in rows], dtype=torch.int32, device="cuda")
    s["keys"] = max(top)
    s["q"] = _randn(g, len(rows), case["Hq"], D).bfloat16()
    return s


# ---------------------------------------------------------------------------
# The operators in plain torch


def _quantise(x, kind):
    """8-bit values (their bits as int8) and fp32 scales of bf16 rows x [..., D]."""
    x = x.double()
    a = x.abs().amax(-1, keepdim=True)
    if kind == "int8":
        s, c = a / 127, torch.round(127 * x / a)
    else:  # the least power of two that brings the row to 448 at most
        m, e = torch.frexp(a)
        e = e - 9 + (m > 0.875)
        s = torch.ldexp(torch.ones_like(a), e)
        c = x / s
    empty, bad = a < 2.0 ** -100, ~a.isfinite()
    c = torch.where(empty | bad, 0, c)
    s = torch.where(bad, float("nan"), torch.where(empty, 1, s))
    return c.float().to(DTYPES[kind]).view(torch.int8), s.float().squeeze(-1)


def _norm_rope(x, w, cs, eps):
    x = x.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    a, b = n.chunk(2, -1)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat([a * c - b * s, b * c + a * s], -1).bfloat16()


def _slots(s):
    """Page and place in the page of rows (q_seq, q_pos)."""
    p = s["q_pos"].long()
    return s["page_table"][s["q_seq"].long(), p // PAGE].long(), p % PAGE


def _take(s, cache, *at):
    """fp32 of a cache's 8-bit values at an index."""
    return s[cache].view(torch.int8)[at].view(DTYPES[s["kind"]]).float()


def _gather(s, cache, scale, keys):
    """fp32 values [sequences, Hkv, keys, D] of a cache, zeros where no page is."""
    pages = -(-keys // PAGE)
    t = s["page_table"][:, :pages].long().clamp(min=0)
    x = _take(s, cache, t) * s[scale][t].unsqueeze(-1)  # [n, pages, Hkv, 16, D]
    return x.transpose(1, 2).reshape(t.shape[0], s["Hkv"], pages * PAGE, s["D"])


def _softmax(z):
    p = torch.exp(z - z.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _decode(s):
    B, Hq, Hkv, D = s["B"], s["Hq"], s["Hkv"], s["D"]
    k = _gather(s, "k_cache", "k_scale", s["max_len"])
    seen = torch.arange(k.shape[2], device="cuda") < s["seq_lens"][:, None]  # [B, keys]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    z = (q @ k.transpose(2, 3)) / math.sqrt(D)
    del k
    p = _softmax(z.masked_fill(~seen[:, None, None, :], float("-inf")))
    v = _gather(s, "v_cache", "v_scale", s["max_len"]).masked_fill_(~seen[:, None, :, None], 0)
    return (p @ v).view(B, Hq, D).bfloat16()


def _prefill(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    T, n, G = s["q"].shape[0], s["page_table"].shape[0], Hq // Hkv
    k = _gather(s, "k_cache", "k_scale", s["keys"])
    L = k.shape[2]
    at = torch.arange(n * L, device="cuda")
    seen = (at // L == s["q_seq"][:, None]) & (at % L <= s["q_pos"][:, None])  # [T, n * L]
    held = seen.any(0)
    k = k.transpose(0, 1).reshape(Hkv, n * L, D)
    q = s["q"].float().view(T, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * T, D)
    z = ((q @ k.transpose(1, 2)) / math.sqrt(D)).view(Hkv, G, T, n * L)
    p = _softmax(z.masked_fill_(~seen, float("-inf"))).view(Hkv, G * T, n * L)
    v = _gather(s, "v_cache", "v_scale", s["keys"]).transpose(0, 1).reshape(Hkv, n * L, D)
    o = (p @ v.masked_fill_(~held[:, None], 0)).view(Hkv, G, T, D)
    return o.permute(2, 0, 1, 3).reshape(T, Hq, D).bfloat16()


def _append_read(s):
    page, at = _slots(s)
    for new, cache, scale in (("k_new", "k_cache", "k_scale"), ("v_new", "v_cache", "v_scale")):
        s[cache].view(torch.int8)[page, :, at], s[scale][page, :, at] = _quantise(s[new], s["kind"])
    k = (_take(s, "k_cache", page, slice(None), at) * s["k_scale"][page, :, at].unsqueeze(-1)).bfloat16()
    v = (_take(s, "v_cache", page, slice(None), at) * s["v_scale"][page, :, at].unsqueeze(-1)).bfloat16()
    return k, v, s["k_scale"], s["v_scale"]


def run(s):
    op = s["op"]
    if own:
        import invariant_deterministic_04_b200 as bi

        if op == "norm":
            return bi.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["cos_sin"], 1e-6,
                                   q_out=torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda"),
                                   k_out=torch.empty(s["k"].shape, dtype=torch.bfloat16, device="cuda"))
        store = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"])
        if op == "append":
            bi.kv_append_q8(s["k_new"], s["v_new"], s["q_seq"], s["q_pos"], *store)
            return (*bi.kv_read_q8(s["q_seq"], s["q_pos"], *store), s["k_scale"], s["v_scale"])
        if op == "decode":
            return bi.attention_decode_q8(s["q"], *store, s["seq_lens"])
        return bi.attention_prefill_q8(s["q"], s["q_seq"], s["q_pos"], *store)
    if op == "norm":
        cs = s["cos_sin"][s["pos"].long()]
        return _norm_rope(s["q"], s["qw"], cs, 1e-6), _norm_rope(s["k"], s["kw"], cs, 1e-6)
    if op == "append":
        return _append_read(s)
    return _decode(s) if op == "decode" else _prefill(s)


# ---------------------------------------------------------------------------
# The definitions in 64 bits


def _row64(s, cache, scale, seq, n):
    """A sequence's first n keys or values in 64 bits, [Hkv, n, D]."""
    pages = s["page_table"][seq, : -(-n // PAGE)].long()
    bits = s[cache].view(torch.int8)[pages]
    x = bits.view(s[cache].dtype).double() * s[scale][pages].double()[..., None]
    return x.permute(1, 0, 2, 3).flatten(1, 2)[:, :n]


def _attend64(q, k, v, D):
    """q [Hq, D] over k, v [Hkv, n, D]."""
    z = torch.einsum("hgd,hnd->hgn", q.double().view(k.shape[0], -1, D), k) * D ** -0.5
    return torch.einsum("hgn,hnd->hgd", torch.softmax(z, -1), v).reshape(-1, D)


def _nearest_e4m3(y):
    """Nearest e4m3 value, ties to even (|y| <= 448): steps of 2^(e-3) with e >= -6."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    D = case["D"]
    if case["op"] == "norm":
        outs = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.double()
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            turn = torch.view_as_complex(s["cos_sin"][s["pos"].long()].double())[:, None, :]
            y = torch.complex(x[..., : D // 2].contiguous(), x[..., D // 2:].contiguous()) * turn
            outs.append(torch.cat([y.real, y.imag], -1))
        return tuple(outs)
    if case["op"] == "append":
        p = s["q_pos"].long()
        page = s["page_table"][s["q_seq"].long(), p // PAGE].long()
        outs, scales = [], []
        for new, scale in (("k_new", "k_scale"), ("v_new", "v_scale")):
            x = s[new].double()
            a = x.abs().max(-1, keepdim=True).values
            if case["kind"] == "int8":
                f = a / 127
                y = torch.round(x * 127 / a) * f
            else:
                f = torch.exp2(torch.ceil(torch.log2(a / 448)))
                y = _nearest_e4m3(x / f) * f
            outs.append(y)
            whole = s[scale].double()
            whole[page, :, p % PAGE] = f[..., 0]
            scales.append(whole)
        return (*outs, *scales)
    if case["op"] == "decode":
        out = []
        for b, n in enumerate(_lens(case)):
            out.append(_attend64(s["q"][b], _row64(s, "k_cache", "k_scale", b, n),
                                 _row64(s, "v_cache", "v_scale", b, n), D))
        return torch.stack(out)
    n, rows = _rows(case)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for seq in range(n):
        mine = [t for t, (a, _) in enumerate(rows) if a == seq]
        pos = torch.tensor([rows[t][1] for t in mine], device="cuda")
        L = int(pos.max()) + 1
        k, v = _row64(s, "k_cache", "k_scale", seq, L), _row64(s, "v_cache", "v_scale", seq, L)
        late = torch.arange(L, device="cuda") > pos[:, None]
        G = case["Hq"] // case["Hkv"]
        for h in range(case["Hq"]):
            z = s["q"][mine, h].double() @ k[h // G].T * D ** -0.5
            out[mine, h] = torch.softmax(z.masked_fill(late, float("-inf")), -1) @ v[h // G]
    return out
