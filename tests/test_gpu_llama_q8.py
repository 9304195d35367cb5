"""The decoder with an 8-bit KV store and per-head norms: the new calls run together as a model
runs them. One layer against a plain 64-bit form that quantises the same rows, and greedy streams
that stay the same under random mixed batching, through the checked binding and the direct calls."""
import numpy as np
import pytest
import torch

import invariant_deterministic_04_b200 as bi
import q8_ref
import synth
from gpu_util import TOL_BF16, dev, max_rel
from invariant_deterministic_04_b200.llama import BiLlama, FastBiLlama, rope_cos_sin, run_repeats, run_schedule

pytestmark = pytest.mark.gpu

CFG = dict(layers=2, hidden=512, heads=8, kv_heads=2, head_dim=64, ffn=1024, vocab=1000, eps=1e-6, theta=10000.0)
KINDS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def weights(cfg, seed, norms):
    w = synth.llama_weights(cfg, seed=seed, device=dev())
    if norms:
        for i, lw in enumerate(w["layers"]):
            lw["q_norm"] = synth.normal_bf16((cfg["head_dim"],), seed + 100 + i, 0.1, 1.0).to(dev())
            lw["k_norm"] = synth.normal_bf16((cfg["head_dim"],), seed + 200 + i, 0.1, 1.0).to(dev())
    return w


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_decoder_layer_matches_64_bits(kind):
    c, D = CFG, CFG["head_dim"]
    nh, nkv = c["heads"], c["kv_heads"]
    w = weights(c, 11, True)
    model = BiLlama(c, w, n_seqs=2, max_pos=64, device=dev(), kv_dtype=KINDS[kind])
    seqs, poss = [0] * 40 + [1] * 25, list(range(40)) + list(range(25))
    toks = list(synth.prompts(1, 65, 1000, seed=12)[0])
    h0 = model.hidden(seqs, poss, toks, n_layers=0).clone()
    h1 = model.hidden(seqs, poss, toks, n_layers=1)
    assert bi.get_device_error() == 0
    lw = w["layers"][0]
    # up to the projections by the library (its own tests cover them), attention and what follows in 64 bits
    qkv = bi.matmul(bi.rmsnorm(h0, lw["attn_norm"], c["eps"]), lw["wqkv"]).cpu()
    T = len(toks)
    q, k, v = (qkv[:, a * D: b * D].reshape(T, b - a, D) for a, b in ((0, nh), (nh, nh + nkv), (nh + nkv, nh + 2 * nkv)))
    pos = torch.tensor(poss, dtype=torch.int32)
    table = rope_cos_sin(64, D, c["theta"], "cpu")
    q, k = (q8_ref.norm_rope(x, lw[n].cpu(), table, pos, c["eps"])[0] for x, n in ((q, "q_norm"), (k, "k_norm")))
    k8, ks = q8_ref.quantise(torch.from_numpy(k).bfloat16(), kind)
    v8, vs = q8_ref.quantise(v, kind)
    K, V = k8 * ks[..., None], v8 * vs[..., None]
    att = np.zeros((T, nh, D))
    for t in range(T):
        mine = [i for i in range(T) if seqs[i] == seqs[t] and poss[i] <= poss[t]]
        att[t] = q8_ref.attend(q[t], K[mine].transpose(1, 0, 2), V[mine].transpose(1, 0, 2), D ** -0.5)[0]
    f = lambda n: synth.to_f64(lw[n])
    h = synth.to_f64(h0) + att.reshape(T, -1) @ f("wo").T
    x = h / np.sqrt((h ** 2).mean(-1, keepdims=True) + c["eps"]) * f("mlp_norm")
    gu = x @ f("wgu").T
    g, u = gu[:, : c["ffn"]], gu[:, c["ffn"]:]
    h = h + (g / (1 + np.exp(-g)) * u) @ f("wdown").T
    assert max_rel(h1, h) <= TOL_BF16


@pytest.mark.parametrize("kind,norms", [("int8", True), ("e4m3", False)])
def test_greedy_streams_identical_under_mixed_batching(kind, norms):
    cfg = dict(CFG, head_dim=128, hidden=512, heads=4, kv_heads=1)
    w = weights(cfg, 21, norms)
    S, P, G = 9, 40, 24
    prompts = synth.prompts(S, P, cfg["vocab"], seed=22)
    res = run_repeats(FastBiLlama, cfg, w, prompts, G, 3, dev(), kv_dtype=KINDS[kind])
    assert res["max_unique"] == 1
    # the same streams from the checked binding, one sequence at a time and under another schedule
    solo = BiLlama(cfg, w, S, P + G, dev(), kv_dtype=KINDS[kind])
    for s in (0, S - 1):
        out = [int(solo.forward([s] * P, list(range(P)), list(prompts[s]), [P - 1])[0])]
        for i in range(G - 1):
            out.append(int(solo.forward([s], [P + i], [out[-1]], [0])[0]))
        assert out == list(res["first"][s]), s
    again, _, _ = run_schedule(BiLlama(cfg, w, S, P + G, dev(), kv_dtype=KINDS[kind]), prompts, G, seed=77, max_batch=4)
    assert np.array_equal(again, res["first"])
    assert bi.get_device_error() == 0


def test_decode_call_continues_what_the_model_prefilled():
    """attention_decode_q8 over the model's own store gives the rows that the model's prefill call computed."""
    w = weights(CFG, 31, True)
    model = BiLlama(CFG, w, n_seqs=3, max_pos=300, device=dev(), kv_dtype=torch.int8)
    rows = [(s, p) for s, n in enumerate((290, 1, 33)) for p in range(n)]
    toks = list(synth.prompts(1, len(rows), 1000, seed=32)[0])
    model.hidden([r[0] for r in rows], [r[1] for r in rows], toks, n_layers=1)
    st = model.store
    q = synth.normal_bf16((3, CFG["heads"], CFG["head_dim"]), 33).to(dev())
    lens = torch.tensor([290, 1, 33], dtype=torch.int32, device=dev())
    a = bi.attention_decode_q8(q, *st.layer(0), lens)
    b = bi.attention_prefill_q8(q, torch.arange(3, dtype=torch.int32, device=dev()), lens - 1, *st.layer(0))
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert bool(torch.isfinite(a.float()).all()) and bi.get_device_error() == 0


def test_store_types():
    with pytest.raises(TypeError, match="kv_dtype"):
        BiLlama(CFG, weights(CFG, 41, False), 1, 16, dev(), kv_dtype=torch.float16)
