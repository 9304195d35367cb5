"""Refusals of the 8-bit store's calls on the CPU: the C ABI's host validation (nothing is
launched) and the binding's own checks, which run before any C call."""
import pytest
import torch

import invariant_deterministic_04_b200 as bi
from invariant_deterministic_04_b200._build import build_library
from test_binding_checks import _bf, _c, _i32, fake  # noqa: F401

OK, NULL, SHAPE, ALIGN, WS, UNSUP = 0, 1, 2, 3, 4, 5
P = 0x10000          # aligned stand-in addresses; host validation never dereferences them
Q = 0x40000000


@pytest.fixture(scope="module")
def L():
    build_library()
    return bi.lib()


def call(f, names, **change):
    """f with `names` (name -> value) in order, some changed."""
    assert not set(change) - set(names)
    return f(*[change.get(n, v) for n, v in names.items()])


APPEND = dict(k=P, v=P, ld=1024, seq=P, pos=P, kc=P, vc=P, ks=P, vs=P, kind=0, pages=10, pt=P, seqs=1, maxp=4, T=3,
              Hkv=8, D=128, st=None)


def test_append_refusals(L):
    f = L.bi_kv_append_q8
    for n in ("k", "v", "seq", "pos", "kc", "vc", "ks", "vs", "pt"):
        assert call(f, APPEND, **{n: None}) == NULL
    for bad in (dict(T=-1), dict(seqs=0), dict(maxp=0), dict(pages=0), dict(Hkv=0), dict(D=0), dict(ld=1023)):
        assert call(f, APPEND, **bad) == SHAPE
    assert call(f, APPEND, kind=2) == UNSUP and call(f, APPEND, kind=-1) == UNSUP
    assert call(f, APPEND, D=96) == UNSUP
    for n in ("k", "v", "kc", "vc", "ks", "vs"):
        assert call(f, APPEND, **{n: P + 8}) == ALIGN
    assert call(f, APPEND, ld=1028) == ALIGN
    assert call(f, APPEND, T=0) == OK


READ = dict(k=Q, v=Q + 0x1000000, ld=1024, seq=P, pos=P, kc=P, vc=P, ks=P, vs=P, kind=1, pages=10, pt=P, seqs=1, maxp=4,
            T=3, Hkv=8, D=128, st=None)


def test_read_refusals(L):
    f = L.bi_kv_read_q8
    for n in ("k", "v", "seq", "pos", "kc", "vc", "ks", "vs", "pt"):
        assert call(f, READ, **{n: None}) == NULL
    assert call(f, READ, ld=512) == SHAPE and call(f, READ, T=-2) == SHAPE
    assert call(f, READ, k=Q + 2) == ALIGN and call(f, READ, ld=1028) == ALIGN
    assert call(f, READ, kind=7) == UNSUP and call(f, READ, D=256) == UNSUP
    assert call(f, READ, v=Q + 2 * 1016) == SHAPE       # the outputs share elements
    assert call(f, READ, k=P + 64) == SHAPE             # an output inside the store
    assert call(f, READ, T=0) == OK


def decode_args(L):
    return dict(q=Q, kc=P, vc=P, ks=P, vs=P, kind=0, pages=100, pt=P, maxp=64, lens=P, out=Q + 0x1000000, B=4, Hq=32,
                Hkv=8, D=128, scale=0.088, ws=P, wsb=L.bi_attention_workspace_size(4, 32, 128, 64), st=None)


def test_decode_refusals(L):
    f, a = L.bi_attention_decode_q8, decode_args(L)
    for n in ("q", "kc", "vc", "ks", "vs", "pt", "lens", "out"):
        assert call(f, a, **{n: None}) == NULL
    for bad in (dict(B=-1), dict(Hq=30), dict(Hq=0), dict(pages=0), dict(maxp=0), dict(scale=float("nan")),
                dict(out=Q + 64), dict(B=1 << 24, wsb=1 << 60)):
        assert call(f, a, **bad) == SHAPE
    assert call(f, a, Hq=34, Hkv=2) == UNSUP            # 17 query heads to a kv-head
    assert call(f, a, D=96) == UNSUP and call(f, a, kind=3) == UNSUP
    assert call(f, a, ws=None) == WS and call(f, a, wsb=a["wsb"] - 1) == WS
    for n in ("q", "kc", "vs", "out", "ws"):
        assert call(f, a, **{n: a[n] + 4}) == ALIGN
    assert call(f, a, B=0, ws=None, wsb=0) == OK


def test_prefill_refusals(L):
    s = L.bi_attention_prefill_q8_workspace_size
    assert s(-1) == 0 and 0 < s(1) <= s(4096)
    f = L.bi_attention_prefill_q8
    a = dict(q=Q, ldq=4096, seq=P, pos=P, kc=P, vc=P, ks=P, vs=P, kind=0, pages=100, pt=P, seqs=2, maxp=64,
             out=Q + 0x1000000, T=10, Hq=32, Hkv=8, D=128, scale=0.088, ws=P, wsb=s(10), st=None)
    for n in ("q", "seq", "pos", "kc", "vc", "ks", "vs", "pt", "out"):
        assert call(f, a, **{n: None}) == NULL
    for bad in (dict(T=-1), dict(seqs=0), dict(ldq=4000), dict(Hq=12), dict(scale=float("inf")), dict(out=Q + 4096)):
        assert call(f, a, **bad) == SHAPE
    assert call(f, a, ldq=4100) == ALIGN and call(f, a, q=Q + 2) == ALIGN and call(f, a, ws=P + 8) == ALIGN
    assert call(f, a, Hq=136) == UNSUP
    assert call(f, a, ws=None) == WS and call(f, a, wsb=s(10) - 1) == WS
    assert call(f, a, T=0, ws=None, wsb=0) == OK


def test_qk_norm_rope_refusals(L):
    f = L.bi_qk_norm_rope
    a = dict(q=Q, ldq=6144, k=Q + 8192, ldk=6144, qw=P, kw=P, pos=P, cs=P, max_pos=384, eps=1e-6, qo=Q, ldqo=6144,
             ko=Q + 8192, ldko=6144, T=5, Hq=32, Hkv=8, D=128, st=None)
    for n in ("q", "k", "qw", "kw", "pos", "cs", "qo", "ko"):
        assert call(f, a, **{n: None}) == NULL
    for bad in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(max_pos=0), dict(eps=float("nan")), dict(eps=-1.0),
                dict(ldq=4088), dict(ldko=1016)):
        assert call(f, a, **bad) == SHAPE
    assert call(f, a, D=96) == UNSUP and call(f, a, D=512) == UNSUP
    assert call(f, a, cs=P + 8) == ALIGN and call(f, a, ldk=6148) == ALIGN and call(f, a, qw=P + 2) == ALIGN
    # in place with another row stride; outputs over the other input, over each other
    assert call(f, a, ldqo=8192) == SHAPE
    assert call(f, a, qo=Q + 8192 - 16) == SHAPE
    assert call(f, a, qo=Q + 0x4000000, ko=Q + 0x4000000 + 4096) == SHAPE
    assert call(f, a, T=0) == OK


# ---------------------------------------------------------------------------
# the binding


def _store(pages=10, Hkv=8, D=128, dtype=torch.int8, rows=3, width=4):
    return [_c(torch.zeros((pages, Hkv, 16, D), dtype=dtype)), _c(torch.zeros((pages, Hkv, 16, D), dtype=dtype)),
            _c(torch.zeros((pages, Hkv, 16))), _c(torch.zeros((pages, Hkv, 16))), _i32(rows, width)]


def test_binding_accepts_the_call_patterns_in_use(fake):
    for dtype in (torch.int8, torch.float8_e4m3fn):
        S = _store(dtype=dtype)
        fused = _bf(3, 48 * 128)
        q, k, v = (fused[:, a * 128: b * 128].view(3, b - a, 128) for a, b in ((0, 32), (32, 40), (40, 48)))
        seq = pos = _i32(3)
        bi.qk_norm_rope(q, k, _bf(128), _bf(128), pos, _c(torch.zeros(64, 64, 2)))
        bi.qk_norm_rope(q, k, _bf(128), _bf(128), pos, _c(torch.zeros(64, 64, 2)), q_out=_bf(3, 32, 128),
                        k_out=_bf(3, 8, 128))
        bi.kv_append_q8(k, v, seq, pos, *S)
        bi.kv_read_q8(seq, pos, *S)
        bi.kv_read_q8(seq, pos, *S, k_out=k, v_out=v)
        bi.attention_decode_q8(_bf(3, 32, 128), *S, _i32(3))
        bi.attention_decode_q8(_bf(2, 56, 128), *S, _i32(3), out=_bf(2, 56, 128),
                               workspace=_c(torch.zeros(4096, dtype=torch.uint8)))
        bi.attention_prefill_q8(q, seq, pos, *S)
    assert {"bi_qk_norm_rope", "bi_kv_append_q8", "bi_kv_read_q8", "bi_attention_decode_q8",
            "bi_attention_prefill_q8"} <= set(fake.calls)


def test_binding_refuses_before_any_call(fake):
    S = _store()
    q, seq = _bf(3, 32, 128), _i32(3)
    k = _bf(3, 8, 128)

    def swap(i, t):
        return S[:i] + [t] + S[i + 1:]

    cases = [
        (TypeError, lambda: bi.attention_decode_q8(q, *_store(dtype=torch.uint8), seq)),
        (TypeError, lambda: bi.attention_decode_q8(q, *swap(1, _store(dtype=torch.float8_e4m3fn)[1]), seq)),
        (TypeError, lambda: bi.attention_decode_q8(q, *swap(2, _bf(10, 8, 16)), seq)),
        (ValueError, lambda: bi.attention_decode_q8(q, *swap(2, _c(torch.zeros(10, 8, 8))), seq)),
        (ValueError, lambda: bi.attention_decode_q8(q, *swap(0, S[0].transpose(0, 1)), seq)),
        (ValueError, lambda: bi.attention_decode_q8(_bf(3, 32, 64), *S, seq)),
        (ValueError, lambda: bi.attention_decode_q8(_bf(4, 32, 128), *S, _i32(4))),      # page_table has 3 rows
        (ValueError, lambda: bi.attention_decode_q8(q, *S, _i32(2))),
        (ValueError, lambda: bi.attention_decode_q8(q, *S, seq, out=_bf(3, 32, 64))),
        (TypeError, lambda: bi.attention_decode_q8(torch.zeros(3, 32, 128, dtype=torch.bfloat16), *S, seq)),
        (ValueError, lambda: bi.attention_prefill_q8(q, _i32(2), seq, *S)),
        (ValueError, lambda: bi.attention_prefill_q8(q.transpose(0, 1), seq, seq, *S)),
        (ValueError, lambda: bi.kv_append_q8(k, _bf(3, 8, 64), seq, seq, *S)),
        (ValueError, lambda: bi.kv_append_q8(_bf(3, 4, 128), _bf(3, 4, 128), seq, seq, *S)),
        (ValueError, lambda: bi.kv_append_q8(k, k, _i32(4), seq, *S)),
        (ValueError, lambda: bi.kv_read_q8(seq, seq, *S, k_out=k)),
        (ValueError, lambda: bi.kv_read_q8(seq, seq, *S, k_out=_bf(2, 8, 128), v_out=_bf(2, 8, 128))),
        (ValueError, lambda: bi.qk_norm_rope(q, _bf(3, 8, 64), _bf(128), _bf(128), seq, _c(torch.zeros(9, 64, 2)))),
        (ValueError, lambda: bi.qk_norm_rope(q, k, _bf(64), _bf(128), seq, _c(torch.zeros(9, 64, 2)))),
        (ValueError, lambda: bi.qk_norm_rope(q, k, _bf(128), _bf(128), _i32(2), _c(torch.zeros(9, 64, 2)))),
        (ValueError, lambda: bi.qk_norm_rope(q, k, _bf(128), _bf(128), seq, _c(torch.zeros(9, 32, 2)))),
        (ValueError, lambda: bi.qk_norm_rope(q, k, _bf(128), _bf(128), seq, _c(torch.zeros(9, 64, 2)),
                                             k_out=_bf(3, 7, 128))),
    ]
    for i, (kind, f) in enumerate(cases):
        with pytest.raises(kind):
            f()
            pytest.fail(f"case {i} was accepted")
    assert not [c for c in fake.calls if not c.endswith("workspace_size")]


def test_long_prefill_batches_of_long_contexts_are_not_refused(L):
    """A prefill keeps no splits in its workspace: rows times splits may pass 31 bits (a decode's may not)."""
    f, T = L.bi_attention_prefill_q8, 1 << 18
    a = dict(q=Q, ldq=4096, seq=P, pos=P, kc=P, vc=P, ks=P, vs=P, kind=0, pages=100, pt=P, seqs=2, maxp=1 << 14,
             out=1 << 44, T=T, Hq=32, Hkv=8, D=128, scale=0.088, ws=P, wsb=16, st=None)
    assert call(f, a) == WS
    d = dict(decode_args(L), B=T, maxp=1 << 14, out=1 << 44, wsb=16)
    assert call(L.bi_attention_decode_q8, d) == SHAPE
    assert call(f, a, maxp=1 << 27) == SHAPE            # positions past 31 bits
