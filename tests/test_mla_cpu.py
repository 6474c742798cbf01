"""Latent attention without a GPU: the entry points' checks, the binding's refusals, and the
64-bit formulas that the GPU tests compare with, against autograd and differences."""
import ctypes

import pytest
import torch

import chunked_linear_attention_chunk_b200 as kda
import mla_ref as ref
from chunked_linear_attention_chunk_b200 import build

OK, INVALID, UNSUPPORTED, ALIGN, ALIAS, CUDA, TIMEOUT, WS = range(8)
BASE = 1 << 40
STEP = 1 << 34  # between made-up addresses


@pytest.fixture(scope="module")
def L():
    build.build()
    return kda.lib()


def P(i, off=0):
    return ctypes.c_void_p(BASE + i * STEP + off)


def _fwd(L, N=2, Tq=100, Tk=120, H=4, dn=128, dr=64, dv=128, dt=kda.KDA_BF16, scale=0.1, cu_q=P(8), cu_k=P(9), q=P(0),
         kv=P(1), kr=P(2), o=P(3), lse=P(4)):
    return L.kda_mla_fwd(N, cu_q, cu_k, Tq, Tk, H, dn, dr, dv, dt, 1, ctypes.c_float(scale), q, kv, kr, o, lse, None)


def test_fwd_validates(L):
    assert _fwd(L, Tq=0) == OK
    for bad in (dict(N=0), dict(Tq=-1), dict(Tk=-1), dict(H=0), dict(dt=9), dict(dt=kda.KDA_E4M3), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(cu_q=None), dict(cu_k=None),
                dict(q=None), dict(kv=None), dict(kr=None), dict(o=None)):
        assert _fwd(L, **bad) == INVALID, bad
    for bad in (dict(dn=64), dict(dr=32), dict(dv=64), dict(dt=kda.KDA_F32), dict(N=70000), dict(H=70000),
                dict(Tk=(1 << 31) - 8)):
        assert _fwd(L, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=P(0, 8)), dict(kv=P(1, 2)), dict(kr=P(2, 8)), dict(o=P(3, 4)), dict(lse=P(4, 2)),
                dict(cu_q=P(8, 1)), dict(cu_k=P(9, 2))):
        assert _fwd(L, **bad) == ALIGN, bad
    for bad in (dict(o=P(0, 1024)), dict(o=P(1)), dict(o=P(2, 64)), dict(lse=P(3, 16)), dict(lse=P(8)), dict(o=P(9))):
        assert _fwd(L, **bad) == ALIAS, bad


def _bwd(L, N=2, Tq=100, Tk=120, H=4, scale=0.1, ws_bytes=None, **kw):
    names = ("cu_q", "cu_k", "q", "kv", "kr", "o", "lse", "dO", "dq", "dkv", "dkr", "ws")
    p = {n: P(i) for i, n in enumerate(names)}
    p.update(kw)
    need = L.kda_mla_bwd_workspace(Tq, Tk, H, 128, 64, 128, kda.KDA_BF16)
    return L.kda_mla_bwd(N, p["cu_q"], p["cu_k"], Tq, Tk, H, 128, 64, 128, kda.KDA_BF16, 1, ctypes.c_float(scale),
                         *(p[n] for n in names[2:]), need if ws_bytes is None else ws_bytes, None)


def test_bwd_validates(L):
    assert _bwd(L, Tq=0, Tk=0) == OK
    for n in ("cu_q", "cu_k", "q", "kv", "kr", "o", "lse", "dO", "dq", "dkv", "dkr"):
        assert _bwd(L, **{n: None}) == INVALID, n
    assert _bwd(L, ws=None) == WS
    assert _bwd(L, ws_bytes=L.kda_mla_bwd_workspace(100, 120, 4, 128, 64, 128, kda.KDA_BF16) - 1) == WS
    for n in ("q", "kv", "kr", "o", "dO", "dq", "dkv", "dkr", "ws"):
        assert _bwd(L, **{n: P(20, 8)}) == ALIGN, n
    for out in ("dq", "dkv", "dkr", "ws"):
        for other in (2, 3, 4, 5, 6, 7):
            assert _bwd(L, **{out: P(other, 64)}) == ALIAS, (out, other)
    assert _bwd(L, dkv=P(8, 16)) == ALIAS and _bwd(L, dkr=P(11, 16)) == ALIAS
    assert L.kda_mla_bwd_workspace(100, 120, 4, 96, 64, 128, kda.KDA_BF16) == 0


def _dec(L, N=3, Sq=1, H=16, G=1, dl=512, dr=64, scale=0.1, cdt=kda.KDA_BF16, pages=10, ps=64, maxp=4, ws_bytes=None,
         q=P(0), cache=P(1), cs=None, bt=P(3), lens=P(4), o=P(5), lse=P(6), ws=P(7), dt=kda.KDA_BF16):
    need = L.kda_mla_decode_workspace(N, Sq, H, G, dl, dr)
    return L.kda_mla_decode(N, Sq, H, G, dl, dr, dt, ctypes.c_float(scale), q, cdt, cache, cs, pages, ps, bt, maxp, lens,
                            o, lse, ws, need if ws_bytes is None else ws_bytes, None)


def test_decode_validates(L):
    for bad in (dict(N=0), dict(Sq=0), dict(H=0), dict(G=0), dict(H=15, G=2), dict(scale=0.0), dict(pages=0),
                dict(ps=0), dict(maxp=0), dict(cdt=7), dict(q=None), dict(cache=None), dict(bt=None), dict(lens=None),
                dict(o=None), dict(cdt=kda.KDA_E4M3), dict(cs=P(2))):
        assert _dec(L, **bad) == INVALID, bad
    for bad in (dict(dl=256), dict(dr=32), dict(dt=kda.KDA_F32), dict(cdt=kda.KDA_F32), dict(ps=8), dict(ps=48),
                dict(ps=100), dict(N=70000), dict(pages=1 << 26), dict(maxp=1 << 26)):
        assert _dec(L, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=P(0, 8)), dict(cache=P(1, 8)), dict(o=P(5, 2)), dict(ws=P(7, 4)), dict(bt=P(3, 2)),
                dict(lens=P(4, 1)), dict(lse=P(6, 3)), dict(cdt=kda.KDA_E4M3, cs=P(2, 2))):
        assert _dec(L, **bad) == ALIGN, bad
    if L.kda_mla_decode_workspace(3, 1, 16, 1, 512, 64) > 0:
        assert _dec(L, ws=None) == WS and _dec(L, ws_bytes=0) == WS
    for bad in (dict(o=P(0)), dict(o=P(1, 64)), dict(lse=P(5)), dict(o=P(3)), dict(lse=P(4)), dict(ws=P(1)),
                dict(cdt=kda.KDA_E4M3, cs=P(5))):
        assert _dec(L, **bad) == ALIAS, bad


def _app(L, N=3, T=20, G=1, dl=512, dr=64, cdt=kda.KDA_BF16, pages=10, ps=64, maxp=4, cu=P(0), x=P(1), lens=P(2), bt=P(3),
         cache=P(4), cs=None, dt=kda.KDA_BF16):
    return L.kda_mla_cache_append(N, cu, T, G, dl, dr, dt, x, lens, bt, maxp, cdt, cache, cs, pages, ps, None)


def test_append_validates(L):
    assert _app(L, T=0) == OK
    for bad in (dict(N=0), dict(T=-1), dict(G=0), dict(cu=None), dict(x=None), dict(lens=None), dict(bt=None),
                dict(cache=None), dict(cdt=kda.KDA_E4M3), dict(cs=P(5)), dict(pages=0)):
        assert _app(L, **bad) == INVALID, bad
    for bad in (dict(dl=128), dict(cdt=kda.KDA_F32), dict(dt=kda.KDA_F32), dict(ps=24), dict(G=2000)):
        assert _app(L, **bad) == UNSUPPORTED, bad
    for bad in (dict(x=P(1, 4)), dict(cache=P(4, 8)), dict(cu=P(0, 2)), dict(cdt=kda.KDA_E4M3, cs=P(5, 1))):
        assert _app(L, **bad) == ALIGN, bad
    for bad in (dict(cache=P(1, 64)), dict(cache=P(3)), dict(cdt=kda.KDA_E4M3, cs=P(4, 64)), dict(cache=P(0)),
                dict(cdt=kda.KDA_E4M3, cs=P(1, 4))):
        assert _app(L, **bad) == ALIAS, bad


def test_role_selftest_validates(L):
    for tries in (0, (1 << 20) + 1):
        assert L.kda_selftest_role_timeout(tries, None) == INVALID


def test_append_selftest_validates(L):
    for limit in (0, 2000001):
        assert L.kda_selftest_append_timeout(limit, 3, P(0), 20, 1, 512, 64, kda.KDA_BF16, P(1), P(2), P(3), 4, kda.KDA_BF16,
                                             P(4), None, 10, 64, None) == INVALID
    assert L.kda_selftest_append_timeout(5, 3, P(0), 20, 1, 512, 64, kda.KDA_BF16, P(1), P(2), P(3), 4, kda.KDA_E4M3, P(4),
                                         None, 10, 64, None) == INVALID


def test_sizes_past_32_bits_are_refused(L):
    """More blocks than a launch takes; a sequence whose last tile would end behind 2^31 rows."""
    assert _fwd(L, N=65535, H=65535) == UNSUPPORTED
    assert _fwd(L, N=65535, Tq=1, H=40000, dt=kda.KDA_BF16) == UNSUPPORTED
    assert _bwd(L, N=65535, H=65535) == UNSUPPORTED
    for call in (_dec, _app):
        assert call(L, ps=16, maxp=(1 << 27) - 1) == UNSUPPORTED
        assert call(L, ps=32, G=2, maxp=1 << 25) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_mla_fwd(z(4, 2, 192), z(4, 2, 256), z(4, 64), cu)
    with pytest.raises(ValueError):
        kda.kda_mla_bwd(z(4, 2, 192), z(4, 2, 256), z(4, 64), z(4, 2, 128), z(4, 2, dt=torch.float32), z(4, 2, 128), cu)
    with pytest.raises(ValueError):
        kda.kda_mla_decode(z(1, 1, 2, 576), z(1, 64, 1, 576), table, lens)
    with pytest.raises(ValueError):
        kda.kda_mla_cache_append(z(1, 1, 576), cu, lens, table, z(1, 64, 1, 576))


@pytest.mark.parametrize("causal", [True, False])
def test_formulas_against_autograd_and_differences(causal):
    """The gradients written out in mla_ref against torch's derivative of the same forward in 64
    bits, and one directional derivative against a central difference."""
    torch.manual_seed(3)
    cq, ck, H = [0, 5, 12], [0, 9, 14], 2
    q, kv, kr = (torch.randn(*s, dtype=torch.float64, requires_grad=True) for s in ((12, H, 192), (14, H, 256), (14, 64)))
    dO = torch.randn(12, H, 128, dtype=torch.float64)

    def forward(q, kv, kr):
        o = []
        for a, b, c, d in zip(cq, cq[1:], ck, ck[1:]):
            vis = ref.visible(b - a, d - c, causal)
            o.append(torch.stack([ref.attention(q[a:b, h], *ref.head_kv(kv[c:d], kr[c:d], h), 0.07, vis)[0]
                                  for h in range(H)], 1))
        return torch.cat(o)

    o = forward(q, kv, kr)
    want = torch.autograd.grad((o * dO).sum(), (q, kv, kr))
    with torch.no_grad():
        ro, lse, _ = ref.fwd(q, kv, kr, cq, ck, 0.07, causal)
        assert torch.allclose(ro, o, atol=1e-13)
        got = ref.bwd(q, kv, kr, ro, lse, dO, cq, ck, 0.07, causal)
        for name, w in zip(("dq", "dkv", "dk_rope"), want):
            assert torch.allclose(got[name][0], w, atol=1e-11), name
        d = torch.randn_like(kr)
        diff = ((forward(q, kv, kr + 1e-6 * d) - forward(q, kv, kr - 1e-6 * d)) * dO).sum() / 2e-6
        assert abs(float(diff - (got["dk_rope"][0] * d).sum())) <= 1e-6 * (1 + abs(float(diff)))


def test_scale_power_of_the_definition():
    assert ref.power_for(448.0) == 1.0 and ref.power_for(449.0) == 2.0 and ref.power_for(0.0) == 2.0 ** -100
    assert ref.power_for(1.75) == 2.0 ** -8 and ref.power_for(1.76) == 2.0 ** -7
