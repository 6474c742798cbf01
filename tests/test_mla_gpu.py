"""Expanded latent attention (kda_mla_fwd, kda_mla_bwd) on the GPU against 64-bit arithmetic."""
import math

import pytest
import torch

import chunked_linear_attention_chunk_b200 as kda
import mla_ref as ref

pytestmark = pytest.mark.gpu


def offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def make(lq, lk, H, seed, std=1.5, spare=0):
    """Packed inputs; `spare` rows of NaN behind the last sequence of both axes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cq, ck = offsets(lq), offsets(lk)

    def rnd(t, *shape, std=1.0):
        x = torch.randn(t + spare, *shape, generator=g, device="cuda") * std
        x[t:] = math.nan
        return x.to(torch.bfloat16)

    x = dict(q=rnd(cq[-1], H, 192, std=std), kv=rnd(ck[-1], H, 256), kr=rnd(ck[-1], 64), dO=rnd(cq[-1], H, 128))
    x["cu_q"], x["cu_k"] = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cq, ck))
    return x, cq, ck


CASES = [
    # lq, lk, H, causal
    ([1], [1], 1, True),
    ([64], [64], 2, True),
    ([127, 129, 1, 128], [127, 129, 1, 128], 3, True),
    ([300, 0, 17, 65], [300, 0, 17, 65], 2, True),
    ([257], [257], 1, False),
    ([5, 130, 64], [700, 131, 64], 2, True),        # keys that were there before
    ([40, 200], [33, 500], 2, False),
    ([200, 10, 7], [60, 3, 0], 2, True),            # more queries than keys: empty rows
    ([9, 3], [0, 70], 1, False),                    # a sequence without keys
    ([0, 0, 4], [10, 0, 9], 2, True),               # sequences without queries
    ([520], [1030], 1, True),
]


@pytest.mark.parametrize("lq,lk,H,causal", CASES)
def test_fwd_matches_64_bits(lq, lk, H, causal):
    x, cq, ck = make(lq, lk, H, seed=11 + sum(lq))
    o, lse = kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"], causal=causal)
    ro, rl, mag = ref.fwd(x["q"], x["kv"], x["kr"], cq, ck, 192 ** -0.5, causal)
    ref.close(o, ro, mag, "o")
    ref.lse_close(lse, rl, 16.0)
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("lq,lk,H,causal", CASES)
def test_bwd_matches_64_bits(lq, lk, H, causal):
    x, cq, ck = make(lq, lk, H, seed=12 + sum(lq))
    o, lse = kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"], causal=causal)
    got = kda.kda_mla_bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], x["cu_q"], x["cu_k"], causal=causal)
    want = ref.bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], cq, ck, 192 ** -0.5, causal)
    for name, (r, mag) in want.items():
        ref.close(got[name], r, mag, name)
    assert kda.kda_device_status() == 0


def test_bwd_matches_differences():
    """<gradient, direction> against a central difference of the 64-bit forward's loss <o, dO>.
    The kernel's gradients carry bfloat16 roundings (each within 2^-7 of its magnitude; their
    products with the direction add like independent terms) and D from the rounded o."""
    x, cq, ck = make([90, 35], [120, 35], 2, seed=31)
    o, lse = kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"])
    got = kda.kda_mla_bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], x["cu_q"], x["cu_k"])
    args = {"dq": x["q"].double(), "dkv": x["kv"].double(), "dk_rope": x["kr"].double()}
    g = torch.Generator(device="cuda").manual_seed(5)
    for name in args:
        d = torch.randn(args[name].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-5

        def loss(sign):
            a = dict(args)
            a[name] = a[name] + sign * eps * d
            return float((ref.fwd(a["dq"], a["dkv"], a["dk_rope"], cq, ck, 192 ** -0.5, True)[0] * x["dO"].double()).sum())

        diff = (loss(1) - loss(-1)) / (2 * eps)
        mine = got[name].double()
        # standard deviation of the sum of independent roundings of at most 2^-7 of each term, five-fold
        tol = 5 * 2.0 ** -7 * float((mine * d).norm()) + 1e-6
        assert abs(float((mine * d).sum()) - diff) <= tol, (name, float((mine * d).sum()), diff, tol)


def test_rows_behind_the_last_sequence_stay():
    """A padded batch: NaN rows behind cu[N] are not read, and outputs there are left as they were."""
    x, cq, ck = make([70, 33], [70, 90], 2, seed=41, spare=150)
    tq, tk = cq[-1], ck[-1]
    o = torch.full((tq + 150, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tq + 150, 2), 7.0, device="cuda")
    kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"], o=o, lse=lse)
    ro, rl, mag = ref.fwd(x["q"], x["kv"], x["kr"], cq, ck, 192 ** -0.5, True)
    ref.close(o[:tq], ro[:tq], mag[:tq], "o")
    assert (o[tq:] == 7.0).all() and (lse[tq:] == 7.0).all()
    out = {"dq": torch.full_like(x["q"], 7.0), "dkv": torch.full_like(x["kv"], 7.0), "dk_rope": torch.full_like(x["kr"], 7.0)}
    got = kda.kda_mla_bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], x["cu_q"], x["cu_k"], out=out)
    want = ref.bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], cq, ck, 192 ** -0.5, True)
    for name, (r, mag) in want.items():
        n = tq if name == "dq" else tk
        ref.close(got[name][:n], r[:n], mag[:n], name)
        assert (got[name][n:] == 7.0).all(), name
    assert kda.kda_device_status() == 0


def test_nan_neighbours_stay_out():
    """NaN rows of one sequence do not reach another that shares a tile with it."""
    x, cq, ck = make([30, 50, 20], [30, 50, 20], 1, seed=43)
    for t in ("q", "kv", "kr", "dO"):
        x[t][30:80] = math.nan
    o, lse = kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"])
    got = kda.kda_mla_bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], x["cu_q"], x["cu_k"])
    for a, b in ((0, 30), (80, 100)):
        sub = [x[t][a:b] for t in ("q", "kv", "kr")]
        ro, rl, mag = ref.fwd(*sub, [0, b - a], [0, b - a], 192 ** -0.5, True)
        ref.close(o[a:b], ro, mag, "o")
        want = ref.bwd(*sub, o[a:b], lse[a:b], x["dO"][a:b], [0, b - a], [0, b - a], 192 ** -0.5, True)
        for name, (r, m) in want.items():
            ref.close(got[name][a:b], r, m, name)


@pytest.mark.parametrize("std", [0.0, 12.0])
def test_flat_and_peaked_softmax(std):
    """All scores equal, and scores tens apart whose maximum moves late in the row."""
    x, cq, ck = make([400], [400], 2, seed=44, std=std)
    if std:
        x["kv"][350:, :, :128] *= 4
    o, lse = kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"])
    ro, rl, mag = ref.fwd(x["q"], x["kv"], x["kr"], cq, ck, 192 ** -0.5, True)
    s_abs = float((x["q"].double().abs().amax(0) @ torch.ones(192, 1, device="cuda", dtype=torch.float64)).max()) if std else 1.0
    # scores of this size: their float32 sums move e^s by 192 2^-24 of the sum of magnitudes
    mag = mag * (1 + 2 ** 8 * (math.expm1(192 * 2.0 ** -24 * s_abs) if std else 0.0))
    ref.close(o, ro, mag, "o")
    ref.lse_close(lse, rl, max(16.0, s_abs))


def test_invalid_offsets_write_nothing():
    x, cq, ck = make([40, 24], [40, 24], 2, seed=45)
    for bad in ([0, 50, 40], [1, 40, 64], [0, 40, 65], [0, -1, 64]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for pair in ((cu, x["cu_k"]), (x["cu_q"], cu)):
            o = torch.full((64, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((64, 2), 7.0, device="cuda")
            kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], *pair, o=o, lse=lse)
            assert kda.kda_device_status() == 1
            assert (o == 7.0).all() and (lse == 7.0).all()
            out = {"dq": torch.full_like(x["q"], 7.0), "dkv": torch.full_like(x["kv"], 7.0),
                   "dk_rope": torch.full_like(x["kr"], 7.0)}
            kda.kda_mla_bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], *pair, out=out)
            assert kda.kda_device_status() == 1
            assert all((t == 7.0).all() for t in out.values())


def test_repeatable_and_captured():
    """Equal calls give equal bits; a captured forward and backward replay on new inputs, and on
    a stream that is not the tensors' own."""
    x, cq, ck = make([333, 71], [400, 71], 3, seed=46)
    y, _, _ = make([333, 71], [400, 71], 3, seed=47)

    def step(z):
        o, lse = kda.kda_mla_fwd(z["q"], z["kv"], z["kr"], z["cu_q"], z["cu_k"])
        return o, lse, kda.kda_mla_bwd(z["q"], z["kv"], z["kr"], o, lse, z["dO"], z["cu_q"], z["cu_k"])

    def same(a, b):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert all(torch.equal(a[2][n], b[2][n]) for n in a[2])

    first, other = step(x), step(y)
    same(step(x), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step(x)
    torch.cuda.current_stream().wait_stream(side)
    same(again, first)
    fixed = {n: t.clone() for n, t in x.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(fixed)
    for z, want in ((x, first), (y, other)):
        for n in fixed:
            fixed[n].copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        same(captured, want)


def test_many_sequences():
    """More sequences than threads of a CTA, most of them short or empty."""
    lq = [(i * 7) % 5 for i in range(700)]
    lk = [n + (i % 3) for i, n in enumerate(lq)]
    x, cq, ck = make(lq, lk, 1, seed=48)
    o, lse = kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"])
    ro, rl, mag = ref.fwd(x["q"], x["kv"], x["kr"], cq, ck, 192 ** -0.5, True)
    ref.close(o, ro, mag, "o")
    got = kda.kda_mla_bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], x["cu_q"], x["cu_k"])
    want = ref.bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], cq, ck, 192 ** -0.5, True)
    for name, (r, m) in want.items():
        ref.close(got[name], r, m, name)


def test_packed_axis_past_32_bit_offsets():
    """The last sequence of packed axes of more than 2^31 numbers; the first one has queries
    without keys, the second keys without queries."""
    T, H, n = 150000, 88, 90
    x, _, _ = make([n], [n], H, seed=51)
    q = torch.empty(T + n, H, 192, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(T + n, H, 256, dtype=torch.bfloat16, device="cuda")
    kr = torch.empty(T + n, 64, dtype=torch.bfloat16, device="cuda")
    q[:T], kv[:T], kr[:T] = 1.0, 1.0, 1.0
    q[T:], kv[T:], kr[T:] = x["q"], x["kv"], x["kr"]
    cu_q, cu_k = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in ([0, T, T, T + n], [0, 0, T, T + n]))
    o, lse = kda.kda_mla_fwd(q, kv, kr, cu_q, cu_k)
    ro, rl, mag = ref.fwd(x["q"], x["kv"], x["kr"], [0, n], [0, n], 192 ** -0.5, True)
    ref.close(o[T:], ro, mag, "o")
    ref.lse_close(lse[T:], rl, 16.0)
    assert (o[T - 5:T] == 0).all() and torch.isneginf(lse[:T]).all()
    dO = torch.ones_like(o)
    dO[T:] = x["dO"]
    got = kda.kda_mla_bwd(q, kv, kr, o, lse, dO, cu_q, cu_k)
    want = ref.bwd(x["q"], x["kv"], x["kr"], o[T:], lse[T:], x["dO"], [0, n], [0, n], 192 ** -0.5, True)
    for name, (r, m) in want.items():
        ref.close(got[name][T:], r, m, name)
        assert (got[name][T - 5:T] == 0).all()
    assert kda.kda_device_status() == 0


def test_no_rows():
    x, cq, ck = make([0, 0], [5, 0], 2, seed=49)
    o, lse = kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"])
    assert o.shape == (0, 2, 128)
    got = kda.kda_mla_bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], x["cu_q"], x["cu_k"])
    assert (got["dkv"] == 0).all() and (got["dk_rope"] == 0).all()
    x, cq, ck = make([6], [0], 2, seed=50)
    o, lse = kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"])
    assert (o == 0).all() and torch.isneginf(lse).all()
    got = kda.kda_mla_bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], x["cu_q"], x["cu_k"])
    assert (got["dq"] == 0).all()
    assert kda.kda_device_status() == 0


def test_bwd_first_step_takes_no_place_early():
    """The first step's weights share their place in shared memory with v on its way to tensor
    memory.  Many tiles of one to three steps, beside another stream's work on the same memory
    system: equal bits every time, and every tile against 64 bits."""
    lens = [(37 * i) % 190 + 1 for i in range(60)]
    x, cq, ck = make(lens, lens, 4, seed=52)
    o, lse = kda.kda_mla_fwd(x["q"], x["kv"], x["kr"], x["cu_q"], x["cu_k"])
    args = (x["q"], x["kv"], x["kr"], o, lse, x["dO"], x["cu_q"], x["cu_k"])
    first = kda.kda_mla_bwd(*args)
    for name, (r, m) in ref.bwd(x["q"], x["kv"], x["kr"], o, lse, x["dO"], cq, ck, 192 ** -0.5, True).items():
        ref.close(first[name], r, m, name)
    a = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            for _ in range(4):
                b.copy_(a)
        got = [kda.kda_mla_bwd(*args) for _ in range(20)]
        torch.cuda.synchronize()
        assert all(torch.equal(g[n], first[n]) for g in got for n in first)
    assert kda.kda_device_status() == 0
