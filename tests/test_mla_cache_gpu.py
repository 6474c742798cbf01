"""The paged latent cache on the GPU: kda_mla_decode against 64-bit arithmetic,
kda_mla_cache_append against the row-by-row definition, and a layer's prefill, append and decode
together."""
import math

import pytest
import torch

import chunked_linear_attention_chunk_b200 as kda
import mla_ref as ref

pytestmark = pytest.mark.gpu


def table_for(lens, ps, g, spare=2):
    need = [-(-n // ps) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device="cuda").to(torch.int32)
    t = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(need):
        t[i, :k] = order[at:at + k]
        at += k
    return t, sum(need) + spare


def make(lens, Sq, H, G, ps, e4m3, seed, std=0.6):
    """Queries and a cache whose rows behind each sequence's end are NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    table, pages = table_for(lens, ps, g)
    c = torch.randn(pages, ps, G, 576, generator=g, device="cuda").to(torch.bfloat16)
    scale = None
    if e4m3:
        scale = torch.exp2(torch.randint(-9, -6, (pages, G), generator=g, device="cuda").float())
        c = (c.float() / scale[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    live = torch.zeros(pages, ps, dtype=torch.bool, device="cuda")
    for i, n in enumerate(lens):
        for j in range(-(-n // ps)):
            live[int(table[i, j]), :min(ps, n - j * ps)] = True
    if e4m3:
        c.view(torch.uint8)[~live] = 0x7F
        scale[~live.any(1)] = math.nan
    else:
        c[~live] = math.nan
    q = (torch.randn(len(lens), Sq, H, 576, generator=g, device="cuda") * std).to(torch.bfloat16)
    return q, c, scale, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


CASES = [
    # lens, Sq, H, G, page size
    ([1], 1, 1, 1, 64),
    ([64], 1, 16, 1, 64),
    ([63, 65, 0, 1, 128], 1, 16, 1, 64),
    ([1000], 1, 32, 1, 64),
    ([5, 700, 33], 2, 32, 1, 16),
    ([130, 0, 2], 3, 5, 1, 32),                # fewer rows than new tokens; 15 columns
    ([200, 97], 1, 64, 1, 128),
    ([150, 31], 1, 128, 1, 64),                # more columns than one tile
    ([300, 77, 500], 1, 24, 2, 32),            # two latent groups
    ([90], 4, 32, 2, 16),
    ([3000, 10, 2500], 1, 16, 1, 192),         # sequences that several CTAs share
    ([260] * 40, 1, 16, 1, 64),
    ([70], 70, 3, 1, 64),                      # many new tokens
    ([3000 + 37 * i for i in range(40)], 1, 32, 1, 64),  # many tiles a CTA, several pieces
    ([2500 + 41 * i for i in range(30)], 2, 32, 1, 16),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,Sq,H,G,ps", CASES)
def test_decode_matches_64_bits(lens, Sq, H, G, ps, e4m3):
    q, c, sc, table, kv_lens = make(lens, Sq, H, G, ps, e4m3, seed=60 + len(lens) + H)
    o, lse = kda.kda_mla_decode(q, c, table, kv_lens, cache_scale=sc)
    ro, rl, mag = ref.decode(q, c, sc, table, lens, 192 ** -0.5)
    ref.close(o, ro, mag, "o")
    ref.lse_close(lse, rl, 32.0)
    assert kda.kda_device_status() == 0


GROUPS = [
    # several latent groups, and more columns a group than one tile holds
    ([130, 5], 1, 144, 2, 64),                 # 72 columns, runs of 8 heads
    ([70, 300], 3, 96, 2, 32),                 # 144 columns
    ([200], 20, 15, 3, 16),                    # 100 columns, single heads
    ([90, 0, 17], 2, 64, 4, 64),               # 32 columns
    ([400, 33], 1, 12, 4, 16),                 # 3 columns
    ([65, 1000], 5, 35, 5, 128),               # 35 columns
    ([500], 80, 64, 2, 64),                    # 2560 columns: 40 tiles
    ([260, 90], 300, 32, 1, 64),               # 9600 columns: more tiles than SMs; more tokens than rows
    ([150 + 7 * i for i in range(30)], 1, 32, 16, 32),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,Sq,H,G,ps", GROUPS)
def test_decode_groups_and_column_tiles(lens, Sq, H, G, ps, e4m3):
    q, c, sc, table, kv_lens = make(lens, Sq, H, G, ps, e4m3, seed=89 + len(lens) + H)
    o, lse = kda.kda_mla_decode(q, c, table, kv_lens, cache_scale=sc)
    ro, rl, mag = ref.decode(q, c, sc, table, lens, 192 ** -0.5)
    ref.close(o, ro, mag, "o")
    ref.lse_close(lse, rl, 32.0)
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("std", [0.0, 6.0])
def test_decode_flat_and_peaked(std, e4m3):
    q, c, sc, table, kv_lens = make([900, 350], 2, 16, 1, 64, e4m3, seed=70, std=std)
    o, lse = kda.kda_mla_decode(q, c, table, kv_lens, cache_scale=sc)
    ro, rl, mag = ref.decode(q, c, sc, table, [900, 350], 192 ** -0.5)
    # |q| |c| summed over a row: 576 * std * 3 or so, times the softmax scale
    s_abs = 576 * 3 * max(std, 0.1) * 192 ** -0.5
    ref.close(o, ro, mag * (1 + 2 ** 8 * math.expm1(576 * 2.0 ** -24 * s_abs)), "o")
    ref.lse_close(lse, rl, max(32.0, s_abs))


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_repeatable_captured_and_on_another_stream(e4m3):
    lens = [1500, 3, 700]
    q, c, sc, table, kv_lens = make(lens, 1, 32, 1, 64, e4m3, seed=71)
    first = kda.kda_mla_decode(q, c, table, kv_lens, cache_scale=sc)
    again = kda.kda_mla_decode(q, c, table, kv_lens, cache_scale=sc)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = kda.kda_mla_decode(q, c, table, kv_lens, cache_scale=sc)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first[0], again[0])
    graph = torch.cuda.CUDAGraph()
    fixed_q, fixed_lens = q.clone(), kv_lens.clone()
    with torch.cuda.graph(graph):
        cap = kda.kda_mla_decode(fixed_q, c, table, fixed_lens, cache_scale=sc)
    for new in (lens, [1400, 0, 640], lens):
        fixed_lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = kda.kda_mla_decode(q, c, table, fixed_lens.clone(), cache_scale=sc)
        assert torch.equal(cap[0], want[0]) and torch.equal(cap[1], want[1])


@pytest.mark.parametrize("e4m3", [False, True])
def test_chained_steps_without_waiting(e4m3):
    """Append, lengthen, decode, twenty times over with one workspace and in place: launches that
    set up early see what the ones before them wrote, as with a synchronisation after each."""
    held, new, H = [700, 5, 130], 1, 32
    g = torch.Generator(device="cuda").manual_seed(78)
    table, pages = table_for([n + 20 for n in held], 32, g)
    rows = torch.randn(20, 3, 1, 576, generator=g, device="cuda").to(torch.bfloat16)
    qs = (torch.randn(20, 3, 1, H, 576, generator=g, device="cuda") * 0.6).to(torch.bfloat16)
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    c0 = torch.randn(pages, 32, 1, 576, generator=g, device="cuda").to(torch.bfloat16)
    ws = torch.empty(kda.kda_mla_decode_workspace(3, 1, H, 1), dtype=torch.uint8, device="cuda")

    cache, sc = c0.clone(), None
    if e4m3:
        c0 = (c0.float() * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        cache, sc = c0.clone(), torch.empty((pages, 1), device="cuda")
    lens0 = torch.tensor(held, dtype=torch.int32, device="cuda")
    lens, q = lens0.clone(), torch.empty_like(qs[0])

    def run(wait):
        got = []
        cache.copy_(c0)
        lens.copy_(lens0)
        if e4m3:
            sc.fill_(2.0 ** -6)
        for i in range(20):
            kda.kda_mla_cache_append(rows[i], cu, lens, table, cache, cache_scale=sc)
            lens.add_(1)
            q.copy_(qs[i])
            for _ in range(2):
                got.append(kda.kda_mla_decode(q, cache, table, lens, cache_scale=sc, workspace=ws))
                if wait:
                    torch.cuda.synchronize()
        return got

    want = run(True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(False)
    graph.replay()
    graph.replay()
    for got in (run(False), captured):
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert kda.kda_device_status() == 0


def test_two_decodes_at_once():
    """Calls on two streams with a workspace each."""
    a = make([2000, 90], 1, 16, 1, 64, False, seed=72)
    b = make([100, 1700, 64], 1, 32, 1, 32, True, seed=73)
    want = [kda.kda_mla_decode(x[0], x[1], x[3], x[4], cache_scale=x[2]) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(kda.kda_mla_decode(x[0], x[1], x[3], x[4], cache_scale=x[2]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for o, l in got[i])


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_long_tail_of_small_weights(e4m3):
    """One row far above the rest: 40000 rows of weight 2^-19 or so of the largest, a twelfth of
    the sum together, and one page between them whose scale is 2^10 times the others'."""
    L, H = 40000, 16
    q, c, sc, table, kv_lens = make([L], 1, H, 1, 64, e4m3, seed=75)
    c[:, :, :, 512:] = 0.0
    q[..., :512] = 0.0
    q[..., 512:] = 0.25
    c[int(table[0, 300]), 17, 0, 512:] = 8.0 if e4m3 else 0.0
    if e4m3:
        sc[table[0].long()] = 2.0 ** -7
        sc[int(table[0, 300])] = 2.0 ** 3
    else:
        c[int(table[0, 300]), 17, 0, 512:] = 64.0
    scale = 19 * math.log(2) / (64 * 0.25 * 64.0)
    o, lse = kda.kda_mla_decode(q, c, table, kv_lens, scale=scale, cache_scale=sc)
    ro, rl, mag = ref.decode(q, c, sc, table, [L], scale)
    ref.close(o, ro, mag, "o")
    ref.lse_close(lse, rl, 32.0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_very_long_tail(e4m3):
    """A row and 384000 rows behind it (sixty pages over and over) of weight 2^-20.5 of its: a fifth
    of the sum.  As many sequences as SMs, so that each is one CTA's."""
    H, ps, times = 2, 64, 100
    n = torch.cuda.get_device_properties(0).multi_processor_count
    q, c, sc, table, _ = make([61 * ps], 1, H, 1, ps, e4m3, seed=79)
    c = c.float().abs().to(c.dtype)  # errors of equal weights add up
    c[:, :, :, 512:] = 0.0
    c[int(table[0, 60]), :, 0, :512] = 0.0
    c[int(table[0, 60]), 17, 0, 512:] = 8.0
    if e4m3:
        sc[:] = 2.0 ** -3
    q[..., :512] = 0.0
    q[..., 512:] = 0.25
    table = torch.cat([table[:, 60:], table[:, :60].repeat(1, times)], 1).contiguous()
    L = table.shape[1] * ps
    scale = 20.5 * math.log(2) / (64 * 0.25 * (1.0 if e4m3 else 8.0))
    o, lse = kda.kda_mla_decode(q.expand(n, -1, -1, -1).contiguous(), c, table.expand(n, -1).contiguous(),
                                torch.full((n,), L, dtype=torch.int32, device="cuda"), scale=scale, cache_scale=sc)
    assert torch.equal(o, o[:1].expand_as(o))
    ro, rl, mag = ref.decode(q, c, sc, table, [L], scale)
    # SLACK counts sums of 576 products; the sum of 384000 weights, 64 at a time in float32, is off by
    # at most 6000 * 2^-24 of itself
    ref.close(o[:1], ro, mag + mag * 2 ** 8 * 6000 * 2.0 ** -24, "o")
    ref.lse_close(lse[:1], rl, 32.0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_reads_a_page_twice_and_no_rows_at_all(e4m3):
    q, c, sc, table, kv_lens = make([256, 130], 1, 16, 1, 64, e4m3, seed=76)
    table[1, 1] = table[1, 0]
    table[0, 3] = table[0, 1]
    o, lse = kda.kda_mla_decode(q, c, table, kv_lens, cache_scale=sc)
    ro, rl, mag = ref.decode(q, c, sc, table, [256, 130], 192 ** -0.5)
    ref.close(o, ro, mag, "o")
    o, lse = kda.kda_mla_decode(q, c, table, torch.zeros_like(kv_lens), cache_scale=sc)
    assert (o == 0).all() and torch.isneginf(lse).all()
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("kind", ["steps", "random"])
@pytest.mark.parametrize("H", [16, 32, 64])
def test_decode_q_far_below_its_largest_number(kind, H):
    """Over an 8-bit cache a number of q is off by at most 2^-22 of its row's largest.  That one
    meets zeros here, and the others, 2^-10 to 2^-30 of it, decide the scores; all of a row's cached
    numbers have one sign, so errors add up."""
    L = 300
    q, c, sc, table, kv_lens = make([L], 1, H, 1, 64, True, seed=85)
    g = torch.Generator(device="cuda").manual_seed(86)
    c = c.float().abs().nan_to_num(0.0).to(torch.float8_e4m3fn)
    c[..., 5] = 0.0
    sc.fill_(2.0 ** -7)
    if kind == "steps":  # 3, 7, 11 or 15 steps of 2^-21
        k = torch.randint(0, 4, (1, 1, H, 576), generator=g, device="cuda")
        x = (4 * k + 3) * 2.0 ** -21
    else:
        x = torch.rand(1, 1, H, 576, generator=g, device="cuda") * torch.exp2(
            -torch.randint(10, 30, (1, 1, H, 576), generator=g, device="cuda").float())
    x[..., 5] = torch.where(torch.arange(H, device="cuda") % 2 == 0, 1.0, 1.9921875)
    q = x.to(torch.bfloat16)
    scale = 2.0 ** 11 if kind == "steps" else 32.0
    o, lse = kda.kda_mla_decode(q, c, table, kv_lens, scale=scale, cache_scale=sc)
    ro, rl, mag = ref.decode(q, c, sc, table, [L], scale)
    rows = ref.rows_of(c, sc, table[0], L)[:, 0].abs()
    some = q.double().abs()[0, 0] * (torch.arange(576, device="cuda") != 5)
    s_abs = (rows @ some.T).amax(0) * scale  # per head
    off = scale * 2.0 ** -22 * q[0, 0, :, 5].double() * rows.sum(1).max() + 576 * 2.0 ** -24 * s_abs
    assert ((lse.double() - rl).abs()[0, 0] <= off + 2.0 ** -20 * (1 + rl.abs()[0, 0])).all()
    ref.close(o, ro, mag * (1 + 2 ** 8 * torch.expm1(2 * off)[:, None]), "o")


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("power", [10, 24, 25, 26, 40, 80])
def test_decode_zeros_beside_large_numbers(H, ps, power):
    """Rows of zeros (scale 2^-100) beside rows of numbers near 2^power whose scores are far below
    or level with them, as the append writes them: their weights, down to 0, times their scale stay
    numbers."""
    L = 4 * ps
    g = torch.Generator(device="cuda").manual_seed(87)
    table = torch.randperm(12, generator=g, device="cuda").to(torch.int32).reshape(3, 4)
    rows = torch.zeros(3, L, 1, 576, device="cuda")
    rows[1:, ps:2 * ps] = (1 + torch.rand(2, ps, 1, 576, generator=g, device="cuda")) * 2.0 ** power
    rows[0] = (1 + torch.rand(L, 1, 576, generator=g, device="cuda")) * 2.0 ** power  # no zeros: one row, of
    rows[0, L // 2 + 3] *= 0.25                                                       # the least, far above the rest
    rows[2, 3 * ps - 7:] = torch.randn(ps + 7, 1, 576, generator=g, device="cuda")
    cache = torch.zeros(12, ps, 1, 576, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.zeros(12, 1, device="cuda")
    cu = torch.arange(4, dtype=torch.int32, device="cuda") * L
    kda.kda_mla_cache_append(rows.reshape(-1, 1, 576).to(torch.bfloat16), cu, torch.zeros(3, dtype=torch.int32, device="cuda"),
                             table, cache, cache_scale=sc)
    q = -torch.rand(3, 1, H, 576, generator=g, device="cuda")
    q[:, :, ::2] = -q[:, :, ::2] * 2.0 ** -power  # every other head: scores of a few hundred, level with the rest
    q = q.to(torch.bfloat16)
    scale = 192 ** -0.5
    o, lse = kda.kda_mla_decode(q, cache, table, torch.full((3,), L, dtype=torch.int32, device="cuda"), scale=scale,
                                cache_scale=sc)
    ro, rl, mag = ref.decode(q, cache, sc, table, [L] * 3, scale)
    # every other head's scores reach 576 * 2 / 13.9 = 83: their float32 sums move e^s by 576 * 2^-24 * 83
    ref.close(o[:, :, ::2], ro[:, :, ::2], mag[:, :, ::2] * (1 + 2 ** 8 * math.expm1(576 * 2.0 ** -24 * 83)), "o, level")
    ref.lse_close(lse[:, :, ::2], rl[:, :, ::2], 83.0)
    # the other heads' large rows have scores of -2^power and less: weights of 0, but for the first sequence's least
    assert torch.isfinite(o[:, :, 1::2]).all()
    ref.close(o[:, :, 1::2], ro[:, :, 1::2], mag[:, :, 1::2], "o, far below")
    ref.lse_close(lse[1:, :, 1::2], rl[1:, :, 1::2], 83.0)
    ref.lse_close(lse[:1, :, 1::2], rl[:1, :, 1::2], float(rl[:1, :, 1::2].abs().max()))
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("H,ps", [(16, 16), (32, 16), (64, 16), (16, 32)])
def test_decode_scales_of_places_without_a_page(H, ps):
    """Tiles that a sequence's pages fill only in part, each in a CTA that held a NaN page's scales
    before: the NaN stays with its own sequence.  Twelve sequences a CTA, every other one of NaN
    pages, the ones between of one page."""
    n = 12 * torch.cuda.get_device_properties(0).multi_processor_count
    lens = [64 if i % 2 == 0 else 1 + i % ps for i in range(n)]
    q, c, sc, table, kv_lens = make(lens, 1, H, 1, ps, True, seed=84)
    sc[table[::2, :64 // ps].reshape(-1).long()] = math.nan
    some = [1, 3, n // 2 + 1, n - 1]
    for _ in range(20):
        o, lse = kda.kda_mla_decode(q, c, table, kv_lens, cache_scale=sc)
        assert torch.isnan(o[::2]).all() and torch.isfinite(o[1::2]).all() and torch.isfinite(lse[1::2]).all()
    ro, rl, mag = ref.decode(q[some], c, sc, table[some], [lens[i] for i in some], 192 ** -0.5)
    ref.close(o[some], ro, mag, "o")
    ref.lse_close(lse[some], rl, 32.0)
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_pool_past_32_bit_offsets(e4m3):
    """Append to and attend over the last pages of a pool of more than 2^32 bytes and numbers."""
    ps, pages, lens = 64, 2 ** 32 // (64 * 576) + 8, [100, 70]
    g = torch.Generator(device="cuda").manual_seed(77)
    cache = torch.empty(pages, ps, 1, 576, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device="cuda")
    sc = torch.zeros(pages, 1, device="cuda") if e4m3 else None
    table = torch.tensor([[pages - 1, pages - 3], [pages - 2, 0]], dtype=torch.int32, device="cuda")
    rows = torch.randn(sum(lens), 1, 576, generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 100, 170], dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    kda.kda_mla_cache_append(rows, cu, zero, table, cache, cache_scale=sc)
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for n, (a, b) in enumerate(((0, 100), (100, 170))):
        held = ref.rows_of(cache, sc, table[n], b - a)
        err = (held - rows[a:b].double()).abs().amax()
        assert float(err) <= (2.0 ** -4 * 8 if e4m3 else 0.0)  # half a step of numbers below 8
    q = (torch.randn(2, 1, 16, 576, generator=g, device="cuda") * 0.6).to(torch.bfloat16)
    o, lse = kda.kda_mla_decode(q, cache, table, kv_lens, cache_scale=sc)
    ro, rl, mag = ref.decode(q, cache, sc, table, lens, 192 ** -0.5)
    ref.close(o, ro, mag, "o")
    ref.lse_close(lse, rl, 32.0)
    assert kda.kda_device_status() == 0


def test_decode_records_bad_lengths_and_pages():
    """Recorded in the status word; the other sequences' results stand."""
    lens = [100, 40, 64]
    q, c, sc, table, kv_lens = make(lens, 1, 16, 1, 64, False, seed=74)
    good = kda.kda_mla_decode(q, c, table, kv_lens)
    for bad_len in (-1, table.shape[1] * 64 + 1):
        l2 = kv_lens.clone()
        l2[1] = bad_len
        o, _ = kda.kda_mla_decode(q, c, table, l2)
        assert kda.kda_device_status() == 1
        assert torch.equal(o[0], good[0][0]) and torch.equal(o[2], good[0][2])
    for page in (-1, c.shape[0]):
        t2 = table.clone()
        t2[0, 1] = page
        o, _ = kda.kda_mla_decode(q, c, t2, kv_lens)
        assert kda.kda_device_status() == 1
        assert torch.equal(o[1], good[0][1]) and torch.equal(o[2], good[0][2])


APPENDS = [
    # rows held, rows new, G, page size
    ([0], [1], 1, 64),
    ([63, 64, 65, 0, 10], [1, 1, 1, 0, 130], 1, 64),
    ([5, 0, 31], [40, 100, 2], 2, 32),
    ([15, 16, 100], [1, 17, 33], 1, 16),
    ([100, 7], [300, 1], 2, 192),
    ([i % 70 for i in range(300)], [i % 3 for i in range(300)], 1, 64),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("held,new,G,ps", APPENDS)
def test_append_matches_the_definition(held, new, G, ps, e4m3):
    """Codes, scales and untouched rows, bit for bit; magnitudes that make some scales grow."""
    g = torch.Generator(device="cuda").manual_seed(80 + len(held))
    table, pages = table_for([a + b for a, b in zip(held, new)], ps, g)
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    rows = torch.randn(cu[-1] + 3, G, 576, generator=g, device="cuda")
    rows *= torch.exp2(torch.randint(-4, 5, (cu[-1] + 3, G, 1), generator=g, device="cuda").float())
    rows = rows.to(torch.bfloat16)
    if cu[-1] > 2:
        rows[1] = 0.0
    c = torch.randn(pages, ps, G, 576, generator=g, device="cuda").to(torch.bfloat16)
    sc = None
    if e4m3:
        sc = torch.exp2(torch.randint(-9, -5, (pages, G), generator=g, device="cuda").float())
        c = (c.float() / sc[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    held_t = torch.tensor(held, dtype=torch.int32, device="cuda")
    want_c, want_s = c.cpu().clone(), None if sc is None else sc.cpu().clone()
    ref.append(rows.cpu(), cu, held, table.cpu(), want_c, want_s)
    kda.kda_mla_cache_append(rows, cu_t, held_t, table, c, cache_scale=sc)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    assert torch.equal(c.cpu().view(torch.uint8), want_c.view(torch.uint8))
    if e4m3:
        assert torch.equal(sc.cpu(), want_s)
    # the same rows again change nothing
    before = c.clone()
    kda.kda_mla_cache_append(rows, cu_t, held_t, table, c, cache_scale=sc)
    assert torch.equal(c.view(torch.uint8), before.view(torch.uint8))


def test_append_extremes():
    """All zeros, the largest and smallest numbers, and a NaN or an infinity, which make the
    scale NaN and the attention over the page NaN."""
    ps = 64
    table = torch.arange(6, dtype=torch.int32, device="cuda")[:, None].contiguous()
    rows = torch.zeros(6, 1, 576, dtype=torch.bfloat16, device="cuda")
    rows[1, 0, 3] = 3.3895313892515355e38
    rows[2, 0, 5] = 1e-38
    rows[3, 0, 7] = math.nan
    rows[4, 0, 9] = -math.inf
    rows[5, 0, :] = 448.0
    c = torch.zeros(6, ps, 1, 576, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.full((6, 1), 5.0, device="cuda")
    cu = torch.arange(7, dtype=torch.int32, device="cuda")
    held = torch.zeros(6, dtype=torch.int32, device="cuda")
    kda.kda_mla_cache_append(rows, cu, held, table, c, cache_scale=sc)
    s = sc[:, 0].cpu().tolist()
    assert s[0] == s[2] == 2.0 ** -100 and s[1] == 2.0 ** 120 and s[5] == 1.0
    assert math.isnan(s[3]) and math.isnan(s[4])
    q = torch.ones(6, 1, 16, 576, dtype=torch.bfloat16, device="cuda")
    o, lse = kda.kda_mla_decode(q, c, table, held + 1, cache_scale=sc)
    assert torch.isnan(o[3]).all() and torch.isnan(o[4]).all()
    assert (o[0] == 0).all() and (o[5] == 448).all() and (o[2] == 0).all()
    # behind a NaN page's rows the scale stays NaN
    kda.kda_mla_cache_append(rows[:1].expand(6, -1, -1).contiguous(), cu, held + 1, table, c, cache_scale=sc)
    assert math.isnan(float(sc[3, 0])) and float(sc[5, 0]) == 1.0


@pytest.mark.parametrize("e4m3", [False, True])
def test_appends_from_threads_with_pages_of_several_sizes(e4m3):
    """Host threads that fill caches of different page sizes at once: every call is launched, and
    every cache holds its rows."""
    import threading
    g = torch.Generator(device="cuda").manual_seed(82)
    errors, made = [], []
    for ps in (16, 64, 32, 128):
        rows = torch.randn(ps, 1, 576, generator=g, device="cuda").to(torch.bfloat16)
        cache = torch.zeros(1, ps, 1, 576, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device="cuda")
        sc = torch.zeros(1, 1, device="cuda") if e4m3 else None
        ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, ps], [0], [[0]])]
        made.append((ps, rows, cache, sc, ints))
    torch.cuda.synchronize()
    start = threading.Barrier(len(made), timeout=60)

    def body(ps, rows, cache, sc, ints):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(4000):
                    kda.kda_mla_cache_append(rows, ints[0], ints[1], ints[2], cache, cache_scale=sc)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (reported below, in the test's own thread)
            errors.append((ps, e))

    threads = [threading.Thread(target=body, args=m) for m in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert kda.kda_device_status() == 0
    for ps, rows, cache, sc, ints in made:
        want_c, want_s = torch.zeros_like(cache, device="cpu"), None if sc is None else torch.zeros(1, 1)
        ref.append(rows.cpu(), [0, ps], [0], ints[2].cpu(), want_c, want_s)
        assert torch.equal(cache.cpu().view(torch.uint8), want_c.view(torch.uint8))


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_whose_rows_do_not_land_writes_nothing(e4m3):
    """The waits run out (20 ms) and say so; cache, scales and the next call are as before."""
    held, new, ps = [5, 0, 31, 64], [40, 100, 2, 1], 32
    g = torch.Generator(device="cuda").manual_seed(83)
    table, pages = table_for([a + b for a, b in zip(held, new)], ps, g)
    cu = torch.tensor([0, 40, 140, 142, 143], dtype=torch.int32, device="cuda")
    held_t = torch.tensor(held, dtype=torch.int32, device="cuda")
    rows = (torch.randn(143, 2, 576, generator=g, device="cuda") * 8).to(torch.bfloat16)
    c = torch.randn(pages, ps, 2, 576, generator=g, device="cuda").to(torch.bfloat16)
    sc = None
    if e4m3:
        sc = torch.full((pages, 2), 2.0 ** -6, device="cuda")
        c = (c.float() * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
    before_c, before_s = c.clone(), None if sc is None else sc.clone()
    assert kda.kda_device_status() == 0
    kda.kda_selftest_append_timeout(20000, rows, cu, held_t, table, c, cache_scale=sc)
    assert kda.kda_device_status() == 6  # KDA_ERR_DEVICE_TIMEOUT
    assert torch.equal(c.view(torch.uint8), before_c.view(torch.uint8))
    assert sc is None or torch.equal(sc, before_s)
    want_c, want_s = c.cpu().clone(), None if sc is None else sc.cpu().clone()
    ref.append(rows.cpu(), cu.tolist(), held, table.cpu(), want_c, want_s)
    kda.kda_mla_cache_append(rows, cu, held_t, table, c, cache_scale=sc)
    torch.cuda.synchronize()
    assert kda.kda_device_status() == 0
    assert torch.equal(c.cpu().view(torch.uint8), want_c.view(torch.uint8))
    assert sc is None or torch.equal(sc.cpu(), want_s)


def test_append_refuses_bad_tables():
    ps = 64
    g = torch.Generator(device="cuda").manual_seed(81)
    rows = torch.randn(6, 1, 576, generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    good = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    for table, held, offs in (
            (torch.tensor([[0], [2]], dtype=torch.int32, device="cuda"), zero, cu),      # no such page
            (torch.tensor([[0], [-1]], dtype=torch.int32, device="cuda"), zero, cu),
            (good, torch.tensor([0, 64], dtype=torch.int32, device="cuda"), cu),         # behind the table
            (good, torch.tensor([0, -5], dtype=torch.int32, device="cuda"), cu)):
        c = torch.zeros(2, ps, 1, 576, dtype=torch.bfloat16, device="cuda")
        kda.kda_mla_cache_append(rows, offs, held, table, c)
        assert kda.kda_device_status() == 1
        assert torch.equal(c[0, :3], rows[:3]) and (c[1] == 0).all()
    for bad in ([0, 4, 3], [0, 3, 7], [1, 3, 6]):
        c = torch.zeros(2, ps, 1, 576, dtype=torch.bfloat16, device="cuda")
        kda.kda_mla_cache_append(rows, torch.tensor(bad, dtype=torch.int32, device="cuda"), zero, good, c)
        assert kda.kda_device_status() == 1
        assert (c == 0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_prefill_append_decode_together(e4m3):
    """A latent-attention layer as a hybrid model runs it: the prompt through the expanded form,
    its latents into the cache, then tokens one at a time in the absorbed form.  Each token's
    result equals attention over the cached rows in 64 bits, with the value projection behind
    it; the prompt's last row equals a decode of the same token up to the projections' roundings."""
    H, ps, lens, steps = 4, 32, [70, 33], 3
    g = torch.Generator(device="cuda").manual_seed(90)
    w_uk = (torch.randn(H, 128, 512, generator=g, device="cuda") / 512 ** 0.5).to(torch.bfloat16)
    w_uv = (torch.randn(H, 128, 512, generator=g, device="cuda") / 512 ** 0.5).to(torch.bfloat16)
    total = [n + steps for n in lens]
    table, pages = table_for(total, ps, g)
    cache = torch.zeros(pages, ps, 1, 576, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device="cuda")
    sc = torch.zeros(pages, 1, device="cuda") if e4m3 else None
    cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    lat = torch.randn(sum(lens), 1, 576, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(sum(lens), H, 192, generator=g, device="cuda").to(torch.bfloat16)
    up = lambda w: torch.einsum("td,hcd->thc", lat[:, 0, :512].float(), w.float())
    kv = torch.cat([up(w_uk), up(w_uv)], -1).to(torch.bfloat16)
    o, lse = kda.kda_mla_fwd(q, kv, lat[:, 0, 512:].contiguous(), cu)
    kda.kda_mla_cache_append(lat, cu, torch.zeros(2, dtype=torch.int32, device="cuda"), table, cache, cache_scale=sc)
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def absorbed(qt):  # [N, H, 192] -> [N, 1, H, 576]
        return torch.cat([torch.einsum("nhc,hcd->nhd", qt[..., :128].float(), w_uk.float()), qt[..., 128:].float()],
                         -1).to(torch.bfloat16)[:, None]

    last = q[cu[1:].long() - 1]
    od, _ = kda.kda_mla_decode(absorbed(last), cache, table, kv_lens, cache_scale=sc)
    od = torch.einsum("nhd,hcd->nhc", od[:, 0].float(), w_uv.float())
    want = o[cu[1:].long() - 1].float()
    # both sides round q or k, v and o to bfloat16 (about 2^-8 each, averaged over the row); the
    # 8-bit cache rounds every latent number by up to 2^-4
    assert float((od - want).norm() / want.norm()) <= (0.08 if e4m3 else 0.02)
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for _ in range(steps):
        new = torch.randn(2, 1, 576, generator=g, device="cuda").to(torch.bfloat16)
        qt = absorbed(torch.randn(2, H, 192, generator=g, device="cuda").to(torch.bfloat16))
        kda.kda_mla_cache_append(new, one, kv_lens, table, cache, cache_scale=sc)
        kv_lens = kv_lens + 1
        od, ld = kda.kda_mla_decode(qt, cache, table, kv_lens, cache_scale=sc)
        ro, rl, mag = ref.decode(qt, cache, sc, table, kv_lens.tolist(), 192 ** -0.5)
        ref.close(od, ro, mag, "o")
        ref.lse_close(ld, rl, 32.0)
    assert kda.kda_device_status() == 0


def test_role_waits_run_out_and_the_context_survives():
    """The waits of the kernels' roles, on barriers that nothing completes, with a short limit: the
    timeout is recorded, nothing acts on what did not come, and the next call is sound.  The time of
    a try, and with it the real limit of 2^20, is of the order of seconds at most."""
    assert kda.kda_device_status() == 0
    kda.kda_selftest_role_timeout(1)  # warm-up
    assert kda.kda_device_status() == 6  # KDA_ERR_DEVICE_TIMEOUT
    ms = []
    for tries in (1 << 10, 1 << 14):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        kda.kda_selftest_role_timeout(tries)
        b.record()
        assert kda.kda_device_status() == 6
        ms.append(a.elapsed_time(b))
        assert ms[-1] > 10.0  # what was on its way gets 10 ms to land
    # three waits run out in a call: the time of one of 2^20 tries from that of 2^14 - 2^10 more in each
    limit_s = (ms[1] - ms[0]) * 1e-3 / 3 * (1 << 20) / ((1 << 14) - (1 << 10))
    assert 0.0 < limit_s < 30.0, (ms, limit_s)
    print("limit of a role's wait: %.2f s" % limit_s)
    q, c, sc, table, kv_lens = make([100], 1, 16, 1, 64, True, seed=88)
    o, lse = kda.kda_mla_decode(q, c, table, kv_lens, cache_scale=sc)
    ro, rl, mag = ref.decode(q, c, sc, table, [100], 192 ** -0.5)
    ref.close(o, ro, mag, "o")
    assert kda.kda_device_status() == 0
