"""Latent-attention operators: the cases that are measured, their plain forms and their
definitions in 64 bits.

The operators are the softmax-attention half of a hybrid model whose other layers are the
chunked linear attention of this library (keys and values of a token come from one latent
vector of 512 numbers and one rotated key of 64 that all heads share):

  fwd     attention over expanded keys and values of packed sequences (prefill)
  bwd     its gradients (training)
  decode  the absorbed form over a paged cache of latent rows, bfloat16 or 8-bit with a
          scale for each page and latent group
  append  writing new rows into such a cache
"""
import math

import torch

own = False

DN, DR, DV = 128, 64, 128  # key part of a head, shared rotated part, value part
DL = 512                   # latent numbers a token
DC = DL + DR               # numbers of a cached row


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a handful of short prompts arriving together: launch latency and ragged tiles
        dict(name="fwd_short_prompts", op="fwd", n=5, q_lo=17, q_hi=301, ctx=0, H=16, causal=True),
        # one document of the 8K stage
        dict(name="fwd_8k", op="fwd", n=1, q_lo=8192, q_hi=8192, ctx=0, H=16, causal=True),
        # a chunk of a long prompt: 2K new tokens behind 14K that are there already
        dict(name="fwd_chunk_of_long_prompt", op="fwd", n=1, q_lo=2047, q_hi=2047, ctx=14401, H=32, causal=True),
        # packed training documents of uneven lengths
        dict(name="bwd_packed_documents", op="bwd", n=6, q_lo=100, q_hi=1500, ctx=0, H=16, causal=True),
        # one training sequence
        dict(name="bwd_8k", op="bwd", n=1, q_lo=8192, q_hi=8192, ctx=0, H=16, causal=True),
        # one user, short context: the latency of a single token
        dict(name="decode_one_user", op="decode", n=1, lo=1000, hi=1000, H=16, G=1, Sq=1, page=64, e4m3=False),
        # a full serving batch (the library's decode workload: 256 sequences, 32 heads)
        dict(name="decode_batch", op="decode", n=256, lo=3000, hi=5000, H=32, G=1, Sq=1, page=64, e4m3=False),
        # few long ragged contexts, two tokens a step (a drafted one and its check)
        dict(name="decode_long_ragged", op="decode", n=23, lo=1, hi=40000, H=32, G=1, Sq=2, page=64, e4m3=False),
        # the serving batch over the 8-bit cache
        dict(name="decode8_batch", op="decode", n=256, lo=3000, hi=5000, H=32, G=1, Sq=1, page=64, e4m3=True),
        # 8-bit, small pages, two latent groups
        dict(name="decode8_groups", op="decode", n=40, lo=1, hi=9000, H=32, G=2, Sq=1, page=32, e4m3=True),
        # a decode step's rows into the 8-bit cache
        dict(name="append8_step", op="append", n=256, lo=1, hi=1, held=5000, G=1, page=64, e4m3=True),
        # a prefill's rows into the 8-bit cache
        dict(name="append8_prefill", op="append", n=16, lo=500, hi=8000, held=300, G=1, page=64, e4m3=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "decode", "decode", "append"])
    if op in ("fwd", "bwd"):
        H = rng.choice([1, 3, 8, 16, 16, 32])
        hi = _log_int(rng, 1, 8000 if op == "fwd" else 6000)
        lo = rng.randint(1, hi)
        # padded score matrices of the plain form stay below those of the largest listed case
        room = 8192 * 8192 * 16 // (H * hi * hi)
        n = max(1, min(_log_int(rng, 1, 64), room // 2))
        ctx = rng.choice([0, 0, _log_int(rng, 1, 12000)])
        if n * H * hi * (hi + ctx) > 8192 * 8192 * 16:
            ctx = 0
        return dict(op=op, n=n, q_lo=lo, q_hi=hi, ctx=ctx, H=H, causal=rng.random() < 0.8)
    if op == "decode":
        G = rng.choice([1, 1, 2])
        H = G * rng.choice([1, 5, 16, 32])
        hi = _log_int(rng, 1, 40000)
        lo = rng.randint(0, hi)
        n = max(1, min(_log_int(rng, 1, 256), 256 * 5000 // (hi * G)))
        return dict(op=op, n=n, lo=lo, hi=hi, H=H, G=G, Sq=rng.choice([1, 1, 2, 3]), page=rng.choice([16, 32, 64, 128]),
                    e4m3=rng.random() < 0.5)
    hi = _log_int(rng, 1, 8000)
    n = max(1, min(_log_int(rng, 1, 256), 80000 // hi))
    return dict(op=op, n=n, lo=rng.randint(0, hi), hi=hi, held=_log_int(rng, 1, 5000), G=rng.choice([1, 1, 2]),
                page=rng.choice([16, 32, 64, 128]), e4m3=rng.random() < 0.7)


def _spread(n, lo, hi):
    """n whole numbers spread over lo..hi, the first of them hi."""
    return [hi - int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def work(case):
    c = case
    if c["op"] in ("fwd", "bwd"):
        lq = _spread(c["n"], c["q_lo"], c["q_hi"])
        pairs = sum(x * (x + c["ctx"]) - (x * (x - 1) // 2 if c["causal"] else 0) for x in lq)
        tq, tk, H = sum(lq), sum(lq) + c["n"] * c["ctx"], c["H"]
        read = 2 * (tq * H * (DN + DR) + tk * H * (DN + DV) + tk * DR)
        rows = 2 * tq * H * DV + 4 * tq * H  # o and lse
        if c["op"] == "fwd":
            return {"bytes": read + rows, "flops": 2 * (DN + DR + DV) * H * pairs}
        return {"bytes": 2 * read + rows + 2 * tq * H * DV, "flops": 2 * (3 * (DN + DR) + 2 * DV) * H * pairs}
    if c["op"] == "decode":
        lens = _spread(c["n"], c["lo"], c["hi"])
        row = c["G"] * DC * (1 if c["e4m3"] else 2)
        q = c["n"] * c["Sq"] * c["H"]
        pairs = sum(max(0, x - s) for x in lens for s in range(c["Sq"])) * c["H"]
        return {"bytes": sum(lens) * row + q * (2 * DC + 2 * DL + 4), "flops": 2 * (DC + DL) * pairs}
    t = sum(_spread(c["n"], c["lo"], c["hi"]))
    return {"bytes": t * c["G"] * DC * (3 if c["e4m3"] else 4), "flops": 2 * t * c["G"] * DC}


# ---------------------------------------------------------------- inputs
def _randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(g, lens, page, n_spare=3):
    """A table of distinct pages in random order for sequences of these lengths (unused entries
    are -1), and how many pages the pool has."""
    need = [-(-x // page) for x in lens]
    total = sum(need) + n_spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    return table, total


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    if c["op"] in ("fwd", "bwd"):
        lq = _spread(c["n"], c["q_lo"], c["q_hi"])
        lk = [x + c["ctx"] for x in lq]
        tq, tk, H = sum(lq), sum(lk), c["H"]
        s.update(lq=lq, lk=lk, cu_q=_ints(_offsets(lq)), cu_k=_ints(_offsets(lk)), scale=(DN + DR) ** -0.5,
                 q=_randn(g, tq, H, DN + DR, std=1.5), kv=_randn(g, tk, H, DN + DV), k_rope=_randn(g, tk, DR))
        if c["op"] == "bwd":  # what a training step holds after its forward pass
            s["dO"] = _randn(g, tq, H, DV)
            s["o"], s["lse"] = _plain_fwd(s)
        return s
    if c["op"] == "decode":
        lens = _spread(c["n"], c["lo"], c["hi"])
        table, pages = _pages(g, lens, c["page"])
        s.update(kv_lens=_ints(lens), block_table=table, scale=(DN + DR) ** -0.5,
                 q=_randn(g, c["n"], c["Sq"], c["H"], DC, std=0.6))
        cache = torch.empty(pages, c["page"], c["G"], DC, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        s["cache"], s["cache_scale"] = _quantised(cache) if c["e4m3"] else (cache, None)
        return s
    new = _spread(c["n"], c["lo"], c["hi"])
    held = _spread(c["n"], 0, c["held"])
    table, pages = _pages(g, [a + b for a, b in zip(new, held)], c["page"])
    rows = _randn(g, sum(new), c["G"], DC)
    cache = torch.empty(pages, c["page"], c["G"], DC, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    # pages differ in magnitude, so that some have to be held at a larger scale after the call
    cache *= torch.exp2(torch.randint(-2, 2, (pages, 1, 1, 1), generator=g, device="cuda")).to(torch.bfloat16)
    s.update(kv_new=rows, cu_new=_ints(_offsets(new)), kv_lens=_ints(held), block_table=table)
    s["cache"], s["cache_scale"] = _quantised(cache) if c["e4m3"] else (cache, None)
    return s


def _power_for(amax):
    """The smallest power of two s >= 2^-100 with amax <= 448 s (NaN where amax is not finite)."""
    m, k = torch.frexp(amax)  # amax = m 2^k, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m <= 0.875, k - 9, k - 8).clamp(min=-100)
    e = torch.where(amax > 0, e, torch.full_like(e, -100))
    return torch.where(torch.isfinite(amax), torch.ldexp(torch.ones_like(amax), e), torch.full_like(amax, math.nan))


def _quantised(cache):
    scale = _power_for(cache.float().abs().amax(dim=(1, 3)))
    return (cache.float() / scale[:, None, :, None]).to(torch.float8_e4m3fn), scale


# ---------------------------------------------------------------- plain forms
def _padded(cu, n_rows):
    """Packed rows to a padded batch: row index [N, L], which of them exist, and of every packed
    row its sequence and place."""
    lens = (cu[1:] - cu[:-1]).long()
    t = torch.arange(n_rows, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), t, right=True)
    place = t - cu.long()[seq]
    return lens, seq, place


def _dense(x, cu, L):
    lens = (cu[1:] - cu[:-1]).long()
    at = torch.arange(L, device=x.device)
    live = at < lens[:, None]
    idx = torch.where(live, cu[:-1].long()[:, None] + at, 0)
    return torch.where(live.view(*live.shape, *[1] * (x.dim() - 1)), x[idx].float(), 0.0), live


def _scores(s):
    """Padded float32 queries, keys, values and masked scores [N, H, Lq, Lk]."""
    Lq, Lk = max(s["lq"]), max(s["lk"])
    q, _ = _dense(s["q"], s["cu_q"], Lq)
    kv, live = _dense(s["kv"], s["cu_k"], Lk)
    kr, _ = _dense(s["k_rope"], s["cu_k"], Lk)
    k = torch.cat([kv[..., :DN], kr[:, :, None].expand(-1, -1, s["H"], -1)], -1)
    q, k, v = q.transpose(1, 2), k.transpose(1, 2), kv[..., DN:].transpose(1, 2)
    sc = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    ok = live[:, None, :]
    if s["causal"]:
        lq, lk = (s["cu_q"][1:] - s["cu_q"][:-1])[:, None, None], (s["cu_k"][1:] - s["cu_k"][:-1])[:, None, None]
        i, j = torch.arange(Lq, device=q.device)[:, None], torch.arange(Lk, device=q.device)
        ok = ok & (j <= i + (lk - lq))
    return q, k, v, sc.masked_fill_(~ok[:, None], -math.inf)


def _plain_fwd(s):
    _, _, v, sc = _scores(s)
    m = sc.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l))[..., 0]
    _, seq, place = _padded(s["cu_q"], s["q"].shape[0])
    return o[seq, :, place].to(torch.bfloat16), lse[seq, :, place].contiguous()


def _plain_bwd(s):
    q, k, v, sc = _scores(s)
    Lq, Lk = max(s["lq"]), max(s["lk"])
    dO, _ = _dense(s["dO"], s["cu_q"], Lq)
    o, _ = _dense(s["o"], s["cu_q"], Lq)
    lse, _ = _dense(s["lse"], s["cu_q"], Lq)
    dO = dO.transpose(1, 2)
    delta = (dO * o.transpose(1, 2)).sum(-1, keepdim=True)
    p = sc.sub_(lse.transpose(1, 2)[..., None].clamp(min=-1e30)).exp_()
    dv = torch.matmul(p.transpose(-1, -2), dO)
    ds = torch.matmul(dO, v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q)
    _, sq, pq = _padded(s["cu_q"], s["q"].shape[0])
    _, sk, pk = _padded(s["cu_k"], s["kv"].shape[0])
    dkv = torch.cat([dk[..., :DN], dv], -1)[sk, :, pk]
    return {"dq": dq[sq, :, pq].to(torch.bfloat16), "dkv": dkv.to(torch.bfloat16),
            "dk_rope": dk[..., DN:].sum(1)[sk, pk].to(torch.bfloat16)}


def _plain_decode(s):
    n, Sq, H, _ = s["q"].shape
    G, page = s["G"], s["page"]
    L = s["block_table"].shape[1] * page
    at = torch.arange(L, device="cuda")
    live = at < s["kv_lens"][:, None]
    table = s["block_table"].clamp(min=0).long()
    c = s["cache"][table].float()
    if s["cache_scale"] is not None:
        c = c * s["cache_scale"][table][:, :, None, :, None]
    c = torch.where(live[:, :, None, None], c.reshape(n, L, G, DC), 0.0).transpose(1, 2)          # [n, G, L, DC]
    q = s["q"].float().view(n, Sq, G, H // G, DC).permute(0, 2, 1, 3, 4).reshape(n, G, -1, DC)    # rows (step, head)
    sc = torch.matmul(q, c.transpose(-1, -2)).mul_(s["scale"]).view(n, G, Sq, H // G, L)
    last = s["kv_lens"][:, None] - Sq + torch.arange(Sq, device="cuda")                           # [n, Sq]
    ok = at <= last[..., None]
    sc = sc.masked_fill_(~ok[:, None, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, G, -1, L), c[..., :DL]).view(n, G, Sq, H // G, DL) / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l))[..., 0]
    return o.permute(0, 2, 1, 3, 4).reshape(n, Sq, H, DL).to(torch.bfloat16), lse.permute(0, 2, 1, 3).reshape(n, Sq, H)


def _plain_append(s):
    new, cache, scale, page = s["kv_new"], s["cache"], s["cache_scale"], s["page"]
    _, seq, place = _padded(s["cu_new"], new.shape[0])
    pos = s["kv_lens"].long()[seq] + place
    to, slot = s["block_table"].long()[seq, pos // page], pos % page
    if scale is None:
        cache[to, slot] = new
        return {"cache": cache}
    # pages that rows of the call go to, and those of them that hold older rows of their sequence
    amax = torch.zeros_like(scale).index_reduce_(0, to, new.float().abs().amax(-1), "amax")
    need = _power_for(amax)
    first = s["kv_lens"].long()
    some = ((s["cu_new"][1:] > s["cu_new"][:-1]) & (first % page > 0))
    mine = torch.where(some, s["block_table"].long().gather(1, (first // page).clamp(max=s["block_table"].shape[1] - 1)[:, None])[:, 0], 0)
    old = torch.where(some[:, None], scale[mine], 0.0)
    now = torch.where(some[:, None], torch.maximum(old, need[mine]), 1.0)
    kept = some[:, None] & (torch.arange(page, device="cuda") < (first % page)[:, None])
    codes = cache[mine].float() * (old / now)[:, None, :, None]
    n_i, s_i = torch.nonzero(kept, as_tuple=True)
    cache.view(torch.uint8)[mine[n_i], s_i] = codes[n_i, s_i].to(torch.float8_e4m3fn).view(torch.uint8)
    need[mine[some]] = now[some]
    scale[to] = need[to]
    cache.view(torch.uint8)[to, slot] = (new.float() / need[to][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return {"cache": cache, "cache_scale": scale}


def run(s):
    if own:
        import chunked_linear_attention_chunk_b200 as kda
        if s["op"] == "fwd":
            return kda.kda_mla_fwd(s["q"], s["kv"], s["k_rope"], s["cu_q"], s["cu_k"], scale=s["scale"], causal=s["causal"])
        if s["op"] == "bwd":
            return kda.kda_mla_bwd(s["q"], s["kv"], s["k_rope"], s["o"], s["lse"], s["dO"], s["cu_q"], s["cu_k"],
                                   scale=s["scale"], causal=s["causal"])
        if s["op"] == "decode":
            return kda.kda_mla_decode(s["q"], s["cache"], s["block_table"], s["kv_lens"], scale=s["scale"],
                                      cache_scale=s["cache_scale"])
        kda.kda_mla_cache_append(s["kv_new"], s["cu_new"], s["kv_lens"], s["block_table"], s["cache"],
                                 cache_scale=s["cache_scale"])
        return {"cache": s["cache"]} if s["cache_scale"] is None else {"cache": s["cache"], "cache_scale": s["cache_scale"]}
    if s["op"] == "fwd":
        return _plain_fwd(s)
    if s["op"] == "bwd":
        return _plain_bwd(s)
    return _plain_decode(s) if s["op"] == "decode" else _plain_append(s)


# ---------------------------------------------------------------- the definitions in 64 bits
def _visible(lq, lk, causal):
    vis = torch.ones(lq, lk, dtype=torch.bool, device="cuda")
    return torch.tril(vis, diagonal=lk - lq) if causal else vis


def _softmax64(x, vis):
    x = torch.where(vis, x, -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.where(vis, torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[..., None]), 0.0), lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        if work(case)["flops"] > 5e12:
            return None
        q, kv, kr = s["q"].double(), s["kv"].double(), s["k_rope"].double()
        back = case["op"] == "bwd"
        o, lse = torch.zeros(q.shape[0], case["H"], DV, dtype=torch.float64, device="cuda"), torch.zeros(
            q.shape[0], case["H"], dtype=torch.float64, device="cuda")
        dq, dkv, dkr = torch.zeros_like(q), torch.zeros_like(kv), torch.zeros_like(kr)
        a = b = 0
        for lq, lk in zip(s["lq"], s["lk"]):
            vis = _visible(lq, lk, case["causal"])
            for h in range(case["H"]):
                qh = q[a:a + lq, h]
                kh = torch.cat([kv[b:b + lk, h, :DN], kr[b:b + lk]], 1)
                vh = kv[b:b + lk, h, DN:]
                sc = qh @ kh.T * s["scale"]
                if not back:
                    p, lse[a:a + lq, h] = _softmax64(sc, vis)
                    o[a:a + lq, h] = p @ vh
                    continue
                given = s["lse"][a:a + lq, h].double()[:, None]
                p = torch.where(vis, torch.exp(sc - given), 0.0)
                do = s["dO"][a:a + lq, h].double()
                ds = s["scale"] * p * (do @ vh.T - (do * s["o"][a:a + lq, h].double()).sum(1, keepdim=True))
                dq[a:a + lq, h] = ds @ kh
                dk = ds.T @ qh
                dkv[b:b + lk, h, :DN] = dk[:, :DN]
                dkv[b:b + lk, h, DN:] = p.T @ do
                dkr[b:b + lk] += dk[:, DN:]
            a, b = a + lq, b + lk
        return {"dq": dq, "dkv": dkv, "dk_rope": dkr} if back else (o, lse)
    if case["op"] == "decode":
        n, Sq, H, G, page = case["n"], case["Sq"], case["H"], case["G"], case["page"]
        o = torch.zeros(n, Sq, H, DL, dtype=torch.float64, device="cuda")
        lse = torch.full((n, Sq, H), -math.inf, dtype=torch.float64, device="cuda")
        for i, L in enumerate(_spread(n, case["lo"], case["hi"])):
            if L == 0:
                continue
            ids = s["block_table"][i, :-(-L // page)].long()
            c = s["cache"][ids].double()
            if case["e4m3"]:
                c = c * s["cache_scale"][ids].double()[:, None, :, None]
            c = c.reshape(-1, G, DC)[:L]
            vis = _visible(Sq, L, True)
            for gr in range(G):
                hs = slice(gr * (H // G), (gr + 1) * (H // G))
                x = torch.einsum("shd,ld->hsl", s["q"][i, :, hs].double(), c[:, gr]) * s["scale"]
                p, l = _softmax64(x, vis)
                o[i, :, hs] = torch.einsum("hsl,ld->shd", p, c[:, gr, :DL])
                lse[i, :, hs] = l.T
        return o, lse
    # append: row by row of the table, with whole-number scales
    page, G = case["page"], case["G"]
    cache, scale = s["cache"].double(), s["cache_scale"]
    new = s["kv_new"].double()
    at = 0
    if scale is not None:
        scale = scale.double()
    for i, (k, held) in enumerate(zip(_spread(case["n"], case["lo"], case["hi"]), _spread(case["n"], 0, case["held"]))):
        done = 0
        while done < k:
            p, slot = s["block_table"][i, (held + done) // page].long(), (held + done) % page
            m = min(page - slot, k - done)
            rows = new[at + done:at + done + m]
            if scale is None:
                cache[p, slot:slot + m] = rows
            else:
                want = torch.exp2(torch.ceil(torch.log2(rows.abs().amax(dim=(0, 2)) / 448.0)).clamp(min=-100))
                if slot:
                    want = torch.maximum(want, scale[p])
                    cache[p, :slot] = (cache[p, :slot] * (scale[p] / want)[:, None]).to(torch.float8_e4m3fn).double()
                scale[p] = want
                cache[p, slot:slot + m] = (rows / want[:, None]).to(torch.float8_e4m3fn).double()
            done += m
        at += k
    return {"cache": cache} if scale is None else {"cache": cache, "cache_scale": scale}
