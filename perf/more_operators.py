"""Cases of the operators around the 8-bit paged cache for long contexts: the norm and position rotation
of queries and keys, attention of a batch that shares prefixes, and attention over the pages that a cheap
score selects (the summaries of the cached keys, the selection, the attention over the selected pages).

``run`` gives an operator's plain form in 32-bit torch operations (64 where angles and sums need it), or,
where ``own`` is set, the call a user makes of the library.  ``exact`` restates the definitions in 64 bits.
"""
import math

import torch

own = False

PAGE = 64  # tokens per cache page
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the queries and keys of packed prompts, read where the fused projection left them: norm of every
        # head, all channels rotated
        dict(name="rotate_prompt", op="rotate", tokens=16384, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             norm=True, stretch=1.0, pos_max=16383, dtype="bf16", fused_qkv=True),
        # a decode step of 256 sequences far into stretched contexts, half of the channels rotated, in pairs of
        # neighbours: latency counts
        dict(name="rotate_step", op="rotate", tokens=256, hq=32, hkv=8, d=128, rot=64, interleaved=True, norm=True,
             stretch=16.0, pos_max=1000000, dtype="bf16", fused_qkv=True),
        # a chat service: 64 users after one system prompt and tools of 8192 tokens
        dict(name="shared_system", op="shared", groups=1, batch=64, draft=1, pages_min=128, pages_max=128, own_max=2048,
             hq=32, hkv=8, d=128, dtype="bf16"),
        # 32 questions about one document of 102400 tokens
        dict(name="shared_document", op="shared", groups=1, batch=32, draft=1, pages_min=1600, pages_max=1600, own_max=512,
             hq=32, hkv=8, d=128, dtype="bf16"),
        # speculative verify of 7 draft tokens: five prefixes of different lengths
        dict(name="shared_window", op="shared", groups=5, batch=40, draft=7, pages_min=3, pages_max=160, own_max=1000,
             hq=32, hkv=4, d=128, dtype="bf16"),
        # a few young sequences, fp32 (verification runs)
        dict(name="shared_f32", op="shared", groups=2, batch=6, draft=1, pages_min=2, pages_max=9, own_max=200, hq=4,
             hkv=2, d=64, dtype="f32"),
        # a decode batch: every sequence's last page got a token
        dict(name="summary_step", op="summary", lens="", start_max=32000, hkv=8, d=128, seqs=256, each=1),
        # the prompts of a batch were appended; some continue a sequence inside a page
        dict(name="summary_prompt", op="summary", lens="8192,5000,1,64,9001,0,4097,6000", start_max=200, hkv=8, d=128,
             seqs=0, each=0),
        # one user with a 102400-token context
        dict(name="select_one", op="select", batch=1, draft=1, len_min=102400, len_max=102400, budget=128, sink=1,
             recent=2, hq=32, hkv=8, d=128, dtype="bf16"),
        # a ragged decode batch of long contexts
        dict(name="select_batch", op="select", batch=64, draft=1, len_min=1, len_max=102400, budget=64, sink=1, recent=2,
             hq=32, hkv=8, d=128, dtype="bf16"),
        # attention over what was selected for one user
        dict(name="attend_one", op="attend", batch=1, draft=1, len_min=102400, len_max=102400, budget=128, hq=32, hkv=8,
             d=128, dtype="bf16"),
        # and for a decode batch
        dict(name="attend_batch", op="attend", batch=64, draft=1, len_min=1, len_max=102400, budget=64, hq=32, hkv=8,
             d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "shared", "shared", "summary", "select", "attend"])
    d = rng.choice([32, 64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8])
    if op == "rotate":
        top = 16384 * 40 * 128 // ((hkv * g + hkv) * d * (2 if dtype == "f32" else 1))
        return dict(op=op, tokens=_log(rng, 1, min(20000, top)), hq=hkv * g, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.7, stretch=rng.choice([1.0, 1.0, 4.0, 32.0]), pos_max=_log(rng, 64, 1000000),
                    dtype=dtype, fused_qkv=rng.random() < 0.5)
    draft = rng.choice([1, 1, 1, 2, 4, 7, 8])
    if op == "shared":
        batch = _log(rng, 2, 128)
        groups = 1 if rng.random() < 0.5 else _log(rng, 1, min(8, batch))
        # no more than the long document's positions, and its products
        top = int(3.2e6 * 8 * 128 / (batch * hkv * d)) // (4 if dtype == "f32" else 1)
        top = min(top, 102400, int(1.3e10 / (batch * draft * hkv * g * d)) // (8 if dtype == "f32" else 1))
        hi = max(1, _log(rng, 64, max(128, top)) // PAGE)
        return dict(op=op, groups=groups, batch=batch, draft=draft, pages_min=rng.choice([0, 1, hi, hi]), pages_max=hi,
                    own_max=_log(rng, draft, 2048), hq=hkv * g, hkv=hkv, d=d, dtype=dtype)
    if op == "summary":
        if rng.random() < 0.5:
            return dict(op=op, lens="", start_max=_log(rng, 64, 32000), hkv=hkv, d=d, seqs=_log(rng, 1, 512),
                        each=rng.choice([1, 1, 2, 7]))
        lens = [_log(rng, 1, 9000) for _ in range(rng.randint(1, 8))]
        while sum(lens) > 32000:
            lens[lens.index(max(lens))] //= 2
        return dict(op=op, lens=",".join(map(str, lens)), start_max=_log(rng, 1, 3000), hkv=hkv, d=d, seqs=0, each=0)
    batch = _log(rng, 1, 64)
    sink, recent = rng.randint(0, 2), rng.randint(2, 4)
    budget = rng.randint(sink + recent, 160)
    if op == "select":
        hi = _log(rng, 64, min(102400, int(64 * 102400 * 8 * 4 / (batch * hkv * g * draft))))
        return dict(op=op, batch=batch, draft=draft, len_min=rng.choice([0, 1, hi // 2]), len_max=hi, budget=budget,
                    sink=sink, recent=recent, hq=hkv * g, hkv=hkv, d=d, dtype=dtype)
    hi = _log(rng, 64, 102400)
    while batch * hkv * min(budget, -(-hi // PAGE)) > 64 * 64 * 8:
        batch = max(1, batch // 2)
    return dict(op=op, batch=batch, draft=draft, len_min=rng.choice([0, 1, hi // 2]), len_max=hi, budget=budget,
                hq=hkv * g, hkv=hkv, d=d, dtype=dtype)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _randint(g, lo, hi, shape):
    """Whole numbers in lo..hi."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int64)


def _unit(amax, most):
    """The smallest power of two u >= 2^-126 with amax <= most u."""
    top, up = math.frexp(most)
    m, e = torch.frexp(amax)
    e = torch.where(m > top, e + 1, e) - up
    return ((torch.where(amax == 0, -126, e).clamp(min=-126) + 127) << 23).to(torch.int32).view(torch.float32)


def _gain(g, heads, d):
    """Channels of a head differ: some are several times larger than others."""
    gain = torch.exp(0.5 * _randn(g, 1, heads, 1, d))
    return gain / gain.square().mean(-1, keepdim=True).sqrt()


def _random_cache(g, pages, heads, d):
    """A cache whose pages hold quantised normal keys and values."""
    made = []
    gain = _gain(g, heads, d)
    for x in (_randn(g, pages, heads, PAGE, d) * gain, _randn(g, pages, heads, d, PAGE)):
        s = _unit(x.abs().amax((2, 3)), 448.0)
        made += [(x / s[:, :, None, None]).to(torch.float8_e4m3fn), s]
        del x
    return made


def _frequencies(rot, stretch):
    """Angles a position: base 10000 to the power -2 i / rot; for a context stretched beyond 8192 positions the
    slow channels (less than 1 turn in 8192) by the stretch, the fast ones (more than 32) not, and between by a ramp."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if stretch == 1.0:
        return f, 1.0
    turns = 8192 * f / (2 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0, 1)
    return f * keep + f / stretch * (1 - keep), 0.1 * math.log(stretch) + 1.0


def _fixed_point(f):
    """Turns a position in units of 2^-64, modulo a turn, as the library's rotation table holds them."""
    whole = [round(x / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for x in f.tolist()]
    return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in whole], dtype=torch.int64, device="cuda")


def _lens(case):
    return [case["each"]] * case["seqs"] if case.get("seqs") else [int(x) for x in case["lens"].split(",")]


def _pages_of(lens):
    return (lens + PAGE - 1) // PAGE


def _random_table(g, held, width):
    """Distinct pages for every sequence's `held` first columns, -1 behind them."""
    B, total = held.shape[0], max(int(held.sum()), 1)
    mine = torch.arange(width, device="cuda") < held[:, None]
    ids = torch.cumsum(mine.reshape(-1).long(), 0).reshape(B, width) - 1
    perm = torch.randperm(total, generator=g, device="cuda")
    return torch.where(mine, perm[ids.clamp(min=0)], torch.full_like(ids, -1)), total


def prepare(case, seed):
    g = _gen(seed)
    op, d = case["op"], case["d"]
    st = {"case": case}
    if op == "rotate":
        T, hq, hkv, dt = case["tokens"], case["hq"], case["hkv"], _DT[case["dtype"]]
        q, k = (2.0 * _randn(g, T, hq, d)).to(dt), (_randn(g, T, hkv, d) * _gain(g, hkv, d)[0, :, 0]).to(dt)
        if case["fused_qkv"]:  # slices of one projection's output
            row = torch.cat([q, k, k], 1)
            q, k = row[:, :hq], row[:, hq:hq + hkv]
        f, factor = _frequencies(case["rot"], case["stretch"])
        st.update(q=q, k=k, pos=_randint(g, 0, case["pos_max"], (T,)).int(), freq=f.cuda(), factor=factor,
                  turns=_fixed_point(f))
        if case["norm"]:
            st.update(qw=1.0 + 0.2 * _randn(g, d), kw=1.0 + 0.2 * _randn(g, d))
    elif op == "shared":
        B, n, D, dt = case["batch"], case["groups"], case["draft"], _DT[case["dtype"]]
        cut = torch.sort(_randint(g, 0, B, (n - 1,))).values
        start = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), B)])
        shared = _randint(g, case["pages_min"], case["pages_max"], (n,))
        own_lens = _randint(g, min(D, case["own_max"]), case["own_max"], (B,))
        group = torch.searchsorted(start[1:].contiguous(), torch.arange(B, device="cuda"), right=True)
        first = shared[group]
        lens = first * PAGE + own_lens
        width = int(_pages_of(lens).max())
        mine, total = _random_table(g, _pages_of(own_lens), int(_pages_of(own_lens).max()))
        before = torch.cumsum(shared, 0) - shared  # the prefixes' pages come behind the sequences' own
        col = torch.arange(width, device="cuda")
        there = (col - first[:, None]).clamp(0, mine.shape[1] - 1)
        table = torch.where(col < first[:, None], total + before[group][:, None] + col, mine.gather(1, there))
        table = torch.where(col < _pages_of(lens)[:, None], table, torch.full_like(table, -1))
        perm = torch.randperm(total + int(shared.sum()), generator=g, device="cuda")
        table = torch.where(table >= 0, perm[table.clamp(min=0)], table)
        kp, ks, vp, vs = _random_cache(g, perm.shape[0], case["hkv"], d)
        st.update(q=(2.0 * _randn(g, B, D, case["hq"], d)).to(dt), lens=lens.int(), table=table.int(),
                  start=start.int(), shared=shared.int(), kp=kp, ks=ks, vp=vp, vs=vs)
    elif op == "summary":
        lens, hkv = _lens(case), case["hkv"]
        n = len(lens)
        start = _randint(g, 0, case["start_max"], (n,))
        size = torch.tensor(lens, device="cuda")
        width = int(_pages_of(start + size).max())
        col = torch.arange(width, device="cuda")
        # the pages that the call looks at are distinct; those before them are one page here
        hit = (col >= (start // PAGE)[:, None]) & (col <= ((start + size - 1) // PAGE)[:, None]) & (size > 0)[:, None]
        ids = torch.cumsum(hit.reshape(-1).long(), 0).reshape(n, width) - 1
        count = sum((PAGE - 1 + x) // PAGE + 1 for x in lens)  # (some pages stay free)
        perm = torch.randperm(count, generator=g, device="cuda")
        kp, ks, vp, vs = _random_cache(g, count + 1, hkv, d)
        st.update(cu=torch.cat([size.new_zeros(1), torch.cumsum(size, 0)]).int(), start=start.int(), tokens=sum(lens),
                  table=torch.where(hit, perm[ids.clamp(min=0)], torch.full_like(ids, count)).int(),
                  kp=kp, ks=ks, vp=vp, vs=vs,
                  bounds=torch.zeros((count + 1, hkv, 2, d), dtype=torch.int8, device="cuda"),
                  unit=torch.ones((count + 1, hkv), device="cuda"))
    else:
        B, D, hq, hkv, dt = case["batch"], case["draft"], case["hq"], case["hkv"], _DT[case["dtype"]]
        lens = _randint(g, case["len_min"], case["len_max"], (B,))
        held = _pages_of(lens)
        width = max(1, (case["len_max"] + PAGE - 1) // PAGE)
        q = (2.0 * _randn(g, B, D, hq, d)).to(dt)
        if op == "select":
            table, total = _random_table(g, held, width)
            # the largest and smallest of 64 normal keys a channel, in steps of the page's unit
            gain = _gain(g, hkv, d)[:, :, 0]
            mid = 0.5 * _randn(g, total, hkv, d)
            hi = (2.4 + mid + 0.4 * _randn(g, total, hkv, d)) * gain
            lo = (-2.4 + mid - 0.4 * _randn(g, total, hkv, d)) * gain
            both = torch.stack([torch.maximum(hi, lo), torch.minimum(hi, lo)], 2)
            unit = _unit(both.abs().amax((2, 3)), 127.0)
            bounds = torch.round(both / unit[:, :, None, None]).to(torch.int8)
            st.update(q=q, lens=lens.int(), table=table.int(), bounds=bounds, unit=unit)
        else:
            K = case["budget"]
            mine = held.clamp(max=K)
            kept = (mine * PAGE - (held * PAGE - lens)).int()
            # for every kv head its own pages, the last one among them, in order
            mark = torch.rand((B, hkv, width), generator=g, device="cuda")
            col = torch.arange(width, device="cuda")
            mark = torch.where(col >= held[:, None, None], torch.full_like(mark, -1.0), mark)
            mark = torch.where(col == held[:, None, None] - 1, torch.full_like(mark, 2.0), mark)
            order = torch.argsort(mark, -1, descending=True)
            pad = torch.zeros((B, hkv, max(0, K - width)), dtype=order.dtype, device="cuda")
            order = torch.cat([order, pad], 2)[:, :, :K]
            behind = torch.arange(K, device="cuda") >= mine[:, None, None]
            index = torch.sort(torch.where(behind, torch.full_like(order, 1 << 30), order), -1).values
            ids, total = _random_table(g, mine.repeat_interleave(hkv), K)
            st.update(q=q, lens=kept, table=ids.view(B, hkv, K).int(),
                      index=torch.where(behind, torch.full_like(index, -1), index).int())
            kp, ks, vp, vs = _random_cache(g, total, hkv, d)
            st.update(kp=kp, ks=ks, vp=vp, vs=vs)
    return st


# ---------------------------------------------------------------- the plain forms

def _plain_rotate(x, pos, freq, factor, interleaved, weight, eps):
    rot = 2 * freq.shape[0]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * weight
    angle = pos.double()[:, None] * freq  # 32 bits lose the angle of a far position
    c, s = (torch.cos(angle) * factor).float()[:, None], (torch.sin(angle) * factor).float()[:, None]
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_attend(q, lens, ids, kp, ks, vp, vs):
    """Attention of q [B, D, hq, d] over the pages ids [B, hkv, P] of each kv head."""
    B, D, hq, d = q.shape
    hkv, P = ids.shape[1], ids.shape[2]
    g = hq // hkv
    head = torch.arange(hkv, device=q.device)[None, :, None]
    ids = ids.long().clamp(min=0)
    k = kp.view(torch.uint8)[ids, head].view(torch.float8_e4m3fn).float() * ks[ids, head][..., None, None]
    qf = q.float().view(B, D, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, D * g, d)
    s = torch.matmul(qf, k.reshape(B, hkv, P * PAGE, d).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    del k
    row = torch.arange(D, device=q.device).repeat_interleave(g)
    limit = lens.long()[:, None] - D + 1 + row[None, :]
    seen = torch.arange(P * PAGE, device=q.device)[None, None, :] < limit[:, :, None]
    s = s.masked_fill(~seen[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    some = total > 0
    p = torch.where(some, p / torch.where(some, total, torch.ones_like(total)), torch.zeros_like(p))
    v = vp.view(torch.uint8)[ids, head].view(torch.float8_e4m3fn).float() * vs[ids, head][..., None, None]
    v = v.transpose(-1, -2).reshape(B, hkv, P * PAGE, d)
    o = torch.matmul(p, v)
    lse = torch.where(some, m + torch.log(total), torch.full_like(total, -math.inf)).squeeze(-1)
    return {"out": o.view(B, hkv, D, g, d).permute(0, 2, 1, 3, 4).reshape(B, D, hq, d).to(q.dtype),
            "lse": lse.view(B, hkv, D, g).permute(0, 2, 1, 3).reshape(B, D, hq)}


def _plain_summary(cu, start, table, kp, ks, bounds, unit):
    n, width = table.shape
    size = (cu[1:] - cu[:-1]).long()
    col = torch.arange(width, device=cu.device)
    end = (start + size)[:, None]
    hit = (col >= (start // PAGE)[:, None]) & (col * PAGE < end) & (size > 0)[:, None]
    page = table.long()[hit]
    fill = (end - col * PAGE).clamp(max=PAGE)[hit]
    k = kp.view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
    there = (torch.arange(PAGE, device=cu.device) < fill[:, None])[:, None, :, None] & ~torch.isnan(k)
    hi = torch.where(there, k, torch.full_like(k, -math.inf)).amax(2)
    lo = torch.where(there, k, torch.full_like(k, math.inf)).amin(2)
    none = torch.isinf(hi)
    both = torch.stack([hi.masked_fill(none, 0.0), lo.masked_fill(none, 0.0)], 2) * ks[page][:, :, None, None]
    step = _unit(both.abs().amax((2, 3)), 127.0)
    return {"bounds": bounds.index_copy(0, page, torch.round(both / step[:, :, None, None]).to(torch.int8)),
            "unit": unit.index_copy(0, page, step)}


def _plain_select(q, lens, table, bounds, unit, budget, sink, recent):
    B, D, hq, d = q.shape
    hkv, P = unit.shape[1], table.shape[1]
    g = hq // hkv
    qf = q.float().view(B, D, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, D * g, d)
    step = _unit(qf.abs().amax(-1), 127.0)
    whole = torch.round(qf / step[..., None])  # whole numbers up to 127, so that every sum below is exact
    ids = table.long().clamp(min=0)
    b = bounds[ids].permute(3, 0, 2, 1, 4).float()  # [2, B, hkv, P, d]
    s = torch.matmul(whole.clamp(min=0), b[0].transpose(-1, -2)) + torch.matmul(whole.clamp(max=0), b[1].transpose(-1, -2))
    score = (s * step[..., None] * unit[ids].transpose(1, 2)[:, :, None]).amax(2)  # [B, hkv, P]
    col = torch.arange(P, device=q.device)
    held = _pages_of(lens.long())[:, None, None]
    stays = (col < sink) | (col >= held - recent)
    score = torch.where(stays, torch.full_like(score, math.inf), score)
    score = torch.where(col < held, score, torch.full_like(score, -math.inf))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    if P < budget:
        order = torch.cat([order, order.new_zeros(B, hkv, budget - P)], -1)
    count = held.clamp(max=budget)
    behind = torch.arange(budget, device=q.device) >= count
    index = torch.sort(torch.where(behind, P, order[..., :budget]), -1).values
    page = table.long()[:, None].expand(B, hkv, P).gather(2, index.clamp(max=P - 1))
    return {"lens": (lens.long() - (held - count)[:, 0, 0] * PAGE).int(),
            "table": torch.where(behind, -1, page).int(), "index": torch.where(behind, -1, index).int()}


def run(state):
    case, st = state["case"], state
    op = case["op"]
    if not own:
        if op == "rotate":
            return {"q": _plain_rotate(st["q"], st["pos"], st["freq"], st["factor"], case["interleaved"], st.get("qw"), 1e-6),
                    "k": _plain_rotate(st["k"], st["pos"], st["freq"], st["factor"], case["interleaved"], st.get("kw"), 1e-6)}
        if op == "shared":
            ids = st["table"][:, None].expand(-1, case["hkv"], -1)
            return _plain_attend(st["q"], st["lens"], ids, st["kp"], st["ks"], st["vp"], st["vs"])
        if op == "summary":
            return _plain_summary(st["cu"], st["start"], st["table"], st["kp"], st["ks"], st["bounds"], st["unit"])
        if op == "select":
            return _plain_select(st["q"], st["lens"], st["table"], st["bounds"], st["unit"], case["budget"], case["sink"],
                                 case["recent"])
        return _plain_attend(st["q"], st["lens"], st["table"], st["kp"], st["ks"], st["vp"], st["vs"])
    from gated_delta_rule_decode_gb300 import attn
    if op == "rotate":
        q, k = attn.norm_rotate(st["q"], st["k"], st["pos"], attn.Rotary(st["turns"], case["interleaved"], st["factor"]),
                                q_weight=st.get("qw"), k_weight=st.get("kw"), eps=1e-6)
        return {"q": q, "k": k}
    if op == "select":
        r = attn.select(st["q"], attn.KeySummary(st["bounds"], st["unit"]), st["lens"], st["table"], case["budget"],
                        case["sink"], case["recent"])
        return {"lens": r.seq_lens, "table": r.block_table, "index": r.index}
    cache = attn.KVCache(st["kp"], st["vp"], st["ks"], st["vs"])
    if op == "shared":
        out, lse = attn.decode_shared(st["q"], cache, st["lens"], st["table"], st["start"], st["shared"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "summary":
        attn.summarise(cache, attn.KeySummary(st["bounds"], st["unit"]), st["cu"], st["tokens"], st["start"], st["table"])
        return {"bounds": st["bounds"], "unit": st["unit"]}
    chosen = attn.Selected(st["lens"], st["table"], st["index"])
    out, lse = attn.decode_selected(st["q"], cache, chosen, return_lse=True)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if op == "summary":  # the keys, their scales, the bounds and units
        lens = _lens(case)
        pages = sum(-(-n // PAGE) for n in lens)
        mean = min(case["start_max"], PAGE - 1) / 2  # positions that a sequence's first page holds already
        tokens = sum(lens) + sum(n > 0 for n in lens) * mean
        return {"bytes": tokens * hkv * d + pages * hkv * (2 * d + 8), "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "rotate":
        return {"bytes": case["tokens"] * ((case["hq"] + hkv) * d * 2 * size + 4), "flops": 0}
    B, D, hq = case["batch"], case["draft"], case["hq"]
    if op == "shared":
        prefix = case["groups"] * (case["pages_min"] + case["pages_max"]) / 2 * PAGE  # positions, each read once
        mine = B * (min(D, case["own_max"]) + case["own_max"]) / 2
        return {"bytes": (prefix + mine) * hkv * (2 * d + 8 / PAGE) + B * D * hq * (2 * d * size + 4),
                "flops": 4 * d * hq * D * (prefix * B / case["groups"] + mine)}
    pages = (case["len_min"] + case["len_max"]) / 2 / PAGE
    if op == "select":  # bounds and units, the queries, the chosen pages' entries
        return {"bytes": B * (pages * (hkv * (2 * d + 4) + 4) + D * hq * d * size + hkv * min(case["budget"], pages) * 8),
                "flops": 4 * B * D * hq * pages * d}
    positions = B * min(case["budget"], pages) * PAGE
    return {"bytes": positions * hkv * (2 * d + 12 / PAGE) + B * D * hq * (2 * d * size + 4),
            "flops": 4 * d * hq * D * positions}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "select":
        return None  # whole numbers all
    st = prepare(case, seed)
    d = case["d"]

    if op == "rotate":
        rot = case["rot"]
        out = {}
        for name, weight in (("q", st.get("qw")), ("k", st.get("kw"))):
            x = st[name].double()
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6) * weight.double()
            # a pair of channels is a complex number that is turned
            turn = torch.polar(torch.full((case["tokens"], 1, rot // 2), st["factor"], dtype=torch.float64, device="cuda"),
                               (st["pos"].double()[:, None] * st["freq"][None, :])[:, None, :])
            if case["interleaved"]:
                z = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
                y = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
                y = torch.cat([z.real, z.imag], -1)
            out[name] = torch.cat([y, x[..., rot:]], -1)
        return out

    # the 256 values of e4m3: sign, 4 exponent bits of bias 7, 3 fraction bits
    values = []
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = math.nan if e == 15 and f == 7 else f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        values.append(-x if b & 128 else x)
    byte = torch.tensor(values, dtype=torch.float64, device="cuda")

    if op == "summary":
        unit = st["unit"].double().clone()
        start, table, cu = st["start"].tolist(), st["table"].tolist(), st["cu"].tolist()
        for n in range(len(start)):
            end = start[n] + cu[n + 1] - cu[n]
            if cu[n + 1] == cu[n]:
                continue
            for c in range(start[n] // PAGE, (end - 1) // PAGE + 1):
                page = table[n][c]
                keys = byte[st["kp"].view(torch.uint8)[page, :, :end - c * PAGE].long()] * st["ks"][page].double()[:, None, None]
                most = keys.abs().amax((1, 2))
                # x = m 2^e with m in [1/2, 1): the power of two at or above x is 2^(e-1) at m = 1/2, else 2^e
                m, e = torch.frexp(most / 127)
                unit[page] = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e).clamp(min=-126))
        return {"bounds": None, "unit": unit}

    B, D, hq, hkv = case["batch"], case["draft"], case["hq"], case["hkv"]
    g = hq // hkv
    out = torch.zeros(B, D, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, D, hq), -math.inf, dtype=torch.float64, device="cuda")
    for n, length in enumerate(st["lens"].tolist()):
        held = -(-length // PAGE)
        if held == 0:
            continue
        for h in range(hkv):
            ids = (st["table"][n, :held] if op == "shared" else st["table"][n, h, :held]).long()
            keys = (byte[st["kp"].view(torch.uint8)[ids, h].long()] * st["ks"][ids, h].double()[:, None, None]).flatten(0, 1)
            vals = byte[st["vp"].view(torch.uint8)[ids, h].long()] * st["vs"][ids, h].double()[:, None, None]
            vals = vals.transpose(1, 2).flatten(0, 1)
            for t in range(D):
                end = length - D + 1 + t
                if end <= 0:
                    continue
                s = st["q"][n, t, h * g:(h + 1) * g].double() @ keys[:end].T / math.sqrt(d)
                top = s.amax(-1, keepdim=True)
                w = torch.exp(s - top)
                total = w.sum(-1)
                out[n, t, h * g:(h + 1) * g] = w @ vals[:end] / total[:, None]
                lse[n, t, h * g:(h + 1) * g] = top.squeeze(-1) + torch.log(total)
    return {"out": out, "lse": lse}
