"""Cases of the softmax-attention operators that sit next to the KDA recurrence in a hybrid model:
attention over packed prompts, the append to an 8-bit paged KV cache, attention over that cache for
single tokens and draft windows, and the eviction of pages by accumulated attention weight.

``run`` gives an operator's plain form in 32-bit torch operations, or, where ``own`` is set, the call
a user makes of the library.  ``exact`` restates the definitions in 64 bits.
"""
import math

import torch

own = False

PAGE = 64          # tokens per cache page
E4M3_MAX = 448.0   # largest finite e4m3 value
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one long prompt (a document, a repository), 8 query heads per kv head
        dict(name="prompt_long", op="prompt", lens="16384", hq=16, hkv=2, d=128, dtype="bf16", fused_qkv=False),
        # a serving batch of mixed prompts, an empty one and a single token among them, read
        # where the fused projection left them
        dict(name="prompt_packed", op="prompt", lens="2048,1,0,777,64,3001,130", hq=32, hkv=8, d=128, dtype="bf16",
             fused_qkv=True),
        # short chat turns, one kv head per query head: latency counts
        dict(name="prompt_short", op="prompt", lens="61,128,17", hq=8, hkv=8, d=64, dtype="bf16", fused_qkv=False),
        # fp32 inputs (verification runs)
        dict(name="prompt_f32", op="prompt", lens="1100,37,400", hq=8, hkv=2, d=64, dtype="f32", fused_qkv=False),
        # the prompts of a batch go into the cache; some continue a sequence inside a page
        dict(name="append_prompt", op="append", lens="8192,5000,1,64,9001,0,4097,6000", start_max=200, hkv=8, d=128,
             dtype="bf16", seqs=0, each=0),
        # every sequence of a decode batch adds its token
        dict(name="append_step", op="append", lens="", start_max=32000, hkv=8, d=128, dtype="bf16", seqs=256, each=1),
        # one user with a 102400-token context
        dict(name="decode_one_long", op="decode", batch=1, draft=1, len_min=102400, len_max=102400, hq=32, hkv=8,
             d=128, dtype="bf16", weights=False),
        # a ragged decode batch that also accumulates the page weights for eviction
        dict(name="decode_batch", op="decode", batch=64, draft=1, len_min=1, len_max=32768, hq=32, hkv=8, d=128,
             dtype="bf16", weights=True),
        # speculative verify: 7 draft tokens a sequence
        dict(name="decode_window", op="decode", batch=32, draft=7, len_min=7, len_max=8192, hq=32, hkv=4, d=128,
             dtype="bf16", weights=False),
        # a few young sequences, fp32
        dict(name="decode_f32", op="decode", batch=4, draft=1, len_min=0, len_max=500, hq=4, hkv=2, d=64,
             dtype="f32", weights=False),
        # a handful of sequences over their budget
        dict(name="evict_small", op="evict", batch=4, pages=64, budget=32, sink=1, recent=4),
        # a decode batch of contexts up to 102400 tokens cut to 32768
        dict(name="evict_batch", op="evict", batch=256, pages=1600, budget=512, sink=2, recent=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "append", "decode", "decode", "evict"])
    if op == "prompt":
        f32 = rng.random() < 0.25
        hkv = rng.choice([1, 2, 3, 4, 8])
        g = rng.choice([1, 2, 3, 4, 5, 8, 16])
        d = rng.choice([32, 64, 64, 128, 128, 128])
        n = rng.randint(1, 6)
        top = (700 if hkv * g > 32 else 1500) if f32 else 4000 if hkv * g > 32 else 9000
        lens = [_log(rng, 1, top) for _ in range(n)]
        while sum(lens) > top:
            lens[lens.index(max(lens))] //= 2
        if rng.random() < 0.2:
            lens.insert(rng.randrange(len(lens) + 1), 0)
        return dict(op=op, lens=",".join(map(str, lens)), hq=hkv * g, hkv=hkv, d=d, dtype="f32" if f32 else "bf16",
                    fused_qkv=rng.random() < 0.5)
    if op == "append":
        hkv, d = rng.choice([1, 2, 4, 5, 8]), rng.choice([32, 64, 128, 128])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if rng.random() < 0.5:
            return dict(op=op, lens="", start_max=_log(rng, 64, 32000), hkv=hkv, d=d, dtype=dtype,
                        seqs=_log(rng, 1, 512), each=rng.choice([1, 1, 2, 7]))
        lens = [_log(rng, 1, 9000) for _ in range(rng.randint(1, 8))]
        while sum(lens) > 32000:
            lens[lens.index(max(lens))] //= 2
        return dict(op=op, lens=",".join(map(str, lens)), start_max=_log(rng, 1, 3000), hkv=hkv, d=d, dtype=dtype,
                    seqs=0, each=0)
    if op == "decode":
        f32 = rng.random() < 0.25
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 3, 4, 6, 8, 16])
        draft = rng.choice([1, 1, 1, 2, 4, 7, 8])
        batch = _log(rng, 1, 128)
        top = min(102400, int(1.0e6 * 8 / (batch * hkv)))
        if draft * g * hkv > 64:
            top = min(top, int(4.0e5 * 64 / (batch * draft * g * hkv)))
        hi = _log(rng, 40, max(64, top))
        return dict(op=op, batch=batch, draft=draft, len_min=rng.choice([0, 1, draft, hi // 2]), len_max=hi, hq=hkv * g,
                    hkv=hkv, d=rng.choice([32, 64, 128, 128, 128]), dtype="f32" if f32 else "bf16",
                    weights=rng.random() < 0.4)
    pages = _log(rng, 8, 1600)
    sink, recent = rng.randint(0, 3), rng.randint(1, 4)
    return dict(op=op, batch=_log(rng, 1, 256), pages=pages, budget=rng.randint(sink + recent, max(sink + recent, pages)),
                sink=sink, recent=recent)


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


def _keys(g, tokens, heads, d, dtype):
    """Keys: unit normal, with some channels several times larger than others."""
    gain = torch.exp(0.5 * _randn(g, heads, d))
    gain = gain / gain.square().mean(-1, keepdim=True).sqrt()
    return (_randn(g, tokens, heads, d) * gain).to(dtype)


def _pow2_scale(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    return ((e + 127) << 23).view(torch.float32)


def _random_cache(g, pages, heads, d):
    """A cache whose pages hold quantised normal keys and values."""
    gain = torch.exp(0.5 * _randn(g, 1, heads, 1, d))
    gain = gain / gain.square().mean(-1, keepdim=True).sqrt()
    made = []
    for x in (_randn(g, pages, heads, PAGE, d) * gain, _randn(g, pages, heads, d, PAGE)):
        s = _pow2_scale(x.abs().amax((2, 3)))
        made += [(x / s[:, :, None, None]).to(torch.float8_e4m3fn), s]
        del x
    return made


def _lens(case):
    return [case["each"]] * case["seqs"] if case.get("seqs") else [int(x) for x in case["lens"].split(",")]


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "prompt":
        lens, hq, hkv, d, dt = _lens(case), case["hq"], case["hkv"], case["d"], _DT[case["dtype"]]
        T = sum(lens)
        q = (2.0 * _randn(g, T, hq, d)).to(dt)
        k, v = _keys(g, T, hkv, d, dt), _randn(g, T, hkv, d).to(dt)
        if case["fused_qkv"]:  # three slices of one projection's output
            row = torch.cat([q, k, v], 1)
            q, k, v = row[:, :hq], row[:, hq:hq + hkv], row[:, hq + hkv:]
        st.update(q=q, k=k, v=v, cu=_cu(lens))
    elif op == "append":
        lens, hkv, d, dt = _lens(case), case["hkv"], case["d"], _DT[case["dtype"]]
        T, n = sum(lens), len(lens)
        start = _randint(g, 0, case["start_max"], (n,))
        need = max((case["start_max"] + x + PAGE - 1) // PAGE + 1 for x in lens)
        # pages that the call touches are distinct; the pages before them stay with their owners,
        # so the table repeats a small pool there
        first, last = start // PAGE, (start + torch.tensor(lens, device="cuda") - 1) // PAGE
        col = torch.arange(need, device="cuda")
        touched = (col >= first[:, None]) & (col <= last[:, None])
        ids = torch.cumsum(touched.reshape(-1).long(), 0).reshape(n, need) - 1
        count = sum((PAGE - 1 + x) // PAGE + 1 for x in lens)
        perm = torch.randperm(count, generator=g, device="cuda")
        table = torch.where(touched, perm[ids.clamp(min=0)], torch.full_like(ids, count))
        kp, ks, vp, vs = _random_cache(g, count + 1, hkv, d)
        ks, vs = ks * 0.5, vs * 0.5  # some pages' scales have to grow
        st.update(k=_keys(g, T, hkv, d, dt), v=_randn(g, T, hkv, d).to(dt), cu=_cu(lens), start=start.int(),
                  table=table.int(), kp=kp, ks=ks, vp=vp, vs=vs)
    elif op == "decode":
        B, D, hq, hkv, d, dt = (case["batch"], case["draft"], case["hq"], case["hkv"], case["d"], _DT[case["dtype"]])
        lens = _randint(g, case["len_min"], case["len_max"], (B,))
        width = (case["len_max"] + PAGE - 1) // PAGE
        held = int(((lens + PAGE - 1) // PAGE).sum())
        owned = torch.arange(width, device="cuda") < ((lens + PAGE - 1) // PAGE)[:, None]
        ids = torch.cumsum(owned.reshape(-1).long(), 0).reshape(B, width) - 1
        perm = torch.randperm(max(held, 1), generator=g, device="cuda")
        table = torch.where(owned, perm[ids.clamp(min=0)], torch.full_like(ids, -1))
        kp, ks, vp, vs = _random_cache(g, max(held, 1), hkv, d)
        st.update(q=(2.0 * _randn(g, B, D, hq, d)).to(dt), lens=lens.int(), table=table.int(), kp=kp, ks=ks, vp=vp,
                  vs=vs)
        if case["weights"]:
            st["weight"] = torch.rand((B, width), generator=g, device="cuda") * owned
    else:
        B, P = case["batch"], case["pages"]
        lens = _randint(g, 1, P * PAGE, (B,))
        perm = torch.randperm(B * P, generator=g, device="cuda").reshape(B, P)
        owned = torch.arange(P, device="cuda") < ((lens + PAGE - 1) // PAGE)[:, None]
        # heavy-tailed weights, rounded so that ties occur
        w = torch.floor(64 * torch.exp(2 * _randn(g, B, P))) / 64
        st.update(lens=lens.int(), table=torch.where(owned, perm, torch.full_like(perm, -1)).int(), weight=w * owned)
    return st


# ---------------------------------------------------------------- the plain forms

def _plain_prompt(q, k, v, cu):
    T, hq, d = q.shape
    hkv = k.shape[1]
    pos = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:].long().contiguous(), pos, right=True)
    seen = (seq[:, None] == seq[None, :]) & (pos[None, :] <= pos[:, None])
    qf = q.float().reshape(T, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    kf, vf = k.float().permute(1, 2, 0), v.float().permute(1, 0, 2)
    s = torch.matmul(qf, kf).mul_(1.0 / math.sqrt(d)).view(hkv, hq // hkv, T, T).masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(hkv, -1, T), vf).view(hkv, hq // hkv, T, d) / l
    lse = (m + torch.log(l)).squeeze(-1)
    return {"out": o.permute(2, 0, 1, 3).reshape(T, hq, d).to(q.dtype), "lse": lse.permute(2, 0, 1).reshape(T, hq)}


def _plain_quantise(x, page, off, keep, pages, scale, token_dim):
    """New rows x [T, H, d] at (page, off) into pages [N, H, ...] with token axis `token_dim`, whose first
    `keep` [N] positions hold earlier tokens; returns the new pages and scales."""
    n, heads = scale.shape
    amax = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    top = torch.zeros(n, heads, device=x.device).index_reduce_(0, page, amax, "amax")
    hit = torch.zeros(n, dtype=torch.bool, device=x.device).index_fill_(0, page, True)
    fresh = _pow2_scale(top)
    new = torch.where((keep > 0)[:, None], torch.maximum(scale, fresh), fresh)
    new = torch.where(hit[:, None], new, scale)
    old = pages.float() * (scale / new)[:, :, None, None]
    place = torch.arange(PAGE, device=x.device)
    kept = (place[None, :] < keep[:, None]) & hit[:, None]
    kept = kept[:, None, :, None] if token_dim == 2 else kept[:, None, None, :]
    full = torch.where(kept, old, pages.float())
    rows = (x / new[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    if token_dim == 2:
        full[page, :, off] = rows
    else:
        full[page, :, :, off] = rows
    return full.to(torch.float8_e4m3fn), new


def _plain_append(k, v, cu, start, table, kp, ks, vp, vs):
    T = k.shape[0]
    i = torch.arange(T, device=k.device)
    seq = torch.searchsorted(cu[1:].long().contiguous(), i, right=True)
    pos = start.long()[seq] + i - cu.long()[seq]
    page, off = table.long()[seq, pos // PAGE], pos % PAGE
    # positions of a page that earlier tokens hold: those before the sequence's start
    keep = torch.zeros(kp.shape[0], dtype=torch.int64, device=k.device)
    keep[page] = (start.long()[seq] - pos // PAGE * PAGE).clamp(0, PAGE)
    kp2, ks2 = _plain_quantise(k.float(), page, off, keep, kp, ks, 2)
    vp2, vs2 = _plain_quantise(v.float(), page, off, keep, vp, vs, 3)
    return {"k_pages": kp2, "k_scale": ks2, "v_pages": vp2, "v_scale": vs2}


def _plain_decode(q, lens, table, kp, ks, vp, vs, weight):
    B, D, hq, d = q.shape
    hkv, P = ks.shape[1], table.shape[1]
    ids = table.long().clamp(min=0)
    k = kp.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * ks[ids][..., None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(B, hkv, P * PAGE, d)
    v = vp.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * vs[ids][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, hkv, P * PAGE, d)
    g = hq // hkv
    qf = q.float().view(B, D, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, D * g, d)
    s = torch.matmul(qf, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    row = torch.arange(D, device=q.device).repeat_interleave(g)
    limit = lens.long()[:, None] - D + 1 + row[None, :]
    seen = torch.arange(P * PAGE, device=q.device)[None, None, :] < limit[:, :, None]
    s = s.masked_fill(~seen[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    some = l > 0
    p = torch.where(some, p / torch.where(some, l, torch.ones_like(l)), torch.zeros_like(p))
    o = torch.matmul(p, v)
    lse = torch.where(some, m + torch.log(l), torch.full_like(l, -math.inf)).squeeze(-1)
    got = {"out": o.view(B, hkv, D, g, d).permute(0, 2, 1, 3, 4).reshape(B, D, hq, d).to(q.dtype),
           "lse": lse.view(B, hkv, D, g).permute(0, 2, 1, 3).reshape(B, D, hq)}
    if weight is not None:
        got["weight"] = weight + p.view(B, hkv * D * g, P, PAGE).sum((1, 3))
    return got


def _plain_evict(lens, table, weight, budget, sink, recent):
    B, P = table.shape
    col = torch.arange(P, device=table.device)
    held = (lens.long() + PAGE - 1) // PAGE
    out = (held - budget).clamp(min=0)
    open_ = (col >= sink) & (col < (held - recent)[:, None])
    key = torch.where(open_, weight, torch.full_like(weight, math.inf))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, col.expand(B, P).contiguous())
    gone = rank >= (P - out)[:, None]
    kept = torch.sort(gone.int(), dim=1, stable=True).indices
    free = torch.sort((~gone).int(), dim=1, stable=True).indices
    past = col >= (P - out)[:, None]
    return {"lens": (lens.long() - out * PAGE).int(),
            "table": torch.where(past, torch.full_like(table, -1), table.gather(1, kept)),
            "weight": torch.where(past, torch.zeros_like(weight), weight.gather(1, kept)),
            "freed": torch.where(col < out[:, None], table.gather(1, free), torch.full_like(table, -1)),
            "count": out.int()}


def run(state):
    case, st = state["case"], state
    op = case["op"]
    if not own:
        if op == "prompt":
            return _plain_prompt(st["q"], st["k"], st["v"], st["cu"])
        if op == "append":
            return _plain_append(st["k"], st["v"], st["cu"], st["start"], st["table"], st["kp"], st["ks"], st["vp"],
                                 st["vs"])
        if op == "decode":
            return _plain_decode(st["q"], st["lens"], st["table"], st["kp"], st["ks"], st["vp"], st["vs"],
                                 st.get("weight"))
        return _plain_evict(st["lens"], st["table"], st["weight"], case["budget"], case["sink"], case["recent"])
    from gated_delta_rule_decode_gb300 import attn
    if op == "prompt":
        out, lse = attn.prefill(st["q"], st["k"], st["v"], st["cu"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "append":
        attn.append(attn.KVCache(st["kp"], st["vp"], st["ks"], st["vs"]), st["k"], st["v"], st["cu"], st["start"],
                    st["table"])
        return {"k_pages": st["kp"], "k_scale": st["ks"], "v_pages": st["vp"], "v_scale": st["vs"]}
    if op == "decode":
        cache = attn.KVCache(st["kp"], st["vp"], st["ks"], st["vs"])
        if "weight" in st:
            out, lse, weight = attn.decode(st["q"], cache, st["lens"], st["table"], return_lse=True,
                                           weight_in=st["weight"], return_weight=True)
            return {"out": out, "lse": lse, "weight": weight}
        out, lse = attn.decode(st["q"], cache, st["lens"], st["table"], return_lse=True)
        return {"out": out, "lse": lse}
    r = attn.evict(st["lens"], st["table"], st["weight"], case["budget"], case["sink"], case["recent"])
    return {"lens": r.seq_lens, "table": r.block_table, "weight": r.weight, "freed": r.freed, "count": r.freed_count}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "evict":  # table and weights in and out, the freed list out, lengths and counts
        return {"bytes": case["batch"] * (case["pages"] * 20 + 12), "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "prompt":
        lens, hq, hkv, d = _lens(case), case["hq"], case["hkv"], case["d"]
        return {"bytes": sum(lens) * ((2 * hq + 2 * hkv) * d * size + 4 * hq),
                "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}
    if op == "append":
        T = sum(_lens(case))
        pages = sum(-(-n // PAGE) for n in _lens(case))
        return {"bytes": T * 2 * case["hkv"] * case["d"] * (size + 1) + pages * case["hkv"] * 8, "flops": 0}
    B, D, hq, hkv, d = case["batch"], case["draft"], case["hq"], case["hkv"], case["d"]
    tokens = B * (case["len_min"] + case["len_max"]) / 2
    held = tokens / PAGE
    return {"bytes": tokens * hkv * 2 * d + held * (8 * hkv + 4 + (8 if case["weights"] else 0))
            + B * D * hq * (2 * d * size + 4), "flops": 4 * d * hq * D * tokens}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "evict":
        weight = torch.zeros(st["weight"].shape, dtype=torch.float64)
        for n, (length, row) in enumerate(zip(st["lens"].tolist(), st["weight"].double().cpu().tolist())):
            held = -(-length // PAGE)
            middle = sorted(range(case["sink"], held - case["recent"]), key=lambda c: (row[c], -c))
            gone = set(middle[:max(0, held - case["budget"])])
            left = [x for c, x in enumerate(row) if c not in gone]
            weight[n, :len(left)] = torch.tensor(left, dtype=torch.float64)
        return {"lens": None, "table": None, "weight": weight, "freed": None, "count": None}

    def table_of_bytes():
        """The 256 values of e4m3: sign, 4 exponent bits of bias 7, 3 fraction bits."""
        values = []
        for b in range(256):
            e, f = (b >> 3) & 15, b & 7
            x = math.nan if e == 15 and f == 7 else f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
            values.append(-x if b & 128 else x)
        return torch.tensor(values, dtype=torch.float64, device="cuda")

    def softmax_rows(scores):
        top = scores.amax(-1, keepdim=True)
        w = (scores - top).exp_()
        return w, w.sum(-1), top.squeeze(-1)

    if op == "prompt":
        lens, hq, hkv, d = _lens(case), case["hq"], case["hkv"], case["d"]
        T = sum(lens)
        if 4 * d * hq * sum(n * n for n in lens) > 6e12:
            return None
        out = torch.empty(T, hq, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(T, hq, dtype=torch.float64, device="cuda")
        at = 0
        for n in lens:
            for h in range(hq):
                kv = h // (hq // hkv)
                keys, vals = st["k"][at:at + n, kv].double(), st["v"][at:at + n, kv].double()
                for lo in range(0, n, 4096):
                    hi = min(n, lo + 4096)
                    s = st["q"][at + lo:at + hi, h].double() @ keys[:hi].T / math.sqrt(d)
                    later = torch.arange(hi, device="cuda")[None, :] > torch.arange(lo, hi, device="cuda")[:, None]
                    w, total, top = softmax_rows(s.masked_fill_(later, -math.inf))
                    out[at + lo:at + hi, h] = w @ vals[:hi] / total[:, None]
                    lse[at + lo:at + hi, h] = top + total.log()
            at += n
        return {"out": out, "lse": lse}

    byte = table_of_bytes()
    if op == "append":
        got = {}
        start, table, cu = st["start"].tolist(), st["table"].tolist(), st["cu"].tolist()
        for x, pages, scale, tag in ((st["k"], st["kp"], st["ks"], "k"), (st["v"], st["vp"], st["vs"], "v")):
            val = byte[pages.view(torch.uint8).long()]
            if tag == "v":
                val = val.transpose(2, 3).contiguous()
            sc = scale.double().clone()
            for n in range(len(start)):
                lo, hi = start[n], start[n] + cu[n + 1] - cu[n]
                if hi == lo:
                    continue
                for c in range(lo // PAGE, (hi - 1) // PAGE + 1):
                    a, b = max(lo, c * PAGE), min(hi, (c + 1) * PAGE)
                    rows = x[cu[n] + a - lo:cu[n] + b - lo].double().transpose(0, 1)
                    # x = m 2^e with m in [1/2, 1): the power of two at or above x is 2^(e-1) at m = 1/2, else 2^e
                    m, e = torch.frexp(rows.abs().amax((1, 2)) / E4M3_MAX)
                    need = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e).clamp(min=-126))
                    page, keep = table[n][c], a - c * PAGE
                    new = torch.maximum(need, sc[page]) if keep else need
                    val[page, :, :keep] *= (sc[page] / new)[:, None, None]
                    val[page, :, keep:keep + b - a] = rows / new[:, None, None]
                    sc[page] = new
            got[tag + "_pages"] = val.transpose(2, 3).contiguous() if tag == "v" else val
            got[tag + "_scale"] = sc
        return got

    B, D, hq, hkv, d = case["batch"], case["draft"], case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    out = torch.zeros(B, D, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, D, hq), -math.inf, dtype=torch.float64, device="cuda")
    weight = st["weight"].double() if "weight" in st else None
    for n, length in enumerate(st["lens"].tolist()):
        held = -(-length // PAGE)
        if held == 0:
            continue
        ids = st["table"][n, :held].long()
        keys = byte[st["kp"].view(torch.uint8)[ids].long()] * st["ks"][ids].double()[..., None, None]
        vals = byte[st["vp"].view(torch.uint8)[ids].long()] * st["vs"][ids].double()[..., None, None]
        keys = keys.transpose(0, 1).reshape(hkv, held * PAGE, d)
        vals = vals.permute(1, 0, 3, 2).reshape(hkv, held * PAGE, d)
        for t in range(D):
            end = length - D + 1 + t
            if end <= 0:
                continue
            for h in range(hkv):
                rows = st["q"][n, t, h * g:(h + 1) * g].double()
                w, total, top = softmax_rows(rows @ keys[h, :end].T / math.sqrt(d))
                out[n, t, h * g:(h + 1) * g] = w @ vals[h, :end] / total[:, None]
                lse[n, t, h * g:(h + 1) * g] = top + total.log()
                if weight is not None:
                    share = torch.zeros(held * PAGE, dtype=torch.float64, device="cuda")
                    share[:end] = (w / total[:, None]).sum(0)
                    weight[n, :held] += share.view(held, PAGE).sum(1)
    return {"out": out, "lse": lse} if weight is None else {"out": out, "lse": lse, "weight": weight}
