"""The operators of the 8-bit latent cache and of block-sparse decode, as measured.

Five operators that belong together: tokens are quantised into the paged 8-bit
cache (append), decode attention reads it (attend), every page gets a mean key
(keys), queries score the pages by them (score), and the best pages of each
query are selected and attended to (sparse).

The plain form (own = False) is elementary torch in 32 bits; with own = True
the same calls go through the framework's public binding.
"""
import math

import torch

own = False

NOPE, ROPE, LORA, VHEAD, PAGE = 128, 64, 512, 128, 64
ROW = LORA + ROPE  # 576 values of a cached token
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
E_MIN, E_MAX = -32, 32  # exponents that a page's scale may have


# ---------------------------------------------------------------- cases
def listed():
    return [
        # Attention over the 8-bit cache.  Two short requests on a 16-head
        # shard: a call whose time is launch latency.
        dict(name="attend_tiny", op="attend", batch=2, q_len=1, heads=16, lo=17, hi=80),
        # One shard of a model split over eight GPUs: bound by the cache's bytes.
        dict(name="attend_tp_shard", op="attend", batch=64, q_len=1, heads=16, lo=4096, hi=4096),
        # All 128 heads on one GPU, requests of very different lengths.
        dict(name="attend_full_head", op="attend", batch=128, q_len=1, heads=128, lo=1000,
             hi=10000),
        # Speculative drafts of four tokens, ragged, one request of four tokens only.
        dict(name="attend_drafts", op="attend", batch=61, q_len=4, heads=128, lo=4, hi=12001),
        # Appending: one new token for each request of a decode batch.
        dict(name="append_decode", op="append", batch=128, lo=64, hi=2000, new=1),
        # Prompts of different lengths written into fresh pages.
        dict(name="append_prefill", op="append", batch=13, lo=512, hi=8190, new=8190),
        # Mean keys: the last page of each request after a decode step (8-bit cache) ...
        dict(name="keys_decode", op="keys", batch=128, lo=64, hi=2000, new=1, fp8=True),
        # ... and every page of fresh prompts (bf16 cache).
        dict(name="keys_prefill", op="keys", batch=13, lo=512, hi=8190, new=8190, fp8=False),
        # Scores: a shard's heads on a few requests, and all heads on long ones.
        dict(name="score_shard", op="score", batch=5, q_len=1, heads=16, lo=700, hi=9000),
        dict(name="score_long", op="score", batch=32, q_len=2, heads=128, lo=4000, hi=65536),
        # Selection and sparse attention: 16 pages of the bf16 cache for a shard's heads ...
        dict(name="sparse_shard", op="sparse", batch=8, q_len=1, heads=16, lo=900, hi=16384,
             top_k=16, first=1, last=1, fp8=False),
        # ... and 33 pages of the 8-bit cache for each of two draft tokens of long requests.
        dict(name="sparse_long", op="sparse", batch=40, q_len=2, heads=128, lo=3, hi=32768,
             top_k=33, first=1, last=2, fp8=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "append", "keys", "score", "sparse"])
    hi = log(80, 16384)
    lo = max(17, log(17, hi))
    c = dict(op=op, lo=min(lo, hi), hi=hi)
    heads, q_len = 16 * rng.randint(1, 8), rng.choice([1, 1, 2, 3, 4, 8])
    if op == "attend":
        most = max(2, min(128, int(5.5e8 / (heads * q_len * hi) / 2)))
        c.update(batch=log(1, most), q_len=q_len, heads=heads)
    elif op == "append":
        c.update(batch=log(1, max(2, min(200, 90000 // hi))), new=rng.choice([1, 1, 5, hi]))
    elif op == "keys":
        c.update(batch=log(1, max(2, min(200, 90000 // hi))), new=rng.choice([1, 1, 7, hi]),
                 fp8=rng.random() < 0.5)
    elif op == "score":
        c.update(batch=log(1, 32), q_len=min(q_len, 2), heads=heads)
    else:
        top_k = log(4, 33)
        c.update(batch=log(1, 40), q_len=min(q_len, 2), heads=heads, top_k=top_k,
                 first=rng.randint(0, 1), last=rng.randint(1, 2), fp8=rng.random() < 0.5)
    return c


def _lens(case):
    """Lengths from lo to hi, evenly spread over their logarithm: the same for every seed
    (which seed gives which request its length differs)."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    if b == 1:
        return [hi]
    return [int(round(math.exp(math.log(lo) + i * (math.log(hi) - math.log(lo)) / (b - 1))))
            for i in range(b)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, its exponent kept within bounds."""
    f, k = torch.frexp(amax)
    e = k - 9 + (f > 0.875).to(k.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return torch.ldexp(torch.ones_like(amax), e)


def _codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = torch.Generator()
    c.manual_seed(seed)
    op, B = case["op"], case["batch"]
    T, H = case.get("q_len", 1), case.get("heads", 16)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    lens = torch.tensor(_lens(case), dtype=torch.int64)[torch.randperm(B, generator=c)]
    lens = lens.clamp(min=T)
    per = [_pages(n) for n in lens.tolist()]
    used, mp = sum(per), _pages(max(case["hi"], T))
    perm = torch.randperm(used, generator=c).to(torch.int32)
    table = torch.full((B, mp), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    s = dict(op=op, table=table.to(dev), lens=lens.to(torch.int32).to(dev),
             B=B, T=T, H=H, scale=SCALE)

    fp8 = case.get("fp8", True)
    if op != "score":
        if fp8:  # a cache in use: standard normal rows, quantised page by page
            kv8 = torch.empty(used, PAGE, ROW, dtype=torch.uint8, device=dev)
            kvs = torch.empty(used, dtype=torch.float32, device=dev)
            for i in range(0, used, 4096):
                n = min(4096, used - i)
                x = torch.randn(n, PAGE, ROW, generator=g, device=dev)
                x = x.to(torch.bfloat16).float()
                kvs[i:i + n] = _scale_of(x.abs().amax(dim=(1, 2)))
                kv8[i:i + n] = _codes(x / kvs[i:i + n, None, None])
            s.update(kv8=kv8, kvs=kvs)
        else:
            s["cache"] = randn(used, PAGE, ROW)
    if op in ("attend", "score", "sparse"):
        s["q"] = randn(B, T, H, ROW if op == "score" else NOPE + ROPE)
    if op in ("attend", "sparse"):
        s["w_uk"] = randn(H, NOPE, LORA, std=1.0 / math.sqrt(NOPE))
        s["w_uv"] = randn(H, LORA, VHEAD, std=1.0 / math.sqrt(LORA))
        s["out"] = torch.empty(B, T, H, VHEAD, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(B, T, H, dtype=torch.float32, device=dev)
    if op in ("append", "keys"):
        new = case["new"]
        s["new"] = lens.clamp(max=new).to(torch.int32).to(dev)
        s["max_new"] = new
    if op == "append":
        # Activations have a few large channels, and tokens of different sizes.
        x = torch.randn(B, new, ROW, generator=g, device=dev)
        x *= torch.exp(0.5 * torch.randn(B, new, 1, generator=g, device=dev))
        x[..., ::97] *= 6.0
        s["rows"] = x.to(torch.bfloat16)
    if op in ("keys", "score"):
        s["keys"] = randn(used, ROW, std=0.125)
    if op == "score":
        s["scores"] = torch.empty(B, T, mp, dtype=torch.float32, device=dev)
    if op == "sparse":
        # Scores of a cheap 16-bit product: equal ones occur.
        s["scores"] = randn(B, T, mp, std=4.0).float()
        s.update(top_k=case["top_k"], first=case["first"], last=case["last"])
        s["sel_table"] = torch.empty(B * T, case["top_k"], dtype=torch.int32, device=dev)
        s["sel_pages"] = torch.empty_like(s["sel_table"])
        s["sel_lens"] = torch.empty(B * T, dtype=torch.int32, device=dev)
    if own:
        from mla_decode_attention_uk_gb300 import binding
        d = binding.Dims(B, T, H, NOPE, ROPE, LORA, VHEAD, PAGE, used, mp)
        s["dims"] = d
        if op == "attend":
            s["handle"] = binding.MlaDecode(d, dev, fp8_kv=True)
        elif op == "sparse":
            ds = binding.Dims(B * T, 1, H, NOPE, ROPE, LORA, VHEAD, PAGE, used, case["top_k"])
            s["handle"] = binding.MlaDecode(ds, dev, fp8_kv=fp8)
    return s


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from mla_decode_attention_uk_gb300 import binding
    op = s["op"]
    if op == "attend":
        m = s["handle"]
        m.plan(s["lens"])
        m.run_fp8kv(s["q"], s["kv8"], s["kvs"], s["table"], s["lens"], s["w_uk"], s["w_uv"],
                    s["scale"], s["out"], s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    if op == "append":
        binding.append_fp8kv(s["dims"], s["rows"], s["kv8"], s["kvs"], s["table"], s["lens"],
                             new_lens=s["new"])
        return dict(values=s["kv8"].view(torch.float8_e4m3fn), scale=s["kvs"])
    if op == "keys":
        if "kv8" in s:
            binding.page_keys_fp8kv(s["dims"], s["kv8"], s["kvs"], s["table"], s["lens"],
                                    s["max_new"], s["keys"], new_lens=s["new"])
        else:
            binding.page_keys(s["dims"], s["cache"], s["table"], s["lens"], s["max_new"],
                              s["keys"], new_lens=s["new"])
        return dict(keys=s["keys"])
    if op == "score":
        binding.score_pages(s["dims"], s["q"], s["keys"], s["table"], s["lens"], s["scores"])
        return dict(scores=s["scores"])
    binding.select_pages(s["dims"], s["scores"], s["table"], s["lens"], s["top_k"], s["first"],
                         s["last"], s["sel_table"], s["sel_lens"], sel_pages=s["sel_pages"])
    m = s["handle"]
    m.plan(s["sel_lens"])
    args = (s["sel_table"], s["sel_lens"], s["w_uk"], s["w_uv"], s["scale"], s["out"], s["lse"])
    if "kv8" in s:
        m.run_fp8kv(s["q"], s["kv8"], s["kvs"], *args)
    else:
        m.run(s["q"], s["cache"], *args)
    return dict(out=s["out"], lse=s["lse"], pages=s["sel_pages"], lens=s["sel_lens"])


# ---------------------------------------------------------------- plain forms
def _gather(s, table):
    """The cached rows of each line of a page table, in 32 bits: [lines, pages * 64, 576]."""
    t = table.clamp(min=0).long()
    if "kv8" in s:
        x = s["kv8"][t].view(torch.float8_e4m3fn).float() * s["kvs"][t][..., None, None]
    else:
        x = s["cache"][t].float()
    return x.view(t.shape[0], -1, ROW)


def _plain_attention(s, q, rows, visible):
    """q [N, T, H, 192], rows [N, L, 576], visible [N, T] keys of each query."""
    lat = torch.einsum("nthk,hkc->nthc", q[..., :NOPE].float(), s["w_uk"].float())
    lat = torch.cat([lat, q[..., NOPE:].float()], dim=-1)
    N, T, H, _ = lat.shape
    x = torch.matmul(lat.view(N, T * H, ROW), rows.transpose(1, 2)).view(N, T, H, -1)
    x = x * s["scale"]
    hidden = torch.arange(rows.shape[1], device=x.device)[None, None, :] >= visible[..., None]
    x = x.masked_fill(hidden[:, :, None, :], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(N, T * H, -1), rows[..., :LORA]).view(N, T, H, LORA) / total
    out = torch.einsum("nthc,hcv->nthv", o, s["w_uv"].float())
    return out.to(torch.bfloat16), (top + torch.log(total)).squeeze(-1)


def _visible(s):
    """Keys that query t of each sequence sees: [B, T]."""
    t = torch.arange(s["T"], device=s["lens"].device)
    return s["lens"].long()[:, None] - s["T"] + t[None, :] + 1


def _touched(s):
    """The pages that hold each sequence's newest tokens: logical numbers, physical
    numbers and whether there is one, [B, most]."""
    length, first = s["lens"].long(), (s["lens"] - s["new"]).long()
    most = min((s["max_new"] + PAGE - 2) // PAGE + 1, s["table"].shape[1])
    logical = (first // PAGE)[:, None] + torch.arange(most, device=length.device)[None, :]
    there = (logical * PAGE < length[:, None]) & (s["new"] > 0)[:, None]
    physical = torch.gather(s["table"].long(), 1, logical.clamp(max=s["table"].shape[1] - 1))
    return length, first, logical, physical, there


def _plain_append(s):
    length, first, logical, physical, there = _touched(s)
    b, j = torch.nonzero(there, as_tuple=True)
    page, logical = physical[b, j], logical[b, j]
    pos = logical[:, None] * PAGE + torch.arange(PAGE, device=page.device)[None, :]
    is_new = (pos >= first[b][:, None]) & (pos < length[b][:, None])
    fresh = first[b] <= logical * PAGE
    at = (pos - first[b][:, None]).clamp(0, s["rows"].shape[1] - 1)
    new = s["rows"][b[:, None], at].float().masked_fill(~is_new[..., None], 0.0)
    old = s["kv8"][page].view(torch.float8_e4m3fn).float() * s["kvs"][page][:, None, None]
    old = old.masked_fill(fresh[:, None, None], 0.0)
    scale = _scale_of(new.abs().amax(dim=(1, 2)))
    scale = torch.where(fresh, scale, torch.maximum(scale, s["kvs"][page]))
    x = torch.where(is_new[..., None], new, old) / scale[:, None, None]
    s["kv8"][page] = _codes(x)
    s["kvs"][page] = scale
    return dict(values=s["kv8"].view(torch.float8_e4m3fn), scale=s["kvs"])


def _plain_keys(s):
    length, _, logical, physical, there = _touched(s)
    b, j = torch.nonzero(there, as_tuple=True)
    page, logical = physical[b, j], logical[b, j]
    rows = _gather(s, page[:, None])
    count = (length[b] - logical * PAGE).clamp(max=PAGE)
    gone = torch.arange(PAGE, device=page.device)[None, :] >= count[:, None]
    mean = rows.masked_fill(gone[..., None], 0.0).sum(dim=1) / count[:, None]
    s["keys"][page] = mean.to(torch.bfloat16)
    return dict(keys=s["keys"])


def _plain_score(s):
    keys = s["keys"][s["table"].clamp(min=0).long()].float()
    B, T, H, _ = s["q"].shape
    x = torch.matmul(s["q"].float().view(B, T * H, ROW), keys.transpose(1, 2))
    x = x.view(B, T, H, -1).amax(dim=2)
    at = torch.arange(x.shape[-1], device=x.device)
    return dict(scores=x.masked_fill(at[None, None, :] * PAGE >= _visible(s)[..., None],
                                     -math.inf))


def _plain_sparse(s):
    B, T, k = s["B"], s["T"], s["top_k"]
    seen = _visible(s).view(B * T)
    count = (seen + PAGE - 1) // PAGE
    x = s["scores"].view(B * T, -1)
    at = torch.arange(x.shape[1], device=x.device)[None, :]
    kept = (at < s["first"]) | (at >= count[:, None] - s["last"])
    x = x.masked_fill(kept, math.inf)
    x = x.masked_fill(at >= count[:, None], -math.inf)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    if order.shape[1] < k:
        order = torch.nn.functional.pad(order, (0, k - order.shape[1]), value=x.shape[1])
    chosen = torch.arange(k, device=x.device)[None, :] < count[:, None]
    pages = order.masked_fill(~chosen, x.shape[1]).sort(dim=1).values
    pages = torch.where(chosen, pages, torch.full_like(pages, -1))
    lens = count.clamp(max=k) * PAGE - (count * PAGE - seen)
    table = s["table"].long().repeat_interleave(T, dim=0)
    table = torch.gather(table, 1, pages.clamp(min=0)).masked_fill(pages < 0, -1)
    q = s["q"].view(B * T, 1, s["H"], NOPE + ROPE)
    out, lse = _plain_attention(s, q, _gather(s, table), lens[:, None])
    return dict(out=out.view(B, T, s["H"], VHEAD), lse=lse.view(B, T, s["H"]),
                pages=pages.to(torch.int32), lens=lens.to(torch.int32))


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "attend":
        out, lse = _plain_attention(state, state["q"], _gather(state, state["table"]),
                                    _visible(state))
        return dict(out=out, lse=lse)
    return dict(append=_plain_append, keys=_plain_keys, score=_plain_score,
                sparse=_plain_sparse)[op](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, B = case["op"], case["batch"]
    T, H = case.get("q_len", 1), case.get("heads", 16)
    lens = [max(n, T) for n in _lens(case)]
    row = ROW if case.get("fp8", True) else 2 * ROW  # bytes of a cached token
    weights = 2 * H * NOPE * LORA * 2
    calls = B * T * H * ((NOPE + ROPE) * 2 + VHEAD * 2 + 4)  # q, out, lse
    bmm = B * T * H * 2 * 2 * NOPE * LORA
    if op == "attend":
        keys = sum(n - T + t + 1 for n in lens for t in range(T)) * H
        return dict(bytes=sum(lens) * row + 8 * sum(map(_pages, lens)) + weights + calls,
                    flops=keys * 2 * (ROW + LORA) + bmm)
    if op in ("append", "keys"):
        new = [min(n, case["new"]) for n in lens]
        pages = sum((n - 1) // PAGE - (n - m) // PAGE + 1 for n, m in zip(lens, new))
        if op == "append":
            return dict(bytes=sum(new) * 3 * ROW + pages * 8, flops=sum(new) * 2 * ROW)
        filled = sum(n - (n - m) // PAGE * PAGE for n, m in zip(lens, new))
        return dict(bytes=filled * row + pages * (2 * ROW + 8), flops=filled * ROW)
    seen = [_pages(n - T + t + 1) for n in lens for t in range(T)]
    held = sum(map(_pages, lens))
    if op == "score":
        return dict(bytes=held * (2 * ROW + 4) + B * T * H * ROW * 2
                    + B * T * _pages(case["hi"]) * 4, flops=sum(seen) * H * 2 * ROW)
    keys = sum(min(p, case["top_k"]) for p in seen) * PAGE
    reads = min(keys, sum(lens))  # a page that two queries select is read once
    return dict(bytes=sum(seen) * 4 + reads * row + weights + calls
                + B * T * case["top_k"] * 8, flops=keys * H * 2 * (ROW + LORA) + bmm)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    f64 = torch.float64
    B, T, H, op = s["B"], s["T"], s["H"], s["op"]
    lens, table = s["lens"].tolist(), s["table"].tolist()

    def page(p):  # the values of physical pages p (a list): [pages, 64, 576]
        p = torch.tensor(p, device="cuda")
        if "kv8" in s:
            x = s["kv8"][p].view(torch.float8_e4m3fn).to(f64)
            return x * s["kvs"][p].to(f64)[:, None, None]
        return s["cache"][p].to(f64)

    def attend(q, rows):  # one query token: q [H, 192], rows [n, 576] that it sees
        lat = torch.bmm(q[:, None, :NOPE].to(f64), s["w_uk"].to(f64))[:, 0]
        x = (lat @ rows[:, :LORA].T + q[:, NOPE:].to(f64) @ rows[:, LORA:].T) * s["scale"]
        lse = torch.logsumexp(x, dim=1)
        o = torch.exp(x - lse[:, None]) @ rows[:, :LORA]
        return torch.bmm(o[:, None], s["w_uv"].to(f64))[:, 0], lse

    if op == "attend":
        out = torch.empty(B, T, H, VHEAD, dtype=f64, device="cuda")
        lse = torch.empty(B, T, H, dtype=f64, device="cuda")
        for b in range(B):
            rows = page(table[b][:_pages(lens[b])]).view(-1, ROW)
            for t in range(T):
                out[b, t], lse[b, t] = attend(s["q"][b, t], rows[:lens[b] - T + t + 1])
        return dict(out=out, lse=lse)
    if op == "append":
        scale = s["kvs"].to(f64).tolist()
        values = s["kv8"].view(torch.float8_e4m3fn).to(f64)
        for b, n in enumerate(s["new"].tolist()):
            i = lens[b] - n
            while i < lens[b]:
                p, stop = table[b][i // PAGE], min(lens[b], (i // PAGE + 1) * PAGE)
                new = s["rows"][b, i - lens[b] + n:stop - lens[b] + n].to(f64)
                top, e = float(new.abs().max()), E_MIN
                while e < E_MAX and 448.0 * 2.0 ** e < top:
                    e += 1
                if i % PAGE:
                    was_scale = scale[p]
                    scale[p] = max(was_scale, 2.0 ** e)
                    held = values[p] * (was_scale / scale[p])
                else:
                    scale[p], held = 2.0 ** e, torch.zeros_like(values[p])
                held[i % PAGE:i % PAGE + stop - i] = new / scale[p]
                values[p] = _nearest_e4m3(held)
                i = stop
        return dict(values=values, scale=torch.tensor(scale, dtype=f64, device="cuda"))
    if op == "keys":
        keys = s["keys"].to(f64)
        for b, n in enumerate(s["new"].tolist()):
            for j in range((lens[b] - n) // PAGE, _pages(lens[b]) if n else 0):
                rows = page([table[b][j]])[0]
                keys[table[b][j]] = rows[:lens[b] - j * PAGE].mean(dim=0)
        return dict(keys=keys)
    if op == "score":
        scores = torch.full(s["scores"].shape, -math.inf, dtype=f64, device="cuda")
        for b in range(B):
            k = s["keys"][torch.tensor(table[b][:_pages(lens[b])], device="cuda").long()].to(f64)
            for t in range(T):
                n = _pages(lens[b] - T + t + 1)
                scores[b, t, :n] = (s["q"][b, t].to(f64) @ k[:n].T).max(dim=0).values
        return dict(scores=scores)
    out = torch.empty(B, T, H, VHEAD, dtype=f64, device="cuda")
    lse = torch.empty(B, T, H, dtype=f64, device="cuda")
    pages = torch.full((B * T, s["top_k"]), -1, dtype=torch.int32)
    new_lens = torch.empty(B * T, dtype=torch.int32)
    scores = s["scores"].cpu()
    for b in range(B):
        for t in range(T):
            seen = lens[b] - T + t + 1
            n, k = _pages(seen), s["top_k"]
            forced = {j for j in range(n) if j < s["first"] or j >= n - s["last"]}
            line = scores[b, t].tolist()
            rest = sorted((j for j in range(n) if j not in forced), key=lambda j: (-line[j], j))
            mine = sorted(list(forced) + rest[:max(0, k - len(forced))]) if n > k \
                else list(range(n))
            pages[b * T + t, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            rows = page([table[b][j] for j in mine]).view(-1, ROW)
            rows = rows[:rows.shape[0] - (n * PAGE - seen)]
            new_lens[b * T + t] = rows.shape[0]
            out[b, t], lse[b, t] = attend(s["q"][b, t], rows)
    return dict(out=out, lse=lse, pages=pages, lens=new_lens)


def _nearest_e4m3(x):
    """x rounded to the nearest value with four significant bits (ties to even), steps of
    2^-9 below 2^-6, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)
