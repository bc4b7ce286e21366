"""The operators around the 4-bit latent cache, as measured.

Five operators that belong together: the norms and the rotation in front of the
cache (prep), quantising new tokens into the paged 4-bit cache (append), decode
attention over it (attend), its pages' mean keys (keys), and reading a cache back
as bf16 rows (gather).

A row of the 4-bit cache holds 512 latent values as E2M1 codes (two to a byte, the
first in the low half), an exponent of four bits for each 16 of them, and 64 RoPE
values as E4M3 codes; a page of 64 rows has one scale.

The plain form (own = False) is elementary torch in 32 bits; with own = True
the same calls go through the framework's public binding.
"""
import math

import torch

own = False

NOPE, ROPE, LORA, VHEAD, PAGE = 128, 64, 512, 128, 64
ROW, QROW = LORA + ROPE, NOPE + ROPE  # values of a cached token, of a query
BLOCK = 16                            # latent values with an exponent of their own
ROW4 = LORA // 2 + LORA // BLOCK // 2 + ROPE  # bytes of a token in the 4-bit cache: 336
SCALE = 1.0 / math.sqrt(QROW)
E_MIN, E_MAX = -32, 32  # exponents that a page's scale may have
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # Attention over the 4-bit cache.  Two short requests on a 16-head
        # shard: a call whose time is launch latency.
        dict(name="attend_tiny", op="attend", batch=2, q_len=1, heads=16, lo=17, hi=80),
        # One shard of a model split over eight GPUs: bound by the cache's bytes.
        dict(name="attend_tp_shard", op="attend", batch=64, q_len=1, heads=16, lo=4096, hi=4096),
        # All 128 heads on one GPU, speculative drafts of four tokens for requests of
        # very different lengths, one of four tokens only.
        dict(name="attend_drafts", op="attend", batch=61, q_len=4, heads=128, lo=4, hi=12001),
        # Appending: one new token for each request of a decode batch.
        dict(name="append_decode", op="append", batch=128, lo=64, hi=2000, new=1),
        # Prompts of different lengths written into fresh pages.
        dict(name="append_prefill", op="append", batch=13, lo=512, hi=8190, new=8190),
        # Mean keys: the last page of each request after a decode step ...
        dict(name="keys_decode", op="keys", batch=128, lo=64, hi=2000, new=1),
        # ... and every page of fresh prompts.
        dict(name="keys_prefill", op="keys", batch=13, lo=512, hi=8190, new=8190),
        # Reading back: a few short prefixes from the 8-bit cache, for a chunk of a
        # prompt that attends to them ...
        dict(name="gather_short", op="gather", batch=3, lo=100, hi=1000, new=1000, cache="fp8"),
        # ... and long ones from the 4-bit cache.
        dict(name="gather_long", op="gather", batch=13, lo=512, hi=8190, new=8190, cache="fp4"),
        # Norms and rotation: one token of two requests, latents into the bf16 cache;
        prep_case("prep_tiny", batch=2, heads=16, lo=17, hi=80, new=1, out="cache"),
        # a decode step of all heads, queries with norms of their own;
        prep_case("prep_full_head", batch=128, heads=128, lo=64, hi=2000, new=1, q_norm=True,
                  out="cache"),
        # prompts of different lengths on a shard's heads, latents cut from a wider
        # projection, into rows for an append.
        prep_case("prep_prefill", batch=7, heads=16, lo=512, hi=8190, new=8190, wide=1024,
                  interleaved=False, out="rows"),
    ]


def prep_case(name, batch, heads, lo, hi, new, out, q_norm=False, wide=0, interleaved=True):
    c = dict(op="prep", batch=batch, heads=heads, lo=lo, hi=hi, new=new, out=out, q_norm=q_norm,
             wide=wide, interleaved=interleaved)
    return dict(c, name=name) if name else c


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "append", "keys", "gather", "prep"])
    hi = log(80, 16384)
    lo = max(17, log(17, hi))
    c = dict(op=op, lo=min(lo, hi), hi=hi)
    heads = 16 * rng.randint(1, 8)
    if op == "attend":
        q_len = rng.choice([1, 1, 2, 3, 4, 8])
        most = max(2, min(128, int(6e7 / (heads * q_len * hi))))
        c.update(batch=log(1, most), q_len=q_len, heads=heads)
        return c
    batch = log(1, max(2, min(200, 36000 // hi)))
    new = rng.choice([1, 1, 5, hi])
    if op == "prep":
        new = min(new, 250000 // heads)
        return prep_case(None, min(batch, max(1, 250000 // (heads * new))), heads, c["lo"], hi, new,
                         rng.choice(["cache", "rows"]), rng.random() < 0.5,
                         rng.choice([0, 8, 1024]), rng.random() < 0.5)
    c.update(batch=batch, new=new)
    if op == "gather":
        c.update(cache=rng.choice(["bf16", "fp8", "fp4"]))
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


# ---------------------------------------------------------------- the formats
def _pow2(e):
    return torch.ldexp(torch.ones(e.shape, device=e.device), e)


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, its exponent kept within bounds."""
    f, k = torch.frexp(amax)
    e = k - 9 + (f > 0.875).to(k.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return _pow2(e)


def _codes8(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _rows4(x):
    """Rows of the 4-bit cache from values in units of their pages' scales: uint8 [.., 336].
    A block's exponent is the smallest j from -8 to 6 with all its values within 7 * 2^j;
    values are rounded to the nearest code, ties to the even one, 6 and up to 6."""
    lat = x[..., :LORA].clamp(-448.0, 448.0).unflatten(-1, (LORA // BLOCK, BLOCK))
    f, k = torch.frexp(lat.abs().amax(dim=-1))
    e = (k - 3 + (f > 0.875).to(k.dtype)).masked_fill(f == 0, -8).clamp(-8, 6)
    a = (lat.abs() / _pow2(e)[..., None]).flatten(-2)
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    code += 8 * torch.signbit(lat).flatten(-2).byte()
    e = (e + 8).to(torch.uint8)
    return torch.cat([code[..., ::2] | (code[..., 1::2] << 4), e[..., ::2] | (e[..., 1::2] << 4),
                      _codes8(x[..., LORA:])], dim=-1)


def _halves(w):
    return torch.stack([w & 15, w >> 4], dim=-1).flatten(-2)


def _values4(w):
    """The values that rows of the 4-bit cache stand for, in units of their pages' scales."""
    n = _halves(w[..., :LORA // 2]).int()
    e = _halves(w[..., LORA // 2:LORA // 2 + LORA // BLOCK // 2]).int() - 8
    # E2M1: a sign, two bits of exponent, one of mantissa (0, 0.5, 1, 1.5, 2, 3, 4, 6).
    x = ((n & 1) + 2 * ((n & 7) > 1)).float() * _pow2(((n >> 1) & 3).clamp(min=1) - 2)
    x = x * (1 - (n >> 3) * 2)
    x = (x.unflatten(-1, (LORA // BLOCK, BLOCK)) * _pow2(e)[..., None]).flatten(-2)
    return torch.cat([x, w[..., ROW4 - ROPE:].contiguous().view(torch.float8_e4m3fn).float()],
                     dim=-1)


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

    def activations(n, width):  # a few large channels, and tokens of different sizes
        x = torch.randn(B, n, width, generator=g, device=dev)
        x *= torch.exp(0.5 * torch.randn(B, n, 1, generator=g, device=dev))
        x[..., ::97] *= 6.0
        return x.to(torch.bfloat16)

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

    kind = case.get("cache", "fp4")
    if op == "prep":
        kind = "bf16" if case["out"] == "cache" else None
    if kind == "bf16":
        s["cache"] = randn(used, PAGE, ROW)
    elif kind:  # a cache in use: standard normal rows, quantised page by page
        name, width = ("kv4", ROW4) if kind == "fp4" else ("kv8", ROW)
        kv = torch.empty(used, PAGE, width, dtype=torch.uint8, device=dev)
        kvs = torch.empty(used, dtype=torch.float32, device=dev)
        for i in range(0, used, 2048):
            n = min(2048, used - i)
            x = torch.randn(n, PAGE, ROW, generator=g, device=dev)
            x = x.to(torch.bfloat16).float()
            kvs[i:i + n] = _scale_of(x.abs().amax(dim=(1, 2)))
            x /= kvs[i:i + n, None, None]
            kv[i:i + n] = _rows4(x) if kind == "fp4" else _codes8(x)
        s.update({name: kv, "kvs": kvs})
    if op == "attend":
        s["q"] = randn(B, T, H, QROW)
        s["w_uk"] = randn(H, NOPE, LORA, std=1.0 / math.sqrt(NOPE))
        s["w_uv"] = randn(H, LORA, VHEAD, std=1.0 / math.sqrt(LORA))
        s["out"] = torch.empty(B, T, H, VHEAD, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(B, T, H, dtype=torch.float32, device=dev)
    else:
        new = case["new"]
        s["new"] = lens.clamp(max=new).to(torch.int32).to(dev)
        s["max_new"] = new
    if op == "append":
        s["rows"] = activations(new, ROW)
    if op == "keys":
        s["keys"] = randn(used, ROW, std=0.125)
    if op == "gather" or (op == "prep" and case["out"] == "rows"):
        s["rows"] = torch.zeros(B, new, ROW, dtype=torch.bfloat16, device=dev)
    if op == "prep":
        s["q"] = randn(B, new, H, QROW)
        s["q_out"] = torch.zeros_like(s["q"])
        # The latents as columns of a projection's output, at its right end.
        s["kv"] = activations(new, case["wide"] + ROW)[..., case["wide"]:]
        s["kv_weight"] = (1.0 + 0.2 * randn(LORA).float()).to(torch.bfloat16)
        s["q_weight"] = (1.0 + 0.2 * randn(QROW).float()).to(torch.bfloat16) \
            if case["q_norm"] else None
        s["interleaved"] = case["interleaved"]
        # cos and sin of every position's angles, made in 64 bits.
        most = mp * PAGE
        freq = 10000.0 ** (-torch.arange(0, ROPE, 2, device=dev, dtype=torch.float64) / ROPE)
        angle = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    if own:
        from mla_decode_attention_uk_gb300 import binding
        d = binding.Dims(B, T, H, NOPE, ROPE, LORA, VHEAD, PAGE, used, mp)
        s["dims"] = d
        if op == "attend":
            s["handle"] = binding.MlaDecode(d, dev, fp8_kv=True)
    return s


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from mla_decode_attention_uk_gb300 import binding
    op = s["op"]
    if op == "attend":
        m = s["handle"]
        m.plan(s["lens"])
        m.run_fp4kv(s["q"], s["kv4"], s["kvs"], s["table"], s["lens"], s["w_uk"], s["w_uv"],
                    s["scale"], s["out"], s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    if op == "append":
        binding.append_fp4kv(s["dims"], s["rows"], s["kv4"], s["kvs"], s["table"], s["lens"],
                             new_lens=s["new"])
        return _parts4(s)
    if op == "keys":
        binding.page_keys_fp4kv(s["dims"], s["kv4"], s["kvs"], s["table"], s["lens"],
                                s["max_new"], s["keys"], new_lens=s["new"])
        return dict(keys=s["keys"])
    if op == "gather":
        if "cache" in s:
            binding.gather(s["dims"], s["cache"], s["table"], s["lens"], s["rows"],
                           new_lens=s["new"])
        elif "kv8" in s:
            binding.gather_fp8kv(s["dims"], s["kv8"], s["kvs"], s["table"], s["lens"], s["rows"],
                                 new_lens=s["new"])
        else:
            binding.gather_fp4kv(s["dims"], s["kv4"], s["kvs"], s["table"], s["lens"], s["rows"],
                                 new_lens=s["new"])
        return dict(rows=s["rows"])
    cached = "cache" in s
    binding.norm_rope(s["dims"], s["lens"], s["cos_sin"], q=s["q"], q_out=s["q_out"],
                      q_weight=s["q_weight"], kv=s["kv"], kv_weight=s["kv_weight"], eps=EPS,
                      rows=None if cached else s["rows"], cache=s["cache"] if cached else None,
                      block_table=s["table"] if cached else None, interleaved=s["interleaved"],
                      new_lens=s["new"])
    return _prepared(s)


def _parts4(s):
    """The 4-bit cache's state: the codes' bytes, which have to be the same (every rounding is
    defined, ties too), the RoPE columns' values and the scales."""
    return dict(codes=s["kv4"][..., :ROW4 - ROPE],
                rope=s["kv4"][..., ROW4 - ROPE:].view(torch.float8_e4m3fn), scale=s["kvs"])


def _prepared(s):
    return dict(q=s["q_out"], latent=s["cache"] if "cache" in s else s["rows"])


# ---------------------------------------------------------------- plain forms
def _read(s, page):
    """The rows of physical pages, in 32 bits: [.., 64, 576]."""
    if "cache" in s:
        return s["cache"][page].float()
    if "kv8" in s:
        x = s["kv8"][page].view(torch.float8_e4m3fn).float()
    else:
        x = _values4(s["kv4"][page])
    return x * s["kvs"][page][..., None, None]


def _plain_attention(s):
    rows = _read(s, s["table"].clamp(min=0).long()).flatten(1, 2)
    q = s["q"]
    lat = torch.einsum("nthk,hkc->nthc", q[..., :NOPE].float(), s["w_uk"].float())
    lat = torch.cat([lat, q[..., NOPE:].float()], dim=-1)
    N, T, H, _ = lat.shape
    x = torch.matmul(lat.view(N, T * H, ROW), rows.transpose(1, 2)).view(N, T, H, -1)
    x = x * s["scale"]
    t = torch.arange(T, device=x.device)
    visible = s["lens"].long()[:, None] - T + t[None, :] + 1
    hidden = torch.arange(rows.shape[1], device=x.device)[None, None, :] >= visible[..., None]
    x = x.masked_fill(hidden[:, :, None, :], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(N, T * H, -1), rows[..., :LORA]).view(N, T, H, LORA) / total
    out = torch.einsum("nthc,hcv->nthv", o, s["w_uv"].float())
    return dict(out=out.to(torch.bfloat16), lse=(top + torch.log(total)).squeeze(-1))


def _touched(s):
    """The pages that hold each sequence's newest tokens, one line each: the sequence, its
    length and the first of those tokens, the page's logical and physical number."""
    length, first = s["lens"].long(), (s["lens"] - s["new"]).long()
    most = min((s["max_new"] + PAGE - 2) // PAGE + 1, s["table"].shape[1])
    logical = (first // PAGE)[:, None] + torch.arange(most, device=length.device)[None, :]
    there = (logical * PAGE < length[:, None]) & (s["new"] > 0)[:, None]
    physical = torch.gather(s["table"].long(), 1, logical.clamp(max=s["table"].shape[1] - 1))
    b, j = torch.nonzero(there, as_tuple=True)
    return b, length[b], first[b], logical[b, j], physical[b, j]


def _plain_append(s):
    b, length, first, logical, page = _touched(s)
    pos = logical[:, None] * PAGE + torch.arange(PAGE, device=page.device)[None, :]
    is_new = (pos >= first[:, None]) & (pos < length[:, None])
    fresh = first <= logical * PAGE
    at = (pos - first[:, None]).clamp(0, s["rows"].shape[1] - 1)
    new = s["rows"][b[:, None], at].float().masked_fill(~is_new[..., None], 0.0)
    old = _read(s, page).masked_fill(fresh[:, None, None], 0.0)
    scale = _scale_of(new.abs().amax(dim=(1, 2)))
    scale = torch.where(fresh, scale, torch.maximum(scale, s["kvs"][page]))
    s["kv4"][page] = _rows4(torch.where(is_new[..., None], new, old) / scale[:, None, None])
    s["kvs"][page] = scale
    return _parts4(s)


def _plain_keys(s):
    _, length, _, logical, page = _touched(s)
    rows = _read(s, page)
    count = (length - logical * PAGE).clamp(max=PAGE)
    gone = torch.arange(PAGE, device=page.device)[None, :] >= count[:, None]
    mean = rows.masked_fill(gone[..., None], 0.0).sum(dim=1) / count[:, None]
    s["keys"][page] = mean.to(torch.bfloat16)
    return dict(keys=s["keys"])


def _newest(s):
    """Which rows of [B, max_new] hold a token, and its position."""
    i = torch.arange(s["max_new"], device=s["lens"].device)[None, :]
    there = i < s["new"][:, None]
    return there, ((s["lens"] - s["new"])[:, None] + i).masked_fill(~there, 0).long()


def _plain_gather(s):
    there, pos = _newest(s)
    page = torch.gather(s["table"].long(), 1, pos // PAGE)[there]
    slot = (pos % PAGE)[there]
    if "cache" in s:
        x = s["cache"][page, slot].float()
    elif "kv8" in s:
        x = s["kv8"][page, slot].view(torch.float8_e4m3fn).float() * s["kvs"][page][:, None]
    else:
        x = _values4(s["kv4"][page, slot]) * s["kvs"][page][:, None]
    s["rows"][there] = x.to(torch.bfloat16)
    return dict(rows=s["rows"])


def _rotate(x, cos, sin, interleaved):
    """x [.., 64] in pairs (2 i, 2 i + 1), or (i, i + 32); cos and sin [.., 32]."""
    a, b = (x[..., ::2], x[..., 1::2]) if interleaved else (x[..., :ROPE // 2],
                                                           x[..., ROPE // 2:])
    pair = a * cos - b * sin, b * cos + a * sin
    return torch.stack(pair, dim=-1).flatten(-2) if interleaved else torch.cat(pair, dim=-1)


def _normed(x, weight):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()


def _plain_prep(s):
    there, pos = _newest(s)
    cos, sin = s["cos_sin"][pos].split(ROPE // 2, dim=-1)
    q = s["q"].float()
    if s["q_weight"] is not None:
        q = _normed(q, s["q_weight"])
    rope = _rotate(q[..., NOPE:], cos[:, :, None], sin[:, :, None], s["interleaved"])
    q = torch.cat([q[..., :NOPE], rope], dim=-1).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(there[..., None, None], q, s["q_out"]))
    kv = s["kv"].float()
    kv = torch.cat([_normed(kv[..., :LORA], s["kv_weight"]),
                    _rotate(kv[..., LORA:], cos, sin, s["interleaved"])], dim=-1)
    kv = kv.to(torch.bfloat16)
    if "cache" in s:
        page = torch.gather(s["table"].long(), 1, pos // PAGE)
        s["cache"][page[there], (pos % PAGE)[there]] = kv[there]
    else:
        s["rows"].copy_(torch.where(there[..., None], kv, s["rows"]))
    return _prepared(s)


def run(state):
    if own:
        return _own(state)
    return dict(attend=_plain_attention, append=_plain_append, keys=_plain_keys,
                gather=_plain_gather, prep=_plain_prep)[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, B = case["op"], case["batch"]
    T, H = case.get("q_len", 1), case.get("heads", 16)
    lens = [max(n, T) for n in _lens(case)]
    if op == "attend":
        weights = 2 * H * NOPE * LORA * 2
        calls = B * T * H * (QROW * 2 + VHEAD * 2 + 4)  # q, out, lse
        bmm = B * T * H * 2 * 2 * NOPE * LORA
        keys = sum(n - T + t + 1 for n in lens for t in range(T)) * H
        return dict(bytes=sum(lens) * ROW4 + 8 * sum(map(_pages, lens)) + weights + calls,
                    flops=keys * 2 * (ROW + LORA) + bmm)
    new = [min(n, case["new"]) for n in lens]
    pages = sum((n - 1) // PAGE - (n - m) // PAGE + 1 for n, m in zip(lens, new))
    if op == "append":
        return dict(bytes=sum(new) * (2 * ROW + ROW4) + pages * 8, flops=sum(new) * 2 * ROW)
    if op == "keys":
        filled = sum(n - (n - m) // PAGE * PAGE for n, m in zip(lens, new))
        return dict(bytes=filled * ROW4 + pages * (2 * ROW + 8), flops=filled * ROW)
    if op == "gather":
        row = dict(bf16=2 * ROW, fp8=ROW, fp4=ROW4)[case["cache"]]
        return dict(bytes=sum(new) * (row + 2 * ROW) + pages * 8, flops=sum(new) * ROW)
    positions = min(sum(new), max(lens))  # a line of cos and sin is read once
    return dict(bytes=sum(new) * (H * QROW + ROW) * 4 + positions * ROPE * 4 + LORA * 2,
                flops=sum(new) * (H * ((QROW * 4 if case["q_norm"] else 0) + ROPE * 3)
                                  + LORA * 4 + ROPE * 3))


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    f64 = torch.float64
    dev = s["lens"].device
    B, T, H, op = s["B"], s["T"], s["H"], s["op"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    e2m1 = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, -0.0, -1, -2, -3, -4, -6, -8, -12], dtype=f64,
                        device=dev) / 2

    def decoded(w):  # rows of the 4-bit cache, in units of their scales
        x = torch.empty(*w.shape[:-1], ROW, dtype=f64, device=dev)
        e = torch.empty(*w.shape[:-1], LORA // BLOCK, dtype=f64, device=dev)
        x[..., 0:LORA:2] = e2m1[(w[..., :256] % 16).long()]
        x[..., 1:LORA:2] = e2m1[(w[..., :256] // 16).long()]
        e[..., 0::2] = (w[..., 256:272] % 16).to(f64)
        e[..., 1::2] = (w[..., 256:272] // 16).to(f64)
        x[..., :LORA] *= (2.0 ** (e - 8)).repeat_interleave(BLOCK, dim=-1)
        x[..., LORA:] = w[..., 272:].contiguous().view(torch.float8_e4m3fn).to(f64)
        return x

    def page(p):  # the values of physical pages p (a list): [pages, 64, 576]
        p = torch.tensor(p, device=dev)
        if "cache" in s:
            return s["cache"][p].to(f64)
        x = s["kv8"][p].view(torch.float8_e4m3fn).to(f64) if "kv8" in s else decoded(s["kv4"][p])
        return x * s["kvs"][p].to(f64)[:, None, None]

    if op == "attend":
        out = torch.empty(B, T, H, VHEAD, dtype=f64, device=dev)
        lse = torch.empty(B, T, H, dtype=f64, device=dev)
        for b in range(B):
            rows = page(table[b][:_pages(lens[b])]).view(-1, ROW)
            for t in range(T):
                c, q = rows[:lens[b] - T + t + 1], s["q"][b, t].to(f64)
                lat = torch.bmm(q[:, None, :NOPE], s["w_uk"].to(f64))[:, 0]
                x = (lat @ c[:, :LORA].T + q[:, NOPE:] @ c[:, LORA:].T) * s["scale"]
                lse[b, t] = torch.logsumexp(x, dim=1)
                o = torch.exp(x - lse[b, t][:, None]) @ c[:, :LORA]
                out[b, t] = torch.bmm(o[:, None], s["w_uv"].to(f64))[:, 0]
        return dict(out=out, lse=lse)
    new = s["new"].tolist()
    if op == "append":
        kv4, kvs = s["kv4"].clone(), s["kvs"].to(f64).tolist()
        for b, n in enumerate(new):
            i = lens[b] - n
            while i < lens[b]:
                p, stop = table[b][i // PAGE], min(lens[b], (i // PAGE + 1) * PAGE)
                rows = s["rows"][b, i - lens[b] + n:stop - lens[b] + n].to(f64)
                top, e = float(rows.abs().max()), E_MIN
                while e < E_MAX and 448.0 * 2.0 ** e < top:
                    e += 1
                at = i % PAGE
                scale = max(kvs[p], 2.0 ** e) if at else 2.0 ** e
                if at and scale != kvs[p]:
                    kv4[p] = _encoded(decoded(kv4[p]) * (kvs[p] / scale))
                elif not at:
                    kv4[p] = 0
                kv4[p, at:at + stop - i] = _encoded(rows / scale)
                kvs[p] = scale
                i = stop
        return dict(codes=kv4[..., :272].clone(),
                    rope=kv4[..., 272:].contiguous().view(torch.float8_e4m3fn).to(f64),
                    scale=torch.tensor(kvs, dtype=f64, device=dev))
    if op == "keys":
        keys = s["keys"].to(f64)
        for b, n in enumerate(new):
            for j in range((lens[b] - n) // PAGE, _pages(lens[b]) if n else 0):
                rows = page([table[b][j]])[0]
                keys[table[b][j]] = rows[:lens[b] - j * PAGE].mean(dim=0)
        return dict(keys=keys)
    if op == "gather":
        rows = s["rows"].to(f64)
        for b, n in enumerate(new):
            rows[b, :n] = page(table[b][:_pages(lens[b])]).view(-1, ROW)[lens[b] - n:lens[b]]
        return dict(rows=rows)
    # Norms and rotation: a pair is a complex number, turned by its position's angle.
    q_out = s["q_out"].to(f64)
    latent = (s["cache"] if "cache" in s else s["rows"]).to(f64)
    table_f64 = s["cos_sin"].to(f64)
    turn = torch.complex(table_f64[:, :ROPE // 2], table_f64[:, ROPE // 2:])

    def turned(x, by):
        if s["interleaved"]:
            z = torch.view_as_complex(x.reshape(*x.shape[:-1], ROPE // 2, 2).contiguous()) * by
            return torch.view_as_real(z).reshape(x.shape)
        z = torch.complex(x[..., :ROPE // 2].contiguous(), x[..., ROPE // 2:].contiguous()) * by
        return torch.cat([z.real, z.imag], dim=-1)

    def normed(x, w):
        return x / torch.sqrt(x.square().sum(dim=-1, keepdim=True) / x.shape[-1] + EPS) * w.to(f64)

    for b, n in enumerate(new):
        at = lens[b] - n
        by = turn[at:lens[b]]
        q = s["q"][b, :n].to(f64)
        if s["q_weight"] is not None:
            q = normed(q, s["q_weight"])
        q_out[b, :n, :, :NOPE] = q[..., :NOPE]
        q_out[b, :n, :, NOPE:] = turned(q[..., NOPE:], by[:, None])
        kv = s["kv"][b, :n].to(f64)
        kv = torch.cat([normed(kv[:, :LORA], s["kv_weight"]), turned(kv[:, LORA:], by)], dim=1)
        if "cache" not in s:
            latent[b, :n] = kv
            continue
        pos = torch.arange(at, lens[b], device=dev)
        latent[s["table"][b].long()[pos // PAGE], pos % PAGE] = kv
    return dict(q=q_out, latent=latent)


def _encoded(x):
    """Rows of the 4-bit cache from values (64 bits) in units of their scales, by search among
    the values that there are."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    lat = x[:, :LORA].clamp(-448, 448).reshape(x.shape[0], LORA // BLOCK, BLOCK)
    top = lat.abs().amax(dim=2)
    e = torch.zeros_like(top)
    for k in range(14):
        e += (top > 7 * 2.0 ** (k - 8)).to(e.dtype)
    away = ((lat.abs() / 2.0 ** (e - 8)[..., None])[..., None] - grid).abs()
    near = away.amin(dim=-1, keepdim=True) == away  # one, or two neighbours
    odd = torch.arange(8, device=x.device) % 2 == 1
    code = (near & ~(odd & (near.sum(dim=-1, keepdim=True) > 1))).to(torch.uint8).argmax(dim=-1)
    code = (code + 8 * torch.signbit(lat)).reshape(x.shape[0], LORA).to(torch.uint8)
    e = e.to(torch.uint8)
    rope = x[:, LORA:]
    step = torch.exp2(torch.floor(torch.log2(rope.abs().clamp(min=2.0 ** -6))) - 3)
    rope = (torch.round(rope / step) * step).clamp(-448.0, 448.0)
    return torch.cat([code[:, 0::2] + 16 * code[:, 1::2], e[:, 0::2] + 16 * e[:, 1::2],
                      rope.to(torch.float8_e4m3fn).view(torch.uint8)], dim=1)
