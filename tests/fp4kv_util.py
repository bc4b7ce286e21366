"""Plain forms of the 4-bit cache's operators for the tests, written from their
definitions (no code of the library)."""
import math

import torch

import fp8kv_util as ref8

PAGE, ROW, ROW4 = 64, 576, 336
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                    dtype=torch.float64)


def _nibbles(w):
    return torch.stack([w % 16, w // 16], dim=-1).flatten(-2).long()


def decode(w):
    """fp64 values of rows [.., 336], in units of their page's scale."""
    e = _nibbles(w[..., 256:272])
    f = torch.where(e == 15, math.nan, torch.exp2(e.double() - 8))
    lat = E2M1[_nibbles(w[..., :256])] * f.repeat_interleave(16, dim=-1)
    return torch.cat([lat, ref8.values(w[..., 272:].contiguous())], dim=-1)


def encode(x):
    """Rows [.., 336] from fp64 values in units of their page's scale."""
    shape = x.shape[:-1]
    lat = x[..., :512].reshape(-1, 32, 16)
    bad = lat.isnan().any(dim=-1)
    lat = lat.nan_to_num(0.0, math.inf, -math.inf).clamp(-448.0, 448.0)
    top = lat.abs().amax(dim=-1)
    e = sum((top > 7.0 * 2.0 ** (k - 8)).long() for k in range(14))
    a = lat.abs() / torch.exp2(e.double() - 8)[..., None]
    # The nearest size, the even code of two that are as near.
    away = (a[..., None] - E2M1[:8]).abs()
    near = away == away.amin(dim=-1, keepdim=True)
    code = torch.full(a.shape, -1, dtype=torch.long)
    for k in (1, 3, 5, 7, 0, 2, 4, 6):
        code[near[..., k]] = k
    code = code + 8 * torch.signbit(lat)
    code[bad] = 0
    e[bad] = 15
    code, e = code.reshape(-1, 512), e.reshape(-1, 32)
    return torch.cat([code[:, ::2] + 16 * code[:, 1::2], e[:, ::2] + 16 * e[:, 1::2],
                      ref8.e4m3(x[..., 512:].reshape(-1, 64)).long()],
                     dim=1).to(torch.uint8).reshape(*shape, ROW4)


def quantise(cache):
    """A whole bf16 cache [pages, 64, 576] -> (rows, scales)."""
    s = torch.tensor([ref8.scale_for(float(p.double().abs().max())) for p in cache],
                     dtype=torch.float64)
    return encode(cache.double() / s[:, None, None]), s.float()


def expand(kv4):
    """The same values as codes of the 8-bit cache."""
    return ref8.e4m3(decode(kv4))


def append(rows, new_lens, block_table, seq_lens, kv4, kv_scale):
    """Reference of the append; returns new (rows, scales)."""
    kv4, kv_scale = kv4.clone(), kv_scale.clone()
    for b, n in enumerate(new_lens):
        L = seq_lens[b]
        for j in range((L - n) // PAGE, (L + PAGE - 1) // PAGE if n else 0):
            p = int(block_table[b, j])
            first, stop = max(L - n, j * PAGE), min(L, (j + 1) * PAGE)
            new = rows[b, first - (L - n):stop - (L - n)].double()
            finite = new[new.isfinite()]
            s = ref8.scale_for(float(finite.abs().max()) if finite.numel() else 0.0)
            if first > j * PAGE:
                s_old = float(kv_scale[p])
                if not 2.0 ** -32 <= s_old <= 2.0 ** 32:
                    s_old = 1.0
                s = max(s, 2.0 ** math.ceil(math.log2(s_old)))
                if s != s_old:
                    kv4[p] = encode(decode(kv4[p]) * (s_old / s))
            else:
                kv4[p] = 0
            kv4[p, first - j * PAGE:stop - j * PAGE] = encode(new / s)
            kv_scale[p] = s
    return kv4, kv_scale


def same(a, b):
    """Rows that are equal, but for which of E4M3's two NaN codes a RoPE value has."""
    ra, rb = a[..., 272:], b[..., 272:]
    nan = (ra & 0x7F) == 0x7F
    return (torch.equal(a[..., :272], b[..., :272]) and torch.equal(nan, (rb & 0x7F) == 0x7F)
            and torch.equal(ra[~nan], rb[~nan]))
