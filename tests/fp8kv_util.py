"""Plain forms of the 8-bit cache's and the sparse decode's operators for the
tests, written from their definitions (no code of the library)."""
import math

import torch

PAGE, ROW = 64, 576


def scale_for(amax):
    """Smallest power of two s with amax <= 448 s, in [2^-32, 2^32]."""
    e = -32
    while e < 32 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def e4m3(x):
    """Codes of fp64 values: four significant bits, ties to even, saturated."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    y = (torch.round(x.nan_to_num(0.0, math.inf, -math.inf) / step.nan_to_num(1.0, 1.0, 1.0))
         * step.nan_to_num(1.0, 1.0, 1.0)).clamp(-448.0, 448.0)
    y = torch.where(x.isnan(), x, y)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def quantise(cache):
    """A whole bf16 cache [pages, 64, 576] -> (codes, scales)."""
    s = torch.tensor([scale_for(float(p.double().abs().max())) for p in cache],
                     dtype=torch.float64)
    return e4m3(cache.double() / s[:, None, None]), s.float()


def append(rows, new_lens, block_table, seq_lens, kv8, kv_scale):
    """Reference of the append; returns new (codes, scales)."""
    kv8, kv_scale = kv8.clone(), kv_scale.clone()
    for b, n in enumerate(new_lens):
        L = seq_lens[b]
        for j in range((L - n) // PAGE, (L + PAGE - 1) // PAGE if n else 0):
            p = int(block_table[b, j])
            first = max(L - n, j * PAGE)
            stop = min(L, (j + 1) * PAGE)
            new = rows[b, first - (L - n):stop - (L - n)].double()
            finite = new[new.isfinite()]
            s = scale_for(float(finite.abs().max()) if finite.numel() else 0.0)
            if first > j * PAGE:
                s_old = float(kv_scale[p])
                if not 2.0 ** -32 <= s_old <= 2.0 ** 32:
                    s_old = 1.0
                s = max(s, 2.0 ** math.ceil(math.log2(s_old)))
                if s != s_old:
                    kv8[p] = e4m3(values(kv8[p]) * (s_old / s))
            else:
                kv8[p] = 0
            kv8[p, first - j * PAGE:stop - j * PAGE] = e4m3(new / s)
            kv_scale[p] = s
    return kv8, kv_scale


def select(scores, block_table, seq_lens, T, top_k, first, last):
    """Reference of the selection: (table, pages, lens)."""
    B = scores.shape[0]
    table = torch.full((B * T, top_k), -1, dtype=torch.int32)
    pages = torch.full((B * T, top_k), -1, dtype=torch.int32)
    lens = torch.zeros(B * T, dtype=torch.int32)
    for b in range(B):
        for t in range(T):
            keys = seq_lens[b] - T + t + 1
            n = (keys + PAGE - 1) // PAGE
            line = [float(x) for x in scores[b, t, :n]]
            line = [(-math.inf, 0) if math.isnan(x) else (x, 1) for x in line]
            if n <= top_k:
                mine = list(range(n))
            else:
                mine = [j for j in range(n) if j < first or j >= n - last]
                rest = [j for j in range(first, n - last)]
                rest.sort(key=lambda j: (-line[j][0], -line[j][1], j))
                mine = sorted(mine + rest[:top_k - first - last])
            i = b * T + t
            pages[i, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            table[i, :len(mine)] = block_table[b][torch.tensor(mine)]
            lens[i] = keys - (n - len(mine)) * PAGE
    return table, pages, lens


# The bounds of the bf16 cache's parity tests (max |d out| 2e-2, mean 2e-3, max
# |d lse| 1e-3) hold weights rounded to bf16, an error e_j of at most 2^-8 of
# each.  Over the 8-bit cache it is at most 2^-7 (two 3-bit terms: the first
# leaves 2^-3 of the weight's power of two, the second 2^-4 of that).  With o_j
# the output that key j alone would give, errors e_j move an output by
#   |sum_j p_j e_j (o_j - o)| <= max |e_j| sum_j p_j |o_j - o|,
# and sum_j p_j |o_j - o| is largest when two keys share the weight: half their
# distance.  Latents are standard normal and the columns of W_UV have norm 1, so
# o_j is standard normal, and over a test's few million pairs two of them are
# less than 6 sqrt(2) = 8.5 apart.  The second 2^-8 adds up to 2^-8 * 8.5 / 2.
OUT_MAX = 2e-2 + 2.0 ** -8 * 8.5 / 2
OUT_MEAN, LSE_MAX = 2e-3, 1e-3


def assert_parity(s, what=""):
    assert math.isfinite(s["out_max"]) and math.isfinite(s["lse_max"]), (what, s)
    assert s["out_max"] <= OUT_MAX and s["out_mean"] <= OUT_MEAN, (what, s)
    assert s["lse_max"] <= LSE_MAX, (what, s)
