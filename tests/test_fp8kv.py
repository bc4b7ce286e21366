"""The 8-bit latent cache: append and attention against 64-bit forms.

A cached value (E4M3 code times a power of two) is exact in bf16, so the fp64
oracle of the bf16 cache is the oracle here too, on the dequantised cache."""
import ctypes
import math

import pytest
import torch

import fp8kv_util as ref
from mla_decode_attention_uk_gb300 import binding
from mla_decode_attention_uk_gb300.inputs import make_inputs, quantize_fp8_blockwise

from fp8kv_util import assert_parity
from parity_util import compare

gpu = pytest.mark.gpu
BF = torch.bfloat16


# ---------------------------------------------------------------- refusals (no GPU)
def good_dims(**kw):
    d = dict(batch=2, q_len=1, num_heads=16, qk_nope=128, qk_rope=64, kv_lora=512, v_head=128,
             page_size=64, num_pages=4, max_pages_per_seq=2)
    d.update(kw)
    return binding.Dims(**d)


OK, ODD2, ODD8 = ctypes.c_void_p(4096), ctypes.c_void_p(4098), ctypes.c_void_p(4104)


def call(name, args, change=None, d=None):
    a = list(args)
    for i, v in (change or {}).items():
        a[i] = v
    return getattr(binding.lib(), name)(ctypes.byref(d or good_dims()), *a)


def test_append_refuses_bad_arguments():
    #       rows max_new new_lens table lens kv8 scale status stream
    args = [OK, 1, OK, OK, OK, OK, OK, OK, None]
    for change in ({0: None}, {0: ODD8}, {1: 0}, {1: -1}, {1: 2 ** 31 - 1}, {2: ODD2}, {3: None},
                   {3: ODD2}, {4: None}, {4: ODD2}, {5: None}, {5: ODD8}, {6: None}, {6: ODD2},
                   {7: ODD2}):
        assert call("mla_decode_append_fp8kv", args, change) == 1, change
    assert call("mla_decode_append_fp8kv", args, d=good_dims(kv_lora=256)) == 2
    assert binding.lib().mla_decode_append_fp8kv(None, *args) == 1


def test_run_and_attend_refuse_bad_arguments():
    sc = ctypes.c_float(0.07)
    #      q kv8 kvs table lens wuk wuv scale out lse ws wbytes stream
    run = [OK, OK, OK, OK, OK, OK, OK, sc, OK, OK, OK, 1 << 30, None]
    for change in ({0: None}, {1: None}, {1: ODD8}, {2: None}, {2: ODD2}, {3: ODD2}, {4: None},
                   {5: ODD8}, {6: None}, {8: ODD8}, {9: None}, {10: None}, {10: ODD8},
                   {7: ctypes.c_float(0.0)}, {7: ctypes.c_float(-1.0)},
                   {7: ctypes.c_float(math.nan)}, {7: ctypes.c_float(math.inf)}):
        assert call("mla_decode_run_fp8kv", run, change) == 1, change
    assert call("mla_decode_run_fp8kv", run, {11: 64}) == 3
    assert call("mla_decode_run_fp8kv", run, d=good_dims(q_len=9)) == 2
    #      kv8 kvs table lens scale lse ws wbytes stream
    att = [OK, OK, OK, OK, sc, OK, OK, 1 << 30, None]
    for change in ({0: None}, {0: ODD8}, {1: None}, {1: ODD2}, {2: None}, {3: ODD2}, {5: None},
                   {6: None}, {6: ODD8}, {4: ctypes.c_float(math.nan)}):
        assert call("mla_decode_attend_fp8kv", att, change) == 1, change
    assert call("mla_decode_attend_fp8kv", att, {7: 64}) == 3
    #       lens ranges ws wbytes stream
    plan = [OK, 5, OK, 1 << 30, None]
    for change in ({0: None}, {1: -1}, {1: 65537}, {2: None}, {2: ODD8}):
        assert call("mla_decode_plan_fp8kv", plan, change) == 1, change
    assert call("mla_decode_plan_fp8kv", plan, {3: 64}) == 3
    assert call("mla_decode_plan_fp8kv", plan, d=good_dims(page_size=16)) == 2


def test_python_calls_check_types_and_shapes():
    d = good_dims()
    kv8, kvs = torch.zeros(4, 64, 576, dtype=torch.uint8), torch.ones(4)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    rows = torch.zeros(2, 3, 576, dtype=BF)
    good = dict(rows=rows, kv8=kv8, kv_scale=kvs, block_table=table, seq_lens=lens)
    for k, v in (("rows", rows.float()), ("rows", rows[:1]), ("rows", rows[:, ::2]),
                 ("kv8", kv8.view(torch.int8)), ("kv8", kv8[:3]), ("kv_scale", kvs.double()),
                 ("kv_scale", kvs[:2]), ("block_table", table.long()), ("block_table", table.t()),
                 ("seq_lens", lens[:1])):
        if k == "block_table" and v.is_contiguous():
            continue
        with pytest.raises(ValueError):
            binding.append_fp8kv(d, **dict(good, **{k: v}))
    with pytest.raises(ValueError):
        binding.append_fp8kv(d, **good, new_lens=lens.long())
    with pytest.raises(ValueError):
        binding.append_fp8kv(d, **good, status=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA device"):
        binding.append_fp8kv(d, **good)  # right shapes, but in host memory


# ---------------------------------------------------------------- append
def pool(pages, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randn(pages, 64, 576, generator=g).to(BF)
    return ref.quantise(c)


def tables(lens, seed, width=None, pages=None):
    per = [(n + 63) // 64 for n in lens]
    total = sum(per) if pages is None else pages
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(total, generator=g).to(torch.int32)
    t = torch.full((len(lens), width or max(max(per), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, total


def run_append(rows, new_lens, table, lens, kv8, kvs, pages, pass_new=True):
    d = good_dims(batch=len(lens), num_pages=pages, max_pages_per_seq=table.shape[1])
    k, s = kv8.cuda(), kvs.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.append_fp8kv(d, rows.cuda(), k, s, table.cuda(),
                         torch.tensor(lens, dtype=torch.int32).cuda(),
                         torch.tensor(new_lens, dtype=torch.int32).cuda() if pass_new else None,
                         status)
    return k.cpu(), s.cpu(), int(status.item())


@gpu
@pytest.mark.parametrize("lens,new,max_new", [
    ([1], [1], 1),                                       # the first token of all
    ([64, 65, 63, 128, 129], [1] * 5, 1),                # around a page's end
    ([200, 64, 70, 1, 5], [200, 64, 6, 1, 0], 200),      # prompts, a chunk, nothing
    ([130, 130, 130], [130, 67, 2], 131),                # whole, from inside a page, two rows
    ([0, 17, 0, 300], [0, 17, 0, 3], 40),                # unused lines of the batch
    ([1000, 513], [999, 512], 1000),
    ([128, 100], [128, 33], 128),                        # a table of two pages
    ([32 + 40, 33 + 40, 95], [32, 0, 31], 32),           # the two kernels' border
    ([33 + 40, 20], [33, 20], 33),
    ([1 + i % 70 for i in range(300)], [(1 + i % 70) // 2 for i in range(300)], 35),
])
def test_append_equals_the_definition(lens, new, max_new):
    # The definition is exact (powers of two, one rounding): codes and scales
    # are equal, in pages that the call leaves alone too.
    table, used = tables(lens, 5)
    kv8, kvs = pool(used + 3, 6)
    g = torch.Generator().manual_seed(7)
    rows = torch.randn(len(lens), max_new, 576, generator=g)
    # Tokens of sizes from 2^-6 to 2^6: scales that grow, and rows that are
    # re-coded to subnormals and to zero.
    rows *= torch.exp2(torch.randint(-6, 7, (len(lens), max_new, 1), generator=g).float())
    rows = rows.to(BF)
    k, s, st = run_append(rows, new, table, lens, kv8, kvs, used + 3)
    rk, rs = ref.append(rows, new, table, lens, kv8, kvs)
    assert st == 0
    assert torch.equal(s, rs)
    assert torch.equal(k, rk)


@gpu
@pytest.mark.parametrize("kind", ["long", "many", "the last ones only", "three times"])
def test_append_of_many_pages(kind):
    # More pages than the buffers of all SMs hold, and more sequences than are
    # looked at together; every page once, whatever order they are filled in.
    lens = {"long": [60000, 41, 30123], "many": [1 + 13 * i % 151 for i in range(1100)],
            "the last ones only": [0] * 515 + [70, 0, 9, 64, 4000],
            "three times": [5000, 700, 9000]}[kind]
    new = [n - (i % 3) * (n // 5) if n > 3 else n for i, n in enumerate(lens)]
    table, used = tables(lens, 21)
    g = torch.Generator().manual_seed(22)
    base = torch.randn(max(new), 576, generator=g).to(BF)
    rows = torch.stack([base.roll(7 * b, 1) * 2.0 ** (b % 5) for b in range(len(lens))])
    kv8 = torch.randint(0, 127, (used, 64, 576), generator=g, dtype=torch.uint8)
    kvs = torch.exp2(torch.randint(-12, -4, (used,), generator=g).float())
    rk, rs = ref.append(rows, new, table, lens, kv8, kvs)
    for _ in range(3 if kind == "three times" else 1):
        k, s, st = run_append(rows, new, table, lens, kv8, kvs, used)
        assert st == 0 and torch.equal(s, rs) and torch.equal(k, rk)


@gpu
def test_append_token_by_token_equals_the_definition_step_by_step():
    steps, B = 70, 3
    table, used = tables([steps + 60] * B, 8)
    kv8, kvs = pool(used, 9)
    rk, rs = kv8.clone(), kvs.clone()
    g = torch.Generator().manual_seed(10)
    for i in range(steps):
        lens = [60 + i + 1, i + 1, max(1, i)]  # the third writes its token a second time
        rows = (torch.randn(B, 1, 576, generator=g) * 2.0 ** (i % 9 - 4)).to(BF)
        kv8, kvs, st = run_append(rows, [1] * B, table, lens, kv8, kvs, used, pass_new=i % 2 == 0)
        rk, rs = ref.append(rows, [1] * B, table, lens, rk, rs)
        assert st == 0 and torch.equal(kvs, rs) and torch.equal(kv8, rk), i


@gpu
def test_append_special_values():
    rows = torch.zeros(1, 6, 576)
    rows[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 1.0])
    rows[0, 1, 0] = 3.0e38          # beyond 448 * 2^32: saturates
    rows[0, 2, 0] = 1.0e-30         # vanishes
    rows[0, 3, 0] = 448.0 * 2.0 ** 32
    rows = rows.to(BF)
    table = torch.tensor([[1]], dtype=torch.int32)
    kv8, kvs = pool(2, 11)
    k, s, st = run_append(rows, [6], table, [6], kv8, kvs, 2)
    rk, rs = ref.append(rows, [6], table, [6], kv8, kvs)
    assert st == 0 and torch.equal(s, rs) and float(s[1]) == 2.0 ** 32
    assert torch.equal(k, rk) or torch.equal(k & 0x7F, rk & 0x7F)  # NaN's sign, zero's sign
    assert k[1, 0, 0] == 0x7E and k[1, 0, 1] == 0xFE and (k[1, 0, 2] & 0x7F) == 0x7F
    # All zeros: the smallest scale, and tokens after them raise it again.
    k, s, st = run_append(torch.zeros(1, 2, 576, dtype=BF), [2], table, [2], kv8, kvs, 2)
    assert st == 0 and float(s[1]) == 2.0 ** -32 and not k[1].any()
    one = torch.ones(1, 1, 576, dtype=BF)
    k, s, st = run_append(one, [1], table, [3], k, s, 2)
    assert st == 0 and float(s[1]) == 2.0 ** -8 and bool((ref.values(k[1, 2]) == 256.0).all())
    # A page of bf16's smallest numbers vanishes under the smallest scale.
    tiny = torch.full((1, 1, 576), 1e-39).to(BF)
    k, s, st = run_append(tiny, [1], table, [1], kv8, kvs, 2)
    assert st == 0 and float(s[1]) == 2.0 ** -32 and not (k[1] & 0x7F).any()


@gpu
@pytest.mark.parametrize("old,status", [
    (1.5 * 2.0 ** -6, 0), (0.75, 0), (1.25 * 2.0 ** -20, 0), (2.0 ** 32, 0), (2.0 ** -32, 0),
    (0.0, 5), (-1.0, 5), (math.nan, 5), (math.inf, 5), (2.0 ** 33, 5), (2.0 ** -33, 5)])
def test_append_to_a_page_of_any_scale(old, status):
    # A cache quantised by others, or never: any positive scale is rounded up to
    # a power of two, one out of range counts as 1.
    table = torch.tensor([[0, 1]], dtype=torch.int32)
    kv8, kvs = pool(2, 16)
    kvs[0] = old
    rows = torch.randn(1, 30, 576, generator=torch.Generator().manual_seed(17)).to(BF)
    k, s, st = run_append(rows, [30], table, [50], kv8, kvs, 2)
    rk, rs = ref.append(rows, [30], table, [50], kv8, kvs)
    assert st == status and torch.equal(s, rs) and torch.equal(k & 0x7F, rk & 0x7F)


@gpu
@pytest.mark.parametrize("lens,new,why", [
    ([129, 20], [1, 1], "past the table"), ([20, 20], [21, 1], "more new tokens than tokens"),
    ([20, 20], [-1, 1], "negative"), ([20, 20], [5, 1], "more than max_new"),
    ([-3, 20], [0, 1], "negative length")])
def test_append_leaves_a_bad_sequence_alone(lens, new, why):
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    kv8, kvs = pool(4, 12)
    rows = torch.randn(2, 4, 576, generator=torch.Generator().manual_seed(13)).to(BF)
    k, s, st = run_append(rows, new, table, lens, kv8, kvs, 4)
    rk, rs = ref.append(rows, [0, new[1]], table, [0, lens[1]], kv8, kvs)
    assert st == 5, why
    assert torch.equal(k, rk) and torch.equal(s, rs)


@gpu
@pytest.mark.parametrize("bad", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_append_skips_a_page_outside_the_pool(bad):
    table = torch.tensor([[0, bad], [2, 3]], dtype=torch.int32)
    kv8, kvs = pool(4, 14)
    rows = torch.randn(2, 128, 576, generator=torch.Generator().manual_seed(15)).to(BF)
    k, s, st = run_append(rows, [100, 100], table, [100, 100], kv8, kvs, 4)
    assert st == 5
    good = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    rk, rs = ref.append(rows, [100, 100], good, [100, 100], kv8, kvs)
    rk[1], rs[1] = kv8[1], kvs[1]
    assert torch.equal(k, rk) and torch.equal(s, rs)


# ---------------------------------------------------------------- attention
def fp8_inputs(inp):
    """The inputs' cache in 8 bits; the inputs then hold the same values in bf16."""
    kv8, kvs = ref.quantise(inp.cache.nan_to_num(0.0))
    inp.cache = (ref.values(kv8) * kvs.double()[:, None, None]).to(BF)
    return inp, kv8, kvs


def run_fp8(inp, kv8, kvs, num_ranges=0, expect=0, m=None):
    g = inp.to(torch.device("cuda"))
    d = binding.dims_for(g.q, g.cache, g.block_table)
    m = m or binding.MlaDecode(d, num_ranges=num_ranges, fp8_kv=True)
    B, T, H = g.q.shape[:3]
    out = torch.full((B, T, H, 128), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((B, T, H), float("nan"), dtype=torch.float32, device="cuda")
    m.plan(g.seq_lens)
    m.run_fp8kv(g.q, kv8.cuda(), kvs.cuda(), g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale,
                out, lse)
    assert m.check() == expect
    return out.cpu(), lse.cpu()


@gpu
@pytest.mark.parametrize("lens", [[1], [2, 63, 64, 65], [17, 80]])
def test_attention_shortest_sequences(lens):
    inp, kv8, kvs = fp8_inputs(make_inputs(len(lens), lens, 1, 16, seed=20))
    out, lse = run_fp8(inp, kv8, kvs)
    assert_parity(compare(inp, out, lse), str(lens))


@gpu
@pytest.mark.parametrize("H,T", [(16, 1), (32, 1), (64, 1), (128, 1), (16, 2), (128, 2), (48, 1),
                                 (80, 1), (96, 2), (112, 2), (16, 4), (128, 3), (64, 8),
                                 (128, 8), (128, 6), (112, 8)])
def test_attention_ragged_lengths_all_rows(H, T):
    lens = [T, 1 + T, 63, 64, 65, 127, 128, 129, 200, 511, 700]
    lens = [max(n, T) for n in lens]
    inp, kv8, kvs = fp8_inputs(make_inputs(len(lens), lens, T, H, seed=100 + H + T))
    out, lse = run_fp8(inp, kv8, kvs)
    assert_parity(compare(inp, out, lse), "H=%d T=%d" % (H, T))


@gpu
@pytest.mark.parametrize("H,T,ranges", [(16, 1, 1), (16, 1, 37), (64, 2, 5), (128, 1, 150),
                                        (128, 4, 9)])
def test_attention_any_split(H, T, ranges):
    inp, kv8, kvs = fp8_inputs(make_inputs(3, [2500, 64, 900], T, H, seed=21))
    out, lse = run_fp8(inp, kv8, kvs, num_ranges=ranges)
    assert_parity(compare(inp, out, lse), "ranges %d" % ranges)


@gpu
@pytest.mark.parametrize("H,T,ranges", [(16, 1, 1), (128, 1, 1), (16, 1, 0), (128, 2, 0), (32, 8, 3)])
def test_attention_many_pieces_of_a_page_or_two(H, T, ranges):
    # Sequences of one to three pages, several (with one range: all) of them to a
    # CTA: query tiles and pages of the next pieces enter the ring while the
    # first are still in work, from the first round of its slots on.
    lens = [max(T, 1 + (37 * i) % 190) for i in range(40 if ranges else 400)]
    lens[0] = T
    inp, kv8, kvs = fp8_inputs(make_inputs(len(lens), lens, T, H, seed=43))
    out, lse = run_fp8(inp, kv8, kvs, num_ranges=ranges)
    assert_parity(compare(inp, out, lse), "ranges %d" % ranges)
    out2, lse2 = run_fp8(inp, kv8, kvs, num_ranges=ranges)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
def test_attention_repeated_runs_give_the_same_bits_while_memory_is_busy():
    # 64 sequences of 64 pages: every SM streams, loads are slow and the pipeline
    # runs out of pages.  Ten runs between copies that evict the cache from L2.
    inp, kv8, kvs = fp8_inputs(make_inputs(64, [4096 - 7 * i for i in range(64)], 1, 16, seed=44))
    g = inp.to(torch.device("cuda"))
    k, s = kv8.cuda(), kvs.cuda()
    m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), fp8_kv=True)
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    results = []
    for i in range(10):
        out = torch.empty(64, 1, 16, 128, dtype=BF, device="cuda")
        lse = torch.empty(64, 1, 16, device="cuda")
        big.fill_(i)
        m.plan(g.seq_lens)
        m.run_fp8kv(g.q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, out, lse)
        results.append((out, lse))
    assert m.check() == 0
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])
    assert_parity(compare(inp, results[0][0].cpu(), results[0][1].cpu()), "64 x 4096")


@gpu
def test_attention_large_batch_takes_the_large_paths():
    lens = torch.randint(1, 400, (300,), generator=torch.Generator().manual_seed(22)).tolist()
    lens = [max(2, n) for n in lens]
    inp, kv8, kvs = fp8_inputs(make_inputs(300, lens, 2, 32, seed=23))
    out, lse = run_fp8(inp, kv8, kvs)
    assert_parity(compare(inp, out, lse), "300 sequences")


@gpu
def test_unused_pages_and_tail_rows_do_not_matter():
    inp, kv8, kvs = fp8_inputs(make_inputs(3, [70, 5, 200], 1, 32, seed=24, spare_pages=2))
    out, lse = run_fp8(inp, kv8, kvs)
    poisoned, scales = kv8.clone(), kvs.clone()
    poisoned[inp.used_pages:] = 0x7F
    scales[inp.used_pages:] = math.nan
    for b, n in enumerate([70, 5, 200]):  # rows past the end: the largest finite code
        poisoned[int(inp.block_table[b, n // 64]), n % 64:] = 0x7E
    out2, lse2 = run_fp8(inp, poisoned, scales)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
def test_pages_in_another_order_give_the_same_bits():
    inp, kv8, kvs = fp8_inputs(make_inputs(4, [700, 64, 65, 300], 2, 64, seed=25))
    out, lse = run_fp8(inp, kv8, kvs)
    perm = torch.randperm(kv8.shape[0], generator=torch.Generator().manual_seed(26))
    inv = torch.argsort(perm).to(torch.int32)
    t = inp.block_table
    inp.block_table = torch.where(t >= 0, inv[t.clamp(min=0).long()], t)
    inp.cache = inp.cache[perm]
    out2, lse2 = run_fp8(inp, kv8[perm], kvs[perm])
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("low,high", [(-12, 2), (-30, 0)])
def test_pages_of_very_different_scales(low, high):
    # Scores stay of the size of ordinary ones (the largest scale is near 1), so
    # small pages have equal weights and values near zero.
    inp = make_inputs(3, [1000, 130, 640], 1, 32, seed=27)
    g = torch.Generator().manual_seed(28)
    e = torch.randint(low, high + 1, (inp.cache.shape[0],), generator=g)
    inp.cache = (inp.cache.float() * torch.exp2(e.float())[:, None, None]).to(BF)
    inp.scale = inp.scale / 2.0 ** max(0, high)
    inp, kv8, kvs = fp8_inputs(inp)
    out, lse = run_fp8(inp, kv8, kvs)
    s = compare(inp, out, lse)
    # Values up to 2^high: the outputs' bounds grow with them.
    assert s["out_max"] <= ref.OUT_MAX * 2.0 ** max(0, high) and s["lse_max"] <= 1e-3, s


@gpu
@pytest.mark.parametrize("H,lens", [(16, [300, 70]), (128, [64] * 90)])
@pytest.mark.parametrize("e", [-12, 9, 13, 16, 24])
def test_queries_of_any_size(e, H, lens):
    # Queries times 2^e and a softmax scale over 2^e: the same scores.  Rows whose
    # absorbed query is far beyond 2^14, in first pieces of a CTA and in later
    # ones (90 sequences x two tiles: one range per CTA pair, 1.2 pieces).
    inp = make_inputs(len(lens), lens, 1, H, seed=46)
    inp.q = (inp.q.float() * 2.0 ** e).to(BF)
    inp.scale = inp.scale / 2.0 ** e
    inp, kv8, kvs = fp8_inputs(inp)
    out, lse = run_fp8(inp, kv8, kvs, num_ranges=20 if H == 128 else 0)
    s = compare(inp, out, lse)
    # The lse's correction for the bf16 query q_lat is the rounding's residual r,
    # |r| <= 2^-9 |q_lat|, stored as E4M3 of 2^10 r: it is below half of E4M3's
    # least number (2^-9) where |q_lat| < 2^-11, and above its largest (448) where
    # |q_lat| > 224.  Every e here is outside of that, so the lse keeps the query's
    # rounding: 2^-9 of a score of 576 terms, whose size is about 1.7, and three
    # times that for the largest of the rows.
    lse_max = 1.7 * 3 * 2.0 ** -9
    assert s["out_max"] <= ref.OUT_MAX and s["out_mean"] <= ref.OUT_MEAN, s
    assert s["lse_max"] <= lse_max, s


@gpu
def test_nan_in_a_visible_token_reaches_its_sequence_only():
    inp, kv8, kvs = fp8_inputs(make_inputs(3, [200, 70, 130], 1, 16, seed=47))
    out0, lse0 = run_fp8(inp, kv8, kvs)
    bad = kv8.clone()
    bad[int(inp.block_table[1, 0]), 11, 500] = 0x7F
    out, lse = run_fp8(inp, bad, kvs)
    assert out[1].isnan().all() and lse[1].isnan().all()
    for b in (0, 2):
        assert torch.equal(out[b], out0[b]) and torch.equal(lse[b], lse0[b])


@gpu
@pytest.mark.parametrize("lens", [[2, 130, 90], [700, 900, 64]])
@pytest.mark.parametrize("H,num_ranges", [(16, 0), (16, 2), (128, 2)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_gives_nan(value, H, num_ranges, lens):
    # In the absorbed part and in the RoPE part, in first pieces of a range and in
    # later ones, split sequences and whole ones.
    inp, kv8, kvs = fp8_inputs(make_inputs(3, lens, 2, H, seed=48))
    out0, lse0 = run_fp8(inp, kv8, kvs, num_ranges=num_ranges)
    inp.q[:, 1, 3, 5] = value
    inp.q[:, 0, H - 1, 140] = value
    out, lse = run_fp8(inp, kv8, kvs, num_ranges=num_ranges)
    changed = torch.zeros_like(lse, dtype=torch.bool)
    changed[:, 1, 3] = changed[:, 0, H - 1] = True
    assert out[changed].isnan().all() and lse[changed].isnan().all()
    assert torch.equal(out[~changed], out0[~changed])
    assert torch.equal(lse[~changed], lse0[~changed])


@gpu
def test_nan_as_the_only_token():
    inp, kv8, kvs = fp8_inputs(make_inputs(2, [1, 65], 1, 16, seed=49))
    bad = kv8.clone()
    for b, k in ((0, 0), (1, 1)):
        bad[int(inp.block_table[b, k]), 0, 500] = 0x7F
    out, lse = run_fp8(inp, bad, kvs)
    assert out.isnan().all() and lse.isnan().all()


@gpu
@pytest.mark.parametrize("n", [4000, 32000])
def test_many_small_weights_next_to_a_large_one(n):
    # One key has a weight of about half the row's sum, the other keys share the
    # rest equally (1 / n each, 2^-13 to 2^-16).  All equal: whatever their
    # rounding is, it is the same for each and must not bias the sum.
    H = 16
    inp = make_inputs(1, [n], 1, H, seed=29)
    inp.q.zero_()
    inp.q[..., 128:] = 1.0             # only the RoPE part of the keys counts
    g = torch.Generator().manual_seed(30)
    v0, v1 = torch.randn(2, 512, generator=g).to(BF)
    inp.cache.zero_()
    inp.cache[..., :512] = v1
    page = int(inp.block_table[0, 10])
    inp.cache[page, 7, :512] = v0
    x = math.log(n) / (64 * inp.scale)  # weight e^(64 x scale) = n
    inp.cache[page, 7, 512:] = x
    inp, kv8, kvs = fp8_inputs(inp)
    out, lse = run_fp8(inp, kv8, kvs)
    s = compare(inp, out, lse)
    # A weight f of the row and a relative error of 2^-7 between the two parts'
    # roundings move the output by f (1 - f) 2^-7 |o0 - o1|, at most 2^-9 |o0 -
    # o1|; o_lat and out are rounded to bf16 (2^-8 each, o_lat's summed over 512
    # products of random sign).  |o0 - o1| stays below 8 for these inputs.
    assert s["out_max"] <= 8 * 2.0 ** -9 + 2 * 4 * 2.0 ** -8, s
    assert s["lse_max"] <= 1e-3, s


@gpu
def test_bad_table_entries_and_scales_are_reported():
    inp, kv8, kvs = fp8_inputs(make_inputs(2, [100, 64], 1, 16, seed=31))
    out0, lse0 = run_fp8(inp, kv8, kvs)
    good = inp.block_table.clone()
    for bad in (-1, kv8.shape[0], 2 ** 31 - 1):
        inp.block_table = good.clone()
        inp.block_table[0, 1] = bad
        out, lse = run_fp8(inp, kv8, kvs, expect=5)
        assert torch.equal(out[1], out0[1]) and torch.equal(lse[1], lse0[1])
        assert out.isfinite().all()
    inp.block_table = good
    for bad in (0.0, -1.0, math.nan, math.inf, 2.0 ** 33):
        scales = kvs.clone()
        scales[int(good[1, 0])] = bad
        out, lse = run_fp8(inp, kv8, scales, expect=5)
        assert torch.equal(out[0], out0[0]) and torch.equal(lse[0], lse0[0])
        assert out.isfinite().all()


@gpu
def test_lengths_out_of_range_are_clamped_and_reported():
    inp, kv8, kvs = fp8_inputs(make_inputs(2, [100, 64], 1, 16, seed=32))
    out0, lse0 = run_fp8(inp, kv8, kvs)
    inp.seq_lens = torch.tensor([100, 0], dtype=torch.int32)
    out, lse = run_fp8(inp, kv8, kvs, expect=5)
    assert torch.equal(out[0], out0[0]) and torch.equal(lse[0], lse0[0])


@gpu
def test_the_plans_for_either_cache_differ_and_serve_both():
    lens = [1 + 13 * i % 700 for i in range(200)]
    inp, kv8, kvs = fp8_inputs(make_inputs(200, lens, 1, 64, seed=45))
    g = inp.to(torch.device("cuda"))
    d = binding.dims_for(g.q, g.cache, g.block_table)
    results = []
    for fp8_kv in (False, True):
        m = binding.MlaDecode(d, fp8_kv=fp8_kv)
        m.plan(g.seq_lens)
        pages = sum((n + 63) // 64 for n in lens)
        assert m.plan_header()[2] == pages + 200 * (6 if fp8_kv else 2)
        for kind in ("bf16", "fp8"):
            out = torch.empty(200, 1, 64, 128, dtype=BF, device="cuda")
            lse = torch.empty(200, 1, 64, device="cuda")
            if kind == "fp8":
                m.run_fp8kv(g.q, kv8.cuda(), kvs.cuda(), g.block_table, g.seq_lens, g.w_uk,
                            g.w_uv, g.scale, out, lse)
            else:
                m.run(g.q, g.cache, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, out, lse)
            assert m.check() == 0
            assert_parity(compare(inp, out.cpu(), lse.cpu()), kind)


@gpu
def test_one_plan_serves_both_caches_and_the_steps_equal_the_run():
    inp, kv8, kvs = fp8_inputs(make_inputs(4, [700, 64, 65, 300], 2, 32, seed=33))
    g = inp.to(torch.device("cuda"))
    k, s = kv8.cuda(), kvs.cuda()
    m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), fp8_kv=True)
    mk = lambda: (torch.empty(4, 2, 32, 128, dtype=BF, device="cuda"),
                  torch.empty(4, 2, 32, device="cuda"))
    m.plan(g.seq_lens)
    (o1, l1), (o2, l2), (o3, l3), (o4, l4) = mk(), mk(), mk(), mk()
    m.run(g.q, g.cache, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, o1, l1)
    m.run_fp8kv(g.q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, o2, l2)
    m.absorb(g.q, g.w_uk)
    m.attend_fp8kv(k, s, g.block_table, g.seq_lens, g.scale, l3)
    m.combine(g.scale, l3)
    m.up_project(g.w_uv, o3)
    assert m.check() == 0
    assert torch.equal(o2, o3) and torch.equal(l2, l3)
    assert (o1.float() - o2.float()).abs().max() <= 2e-2 + ref.OUT_MAX and (l1 - l2).abs().max() <= 2e-3
    # FP8 weights through the step calls.
    uk8, uks = quantize_fp8_blockwise(inp.w_uk)
    uv8, uvs = quantize_fp8_blockwise(inp.w_uv)
    dq = lambda w, sc: (w.view(torch.float8_e4m3fn).float()
                        * sc.repeat_interleave(128, 1).repeat_interleave(128, 2)).to(BF)
    m.absorb_fp8w(g.q, uk8.cuda(), uks.cuda())
    m.attend_fp8kv(k, s, g.block_table, g.seq_lens, g.scale, l4)
    m.combine(g.scale, l4)
    m.up_project_fp8w(uv8.cuda(), uvs.cuda(), o4)
    assert m.check() == 0
    inp.w_uk, inp.w_uv = dq(uk8, uks), dq(uv8, uvs)
    assert_parity(compare(inp, o4.cpu(), l4.cpu()), "FP8 weights and cache")


@gpu
def test_captured_and_replayed_on_another_stream_with_new_inputs():
    inp, kv8, kvs = fp8_inputs(make_inputs(5, [300, 64, 1, 130, 70], 1, 48, seed=34))
    out0, lse0 = run_fp8(inp, kv8, kvs)
    g = inp.to(torch.device("cuda"))
    k, s = kv8.cuda(), kvs.cuda()
    m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), fp8_kv=True)
    rows = torch.randn(5, 1, 576, generator=torch.Generator().manual_seed(35)).to(BF).cuda()
    out = torch.empty(5, 1, 48, 128, dtype=BF, device="cuda")
    lse = torch.empty(5, 1, 48, device="cuda")
    stream = torch.cuda.Stream()

    def step():
        binding.append_fp8kv(m.dims, rows, k, s, g.block_table, g.seq_lens)
        m.plan(g.seq_lens)
        m.run_fp8kv(g.q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, out, lse)

    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    torch.cuda.synchronize()
    for seed in (36, 37):  # other tokens, other queries, other lengths
        gen = torch.Generator().manual_seed(seed)
        new = (torch.randn(5, 1, 576, generator=gen) * 2.0).to(BF)
        inp.q = torch.randn(5, 1, 48, 192, generator=gen).to(BF)
        inp.seq_lens = torch.tensor([299, 63, 1, 129 - (seed & 1), 65], dtype=torch.int32)
        k.copy_(kv8)
        s.copy_(kvs)
        rows.copy_(new)
        g.q.copy_(inp.q)
        g.seq_lens.copy_(inp.seq_lens)
        graph.replay()
        torch.cuda.synchronize()
        rk, rs = ref.append(new, [1] * 5, inp.block_table, inp.seq_lens.tolist(), kv8, kvs)
        assert torch.equal(k.cpu(), rk) and torch.equal(s.cpu(), rs)
        inp.cache = (ref.values(rk) * rs.double()[:, None, None]).to(BF)
        assert m.check() == 0
        assert_parity(compare(inp, out.cpu(), lse.cpu()), "replay %d" % seed)


@gpu
def test_two_calls_at_once_on_two_streams():
    cases = []
    for seed in (38, 39):
        inp, kv8, kvs = fp8_inputs(make_inputs(6, [900, 64, 65, 300, 1, 511], 1, 64, seed=seed))
        cases.append((inp, kv8, kvs, *run_fp8(inp, kv8, kvs)))
    dev = torch.device("cuda")
    live = []
    for inp, kv8, kvs, _, _ in cases:
        g = inp.to(dev)
        m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), fp8_kv=True)
        live.append((g, kv8.cuda(), kvs.cuda(), m, torch.empty(6, 1, 64, 128, dtype=BF, device=dev),
                     torch.empty(6, 1, 64, device=dev), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, k, s, m, out, lse, st in live:
            with torch.cuda.stream(st):
                m.plan(g.seq_lens)
                m.run_fp8kv(g.q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, out,
                            lse)
    torch.cuda.synchronize()
    for (_, _, _, out0, lse0), (_, _, _, _, out, lse, _) in zip(cases, live):
        assert torch.equal(out.cpu(), out0) and torch.equal(lse.cpu(), lse0)


@gpu
def test_cache_offsets_beyond_32_bits():
    # 130,000 pages of 36,864 codes: 4.8 GB; the sequences' pages lie at its end
    # and its start.
    pages = 130000
    inp, kv8, kvs = fp8_inputs(make_inputs(2, [200, 70], 1, 16, seed=40))
    used = kv8.shape[0]
    big = torch.zeros(pages, 64, 576, dtype=torch.uint8, device="cuda")
    scale = torch.ones(pages, device="cuda")
    where = torch.tensor([pages - 1, 0, pages - 2, 1, pages - 3, 2][:used])
    big[where.cuda()] = kv8.cuda()
    scale[where.cuda()] = kvs.cuda()
    g = inp.to(torch.device("cuda"))
    t = inp.block_table
    table = torch.where(t >= 0, where[t.clamp(min=0).long()].to(torch.int32), t).cuda()
    d = binding.Dims(2, 1, 16, 128, 64, 512, 128, 64, pages, table.shape[1])
    m = binding.MlaDecode(d, fp8_kv=True)
    out = torch.empty(2, 1, 16, 128, dtype=BF, device="cuda")
    lse = torch.empty(2, 1, 16, device="cuda")
    m.plan(g.seq_lens)
    m.run_fp8kv(g.q, big, scale, table, g.seq_lens, g.w_uk, g.w_uv, g.scale, out, lse)
    assert m.check() == 0
    assert_parity(compare(inp, out.cpu(), lse.cpu()), "large pool")
    rows = torch.randn(2, 1, 576, generator=torch.Generator().manual_seed(41)).to(BF)
    binding.append_fp8kv(d, rows.cuda(), big, scale, table, g.seq_lens)
    rk, rs = ref.append(rows, [1, 1], inp.block_table, [200, 70], kv8, kvs)
    assert torch.equal(big[where.cuda()].cpu(), rk) and torch.equal(scale[where.cuda()].cpu(), rs)


@gpu
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("B,H,ranges", [(24, 16, 1), (24, 128, 1), (160, 16, 2), (40, 64, 0)])
def test_runs_of_other_queries_back_to_back_on_one_plan(fp8, B, H, ranges):
    # A plan serves every layer of a step.  The absorb step of a run starts while
    # the run before it is at work, whose attention reads the absorbed query of
    # one sequence after the other (with one range on a single SM, the others
    # being free): every run must see its own queries, bit for bit.
    inp = make_inputs(B, [500 + 37 * i % 300 for i in range(B)], 1, H, seed=80)
    inp, kv8, kvs = fp8_inputs(inp)
    g = inp.to(torch.device("cuda"))
    k, s = kv8.cuda(), kvs.cuda()
    m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), num_ranges=ranges,
                          fp8_kv=fp8)
    gen = torch.Generator().manual_seed(81)
    queries = [torch.randn(B, 1, H, 192, generator=gen).to(BF).cuda() for _ in range(4)]
    mk = lambda: [(torch.zeros(B, 1, H, 128, dtype=BF, device="cuda"),
                   torch.zeros(B, 1, H, device="cuda")) for _ in queries]

    def run(q, out, lse):
        tail = (g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, out, lse)
        m.run_fp8kv(q, k, s, *tail) if fp8 else m.run(q, g.cache, *tail)

    alone, together = mk(), mk()
    m.plan(g.seq_lens)
    for q, (out, lse) in zip(queries, alone):
        run(q, out, lse)
        torch.cuda.synchronize()
    for _ in range(5):
        for q, (out, lse) in zip(queries, together):
            run(q, out, lse)
    assert m.check() == 0
    for (o1, l1), (o2, l2) in zip(alone, together):
        assert torch.equal(o1, o2) and torch.equal(l1, l2)


@gpu
@pytest.mark.parametrize("H,ranges", [(16, 1), (16, 3), (128, 1)])
def test_a_maximum_that_rises_with_every_page_of_many_pieces(H, ranges):
    # Scores that grow by more than the lazy maximum's slack from page to page:
    # every page but a piece's first rescales the output, behind the product of
    # the page before, while the next piece's query tile and its terms take the
    # slots that this product frees.  Pieces of three to six pages, many to a CTA.
    lens = [64 * (3 + i % 4) - i % 7 for i in range(48)]
    inp = make_inputs(len(lens), lens, 1, H, seed=82)
    inp.q[..., :128] = 0.0
    inp.q[..., 128:] = 1.0
    inp.cache[..., 512:] = 0.0
    for b, n in enumerate(lens):
        for j in range((n + 63) // 64):
            # 64 products of 2 j, times 1 / sqrt(192): 9.2 a page, 8 ln 2 = 5.5.
            inp.cache[int(inp.block_table[b, j]), :, 512:] = 2.0 * j
    inp, kv8, kvs = fp8_inputs(inp)
    out, lse = run_fp8(inp, kv8, kvs, num_ranges=ranges)
    assert_parity(compare(inp, out, lse), "ranges %d" % ranges)
    for _ in range(20):
        out2, lse2 = run_fp8(inp, kv8, kvs, num_ranges=ranges)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("H,lens", [(16, [300, 70]), (128, [64] * 90)])
@pytest.mark.parametrize("e", [-100, -80, -50, -40, -36, 36, 40, 41, 44, 60, 90, 110])
def test_queries_of_extreme_size(e, H, lens):
    # As test_queries_of_any_size, towards the ends of bf16's range.
    inp = make_inputs(len(lens), lens, 1, H, seed=46)
    inp.q = (inp.q.float() * 2.0 ** e).to(BF)
    inp.scale = inp.scale / 2.0 ** e
    inp, kv8, kvs = fp8_inputs(inp)
    out, lse = run_fp8(inp, kv8, kvs, num_ranges=20 if H == 128 else 0)
    s = compare(inp, out, lse)
    # The bound of the lse: as there.
    assert s["out_max"] <= ref.OUT_MAX and s["out_mean"] <= ref.OUT_MEAN, s
    assert s["lse_max"] <= 1.7 * 3 * 2.0 ** -9, s


def test_run_and_attend_check_every_tensor(monkeypatch):
    # (In host memory: a call whose tensors are right is refused for that alone.)
    monkeypatch.setattr(binding, "workspace_size", lambda d, ranges=0: 4096)
    B, T, H = 2, 2, 16
    m = binding.MlaDecode(good_dims(q_len=T), device=torch.device("cpu"))
    good = dict(q=torch.zeros(B, T, H, 192, dtype=BF),
                kv8=torch.zeros(4, 64, 576, dtype=torch.uint8), kv_scale=torch.ones(4),
                block_table=torch.zeros(B, 2, dtype=torch.int32),
                seq_lens=torch.ones(B, dtype=torch.int32),
                w_uk=torch.zeros(H, 128, 512, dtype=BF), w_uv=torch.zeros(H, 512, 128, dtype=BF),
                out=torch.zeros(B, T, H, 128, dtype=BF), lse=torch.zeros(B, T, H))
    attend = ("kv8", "kv_scale", "block_table", "seq_lens", "lse")

    def refused(name, **change):
        a = dict(good, **change)
        with pytest.raises(ValueError, match="^%s: " % name):
            m.run_fp8kv(scale=0.07, **a)
        if name in attend:
            with pytest.raises(ValueError, match="^%s: " % name):
                m.attend_fp8kv(scale=0.07, **{k: a[k] for k in attend})

    for name, t in good.items():
        refused(name, **{name: None})
        refused(name, **{name: t.double()})                          # another type
        refused(name, **{name: t[:-1]})                              # too short
        refused(name, **{name: torch.cat([t, t])[::2]})              # strided
        refused(name, **{name: torch.cat([t, t])})                   # too long
    refused("w_uk", w_uk=good["w_uv"])
    with pytest.raises(ValueError, match="^kv8: .*CUDA device"):
        m.run_fp8kv(scale=0.07, **good)
    with pytest.raises(ValueError, match="^kv8: .*CUDA device"):
        m.attend_fp8kv(scale=0.07, **{k: good[k] for k in attend})
    # [B, T, ...] for a handle of B * T sequences of one token.
    m = binding.MlaDecode(good_dims(batch=B * T), device=torch.device("cpu"))
    good.update(block_table=torch.zeros(B * T, 2, dtype=torch.int32),
                seq_lens=torch.ones(B * T, dtype=torch.int32))
    refused("kv8")


@gpu
def test_a_refused_run_enqueues_nothing():
    inp, kv8, kvs = fp8_inputs(make_inputs(2, [70, 5], 1, 16, seed=83))
    g = inp.to(torch.device("cuda"))
    m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), fp8_kv=True)
    out = torch.full((2, 1, 16, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((2, 1, 16), 7.0, device="cuda")
    k, s = kv8.cuda(), kvs.cuda()
    m.plan(g.seq_lens)
    for q, o in ((g.q.float(), out), (g.q[:1], out), (g.q, out[:, :, :8]), (g.q.cpu(), out)):
        with pytest.raises(ValueError):
            m.run_fp8kv(q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, o, lse)
    assert m.check() == 0 and (out == 7.0).all() and (lse == 7.0).all()


def test_missing_tensors_and_other_ranks_are_refused_by_name():
    d = good_dims()
    kv8, kvs = torch.zeros(4, 64, 576, dtype=torch.uint8), torch.ones(4)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    keys, query = torch.zeros(4, 576, dtype=BF), torch.zeros(2, 1, 16, 576, dtype=BF)
    scores, sel = torch.zeros(2, 1, 2), torch.zeros(2, 2, dtype=torch.int32)
    rows = torch.zeros(2, 3, 576, dtype=BF)
    for bad in (None, rows[0, 0], rows[None], torch.zeros((), dtype=BF)):
        with pytest.raises(ValueError, match="^rows: "):
            binding.append_fp8kv(d, bad, kv8, kvs, table, lens)
    for fn, args in ((binding.append_fp8kv, (rows, kv8, kvs, table, lens)),
                     (binding.page_keys, (kv8.to(BF), table, lens, 1, keys)),
                     (binding.page_keys_fp8kv, (kv8, kvs, table, lens, 1, keys)),
                     (binding.score_pages, (query, keys, table, lens, scores)),
                     (binding.select_pages, (scores, table, lens, 2, 1, 1, sel, lens))):
        for i, a in enumerate(args):
            if isinstance(a, torch.Tensor):
                with pytest.raises(ValueError, match="got None"):
                    fn(d, *args[:i], None, *args[i + 1:])


@gpu
@pytest.mark.parametrize("old", [1.5 * 2.0 ** -6, 0.75, 1.25 * 2.0 ** -20, 1.9, 0.0, math.nan])
def test_append_under_another_scale_keeps_every_sign(old):
    # Rows that stay are re-coded under a scale that is not a power of two: signs
    # too, those of values that vanish among them.
    table = torch.tensor([[0, 1]], dtype=torch.int32)
    kv8, kvs = pool(2, 16)
    kv8[0, 3, :256] = torch.arange(256, dtype=torch.uint8)  # every code
    kvs[0] = old
    rows = torch.randn(1, 30, 576, generator=torch.Generator().manual_seed(17)).to(BF)
    rows[0, 5, :4] = torch.tensor([0.0, -0.0, 1e-30, -1e-30])
    k, s, _ = run_append(rows, [30], table, [50], kv8, kvs, 2)
    rk, rs = ref.append(rows, [30], table, [50], kv8, kvs)
    nan = (rk & 0x7F) == 0x7F  # (a NaN's sign is nobody's)
    assert torch.equal(s, rs) and torch.equal(k[~nan], rk[~nan])
    assert ((k[nan] & 0x7F) == 0x7F).all()
    assert bool((k[0, 25, :4] == torch.tensor([0x00, 0x80, 0x00, 0x80], dtype=torch.uint8)).all())


@gpu
def test_append_of_special_values_keeps_signs():
    rows = torch.zeros(1, 6, 576)
    rows[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, -1.0])
    rows[0, 1, :2] = torch.tensor([3.0e38, -3.0e38])
    rows[0, 2, :3] = torch.tensor([1.0e-30, -1.0e-30, -0.0])
    rows[0, 3, :2] = torch.tensor([448.0 * 2.0 ** 32, -448.0 * 2.0 ** 32])
    rows = rows.to(BF)
    table = torch.tensor([[1]], dtype=torch.int32)
    kv8, kvs = pool(2, 11)
    k, s, st = run_append(rows, [6], table, [6], kv8, kvs, 2)
    rk, rs = ref.append(rows, [6], table, [6], kv8, kvs)
    nan = (rk & 0x7F) == 0x7F
    assert st == 0 and torch.equal(s, rs) and torch.equal(k[~nan], rk[~nan])
    assert int(nan.sum()) == 1 and (k[1, 0, 2] & 0x7F) == 0x7F
    assert k[1, 2, :4].tolist() == [0x00, 0x80, 0x80, 0x00]
