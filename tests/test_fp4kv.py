"""The 4-bit latent cache: append, attention, page keys, reading back (from every
cache), against 64-bit forms."""
import ctypes
import math

import pytest
import torch

import fp4kv_util as ref
import fp8kv_util as ref8
from fp8kv_util import assert_parity
from mla_decode_attention_uk_gb300 import binding
from mla_decode_attention_uk_gb300.inputs import make_inputs
from parity_util import compare
from test_fp8kv import ODD2, ODD8, OK, call, good_dims, run_fp8, tables

gpu = pytest.mark.gpu
BF = torch.bfloat16


def cuda_ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# ---------------------------------------------------------------- the format (no GPU)
def test_every_value_is_one_of_e4m3():
    for e in range(15):
        x = ref.E2M1 * 2.0 ** (e - 8)
        assert torch.equal(ref8.values(ref8.e4m3(x)), x)


def test_the_reference_rounds_to_the_nearest_value():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(50, 576, generator=g, dtype=torch.float64)
    x *= torch.exp2(torch.randint(-12, 8, (50, 576), generator=g).double())
    x[0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.75, -1.25,
                              -1.75, -2.5, -3.5, -5.0, -7.0]) / 256
    y = ref.decode(ref.encode(x))
    assert torch.equal(ref.encode(y), ref.encode(y).clone())
    assert torch.equal(ref.decode(ref.encode(y)), y)  # what it stands for stays
    assert torch.equal(y[0, :16] * 256, torch.tensor([0, 1, 1, 2, 2, 4, 4, 6, 0, -1, -1, -2, -2,
                                                      -4, -4, -6], dtype=torch.float64))
    top = x[:, :512].reshape(50, 32, 16).abs().amax(dim=2)
    j = torch.ceil(torch.log2(top / 7)).clamp(-8, 6)
    err = (x - y)[:, :512].reshape(50, 32, 16).abs()
    # Half of the top step, 2 * 2^j; half of the least one where 4 * 2^j is not reached.
    assert bool((err <= torch.exp2(j)[..., None]).all() | (top > 448).any())


def test_quantising_what_was_quantised_keeps_its_values_and_settles():
    # A block's exponent may fall the first time (its largest value was rounded down to where
    # a smaller unit holds it), the values do not move, and the second time nothing does.
    g = torch.Generator().manual_seed(2)
    x = torch.randn(200, 576, generator=g, dtype=torch.float64)
    x *= torch.exp2(torch.randint(-12, 8, (200, 576), generator=g).double())
    once = ref.encode(x)
    twice = ref.encode(ref.decode(once))
    assert torch.equal(ref.decode(twice), ref.decode(once))
    assert torch.equal(ref.encode(ref.decode(twice)), twice)


# ---------------------------------------------------------------- refusals (no GPU)
def test_append_refuses_bad_arguments():
    #       rows max_new new_lens table lens kv4 scale status stream
    args = [OK, 1, OK, OK, OK, OK, OK, OK, None]
    for change in ({0: None}, {0: ODD8}, {1: 0}, {1: -1}, {1: 2 ** 31 - 1}, {2: ODD2}, {3: None},
                   {3: ODD2}, {4: None}, {4: ODD2}, {5: None}, {5: ODD8}, {6: None}, {6: ODD2},
                   {7: ODD2}):
        assert call("mla_decode_append_fp4kv", args, change) == 1, change
    assert call("mla_decode_append_fp4kv", args, d=good_dims(kv_lora=256)) == 2
    assert binding.lib().mla_decode_append_fp4kv(None, *args) == 1


def test_run_and_attend_refuse_bad_arguments():
    sc = ctypes.c_float(0.07)
    #      q kv4 kvs table lens wuk wuv scale out lse ws wbytes stream
    run = [OK, OK, OK, OK, OK, OK, OK, sc, OK, OK, OK, 1 << 30, None]
    for change in ({0: None}, {1: None}, {1: ODD8}, {2: None}, {2: ODD2}, {3: ODD2}, {4: None},
                   {5: ODD8}, {6: None}, {8: ODD8}, {9: None}, {10: None}, {10: ODD8},
                   {7: ctypes.c_float(0.0)}, {7: ctypes.c_float(-1.0)},
                   {7: ctypes.c_float(math.nan)}, {7: ctypes.c_float(math.inf)}):
        assert call("mla_decode_run_fp4kv", run, change) == 1, change
    assert call("mla_decode_run_fp4kv", run, {11: 64}) == 3
    assert call("mla_decode_run_fp4kv", run, d=good_dims(q_len=9)) == 2
    #      kv4 kvs table lens scale lse ws wbytes stream
    att = [OK, OK, OK, OK, sc, OK, OK, 1 << 30, None]
    for change in ({0: None}, {0: ODD8}, {1: None}, {1: ODD2}, {2: None}, {3: ODD2}, {5: None},
                   {6: None}, {6: ODD8}, {4: ctypes.c_float(math.nan)}):
        assert call("mla_decode_attend_fp4kv", att, change) == 1, change
    assert call("mla_decode_attend_fp4kv", att, {7: 64}) == 3


@pytest.mark.parametrize("name", ["gather", "gather_fp8kv", "gather_fp4kv", "page_keys_fp4kv"])
def test_gather_and_keys_refuse_bad_arguments(name):
    name = "mla_decode_" + name
    quantised = name != "mla_decode_gather"
    #      cache (scale) table lens max_new new_lens dst status stream
    args = [OK] + [OK] * quantised + [OK, OK, 1, OK, OK, OK, None]
    k = int(quantised)
    changes = [{0: None}, {0: ODD8}, {1 + k: None}, {1 + k: ODD2}, {2 + k: None}, {2 + k: ODD2},
               {3 + k: 0}, {3 + k: -7}, {3 + k: 2 ** 31 - 1}, {4 + k: ODD2}, {5 + k: None},
               {5 + k: ODD8}, {6 + k: ODD2}] + [{1: None}, {1: ODD2}] * quantised
    for change in changes:
        assert call(name, args, change) == 1, change
    assert call(name, args, d=good_dims(page_size=32)) == 2
    assert getattr(binding.lib(), name)(None, *args) == 1


def test_python_calls_check_types_and_shapes():
    d = good_dims()
    kv4, kvs = torch.zeros(4, 64, 336, dtype=torch.uint8), torch.ones(4)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    rows, keys = torch.zeros(2, 3, 576, dtype=BF), torch.zeros(4, 576, dtype=BF)
    cache = torch.zeros(4, 64, 576, dtype=BF)
    kv8 = torch.zeros(4, 64, 576, dtype=torch.uint8)
    common = dict(block_table=table, seq_lens=lens)
    q4 = dict(kv4=kv4, kv_scale=kvs, **common)
    calls = [(binding.append_fp4kv, dict(rows=rows, **q4)),
             (binding.gather_fp4kv, dict(rows=rows, **q4)),
             (binding.gather_fp8kv, dict(rows=rows, kv8=kv8, kv_scale=kvs, **common)),
             (binding.gather, dict(rows=rows, cache=cache, **common)),
             (binding.page_keys_fp4kv, dict(max_new=1, keys=keys, **q4))]
    for f, good in calls:
        for k, v in (("rows", rows.float()), ("rows", rows[:1]), ("rows", rows[:, ::2]),
                     ("rows", None), ("kv4", kv4.view(torch.int8)), ("kv4", kv4[:3]), ("kv4", kv8),
                     ("kv8", kv4), ("cache", cache.half()), ("cache", cache[:3]),
                     ("kv_scale", kvs.double()), ("kv_scale", kvs[:2]), ("keys", keys.float()),
                     ("block_table", table.long()), ("seq_lens", lens[:1]), ("seq_lens", None)):
            if k in good:
                with pytest.raises(ValueError):
                    f(d, **dict(good, **{k: v}))
        with pytest.raises(ValueError):
            f(d, **good, new_lens=lens.long())
        with pytest.raises(ValueError):
            f(d, **good, status=torch.zeros(2, dtype=torch.int32))
        with pytest.raises(ValueError, match="CUDA device"):
            f(d, **good)  # right shapes, but in host memory


# ---------------------------------------------------------------- append
def pool(pages, seed):
    g = torch.Generator().manual_seed(seed)
    return ref.quantise(torch.randn(pages, 64, 576, generator=g).to(BF))


def run_append(rows, new_lens, table, lens, kv4, kvs, pages, pass_new=True):
    d = good_dims(batch=len(lens), num_pages=pages, max_pages_per_seq=table.shape[1])
    k, s = kv4.cuda(), kvs.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.append_fp4kv(d, rows.cuda(), k, s, table.cuda(), cuda_ints(lens),
                         cuda_ints(new_lens) if pass_new else None, status)
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
    # Every rounding is defined, ties too: bytes and scales are equal, in pages that
    # the call leaves alone too.
    table, used = tables(lens, 5)
    kv4, kvs = pool(used + 3, 6)
    g = torch.Generator().manual_seed(7)
    rows = torch.randn(len(lens), max_new, 576, generator=g)
    # Tokens of sizes from 2^-9 to 2^9, and columns too: scales that grow, blocks at
    # the end of the exponents' range, rows that are quantised again and vanish.
    rows *= torch.exp2(torch.randint(-9, 10, (len(lens), max_new, 1), generator=g).float())
    rows *= torch.exp2(torch.randint(-9, 1, (1, 1, 576), generator=g).float())
    rows = rows.to(BF)
    k, s, st = run_append(rows, new, table, lens, kv4, kvs, used + 3)
    rk, rs = ref.append(rows, new, table, lens, kv4, kvs)
    assert st == 0
    assert torch.equal(s, rs)
    assert torch.equal(k, rk)


@gpu
@pytest.mark.parametrize("kind", ["long", "many", "the last ones only"])
def test_append_of_many_pages(kind):
    lens = {"long": [30000, 41, 12123], "many": [1 + 13 * i % 151 for i in range(700)],
            "the last ones only": [0] * 515 + [70, 0, 9, 64, 4000]}[kind]
    new = [n - (i % 3) * (n // 5) if n > 3 else n for i, n in enumerate(lens)]
    table, used = tables(lens, 21)
    g = torch.Generator().manual_seed(22)
    base = torch.randn(max(new), 576, generator=g).to(BF)
    rows = torch.stack([base.roll(7 * b, 1) * 2.0 ** (b % 5) for b in range(len(lens))])
    kv4 = torch.randint(0, 256, (used, 64, 336), generator=g, dtype=torch.uint8)
    kvs = torch.exp2(torch.randint(-12, -4, (used,), generator=g).float())
    rk, rs = ref.append(rows, new, table, lens, kv4, kvs)
    k, s, st = run_append(rows, new, table, lens, kv4, kvs, used)
    assert st == 0 and torch.equal(s, rs) and ref.same(k, rk)


@gpu
def test_append_token_by_token_equals_the_definition_step_by_step():
    steps, B = 70, 3
    table, used = tables([steps + 60] * B, 8)
    kv4, kvs = pool(used, 9)
    rk, rs = kv4.clone(), kvs.clone()
    g = torch.Generator().manual_seed(10)
    for i in range(steps):
        lens = [60 + i + 1, i + 1, max(1, i)]  # the third writes its token a second time
        rows = (torch.randn(B, 1, 576, generator=g) * 2.0 ** (i % 9 - 4)).to(BF)
        kv4, kvs, st = run_append(rows, [1] * B, table, lens, kv4, kvs, used, pass_new=i % 2 == 0)
        rk, rs = ref.append(rows, [1] * B, table, lens, rk, rs)
        assert st == 0 and torch.equal(kvs, rs) and torch.equal(kv4, rk), i


@gpu
def test_append_special_values():
    rows = torch.zeros(1, 8, 576)
    rows[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 1.0])
    rows[0, 0, 16:20] = torch.tensor([math.inf, -math.inf, 1.0, 2.0 ** 33])
    rows[0, 0, 512:516] = torch.tensor([math.inf, -math.inf, math.nan, 1.0])
    rows[0, 1, 0] = 3.0e38          # beyond 448 * 2^32: saturates
    rows[0, 2, 0] = 1.0e-30         # vanishes
    rows[0, 3, 0] = 448.0 * 2.0 ** 32
    rows[0, 4, 40] = math.nan       # the second half of a block
    rows[0, 5] = -1e-38             # no normal number of fp32
    rows[0, 6] = torch.arange(576) / 64 * 2.0 ** 32
    rows[0, 7] = -torch.arange(576) / 64 * 2.0 ** 27
    rows = rows.to(BF)
    table = torch.tensor([[1]], dtype=torch.int32)
    kv4, kvs = pool(2, 11)
    k, s, st = run_append(rows, [8], table, [8], kv4, kvs, 2)
    rk, rs = ref.append(rows, [8], table, [8], kv4, kvs)
    assert st == 0 and torch.equal(s, rs) and float(s[1]) == 2.0 ** 32
    assert ref.same(k, rk)
    v = ref.decode(k[1])
    assert v[0, :16].isnan().all() and v[4, 32:48].isnan().all() and not v[4, 48:].isnan().any()
    assert v[0, 16] == 384 and v[0, 17] == -384 and v[0, 512] == 448 and v[0, 514].isnan()
    # All zeros: the smallest scale, and tokens after them raise it again.
    k, s, st = run_append(torch.zeros(1, 2, 576, dtype=BF), [2], table, [2], kv4, kvs, 2)
    assert st == 0 and float(s[1]) == 2.0 ** -32 and not k[1].any()
    one = torch.ones(1, 1, 576, dtype=BF)
    k, s, st = run_append(one, [1], table, [3], k, s, 2)
    assert st == 0 and float(s[1]) == 2.0 ** -8 and bool((ref.decode(k[1, 2]) == 256.0).all())
    # A page of bf16's smallest numbers vanishes under the smallest scale.
    tiny = torch.full((1, 1, 576), 1e-39).to(BF)
    k, s, st = run_append(tiny, [1], table, [1], kv4, kvs, 2)
    assert st == 0 and float(s[1]) == 2.0 ** -32 and not ref.decode(k[1]).any()


@gpu
@pytest.mark.parametrize("old,status", [
    (1.5 * 2.0 ** -6, 0), (0.75, 0), (1.2345678 * 2.0 ** -20, 0), (2.0 ** 32, 0), (2.0 ** -32, 0),
    (0.0, 5), (-1.0, 5), (math.nan, 5), (math.inf, 5), (2.0 ** 33, 5), (2.0 ** -33, 5)])
def test_append_to_a_page_of_any_scale(old, status):
    # A cache quantised by others (any bytes, NaN blocks among them), or never: any
    # positive scale is rounded up to a power of two, one out of range counts as 1.
    table = torch.tensor([[0, 1]], dtype=torch.int32)
    g = torch.Generator().manual_seed(16)
    kv4, kvs = torch.randint(0, 256, (2, 64, 336), generator=g, dtype=torch.uint8), torch.ones(2)
    kvs[0] = old
    rows = torch.randn(1, 30, 576, generator=g).to(BF)
    k, s, st = run_append(rows, [30], table, [50], kv4, kvs, 2)
    rk, rs = ref.append(rows, [30], table, [50], kv4, kvs)
    assert st == status and torch.equal(s, rs) and ref.same(k, rk)


@gpu
@pytest.mark.parametrize("lens,new,why", [
    ([129, 20], [1, 1], "past the table"), ([20, 20], [21, 1], "more new tokens than tokens"),
    ([20, 20], [-1, 1], "negative"), ([20, 20], [5, 1], "more than max_new"),
    ([-3, 20], [0, 1], "negative length")])
def test_append_leaves_a_bad_sequence_alone(lens, new, why):
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    kv4, kvs = pool(4, 12)
    rows = torch.randn(2, 4, 576, generator=torch.Generator().manual_seed(13)).to(BF)
    k, s, st = run_append(rows, new, table, lens, kv4, kvs, 4)
    rk, rs = ref.append(rows, [0, new[1]], table, [0, lens[1]], kv4, kvs)
    assert st == 5, why
    assert torch.equal(k, rk) and torch.equal(s, rs)


@gpu
@pytest.mark.parametrize("bad", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_append_skips_a_page_outside_the_pool(bad):
    table = torch.tensor([[0, bad], [2, 3]], dtype=torch.int32)
    kv4, kvs = pool(4, 14)
    rows = torch.randn(2, 128, 576, generator=torch.Generator().manual_seed(15)).to(BF)
    k, s, st = run_append(rows, [100, 100], table, [100, 100], kv4, kvs, 4)
    assert st == 5
    good = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    rk, rs = ref.append(rows, [100, 100], good, [100, 100], kv4, kvs)
    rk[1], rs[1] = kv4[1], kvs[1]
    assert torch.equal(k, rk) and torch.equal(s, rs)


# ---------------------------------------------------------------- reading back, page keys
def any_cache(kind, pages, seed):
    """(tensors of a cache of any bytes, what its pages stand for in fp64)."""
    g = torch.Generator().manual_seed(seed)
    if kind == "bf16":
        c = torch.randn(pages, 64, 576, generator=g).to(BF)
        return [c], c.double()
    s = torch.exp2(torch.randint(-9, 9, (pages,), generator=g).float())
    s[::5] *= 1.2345678  # by others: no power of two
    width = 576 if kind == "fp8" else 336
    kv = torch.randint(0, 256, (pages, 64, width), generator=g, dtype=torch.uint8)
    v = ref8.values(kv) if kind == "fp8" else ref.decode(kv)
    return [kv, s], v * s.double()[:, None, None]


def run_gather(kind, tensors, table, lens, new, max_new):
    d = good_dims(batch=len(lens), num_pages=tensors[0].shape[0],
                  max_pages_per_seq=table.shape[1])
    f = dict(bf16=binding.gather, fp8=binding.gather_fp8kv, fp4=binding.gather_fp4kv)[kind]
    rows = torch.full((len(lens), max_new, 576), 7.0, dtype=BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    f(d, *[t.cuda() for t in tensors], table.cuda(), cuda_ints(lens), rows,
      cuda_ints(new) if new is not None else None, status)
    return rows.cpu(), int(status.item())


GATHERS = [([1], None, 1), ([64, 65, 63, 128, 129], [1] * 5, 1),
           ([200, 64, 70, 1, 5, 0], [200, 64, 6, 1, 0, 0], 203),
           ([130, 130, 130], [130, 67, 2], 131), ([1000, 513], [999, 512], 1000),
           ([5000, 17], [4999, 17], 5000)]


@gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("lens,new,max_new", GATHERS)
def test_gather_equals_the_cache(kind, lens, new, max_new):
    table, used = tables(lens, 61)
    tensors, values = any_cache(kind, used + 2, 62)
    rows, st = run_gather(kind, tensors, table, lens, new, max_new)
    assert st == 0
    want = torch.full((len(lens), max_new, 576), 7.0, dtype=BF)
    for b, n in enumerate(new or [max_new] * len(lens)):
        pages = table[b, :(lens[b] + 63) // 64].long()
        # A product of fp32 rounded to bf16: fp64 rounded once to fp32 gives the same.
        want[b, :n] = values[pages].reshape(-1, 576)[lens[b] - n:lens[b]].float().to(BF)
    assert torch.equal(rows.isnan(), want.isnan())
    assert torch.equal(rows.nan_to_num(0.0), want.nan_to_num(0.0))


def bf16_once(x):
    """fp64 values (normal numbers of bf16, or zero) to bf16, ties to even, in one step
    (torch goes by way of fp32)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -120))) - 7)
    return (torch.round(x / step) * step).to(BF)


def scales_next_to_ties(mantissa, count):
    """Scales in [1, 2) whose product with mantissa / 8 fp32 rounds onto a tie of bf16 and,
    rounded on from there, to another value than its own nearest."""
    s = torch.arange(2 ** 23, 2 ** 24)
    p = s * mantissa
    s = s[(p.float().long() != p) & (p.float().view(torch.int32) % 2 ** 16 == 2 ** 15)].double()
    s = s * 2.0 ** -23
    x = s * (mantissa / 8)
    s = s[x.float().to(BF) != bf16_once(x)]
    assert len(s) >= count
    return s[:count].float()


@gpu
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_gather_rounds_once(kind):
    # Codes of every mantissa under scales for which one of their products is next to a tie.
    s = torch.cat([scales_next_to_ties(m, 8) for m in (range(9, 16) if kind == "fp8" else [12])])
    s = torch.cat([s, s * 2.0 ** -9, s * 2.0 ** 14])
    pages, g = len(s), torch.Generator().manual_seed(69)
    kv = torch.randint(0, 256, (pages, 64, 576 if kind == "fp8" else 336), generator=g,
                       dtype=torch.uint8)
    if kind == "fp4":
        kv[..., 256:272] &= 0x77  # no NaN blocks
        kv[..., 272:] &= 0xF7
    kv[(kv == 0x7F) | (kv == 0xFF)] = 0x3F
    values = ref8.values(kv) if kind == "fp8" else ref.decode(kv)
    exact = values * s.double()[:, None, None]
    table, lens = torch.arange(pages, dtype=torch.int32)[None], [64 * pages]
    rows, st = run_gather(kind, [kv, s], table, lens, None, lens[0])
    assert st == 0
    want = bf16_once(exact).reshape(1, -1, 576)
    assert bool((exact.float().to(BF).reshape(1, -1, 576) != want).any())
    assert torch.equal(rows, want)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_gather_reports_bad_lines_and_leaves_their_rows(kind):
    table, used = tables([130, 130], 63)
    tensors, values = any_cache(kind, used, 64)
    for lens, new in (([200, 130], [130, 130]), ([130, 130], [-1, 130]), ([130, 130], [131, 130]),
                      ([-1, 130], [0, 130]), ([20, 130], [21, 130])):
        rows, st = run_gather(kind, tensors, table, lens, new, 130)
        assert st == 5 and bool((rows[0] == 7).all()) and not bool((rows[1] == 7).all())
    for bad in (-1, used, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 1] = bad
        rows, st = run_gather(kind, tensors, t, [130, 130], None, 130)
        good, _ = run_gather(kind, tensors, table, [130, 130], None, 130)
        assert st == 5 and bool((rows[0, 64:128] == 7).all())
        for x, y in ((rows[0, :64], good[0, :64]), (rows[0, 128:], good[0, 128:]),
                     (rows[1], good[1])):
            assert torch.equal(x.nan_to_num(0.0), y.nan_to_num(0.0))
    if kind != "bf16":
        for bad in (0.0, -1.0, math.nan, math.inf, 2.0 ** 33):
            s = tensors[1].clone()
            s[int(table[0, 0])] = bad
            one = s.clone()
            one[int(table[0, 0])] = 1.0
            rows, st = run_gather(kind, [tensors[0], s], table, [130, 130], None, 130)
            want, st1 = run_gather(kind, [tensors[0], one], table, [130, 130], None, 130)
            assert st == 5 and st1 == 0
            assert torch.equal(rows.nan_to_num(0.0), want.nan_to_num(0.0))


@gpu
def test_page_keys_are_the_means_of_the_filled_rows():
    lens, new = [1, 64, 65, 200, 130, 5], [1, 64, 1, 137, 3, 0]
    table, used = tables(lens, 65)
    kv4, kvs = pool(used + 1, 66)
    kvs[0] *= 1.5
    d = good_dims(batch=len(lens), num_pages=used + 1, max_pages_per_seq=table.shape[1])
    keys = torch.full((used + 1, 576), 7.0, dtype=BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.page_keys_fp4kv(d, kv4.cuda(), kvs.cuda(), table.cuda(), cuda_ints(lens), 137, keys,
                            cuda_ints(new), status)
    assert int(status.item()) == 0
    values = ref.decode(kv4) * kvs.double()[:, None, None]
    want = torch.full((used + 1, 576), 7.0, dtype=torch.float64)
    size = torch.zeros(used + 1, 576, dtype=torch.float64)
    for b, n in enumerate(new):
        for j in range((lens[b] - n) // 64, (lens[b] + 63) // 64 if n else 0):
            p = int(table[b, j])
            filled = values[p, :lens[b] - 64 * j]
            want[p], size[p] = filled.mean(dim=0), filled.abs().mean(dim=0)
    # bf16's rounding of the mean, and fp32's of at most 64 sums and two products.
    bound = want.abs() * 2.0 ** -8 + size * 66 * 2.0 ** -24
    assert bool(((keys.cpu().double() - want).abs() <= bound).all())


# ---------------------------------------------------------------- attention
def fp4_inputs(inp):
    """The inputs' cache in 4 bits; the inputs then hold the same values in bf16."""
    kv4, kvs = ref.quantise(inp.cache.nan_to_num(0.0))
    inp.cache = (ref.decode(kv4) * kvs.double()[:, None, None]).to(BF)
    return inp, kv4, kvs


def run_fp4(inp, kv4, kvs, num_ranges=0, expect=0):
    g = inp.to(torch.device("cuda"))
    m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), num_ranges=num_ranges,
                          fp8_kv=True)
    B, T, H = g.q.shape[:3]
    out = torch.full((B, T, H, 128), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((B, T, H), float("nan"), dtype=torch.float32, device="cuda")
    m.plan(g.seq_lens)
    m.run_fp4kv(g.q, kv4.cuda(), kvs.cuda(), g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale,
                out, lse)
    assert m.check() == expect
    return out.cpu(), lse.cpu()


@gpu
@pytest.mark.parametrize("lens", [[1], [2, 63, 64, 65], [17, 80]])
def test_attention_shortest_sequences(lens):
    inp, kv4, kvs = fp4_inputs(make_inputs(len(lens), lens, 1, 16, seed=20))
    out, lse = run_fp4(inp, kv4, kvs)
    assert_parity(compare(inp, out, lse), str(lens))


@gpu
@pytest.mark.parametrize("H,T", [(16, 1), (32, 1), (64, 1), (128, 1), (16, 2), (128, 2), (48, 1),
                                 (80, 1), (96, 2), (16, 4), (128, 3), (64, 8), (112, 8)])
def test_attention_ragged_lengths_all_rows(H, T):
    lens = [max(n, T) for n in (T, 1 + T, 63, 64, 65, 127, 128, 129, 200, 511, 700)]
    inp, kv4, kvs = fp4_inputs(make_inputs(len(lens), lens, T, H, seed=100 + H + T))
    out, lse = run_fp4(inp, kv4, kvs)
    assert_parity(compare(inp, out, lse), "H=%d T=%d" % (H, T))


@gpu
@pytest.mark.parametrize("H,T,ranges", [(16, 1, 1), (16, 1, 37), (64, 2, 5), (128, 1, 150),
                                        (128, 4, 9)])
def test_attention_any_split(H, T, ranges):
    inp, kv4, kvs = fp4_inputs(make_inputs(3, [2500, 64, 900], T, H, seed=21))
    out, lse = run_fp4(inp, kv4, kvs, num_ranges=ranges)
    assert_parity(compare(inp, out, lse), "ranges %d" % ranges)


@gpu
@pytest.mark.parametrize("H,T,ranges", [(16, 1, 1), (128, 1, 1), (16, 1, 0), (128, 2, 0),
                                        (32, 8, 3)])
def test_attention_many_pieces_of_a_page_or_two(H, T, ranges):
    # Several sequences of one to three pages (with one range: all) to a CTA: query
    # tiles and pages of the next pieces enter the rings while the first are in work.
    lens = [max(T, 1 + (37 * i) % 190) for i in range(40 if ranges else 400)]
    lens[0] = T
    inp, kv4, kvs = fp4_inputs(make_inputs(len(lens), lens, T, H, seed=43))
    out, lse = run_fp4(inp, kv4, kvs, num_ranges=ranges)
    assert_parity(compare(inp, out, lse), "ranges %d" % ranges)
    out2, lse2 = run_fp4(inp, kv4, kvs, num_ranges=ranges)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("H,T,ranges", [(16, 1, 0), (128, 1, 3), (64, 2, 0), (80, 3, 2)])
def test_attention_equals_the_8_bit_cache_of_the_same_values(H, T, ranges):
    # Blocks of every exponent, values of every code, scales that are no powers of two.
    inp = make_inputs(4, [max(T, n) for n in (1, 200, 900, 65)], T, H, seed=45)
    g = torch.Generator().manual_seed(46)
    kv4 = torch.randint(0, 256, (inp.cache.shape[0], 64, 336), generator=g, dtype=torch.uint8)
    kv4[..., 256:272] = torch.randint(0, 15, kv4[..., 256:272].shape, generator=g) + \
        16 * torch.randint(0, 15, kv4[..., 256:272].shape, generator=g)
    kv4[..., 272:] %= 0x70
    kvs = torch.rand(kv4.shape[0], generator=g) * 2.0 ** -7 + 2.0 ** -8
    out, lse = run_fp4(inp, kv4, kvs, num_ranges=ranges)
    out8, lse8 = run_fp8(inp, ref.expand(kv4), kvs, num_ranges=ranges)
    assert out.isfinite().all()
    assert torch.equal(out, out8) and torch.equal(lse, lse8)


@gpu
@pytest.mark.parametrize("H,T,ranges", [(16, 1, 1), (16, 1, 0), (32, 1, 2), (128, 1, 1),
                                        (80, 2, 5), (128, 8, 1)])
def test_attention_pieces_that_end_as_the_next_query_is_due(H, T, ranges):
    # Hundreds of pieces of one page (and a few more) to a CTA: each time the warps that
    # expand pages have done their last one, the slots of the next query's tile become free.
    lens = [max(T, 64 * (1 + (i % 11 == 3) * (i % 4)) - 5 * i % 63) for i in range(300)]
    inp, kv4, kvs = fp4_inputs(make_inputs(len(lens), lens, T, H, seed=49))
    out, lse = run_fp4(inp, kv4, kvs, num_ranges=ranges)
    out8, lse8 = run_fp8(inp, ref.expand(kv4), kvs, num_ranges=ranges)
    assert torch.equal(out, out8) and torch.equal(lse, lse8)
    g = inp.to(torch.device("cuda"))
    k, s = kv4.cuda(), kvs.cuda()
    m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), num_ranges=ranges,
                          fp8_kv=True)
    m.plan(g.seq_lens)
    for _ in range(50):
        got, got_lse = torch.zeros_like(g.q[..., :128]), torch.zeros(lse.shape, device="cuda")
        m.run_fp4kv(g.q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, got, got_lse)
        assert m.check() == 0
        assert torch.equal(got.cpu(), out) and torch.equal(got_lse.cpu(), lse)


@gpu
def test_attention_repeated_runs_give_the_same_bits_while_memory_is_busy():
    inp, kv4, kvs = fp4_inputs(make_inputs(64, [4096 - 7 * i for i in range(64)], 1, 16, seed=44))
    g = inp.to(torch.device("cuda"))
    k, s = kv4.cuda(), kvs.cuda()
    m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), fp8_kv=True)
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    results = []
    for i in range(10):
        out = torch.empty(64, 1, 16, 128, dtype=BF, device="cuda")
        lse = torch.empty(64, 1, 16, device="cuda")
        big.fill_(i)
        m.plan(g.seq_lens)
        m.run_fp4kv(g.q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, out, lse)
        results.append((out, lse))
    assert m.check() == 0
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])
    assert_parity(compare(inp, results[0][0].cpu(), results[0][1].cpu()), "64 x 4096")


@gpu
def test_unused_pages_and_tail_rows_do_not_matter():
    inp, kv4, kvs = fp4_inputs(make_inputs(3, [70, 5, 200], 1, 32, seed=24, spare_pages=2))
    out, lse = run_fp4(inp, kv4, kvs)
    poisoned, scales = kv4.clone(), kvs.clone()
    poisoned[inp.used_pages:] = 0xFF
    scales[inp.used_pages:] = math.nan
    for b, n in enumerate([70, 5, 200]):  # rows past the end: the largest finite values
        tail = poisoned[int(inp.block_table[b, n // 64]), n % 64:]
        tail[:, :256], tail[:, 256:272], tail[:, 272:] = 0x77, 0xEE, 0x7E
    out2, lse2 = run_fp4(inp, poisoned, scales)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("H,T", [(16, 1), (128, 1), (64, 3)])
def test_nan_past_the_length_does_not_matter(H, T):
    lens = [T, 70, 5, 200, 127, 64]
    inp, kv4, kvs = fp4_inputs(make_inputs(len(lens), lens, T, H, seed=25))
    out, lse = run_fp4(inp, kv4, kvs)
    poisoned = kv4.clone()
    for b, n in enumerate(lens):
        if n % 64:
            poisoned[int(inp.block_table[b, n // 64]), n % 64:] = 0xFF
    out2, lse2 = run_fp4(inp, poisoned, kvs)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("where", ["block", "rope"])
def test_nan_in_a_visible_token_reaches_its_sequence_only(where):
    inp, kv4, kvs = fp4_inputs(make_inputs(3, [200, 70, 130], 1, 16, seed=47))
    out0, lse0 = run_fp4(inp, kv4, kvs)
    bad = kv4.clone()
    row = bad[int(inp.block_table[1, 0]), 11]
    row[271 if where == "block" else 300] = 0xF3 if where == "block" else 0x7F
    out, lse = run_fp4(inp, bad, kvs)
    assert out[1].isnan().all() and lse[1].isnan().all()
    for b in (0, 2):
        assert torch.equal(out[b], out0[b]) and torch.equal(lse[b], lse0[b])


@gpu
def test_bad_table_entries_and_scales_are_reported():
    inp, kv4, kvs = fp4_inputs(make_inputs(2, [100, 64], 1, 16, seed=31))
    out0, lse0 = run_fp4(inp, kv4, kvs)
    good = inp.block_table.clone()
    for bad in (-1, kv4.shape[0], 2 ** 31 - 1):
        inp.block_table = good.clone()
        inp.block_table[0, 1] = bad
        out, lse = run_fp4(inp, kv4, kvs, expect=5)
        assert torch.equal(out[1], out0[1]) and torch.equal(lse[1], lse0[1])
        assert out.isfinite().all()
    inp.block_table = good
    for bad in (0.0, -1.0, math.nan, math.inf, 2.0 ** 33):
        scales = kvs.clone()
        scales[int(good[1, 0])] = bad
        out, lse = run_fp4(inp, kv4, scales, expect=5)
        assert torch.equal(out[0], out0[0]) and torch.equal(lse[0], lse0[0])
        assert out.isfinite().all()


@gpu
def test_a_cache_beyond_two_gigabytes():
    # Pages on both sides of byte offset 2^31 and 2^32 of the pool.
    pages = (1 << 32) // (64 * 336) + 4
    inp = make_inputs(1, [64 * 4], 1, 16, seed=32)
    small, scales = ref.quantise(inp.cache[:4].nan_to_num(0.0))
    inp.cache = (ref.decode(small) * scales.double()[:, None, None]).to(BF)
    at = [0, (1 << 31) // (64 * 336), (1 << 32) // (64 * 336), pages - 1]
    kv4 = torch.zeros(pages, 64, 336, dtype=torch.uint8, device="cuda")
    kvs = torch.ones(pages, device="cuda")
    t = torch.tensor([at], dtype=torch.int32)
    order = [int(p) for p in inp.block_table[0, :4]]
    kv4[torch.tensor(at)] = small[order].cuda()
    kvs[torch.tensor(at)] = scales[order].cuda()
    d = good_dims(batch=1, num_pages=pages, max_pages_per_seq=4)
    rows = torch.zeros(1, 256, 576, dtype=BF, device="cuda")
    binding.gather_fp4kv(d, kv4, kvs, t.cuda(), cuda_ints([256]), rows)
    assert torch.equal(rows.cpu()[0], inp.cache[order].reshape(256, 576))
    g = inp.to(torch.device("cuda"))
    m = binding.MlaDecode(d, fp8_kv=True)
    out = torch.empty(1, 1, 16, 128, dtype=BF, device="cuda")
    lse = torch.empty(1, 1, 16, device="cuda")
    m.plan(g.seq_lens)
    m.run_fp4kv(g.q, kv4, kvs, t.cuda(), g.seq_lens, g.w_uk, g.w_uv, g.scale, out, lse)
    assert m.check() == 0
    assert_parity(compare(inp, out.cpu(), lse.cpu()), "far pages")
    new = rows[:, -70:].contiguous()
    kv4[at[2]], kv4[at[3]] = 0, 0
    binding.append_fp4kv(d, new, kv4, kvs, t.cuda(), cuda_ints([256]))
    binding.gather_fp4kv(d, kv4, kvs, t.cuda(), cuda_ints([256]), rows[:, :64].contiguous())
    assert torch.equal(ref.decode(kv4[at[3]].cpu()) * float(kvs[at[3]]),
                       inp.cache[order[3]].double())


@gpu
def test_append_to_pages_beyond_two_gigabytes_equals_the_definition():
    # Pages on both sides of byte offset 2^31 and 2^32 of the pool; 70 new tokens in the last
    # two of them: six rows behind 58 that stay, and a page that starts afresh.
    pages = (1 << 32) // (64 * 336) + 4
    at = [0, (1 << 31) // (64 * 336), (1 << 32) // (64 * 336), pages - 1]
    kv4, kvs = pool(4, 17)
    rows = (torch.randn(1, 70, 576, generator=torch.Generator().manual_seed(18)) * 64).to(BF)
    far, far_s = torch.zeros(pages, 64, 336, dtype=torch.uint8, device="cuda"), torch.ones(pages)
    where = torch.tensor(at)
    far[where], far_s[where] = kv4.cuda(), kvs
    far_s = far_s.cuda()
    d = good_dims(batch=1, num_pages=pages, max_pages_per_seq=4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.tensor([at], dtype=torch.int32).cuda()
    binding.append_fp4kv(d, rows.cuda(), far, far_s, table, cuda_ints([256]), status=status)
    near = torch.arange(4, dtype=torch.int32)[None]
    rk, rs = ref.append(rows, [70], near, [256], kv4, kvs)
    assert int(status.item()) == 0
    assert torch.equal(far[where].cpu(), rk) and torch.equal(far_s[where].cpu(), rs)
    # Nothing else was written, and what was is read back.
    assert int(far.any(dim=2).any(dim=1).sum()) == 4
    assert int((far_s != 1).sum()) == int((rs != 1).sum())
    got = torch.full((1, 256, 576), 7.0, dtype=BF, device="cuda")
    binding.gather_fp4kv(d, far, far_s, table, cuda_ints([256]), got)
    want = (ref.decode(rk) * rs.double()[:, None, None]).to(BF)
    assert torch.equal(got.cpu().view(4, 64, 576), want)


@gpu
def test_one_plan_serves_every_cache_and_the_steps_equal_the_run():
    inp, kv4, kvs = fp4_inputs(make_inputs(4, [700, 64, 65, 300], 2, 32, seed=33))
    g = inp.to(torch.device("cuda"))
    k, s = kv4.cuda(), kvs.cuda()
    for fp8_kv in (True, False):  # a plan of either balance
        m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), fp8_kv=fp8_kv)
        (o1, l1), (o2, l2), (o3, l3) = [(torch.empty(4, 2, 32, 128, dtype=BF, device="cuda"),
                                         torch.empty(4, 2, 32, device="cuda")) for _ in range(3)]
        m.plan(g.seq_lens)
        m.run(g.q, g.cache, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, o1, l1)
        m.run_fp4kv(g.q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, o2, l2)
        m.absorb(g.q, g.w_uk)
        m.attend_fp4kv(k, s, g.block_table, g.seq_lens, g.scale, l3)
        m.combine(g.scale, l3)
        m.up_project(g.w_uv, o3)
        assert m.check() == 0
        assert torch.equal(o2, o3) and torch.equal(l2, l3)
        # The bf16 cache holds the same values: the two parity bounds together.
        assert float((o1.float() - o2.float()).abs().max()) <= 2e-2 + ref8.OUT_MAX
        assert float((l1 - l2).abs().max()) <= 2e-3


@gpu
@pytest.mark.parametrize("B,H,ranges", [(24, 16, 1), (24, 128, 1), (160, 16, 2), (40, 64, 0)])
def test_runs_of_other_queries_back_to_back_on_one_plan(B, H, ranges):
    lens = [500 + 37 * i % 300 for i in range(B)]
    inp, kv4, kvs = fp4_inputs(make_inputs(B, lens, 1, H, seed=80))
    g = inp.to(torch.device("cuda"))
    k, s = kv4.cuda(), kvs.cuda()
    m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), num_ranges=ranges,
                          fp8_kv=True)
    gen = torch.Generator().manual_seed(81)
    queries = [torch.randn(B, 1, H, 192, generator=gen).to(BF).cuda() for _ in range(4)]
    alone, together = [[(torch.zeros(B, 1, H, 128, dtype=BF, device="cuda"),
                         torch.zeros(B, 1, H, device="cuda")) for _ in queries] for _ in range(2)]

    def run(q, out, lse):
        m.run_fp4kv(q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, out, lse)

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
@pytest.mark.parametrize("H,T,ranges", [(16, 1, 1), (16, 1, 3), (128, 1, 1), (80, 1, 2)])
def test_a_maximum_that_rises_with_every_page_of_many_pieces(H, T, ranges):
    # Scores that grow by more than the lazy maximum's slack from page to page: every
    # page but a piece's first rescales the output, while the next pieces' pages are
    # expanded and their query tiles take the slots that become free.
    lens = [64 * (3 + i % 4) - i % 7 for i in range(48)]
    inp = make_inputs(len(lens), lens, T, H, seed=82)
    inp.q[..., :128] = 0.0
    inp.q[..., 128:] = 1.0
    inp.cache[..., 512:] = 0.0
    for b, n in enumerate(lens):
        for j in range((n + 63) // 64):
            # 64 products of 2 j, times 1 / sqrt(192): 9.2 a page, 8 ln 2 = 5.5.
            inp.cache[int(inp.block_table[b, j]), :, 512:] = 2.0 * j
    inp, kv4, kvs = fp4_inputs(inp)
    out, lse = run_fp4(inp, kv4, kvs, num_ranges=ranges)
    assert_parity(compare(inp, out, lse), "ranges %d" % ranges)
    for _ in range(20):
        out2, lse2 = run_fp4(inp, kv4, kvs, num_ranges=ranges)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("low,high", [(-12, 2), (-30, 0)])
def test_pages_of_very_different_scales(low, high):
    inp = make_inputs(3, [1000, 130, 640], 1, 32, seed=27)
    g = torch.Generator().manual_seed(28)
    e = torch.randint(low, high + 1, (inp.cache.shape[0],), generator=g)
    inp.cache = (inp.cache.float() * torch.exp2(e.float())[:, None, None]).to(BF)
    inp.scale = inp.scale / 2.0 ** max(0, high)
    inp, kv4, kvs = fp4_inputs(inp)
    out, lse = run_fp4(inp, kv4, kvs)
    s = compare(inp, out, lse)
    # Values up to 2^high: the outputs' bounds grow with them.
    assert s["out_max"] <= ref8.OUT_MAX * 2.0 ** max(0, high) and s["lse_max"] <= 1e-3, s


@gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_gives_nan(value):
    for H, num_ranges, lens in ((16, 0, [2, 130, 90]), (128, 2, [700, 900, 64])):
        inp, kv4, kvs = fp4_inputs(make_inputs(3, lens, 2, H, seed=48))
        out0, lse0 = run_fp4(inp, kv4, kvs, num_ranges=num_ranges)
        inp.q[:, 1, 3, 5] = value
        inp.q[:, 0, H - 1, 140] = value
        out, lse = run_fp4(inp, kv4, kvs, num_ranges=num_ranges)
        changed = torch.zeros_like(lse, dtype=torch.bool)
        changed[:, 1, 3] = changed[:, 0, H - 1] = True
        assert out[changed].isnan().all() and lse[changed].isnan().all()
        assert torch.equal(out[~changed], out0[~changed])
        assert torch.equal(lse[~changed], lse0[~changed])


@gpu
def test_lengths_out_of_range_are_clamped_and_reported():
    inp, kv4, kvs = fp4_inputs(make_inputs(2, [100, 64], 1, 16, seed=32))
    out0, lse0 = run_fp4(inp, kv4, kvs)
    inp.seq_lens = torch.tensor([100, 0], dtype=torch.int32)
    out, lse = run_fp4(inp, kv4, kvs, expect=5)
    assert torch.equal(out[0], out0[0]) and torch.equal(lse[0], lse0[0])


@gpu
def test_two_calls_at_once_on_two_streams():
    # Attention on one stream, appends, keys and reading back of other caches on others.
    cases = []
    for seed in (38, 39):
        inp, kv4, kvs = fp4_inputs(make_inputs(6, [900, 64, 65, 300, 1, 511], 1, 64, seed=seed))
        cases.append((inp, kv4, kvs, *run_fp4(inp, kv4, kvs)))
    dev = torch.device("cuda")
    live = []
    for inp, kv4, kvs, _, _ in cases:
        g = inp.to(dev)
        m = binding.MlaDecode(binding.dims_for(g.q, g.cache, g.block_table), fp8_kv=True)
        live.append((g, kv4.cuda(), kvs.cuda(), m, torch.empty(6, 1, 64, 128, dtype=BF, device=dev),
                     torch.empty(6, 1, 64, device=dev), torch.cuda.Stream(),
                     torch.zeros(6, 900, 576, dtype=BF, device=dev),
                     torch.zeros(kv4.shape[0], 576, dtype=BF, device=dev)))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, k, s, m, out, lse, st, rows, keys in live:
            with torch.cuda.stream(st):
                binding.gather_fp4kv(m.dims, k, s, g.block_table, g.seq_lens, rows, g.seq_lens)
                binding.append_fp4kv(m.dims, rows, k, s, g.block_table, g.seq_lens, g.seq_lens)
                binding.page_keys_fp4kv(m.dims, k, s, g.block_table, g.seq_lens, 900, keys,
                                        g.seq_lens)
                m.plan(g.seq_lens)
                m.run_fp4kv(g.q, k, s, g.block_table, g.seq_lens, g.w_uk, g.w_uv, g.scale, out,
                            lse)
    torch.cuda.synchronize()
    for (inp, kv4, kvs, out0, lse0), (_, k, s, m, out, lse, _, _, _) in zip(cases, live):
        assert m.check() == 0
        # What is read back and appended again keeps its values, whatever the page's scale
        # becomes (it may shrink with the largest value's rounding).
        v = ref.decode(k.cpu()) * s.cpu().double()[:, None, None]
        w = ref.decode(kv4) * kvs.double()[:, None, None]
        for b, n in enumerate(inp.seq_lens.tolist()):
            pages = inp.block_table[b, :(n + 63) // 64].long()
            assert torch.equal(v[pages].reshape(-1, 576)[:n], w[pages].reshape(-1, 576)[:n])
        s2 = compare(inp, out.cpu(), lse.cpu())
        assert_parity(s2, "two streams")


@gpu
@pytest.mark.parametrize("kind", ["fp4", "fp8", "bf16"])
@pytest.mark.parametrize("B,max_new", [(256, 65), (3, 200), (256, 300), (257, 300), (255, 200)])
def test_gather_and_keys_with_and_without_a_list(kind, B, max_new):
    # The page keys of up to 256 sequences with many pages go by a list of them.
    lens = [(37 * i) % (max_new + 30) for i in range(B)]
    new = [min(n, max_new) - (i % 3 == 0 and n > 0) for i, n in enumerate(lens)]
    table, used = tables(lens, 67)
    tensors, values = any_cache(kind, used + 1, 68)
    if kind != "bf16":  # finite ones, for the means
        if kind == "fp8":
            tensors[0] %= 0x70
            values = ref8.values(tensors[0]) * tensors[1].double()[:, None, None]
        else:
            tensors[0][..., 256:272] &= 0x77
            tensors[0][..., 272:] %= 0x70
            values = ref.decode(tensors[0]) * tensors[1].double()[:, None, None]
    rows, st = run_gather(kind, tensors, table, lens, new, max_new)
    assert st == 0
    want = torch.full((B, max_new, 576), 7.0, dtype=BF)
    keys, size = torch.full((2, used + 1, 576), 7.0, dtype=torch.float64)
    for b, n in enumerate(new):
        if n == 0:
            continue
        pages = table[b, :(lens[b] + 63) // 64].long()
        want[b, :n] = values[pages].reshape(-1, 576)[lens[b] - n:lens[b]].float().to(BF)
        for j in range((lens[b] - n) // 64, len(pages)):
            filled = values[pages[j], :lens[b] - 64 * j]
            keys[pages[j]], size[pages[j]] = filled.mean(dim=0), filled.abs().mean(dim=0)
    assert torch.equal(rows, want)
    d = good_dims(batch=B, num_pages=used + 1, max_pages_per_seq=table.shape[1])
    f = dict(bf16=binding.page_keys, fp8=binding.page_keys_fp8kv, fp4=binding.page_keys_fp4kv)[kind]
    got = torch.full((used + 1, 576), 7.0, dtype=BF, device="cuda")
    f(d, *[t.cuda() for t in tensors], table.cuda(), cuda_ints(lens), max_new, got, cuda_ints(new))
    # As in test_page_keys_are_the_means_of_the_filled_rows.
    bound = keys.abs() * 2.0 ** -8 + size * 66 * 2.0 ** -24
    assert bool(((got.cpu().double() - keys).abs() <= bound).all())


def test_run_and_attend_check_every_tensor(monkeypatch):
    # (In host memory: a call whose tensors are right is refused for that alone.)
    monkeypatch.setattr(binding, "workspace_size", lambda d, ranges=0: 4096)
    B, T, H = 2, 2, 16
    m = binding.MlaDecode(good_dims(q_len=T), device=torch.device("cpu"))
    good = dict(q=torch.zeros(B, T, H, 192, dtype=BF),
                kv4=torch.zeros(4, 64, 336, dtype=torch.uint8), kv_scale=torch.ones(4),
                block_table=torch.zeros(B, 2, dtype=torch.int32),
                seq_lens=torch.ones(B, dtype=torch.int32),
                w_uk=torch.zeros(H, 128, 512, dtype=BF), w_uv=torch.zeros(H, 512, 128, dtype=BF),
                out=torch.zeros(B, T, H, 128, dtype=BF), lse=torch.zeros(B, T, H))
    attend = ("kv4", "kv_scale", "block_table", "seq_lens", "lse")

    def refused(name, **change):
        a = dict(good, **change)
        with pytest.raises(ValueError, match="^%s: " % name):
            m.run_fp4kv(scale=0.07, **a)
        if name in attend:
            with pytest.raises(ValueError, match="^%s: " % name):
                m.attend_fp4kv(scale=0.07, **{k: a[k] for k in attend})

    for name, t in good.items():
        refused(name, **{name: None})
        refused(name, **{name: t.double()})                          # another type
        refused(name, **{name: t[:-1]})                              # too short
        refused(name, **{name: torch.cat([t, t])[::2]})              # strided
    refused("kv4", kv4=torch.zeros(4, 64, 576, dtype=torch.uint8))   # the 8-bit cache
    with pytest.raises(ValueError, match="^kv4: .*CUDA device"):
        m.run_fp4kv(scale=0.07, **good)
    with pytest.raises(ValueError, match="^kv4: .*CUDA device"):
        m.attend_fp4kv(scale=0.07, **{k: good[k] for k in attend})
