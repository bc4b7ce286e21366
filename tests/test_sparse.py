"""Block-sparse decode: page keys, scores, selection, and the decode on them."""
import ctypes
import math
import threading

import pytest
import torch

import fp8kv_util as ref
import oracle
from mla_decode_attention_uk_gb300 import binding
from mla_decode_attention_uk_gb300.inputs import make_inputs

gpu = pytest.mark.gpu
BF = torch.bfloat16
OK, ODD2, ODD8 = ctypes.c_void_p(4096), ctypes.c_void_p(4098), ctypes.c_void_p(4104)


def dims(B, T=1, H=16, pages=4, width=2):
    return binding.Dims(B, T, H, 128, 64, 512, 128, 64, pages, width)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


# ---------------------------------------------------------------- refusals (no GPU)
def test_refusals():
    L = binding.lib()
    d = ctypes.byref(dims(2))
    bad = ctypes.byref(binding.Dims(2, 1, 16, 128, 64, 256, 128, 64, 4, 2))
    cases = {
        # cache table lens max_new new_lens keys status stream
        "mla_decode_page_keys": ([OK, OK, OK, 1, OK, OK, OK, None],
                                 [{0: None}, {0: ODD8}, {1: None}, {1: ODD2}, {2: None}, {2: ODD2},
                                  {3: 0}, {3: 2 ** 31 - 1}, {4: ODD2}, {5: None}, {5: ODD8},
                                  {6: ODD2}]),
        # kv8 scale table lens max_new new_lens keys status stream
        "mla_decode_page_keys_fp8kv": ([OK, OK, OK, OK, 1, OK, OK, OK, None],
                                       [{0: None}, {0: ODD8}, {1: None}, {1: ODD2}, {2: None},
                                        {3: None}, {4: -1}, {6: None}, {7: ODD2}]),
        # query keys table lens scores status stream
        "mla_decode_score_pages": ([OK, OK, OK, OK, OK, OK, None],
                                   [{0: None}, {0: ODD8}, {1: None}, {1: ODD8}, {2: None},
                                    {2: ODD2}, {3: None}, {3: ODD2}, {4: None}, {4: ODD2},
                                    {5: ODD2}]),
        # scores table lens top_k first last sel_table sel_pages sel_lens status stream
        "mla_decode_select_pages": ([OK, OK, OK, 4, 1, 1, OK, OK, OK, OK, None],
                                    [{0: None}, {0: ODD2}, {1: None}, {2: None}, {3: 0}, {3: 1},
                                     {3: -2 ** 31}, {3: 2 ** 31 - 1}, {4: -1}, {4: 4}, {5: 0},
                                     {5: -1}, {5: 4}, {4: 2 ** 31 - 1}, {6: None}, {6: ODD2},
                                     {7: ODD2}, {8: None}, {8: ODD2}, {9: ODD2}]),
    }
    for name, (args, changes) in cases.items():
        fn = getattr(L, name)
        for change in changes:
            a = list(args)
            for i, v in change.items():
                a[i] = v
            assert fn(d, *a) == 1, (name, change)
        assert fn(bad, *args) == 2, name
        assert fn(None, *args) == 1, name


def test_python_calls_check_types_and_shapes():
    d = dims(2, T=2)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), i32([2, 2])
    q, keys = torch.zeros(2, 2, 16, 576, dtype=BF), torch.zeros(4, 576, dtype=BF)
    scores = torch.zeros(2, 2, 2)
    sel, sl = torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.score_pages(d, q[:, :1], keys, table, lens, scores)
    with pytest.raises(ValueError):
        binding.score_pages(d, q, keys.float(), table, lens, scores)
    with pytest.raises(ValueError):
        binding.score_pages(d, q, keys, table, lens, scores[:, :, :1])
    with pytest.raises(ValueError):
        binding.select_pages(d, scores, table, lens, 4, 1, 1, sel, sl)
    with pytest.raises(ValueError):
        binding.select_pages(d, scores, table, lens, 3, 1, 1, sel, sl[:2])
    with pytest.raises(ValueError):
        binding.select_pages(d, scores, table, lens, 3, 1, 1, sel, sl, sel_pages=sel.long())
    with pytest.raises(ValueError):
        binding.page_keys(d, torch.zeros(4, 64, 576), table, lens, 1, keys)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.score_pages(d, q, keys, table, lens, scores)  # in host memory
    with pytest.raises(ValueError):
        binding.page_keys_fp8kv(d, torch.zeros(4, 64, 576, dtype=torch.uint8), torch.ones(3),
                                table, lens, 1, keys)


# ---------------------------------------------------------------- page keys
@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,new,max_new", [
    ([1], [1], 1), ([64, 65, 63, 128], [1, 1, 1, 1], 1), ([0, 200, 130], [0, 200, 67], 200),
    ([500, 77, 64], [3, 77, 0], 100)])
def test_page_keys_are_the_mean_rows(fp8, lens, new, max_new):
    inp = make_inputs(len(lens), lens, 1, 16, seed=50, spare_pages=1)
    pages, width = inp.cache.shape[0], inp.block_table.shape[1]
    cache = inp.cache.nan_to_num(0.0)
    kv8, kvs = ref.quantise(cache)
    keys = torch.full((pages, 576), 7.0, dtype=BF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = keys.cuda()
    d = dims(len(lens), pages=pages, width=width)
    args = (inp.block_table.cuda(), i32(lens).cuda(), max_new, k, i32(new).cuda(), status)
    if fp8:
        binding.page_keys_fp8kv(d, kv8.cuda(), kvs.cuda(), *args)
        cache = ref.values(kv8) * kvs.double()[:, None, None]
    else:
        binding.page_keys(d, cache.cuda(), *args)
    assert int(status.item()) == 0
    want = keys.double()
    for b, n in enumerate(new):
        for j in range((lens[b] - n) // 64, (lens[b] + 63) // 64 if n else 0):
            p = int(inp.block_table[b, j])
            want[p] = cache[p, :min(64, lens[b] - j * 64)].double().mean(dim=0)
    # fp32 sums of up to 64 values below 6 (2^-24 each, of partial sums up to
    # 64), then one rounding to bf16.
    err = (k.cpu().double() - want).abs()
    assert (err <= want.abs() * 2.0 ** -8 + 64 * 6 * 2.0 ** -24).all()


@gpu
@pytest.mark.parametrize("lens,new", [([129, 20], [1, 1]), ([20, 20], [21, 1]), ([20, 20], [-1, 1]),
                                      ([-5, 20], [0, 1])])
def test_page_keys_leave_a_bad_sequence_alone(lens, new):
    cache = torch.randn(4, 64, 576, generator=torch.Generator().manual_seed(51)).to(BF)
    table = i32([[0, 1], [2, -7]])
    keys = torch.zeros(4, 576, dtype=BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.page_keys(dims(2), cache.cuda(), table.cuda(), i32(lens).cuda(), 1, keys,
                      i32(new).cuda(), status)
    assert int(status.item()) == 5
    assert not keys[[0, 1, 3]].any() and bool(keys[2].any())
    status.zero_()
    keys.zero_()
    binding.page_keys(dims(2), cache.cuda(), table.cuda(), i32([5, 70]).cuda(), 1, keys, None,
                      status)  # the second sequence's page is not in the pool
    assert int(status.item()) == 5 and not keys[1:].any() and bool(keys[0].any())


@gpu
@pytest.mark.parametrize("scale", [0.0, -2.0, math.nan, math.inf, 2.0 ** 33, 2.0 ** -33])
def test_page_keys_of_a_page_with_a_bad_scale(scale):
    # Taken as 1 and reported, as the attention does.
    kv8, kvs = ref.quantise(torch.randn(2, 64, 576, generator=torch.Generator().manual_seed(56)))
    args = (i32([[0, 1]]).cuda(), i32([100]).cuda(), 100)
    got, status = [], []
    for first in (scale, 1.0):
        kvs[0] = first
        got.append(torch.zeros(2, 576, dtype=BF, device="cuda"))
        status.append(torch.zeros(1, dtype=torch.int32, device="cuda"))
        binding.page_keys_fp8kv(dims(1, pages=2, width=2), kv8.cuda(), kvs.cuda(), *args, got[-1],
                                None, status[-1])
    assert [int(x.item()) for x in status] == [5, 0]
    assert torch.equal(got[0], got[1]) and bool(got[0][0].any())


# ---------------------------------------------------------------- scores
@gpu
@pytest.mark.parametrize("B,T,H,lens,width", [
    (1, 1, 16, [1], 1), (3, 1, 16, [64, 65, 4000], 70), (2, 2, 48, [130, 8200], 129),
    (4, 8, 128, [8, 71, 4095, 1000], 64), (2, 3, 112, [3, 12000], 200)])
def test_scores_are_the_largest_head_product(B, T, H, lens, width):
    g = torch.Generator().manual_seed(52)
    pages = sum((n + 63) // 64 for n in lens) + 1
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = (n + 63) // 64
        table[b, :m] = perm[at:at + m]
        at += m
    q = torch.randn(B, T, H, 576, generator=g).to(BF)
    keys = (torch.randn(pages, 576, generator=g) * 0.3).to(BF)
    keys[perm[-1].item()] = math.nan  # in no sequence
    scores = torch.full((B, T, width), 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.score_pages(dims(B, T, H, pages, width), q.cuda(), keys.cuda(), table.cuda(),
                        i32(lens).cuda(), scores, status)
    assert int(status.item()) == 0
    got = scores.cpu().double()
    for b in range(B):
        for t in range(T):
            n = (lens[b] - T + t + 64) // 64
            assert (got[b, t, n:] == -math.inf).all()
            k = keys[table[b, :n].long()].double()
            want = (q[b, t].double() @ k.T).max(dim=0).values
            # 576 exact products summed in fp32: at most 2^-23 a step of sums
            # that stay below sum |q| |k| (about 0.2 * 576); 2^-14 is four
            # times that.
            assert ((got[b, t, :n] - want).abs() <= 2.0 ** -14 * 4).all()


@gpu
def test_scores_with_bad_lengths_pages_and_nan():
    q = torch.randn(2, 1, 16, 576, generator=torch.Generator().manual_seed(53)).to(BF)
    keys = torch.randn(4, 576, generator=torch.Generator().manual_seed(54)).to(BF)
    table = i32([[0, 1], [2, 9]])
    scores = torch.empty(2, 1, 2, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.score_pages(dims(2), q.cuda(), keys.cuda(), table.cuda(), i32([100, 100]).cuda(),
                        scores, status)
    assert int(status.item()) == 5 and scores.isfinite().all()
    status.zero_()
    binding.score_pages(dims(2), q.cuda(), keys.cuda(), i32([[0, 1], [2, 3]]).cuda(),
                        i32([0, 500]).cuda(), scores, status)
    assert int(status.item()) == 5
    assert scores[0, 0, 1] == -math.inf and scores[1].isfinite().all()
    q[0, 0, 3] = math.nan  # one head's products count as -infinity
    q[1] = math.nan
    binding.score_pages(dims(2), q.cuda(), keys.cuda(), i32([[0, 1], [2, 3]]).cuda(),
                        i32([128, 128]).cuda(), scores, None)
    want = (q[0, 0, [h for h in range(16) if h != 3]].double() @ keys[:2].double().T).amax(0)
    assert (scores[0, 0].cpu().double() - want).abs().max() <= 1e-3
    assert (scores[1] == -math.inf).all()


# ---------------------------------------------------------------- selection
def run_select(scores, table, lens, T, top_k, first, last, status=None, pages_out=True):
    B, _, width = scores.shape
    d = dims(B, T, 16, int(table.max()) + 1, width)
    st = torch.full((B * T, top_k), 77, dtype=torch.int32, device="cuda")
    sp = torch.full((B * T, top_k), 77, dtype=torch.int32, device="cuda")
    sl = torch.full((B * T,), 77, dtype=torch.int32, device="cuda")
    binding.select_pages(d, scores.cuda(), table.cuda(), i32(lens).cuda(), top_k, first, last, st,
                         sl, sel_pages=sp if pages_out else None, status=status)
    return st.cpu(), sp.cpu(), sl.cpu()


def table_of(B, width, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(B * width, generator=g).to(torch.int32).view(B, width)


@gpu
@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "special"])
@pytest.mark.parametrize("lens,T,width,top_k,first,last", [
    ([1], 1, 1, 1, 0, 1), ([64, 65, 640], 1, 10, 3, 1, 1), ([640, 641, 63], 2, 11, 2, 1, 1),
    ([9000, 8, 16384], 8, 256, 16, 0, 1), ([16383, 5000, 20000], 3, 313, 33, 2, 3),
    ([64 * 1500, 64 * 257 + 1], 1, 1500, 300, 1, 2), ([40000], 1, 700, 699, 0, 1),
    ([128, 100], 1, 2, 5, 2, 3),
    ([64 * 2048, 64 * 2049, 64 * 5000 - 1], 1, 5000, 70, 1, 1)])  # keys that do not fit the CTA
def test_selection_equals_the_definition(kind, lens, T, width, top_k, first, last):
    g = torch.Generator().manual_seed(55)
    B = len(lens)
    s = torch.randn(B, T, width, generator=g) * 5
    if kind == "ties":
        s = s.round()
        s[s == 0] *= torch.where(torch.rand(s[s == 0].shape, generator=g) < 0.5, -1.0, 1.0)
    elif kind == "equal":
        s.fill_(-2.5)
    elif kind == "special":
        pick = torch.randint(0, 5, s.shape, generator=g)
        for i, v in enumerate((math.nan, math.inf, -math.inf, 3.4e38, 1e-45)):
            s[pick == i] = torch.where(torch.rand(s[pick == i].shape, generator=g) < 0.7,
                                       torch.tensor(v), s[pick == i])
    table = table_of(B, width, 56)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st, sp, sl = run_select(s, table, lens, T, top_k, first, last, status)
    rt, rp, rl = ref.select(s, table, lens, T, top_k, first, last)
    assert int(status.item()) == 0
    assert torch.equal(sp, rp)
    assert torch.equal(st, rt)
    assert torch.equal(sl, rl)
    st2, sp2, sl2 = run_select(s, table, lens, T, top_k, first, last, pages_out=False)
    assert torch.equal(st2, rt) and torch.equal(sl2, rl) and (sp2 == 77).all()


@gpu
def test_selection_clamps_and_reports_bad_lengths():
    s = torch.randn(2, 1, 6, generator=torch.Generator().manual_seed(57))
    table = table_of(2, 6, 58)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st, sp, sl = run_select(s, table, [0, 1000], 1, 3, 1, 1, status)
    rt, rp, rl = ref.select(s, table, [1, 384], 1, 3, 1, 1)
    assert int(status.item()) == 5
    assert torch.equal(st, rt) and torch.equal(sp, rp) and torch.equal(sl, rl)


# ---------------------------------------------------------------- together
def expected(q, cache, w_uk, w_uv, scale, table, lens):
    o, l, _ = oracle.decode(q, cache, table, lens, w_uk, w_uv, scale)
    return torch.from_numpy(o).view(*q.shape[:3], 128), torch.from_numpy(l).view(*q.shape[:3])


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H", [(1, 16), (2, 64), (3, 128)])
def test_append_score_select_and_decode_together(fp8, T, H):
    B, top_k = 4, 6
    lens = [2000, 64 + T, T, 1100]
    inp = make_inputs(B, lens, T, H, seed=60 + H)
    pages, width = inp.cache.shape[0], inp.block_table.shape[1]
    g = inp.to(torch.device("cuda"))
    d = binding.Dims(B, T, H, 128, 64, 512, 128, 64, pages, width)
    keys = torch.zeros(pages, 576, dtype=BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    max_len = max(lens)
    if fp8:
        kv8 = torch.full((pages, 64, 576), 0x7F, dtype=torch.uint8, device="cuda")
        kvs = torch.full((pages,), math.nan, device="cuda")
        rows = torch.zeros(B, max_len, 576, dtype=BF)
        for b, n in enumerate(lens):
            flat = inp.cache[inp.block_table[b, :(n + 63) // 64].long()].view(-1, 576)
            rows[b, :n] = flat[:n]
        binding.append_fp8kv(d, rows.cuda(), kv8, kvs, g.block_table, g.seq_lens, g.seq_lens,
                             status)
        binding.page_keys_fp8kv(d, kv8, kvs, g.block_table, g.seq_lens, max_len, keys, g.seq_lens,
                                status)
        cache = (ref.values(kv8.cpu()) * kvs.cpu().double()[:, None, None]).to(BF)
    else:
        binding.page_keys(d, g.cache, g.block_table, g.seq_lens, max_len, keys, g.seq_lens,
                          status)
        cache = inp.cache
    ds = binding.Dims(B * T, 1, H, 128, 64, 512, 128, 64, pages, top_k)
    m = binding.MlaDecode(ds, fp8_kv=fp8)
    scores = torch.empty(B, T, width, device="cuda")
    st = torch.empty(B * T, top_k, dtype=torch.int32, device="cuda")
    sl = torch.empty(B * T, dtype=torch.int32, device="cuda")
    out = torch.empty(B * T, 1, H, 128, dtype=BF, device="cuda")
    lse = torch.empty(B * T, 1, H, device="cuda")
    m.absorb(g.q.view(B * T, 1, H, 192), g.w_uk)
    q_lat = m.q_lat().view(B, T, H, 576)
    binding.score_pages(d, q_lat, keys, g.block_table, g.seq_lens, scores, status)
    binding.select_pages(d, scores, g.block_table, g.seq_lens, top_k, 1, 1, st, sl, None, status)
    m.plan(sl)
    args = (st, sl, g.w_uk, g.w_uv, g.scale, out, lse)
    if fp8:
        m.run_fp8kv(g.q, kv8, kvs, *args)
    else:
        m.run(g.q, g.cache, *args)
    assert m.check() == 0 and int(status.item()) == 0
    rt, _, rl = ref.select(scores.cpu(), inp.block_table, lens, T, top_k, 1, 1)
    assert torch.equal(st.cpu(), rt) and torch.equal(sl.cpu(), rl)
    o, l = expected(inp.q.view(B * T, 1, H, 192), cache, inp.w_uk, inp.w_uv, inp.scale, rt, rl)
    err = (out.cpu().double() - o).abs()
    assert err.max() <= ref.OUT_MAX and err.mean() <= ref.OUT_MEAN
    assert (lse.cpu().double() - l).abs().max() <= 1e-3
    # Sequences whose pages are all selected attend to everything.
    full, full_lse = expected(inp.q, cache, inp.w_uk, inp.w_uv, inp.scale, inp.block_table,
                              inp.seq_lens)
    for b in (1, 2):
        assert (out.view(B, T, H, 128)[b].cpu().double() - full[b]).abs().max() <= ref.OUT_MAX


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H", [(1, 16), (2, 128)])
def test_one_absorb_serves_scores_and_attention(fp8, T, H):
    # absorb, scores, selection, plan, attention and the rest: bit for bit a run's
    # results, which absorbs for itself.
    B, top_k, lens = 3, 5, [900, 64 + T, 1500]
    inp = make_inputs(B, lens, T, H, seed=65)
    pages, width = inp.cache.shape[0], inp.block_table.shape[1]
    g = inp.to(torch.device("cuda"))
    d = binding.Dims(B, T, H, 128, 64, 512, 128, 64, pages, width)
    keys = torch.zeros(pages, 576, dtype=BF, device="cuda")
    kv8, kvs = (x.cuda() for x in ref.quantise(inp.cache.nan_to_num(0.0)))
    binding.page_keys_fp8kv(d, kv8, kvs, g.block_table, g.seq_lens, max(lens), keys, g.seq_lens)
    m = binding.MlaDecode(binding.Dims(B * T, 1, H, 128, 64, 512, 128, 64, pages, top_k),
                          fp8_kv=fp8)
    scores = torch.empty(B, T, width, device="cuda")
    st = torch.empty(B * T, top_k, dtype=torch.int32, device="cuda")
    sl = torch.empty(B * T, dtype=torch.int32, device="cuda")
    q = g.q.view(B * T, 1, H, 192)
    got = [(torch.zeros(B * T, 1, H, 128, dtype=BF, device="cuda"),
            torch.zeros(B * T, 1, H, device="cuda")) for _ in range(2)]
    m.absorb(q, g.w_uk)
    binding.score_pages(d, m.q_lat().view(B, T, H, 576), keys, g.block_table, g.seq_lens, scores)
    binding.select_pages(d, scores, g.block_table, g.seq_lens, top_k, 1, 1, st, sl)
    m.plan(sl)
    out, lse = got[0]
    if fp8:
        m.attend_fp8kv(kv8, kvs, st, sl, g.scale, lse)
    else:
        m.attend(g.cache, st, sl, g.scale, lse)
    m.combine(g.scale, lse)
    m.up_project(g.w_uv, out)
    assert m.check() == 0
    out, lse = got[1]
    args = (st, sl, g.w_uk, g.w_uv, g.scale, out, lse)
    if fp8:
        m.run_fp8kv(q, kv8, kvs, *args)
    else:
        m.run(q, g.cache, *args)
    assert m.check() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert bool(got[0][0].any()) and got[0][1].isfinite().all()


@gpu
def test_the_whole_chain_captured_and_replayed_on_another_stream():
    B, T, H, top_k = 3, 2, 32, 4
    inp = make_inputs(B, [900, 300, 130], T, H, seed=70)
    pages, width = inp.cache.shape[0], inp.block_table.shape[1]
    g = inp.to(torch.device("cuda"))
    d = binding.Dims(B, T, H, 128, 64, 512, 128, 64, pages, width)
    m = binding.MlaDecode(binding.Dims(B * T, 1, H, 128, 64, 512, 128, 64, pages, top_k),
                          fp8_kv=True)
    kv8, kvs = (x.cuda() for x in ref.quantise(inp.cache))
    rows = torch.zeros(B, T, 576, dtype=BF, device="cuda")
    keys = torch.zeros(pages, 576, dtype=BF, device="cuda")
    scores = torch.empty(B, T, width, device="cuda")
    st = torch.empty(B * T, top_k, dtype=torch.int32, device="cuda")
    sl = torch.empty(B * T, dtype=torch.int32, device="cuda")
    out = torch.empty(B * T, 1, H, 128, dtype=BF, device="cuda")
    lse = torch.empty(B * T, 1, H, device="cuda")
    q_lat = m.q_lat().view(B, T, H, 576)
    # The pages that were there before this step.
    binding.page_keys_fp8kv(d, kv8, kvs, g.block_table, g.seq_lens, 900, keys, g.seq_lens)

    def step():
        binding.append_fp8kv(d, rows, kv8, kvs, g.block_table, g.seq_lens)
        binding.page_keys_fp8kv(d, kv8, kvs, g.block_table, g.seq_lens, T, keys)
        m.absorb(g.q.view(B * T, 1, H, 192), g.w_uk)
        binding.score_pages(d, q_lat, keys, g.block_table, g.seq_lens, scores)
        binding.select_pages(d, scores, g.block_table, g.seq_lens, top_k, 1, 1, st, sl)
        m.plan(sl)
        m.run_fp8kv(g.q, kv8, kvs, st, sl, g.w_uk, g.w_uv, g.scale, out, lse)

    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    saved = kv8.clone(), kvs.clone(), keys.clone()
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    torch.cuda.synchronize()
    for seed, lens in ((71, [900, 300, 130]), (72, [850, 257, 66]), (73, [64, 2, 129])):
        gen = torch.Generator().manual_seed(seed)
        new = torch.randn(B, T, 576, generator=gen).to(BF)
        q = torch.randn(B, T, H, 192, generator=gen).to(BF)
        for x, y in zip((kv8, kvs, keys), saved):
            x.copy_(y)
        rows.copy_(new)
        g.q.copy_(q)
        g.seq_lens.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert m.check() == 0
        rk, rs = ref.append(new, [T] * B, inp.block_table, lens, saved[0].cpu(), saved[1].cpu())
        assert torch.equal(kv8.cpu(), rk) and torch.equal(kvs.cpu(), rs)
        rt, _, rl = ref.select(scores.cpu(), inp.block_table, lens, T, top_k, 1, 1)
        assert torch.equal(st.cpu(), rt) and torch.equal(sl.cpu(), rl)
        cache = (ref.values(rk) * rs.double()[:, None, None]).to(BF)
        o, l = expected(q.view(B * T, 1, H, 192), cache, inp.w_uk, inp.w_uv, inp.scale, rt, rl)
        err = (out.cpu().double() - o).abs()
        assert err.max() <= ref.OUT_MAX and err.mean() <= ref.OUT_MEAN
        assert (lse.cpu().double() - l).abs().max() <= 1e-3


@gpu
def test_scores_of_other_shapes_from_several_host_threads():
    # Shapes whose kernels take different amounts of shared memory (16, 64 and 128
    # rows of queries), called at once from six threads.  (Through the C entry: the
    # interpreter lets go of its lock there only.)
    g = torch.Generator().manual_seed(75)
    table, lens = i32([[0, 1], [2, 3]]).cuda(), i32([100, 128]).cuda()
    keys = torch.randn(4, 576, generator=g).to(BF).cuda()
    cases = []
    for H in (16, 64, 128) * 2:
        q = torch.randn(2, 1, H, 576, generator=g).to(BF).cuda()
        want, got = torch.empty(2, 1, 2, device="cuda"), torch.empty(2, 1, 2, device="cuda")
        binding.score_pages(dims(2, 1, H), q, keys, table, lens, want)
        cases.append((H, q, want, got, torch.cuda.Stream()))
    torch.cuda.synchronize()
    start, codes = threading.Barrier(len(cases)), []

    def work(H, q, want, got, stream):
        fn, d = binding.lib().mla_decode_score_pages, dims(2, 1, H)
        args = (ctypes.byref(d), q.data_ptr(), keys.data_ptr(), table.data_ptr(),
                lens.data_ptr(), got.data_ptr(), None, stream.cuda_stream)
        torch.cuda.set_device(0)
        start.wait()
        codes.extend(c for c in (fn(*args) for _ in range(5000)) if c)

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not codes, (len(codes), set(codes))
    for _, _, want, got, _ in cases:
        assert torch.equal(got, want)
