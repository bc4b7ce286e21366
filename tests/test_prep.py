"""Norms and rotation in front of the cache, against their formulas in 64 bits, and
the whole chain over the 4-bit cache."""
import ctypes
import math
import random

import pytest
import torch

import fp4kv_util as ref
from mla_decode_attention_uk_gb300 import binding
from test_fp8kv import ODD2, ODD8, OK, call, good_dims, tables

gpu = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


# ---------------------------------------------------------------- refusals (no GPU)
class Args(ctypes.Structure):
    P, I64 = ctypes.c_void_p, ctypes.c_int64
    _fields_ = [("q", P), ("q_stride", I64), ("q_weight", P), ("kv", P), ("kv_stride", I64),
                ("kv_weight", P), ("cos_sin", P), ("positions", P), ("new_lens", P),
                ("seq_lens", P), ("q_out", P), ("rows", P), ("kv_cache", P), ("block_table", P),
                ("status", P), ("eps", ctypes.c_float), ("max_position", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("max_new", ctypes.c_int32)]


def test_refuses_bad_arguments():
    good = {name: OK for name, kind in Args._fields_ if kind is ctypes.c_void_p}
    good.update(q_stride=16 * 192, kv_stride=576, eps=EPS, max_position=9, interleaved=1, max_new=1)

    def code(d=None, **change):
        return call("mla_decode_norm_rope", [ctypes.byref(Args(**dict(good, **change))), None], d=d)

    pointers = ("q", "kv", "q_weight", "kv_weight", "cos_sin", "q_out", "rows", "kv_cache")
    bad = [{name: ODD8} for name in pointers]
    bad += [{name: ODD2} for name in ("positions", "new_lens", "seq_lens", "block_table", "status")]
    bad += [{name: None} for name in ("cos_sin", "seq_lens", "q_out", "block_table")]
    bad += [{"q_stride": n} for n in (16 * 192 - 8, 16 * 192 + 4, -16 * 192)]
    bad += [{"kv_stride": n} for n in (568, 580, -576)]
    # In place, but with gaps on one side only.
    bad += [{"q_stride": 16 * 192 + 8}, {"kv_stride": 584}]
    bad += [{"eps": x} for x in (0.0, -1.0, math.nan, math.inf)]
    bad += [{"max_position": 0}, {"max_position": -1}, {"interleaved": 2}, {"interleaved": -1},
            {"max_new": 0}, {"max_new": -1}, {"max_new": 2 ** 30}]  # (more than 2^30 tasks)
    no_q, no_kv = dict(q=None, q_out=None, q_weight=None), dict(kv=None, kv_weight=None, rows=None,
                                                               kv_cache=None)
    # Outputs and weights without their input, and nowhere to write the latents.
    bad += [dict(no_q, q_out=OK), dict(no_q, q_weight=OK), dict(no_kv, kv_weight=OK),
            dict(no_kv, rows=OK), dict(no_kv, kv_cache=OK), {"rows": None, "kv_cache": None},
            {**no_q, **no_kv}]
    for change in bad:
        assert code(**change) == 1, change
    assert call("mla_decode_norm_rope", [None, None]) == 1
    assert code(d=good_dims(qk_rope=32)) == 2
    assert binding.lib().mla_decode_norm_rope(None, ctypes.byref(Args(**good)), None) == 1


def test_refuses_outputs_over_other_tokens_or_each_other():
    # Against every token's bytes, with the four tensors at places near each other.  (Without
    # a device a call whose arguments are right ends there, with 4.)
    if torch.cuda.is_available():
        pytest.skip("addresses that are not memory")
    rng = random.Random(5)
    H, row, lat = 16, 16 * 192, 576

    def tokens(at, stride, length, n):
        return [(at + 2 * stride * i, at + 2 * (stride * i + length)) for i in range(n)]

    def meet(x, y):
        return any(a < d and c < b for a, b in x for c, d in y)

    refused = 0
    for _ in range(4000):
        B, T = rng.randint(1, 2), rng.randint(1, 3)
        n = B * T
        span = rng.choice((400, 4000, 40000))
        place = lambda: 1 << 20 | 16 * rng.randint(0, span)  # noqa: E731
        x = dict(q=place(), kv=place(), q_out=place(), rows=place(),
                 q_stride=row + 8 * rng.choice((0, 0, 8, 144, 1000, 5000)),
                 kv_stride=lat + 8 * rng.choice((0, 0, 8, 400, 5000)))
        if rng.random() < 0.4:
            x["q_out"] = x["q"]
        if rng.random() < 0.4:
            x["rows"] = x["kv"]
        q, kv = tokens(x["q"], x["q_stride"], row, n), tokens(x["kv"], x["kv_stride"], lat, n)
        q_out, rows = tokens(x["q_out"], row, row, n), tokens(x["rows"], lat, lat, n)
        bad = (q_out != q and meet(q_out, q)) or (rows != kv and meet(rows, kv))
        bad = bad or meet(q_out, kv) or meet(rows, q) or meet(q_out, rows)
        # (One token is in place whatever the stride, but the strides have to say so.)
        bad = bad or (x["q_out"] == x["q"] and x["q_stride"] != row)
        bad = bad or (x["rows"] == x["kv"] and x["kv_stride"] != lat)
        args = Args(q_weight=OK, kv_weight=OK, cos_sin=OK, seq_lens=OK, eps=EPS, max_position=9,
                    interleaved=1, max_new=T, **x)
        got = call("mla_decode_norm_rope", [ctypes.byref(args), None],
                   d=good_dims(batch=B, num_heads=H))
        assert got == (1 if bad else 4), x
        refused += bad
    assert 1000 < refused < 3800


def test_python_call_checks_types_and_shapes():
    d = good_dims()
    q, kv = torch.zeros(2, 3, 16, 192, dtype=BF), torch.zeros(2, 3, 576, dtype=BF)
    good = dict(seq_lens=torch.ones(2, dtype=torch.int32), cos_sin=torch.zeros(9, 64), q=q,
                q_out=q, kv=kv, rows=kv, q_weight=torch.ones(192, dtype=BF),
                kv_weight=torch.ones(512, dtype=BF), cache=torch.zeros(4, 64, 576, dtype=BF),
                block_table=torch.zeros(2, 2, dtype=torch.int32),
                positions=torch.zeros(2, 3, dtype=torch.int32),
                new_lens=torch.ones(2, dtype=torch.int32),
                status=torch.zeros(1, dtype=torch.int32))
    wide = torch.zeros(2, 3, 700, dtype=BF)
    for k, v in (("q", q.float()), ("q", q[:1]), ("q", q.transpose(0, 1)), ("q", q[..., :128]),
                 ("q", torch.zeros(2, 5, 16, 192, dtype=BF)[:, :3]),  # uneven: a gap per batch
                 ("q", torch.zeros(2, 3, 32, 192, dtype=BF)[:, :, ::2]),
                 ("kv", kv.float()), ("kv", kv[:, :2]), ("kv", wide[..., 4:580]),
                 ("q_out", q.float()), ("q_out", None), ("q_out", q[:, :1]),
                 ("q_weight", torch.ones(128, dtype=BF)), ("kv_weight", torch.ones(512)),
                 ("rows", kv[:, :2]), ("cos_sin", torch.zeros(9, 32)), ("cos_sin", None),
                 ("cos_sin", torch.zeros(9, 64, dtype=torch.float64)),
                 ("cache", good["cache"][:3]), ("block_table", good["block_table"].long()),
                 ("positions", good["positions"][:1]), ("new_lens", good["new_lens"].long()),
                 ("status", torch.zeros(2, dtype=torch.int32)), ("seq_lens", None),
                 ("seq_lens", good["seq_lens"][:1])):
        with pytest.raises(ValueError):
            binding.norm_rope(d, **dict(good, **{k: v}))
    with pytest.raises(ValueError, match="CUDA device"):
        binding.norm_rope(d, **good)  # right shapes, but in host memory
    for k in ("seq_lens", "cos_sin"):
        with pytest.raises(ValueError, match=k):
            binding.norm_rope(d, **dict(good, kv=torch.zeros(2, 3, 704, dtype=BF)[..., :576],
                                        **{k: None}))


# ---------------------------------------------------------------- the formulas
def cos_sin_table(n):
    a = torch.arange(n, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def normed(x, w):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w.double()


def rotated(x, cs, interleaved):
    """x [.., 64] and lines of cos and sin [.., 64], fp64; also the sum of the two
    products' sizes."""
    c, s = cs[..., :32], cs[..., 32:]
    i, j = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    y, size = torch.empty_like(x), torch.empty_like(x)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    size[..., i] = (x[..., i] * c).abs() + (x[..., j] * s).abs()
    size[..., j] = (x[..., j] * c).abs() + (x[..., i] * s).abs()
    return y, size


def assert_rounded(got, want, size, what):
    """bf16's rounding, half a step: 2^-8 of the value; and fp32's in front of it: the
    sum of up to 512 squares and its root, two products and a rotation, at most 2^-24
    each (512 additions in any order: 512 / 2 of them under the root), relative to the
    sizes of a rotation's products."""
    bound = want.abs() * 2.0 ** -8 + size * (512 / 2 + 8) * 2.0 ** -24 + 2.0 ** -134
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), (what, float((off - bound).max()))


def check(B=3, H=16, lens=(5, 70, 130), new=(1, 70, 67), max_new=70, q_norm=True, kv_norm=True,
          interleaved=True, wide_q=0, wide_kv=0, to="both", positions=None, scale=1.0, seed=1,
          in_place=False):
    g = torch.Generator().manual_seed(seed)
    lens, new = list(lens), list(new)
    table, used = tables(lens, seed + 1)
    d = good_dims(batch=B, num_heads=H, num_pages=used + 1, max_pages_per_seq=table.shape[1])

    def randn(*shape):
        return (torch.randn(*shape, generator=g) * scale).to(BF)

    q_all, kv_all = randn(B, max_new, H * 192 + wide_q), randn(B, max_new, 576 + wide_kv)
    qw, kvw = randn(192) if q_norm else None, randn(512) if kv_norm else None
    cs = cos_sin_table(300)
    pos = torch.randint(0, 300, (B, max_new), generator=g, dtype=torch.int32) \
        if positions == "random" else None
    dq, dkv = q_all.cuda(), kv_all.cuda()
    q = dq[..., wide_q:].unflatten(-1, (H, 192))
    kv = dkv[..., wide_kv:]
    q_out = q if in_place else torch.full((B, max_new, H, 192), 7.0, dtype=BF, device="cuda")
    rows = None
    if to != "cache":
        rows = kv if in_place else torch.full((B, max_new, 576), 7.0, dtype=BF, device="cuda")
    cache = torch.full((used + 1, 64, 576), 7.0, dtype=BF, device="cuda") if to != "rows" else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    put = lambda t: None if t is None else t.cuda()  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    binding.norm_rope(d, ints(lens), cs.cuda(), q=q, q_out=q_out, q_weight=put(qw), kv=kv,
                      kv_weight=put(kvw), rows=rows, cache=cache,
                      block_table=table.cuda() if cache is not None else None, eps=EPS,
                      interleaved=interleaved, positions=put(pos), new_lens=ints(new),
                      status=status)
    assert int(status.item()) == 0
    q64 = q_all[..., wide_q:].unflatten(-1, (H, 192)).double()
    kv64 = kv_all[..., wide_kv:].double()
    kept = torch.full((used + 1, 64), True)
    for b, n in enumerate(new):
        at = pos[b, :n].long() if pos is not None else torch.arange(lens[b] - n, lens[b])
        line = cs.double()[at]
        x = normed(q64[b, :n], qw) if q_norm else q64[b, :n]
        rope, size = rotated(x[..., 128:], line[:, None], interleaved)
        got = q_out[b, :n].cpu()
        assert_rounded(got[..., 128:], rope, size, "q rope")
        if q_norm:
            assert_rounded(got[..., :128], x[..., :128], x[..., :128].abs(), "q nope")
        else:
            assert torch.equal(got[..., :128].double(), x[..., :128])
        y = normed(kv64[b, :n, :512], kvw) if kv_norm else kv64[b, :n, :512]
        rope, size = rotated(kv64[b, :n, 512:], line, interleaved)
        got = []
        if rows is not None:
            got.append(rows[b, :n].cpu())
        if cache is not None:
            p = torch.arange(lens[b] - n, lens[b])
            pages = table[b].long()[p // 64]
            got.append(cache.cpu()[pages, p % 64])
            kept[pages, p % 64] = False
        for x in got:
            assert_rounded(x[:, 512:], rope, size, "k rope")
            if kv_norm:
                assert_rounded(x[:, :512], y, y.abs(), "latent")
            else:
                assert torch.equal(x[:, :512].double(), y)
        # Rows behind a sequence's tokens stay as they were.
        if in_place:
            assert torch.equal(q_out[b, n:].cpu().double(), q64[b, n:])
            assert rows is None or torch.equal(rows[b, n:].cpu().double(), kv64[b, n:])
        else:
            assert bool((q_out[b, n:] == 7).all())
            assert rows is None or bool((rows[b, n:] == 7).all())
    if cache is not None:
        assert bool((cache.cpu()[kept] == 7).all())
    if rows is not None and cache is not None and not in_place:
        for b, n in enumerate(new):
            p = torch.arange(lens[b] - n, lens[b])
            assert torch.equal(rows[b, :n].cpu(), cache.cpu()[table[b].long()[p // 64], p % 64])


@gpu
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("q_norm,kv_norm", [(True, True), (False, True), (False, False)])
@pytest.mark.parametrize("to", ["rows", "cache", "both"])
def test_equals_the_formulas(interleaved, q_norm, kv_norm, to):
    check(interleaved=interleaved, q_norm=q_norm, kv_norm=kv_norm, to=to)


@gpu
@pytest.mark.parametrize("B,H,lens,new,max_new", [
    (1, 16, [1], [1], 1), (1, 128, [64], [1], 1), (2, 16, [17, 80], [1, 1], 1),
    (5, 48, [64, 65, 0, 128, 129], [1, 0, 0, 1, 1], 1), (3, 112, [8, 200, 64], [8, 3, 5], 8),
    (1, 16, [299], [299], 299), (70, 16, [1 + i for i in range(70)], [1] * 70, 1),
    (300, 128, [3] * 300, [3] * 300, 3)])
def test_batches_heads_and_lengths(B, H, lens, new, max_new):
    check(B=B, H=H, lens=lens, new=new, max_new=max_new, seed=2)


@gpu
@pytest.mark.parametrize("wide_q,wide_kv", [(0, 8), (8, 0), (576, 1024), (192, 64)])
def test_columns_of_wider_projections(wide_q, wide_kv):
    check(wide_q=wide_q, wide_kv=wide_kv, seed=3)


@gpu
@pytest.mark.parametrize("wide_q,wide_kv", [(0, 8), (8, 0), (576, 1024)])
@pytest.mark.parametrize("B,max_new", [(1, 1), (1, 5), (4, 1), (4, 3), (4, 64), (3, 65)])
def test_columns_of_wider_projections_of_few_tokens(wide_q, wide_kv, B, max_new):
    lens = [max_new + 3 * i for i in range(B)]
    check(B=B, lens=lens, new=[max_new - (i == 1) for i in range(B)], max_new=max_new,
          wide_q=wide_q, wide_kv=wide_kv, seed=9)


@gpu
@pytest.mark.parametrize("B", [255, 256, 257])
@pytest.mark.parametrize("max_new", [64, 65])
def test_with_and_without_a_list(B, max_new):
    # Up to 256 sequences go by a list of their tokens from 16,384 on, which many of them
    # do not have.
    lens = [(37 * i) % (max_new + 30) for i in range(B)]
    check(B=B, lens=lens, new=[min(n, max_new) if i % 4 else 0 for i, n in enumerate(lens)],
          max_new=max_new, to="both", seed=10)


@gpu
@pytest.mark.parametrize("max_new", [1, 70])
def test_queries_alone_and_latents_alone(max_new):
    g = torch.Generator().manual_seed(11)
    d = good_dims(batch=2, num_heads=32, num_pages=4, max_pages_per_seq=2)
    q = torch.randn(2, max_new, 32, 192, generator=g).to(BF).cuda()
    kv = torch.randn(2, max_new, 576, generator=g).to(BF).cuda()
    lens = torch.tensor([max_new, max_new + 20], dtype=torch.int32).cuda()
    cs, w = cos_sin_table(128).cuda(), torch.randn(512, generator=g).to(BF).cuda()
    both = torch.empty_like(q), torch.empty_like(kv)
    binding.norm_rope(d, lens, cs, q=q, q_out=both[0], kv=kv, kv_weight=w, rows=both[1])
    alone = torch.empty_like(q), torch.empty_like(kv)
    binding.norm_rope(d, lens, cs, q=q, q_out=alone[0])
    binding.norm_rope(d, lens, cs, kv=kv, kv_weight=w, rows=alone[1])
    assert torch.equal(both[0], alone[0]) and torch.equal(both[1], alone[1])


@gpu
@pytest.mark.parametrize("interleaved", [True, False])
def test_given_positions_and_in_place(interleaved):
    check(positions="random", interleaved=interleaved, seed=4)
    check(in_place=True, interleaved=interleaved, seed=5)
    check(in_place=True, q_norm=False, kv_norm=False, to="rows", interleaved=interleaved, seed=6)


@gpu
def test_outputs_over_a_wider_projection_are_refused_and_leave_it():
    B, T, H = 2, 3, 16
    g = torch.Generator().manual_seed(12)
    wide = torch.randn(B, T, H * 192 + 576, generator=g).to(BF).cuda()
    q, kv = wide[..., :H * 192].unflatten(-1, (H, 192)), wide[..., H * 192:]
    flat, before = wide.view(-1), wide.clone()
    q_out = flat[:B * T * H * 192].view(B, T, H, 192)
    rows = flat[-B * T * 576:].view(B, T, 576)
    d = good_dims(batch=B, num_heads=H)
    lens, cs = torch.full((B,), T, dtype=torch.int32).cuda(), cos_sin_table(9).cuda()
    over_q = flat[:B * T * 576].view(B, T, 576)
    for change in (dict(q_out=q_out), dict(rows=rows), dict(rows=over_q)):
        a = dict(dict(q=q, kv=kv, q_out=torch.empty_like(q_out), rows=torch.empty_like(rows)),
                 **change)
        with pytest.raises(binding.MlaDecodeError, match="INVALID_ARG"):
            binding.norm_rope(d, lens, cs, **a)
    assert torch.equal(wide, before)


@gpu
@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** 40])
def test_rows_of_any_size(scale):
    # Far below eps's root (the norm is then a factor of 1000) and far above.
    check(scale=scale, seed=7)


@gpu
def test_a_row_of_zeros_and_rows_that_are_not_finite():
    d = good_dims(batch=1, num_pages=1, max_pages_per_seq=1)
    q = torch.ones(1, 6, 16, 192, dtype=BF, device="cuda")
    kv = torch.ones(1, 6, 576, dtype=BF, device="cuda")
    q[0, 0], kv[0, 0] = 0, 0
    q[0, 1, 3, 5], kv[0, 2, 7], kv[0, 3, 570], kv[0, 4, 0] = math.nan, math.nan, math.inf, math.inf
    w = torch.ones(192, dtype=BF, device="cuda"), torch.ones(512, dtype=BF, device="cuda")
    q_out, rows = torch.empty_like(q), torch.empty_like(kv)
    binding.norm_rope(d, torch.tensor([6], dtype=torch.int32).cuda(), cos_sin_table(6).cuda(), q=q,
                      q_out=q_out, q_weight=w[0], kv=kv, kv_weight=w[1], rows=rows)
    assert not q_out[0, 0].any() and not rows[0, 0].any()
    nan = q_out.isnan().any(dim=-1).cpu()[0]
    assert bool(nan[1, 3]) and int(nan.sum()) == 1
    assert rows[0, 2, :512].isnan().all() and not rows[0, 2, 512:].isnan().any()
    assert not rows[0, 3, :512].isnan().any() and not rows[0, 3, 512:].isfinite().all()
    assert rows[0, 4, 0].isnan() and not rows[0, 4, 1:512].any() and rows[0, 4, 512:].any()
    assert rows[0, 5].isfinite().all()


@gpu
@pytest.mark.parametrize("new", [None, [5]])
def test_tokens_and_pages_beyond_two_gigabytes(new):
    # Tokens 2^29 elements (2^30 bytes) apart, and pages on both sides of byte 2^31 and 2^32.
    gap, pages = 1 << 29, (1 << 32) // (64 * 576 * 2) + 3
    at = [(1 << 31) // (64 * 576 * 2), (1 << 32) // (64 * 576 * 2), pages - 1]
    d = good_dims(batch=1, num_heads=16, num_pages=pages, max_pages_per_seq=3)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(1, 5, 16, 192, generator=g).to(BF)
    kv = torch.randn(1, 5, 576, generator=g).to(BF)
    far_q = torch.empty(4 * gap + 16 * 192, dtype=BF, device="cuda")
    far_kv = torch.empty(4 * gap + 576, dtype=BF, device="cuda")
    far_q = far_q.as_strided((1, 5, 16, 192), (5 * gap, gap, 192, 1))
    far_kv = far_kv.as_strided((1, 5, 576), (5 * gap, gap, 1))
    far_q.copy_(q)
    far_kv.copy_(kv)
    cache = torch.zeros(pages, 64, 576, dtype=BF, device="cuda")
    table = torch.tensor([at], dtype=torch.int32, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    cs = cos_sin_table(140).cuda()
    for first in (62, 126):  # (the third token is in the next page)
        want_q, want_rows = torch.empty_like(q).cuda(), torch.empty_like(kv).cuda()
        got_q, got_rows = torch.zeros_like(want_q), torch.zeros_like(want_rows)
        binding.norm_rope(d, ints([first + 5]), cs, q=q.cuda(), q_out=want_q, kv=kv.cuda(),
                          rows=want_rows)
        binding.norm_rope(d, ints([first + 5]), cs, q=far_q, q_out=got_q, kv=far_kv, cache=cache,
                          block_table=table, new_lens=None if new is None else ints(new))
        binding.gather(d, cache, table, ints([first + 5]), got_rows)
        assert torch.equal(got_q, want_q) and torch.equal(got_rows, want_rows)
        for i in range(5):
            p = first + i
            assert torch.equal(cache[at[p // 64], p % 64], want_rows[0, i])


@gpu
def test_reports_bad_positions_lengths_and_pages():
    B, n = 3, 4
    d = good_dims(batch=B, num_pages=6, max_pages_per_seq=2)
    g = torch.Generator().manual_seed(8)
    q = torch.randn(B, n, 16, 192, generator=g).to(BF).cuda()
    kv = torch.randn(B, n, 576, generator=g).to(BF).cuda()
    table = torch.arange(6, dtype=torch.int32).view(3, 2).cuda()
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    positions = torch.randint(0, 50, (B, n), generator=g, dtype=torch.int32)

    def run(lens=(66, 66, 66), new=(4, 4, 4), pos=positions, table=table, cos_sin=50):
        q_out, rows = torch.full_like(q, 7.0), torch.full_like(kv, 7.0)
        cache = torch.full((6, 64, 576), 7.0, dtype=BF, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        binding.norm_rope(d, ints(lens), cos_sin_table(cos_sin).cuda(), q=q, q_out=q_out, kv=kv,
                          rows=rows, cache=cache, block_table=table,
                          positions=pos if pos is None else pos.cuda(), new_lens=ints(new),
                          status=status)
        return q_out, rows, cache, int(status.item())

    good = run()
    assert good[3] == 0
    for bad in (-1, 50, 2 ** 31 - 1, -2 ** 31):
        p = positions.clone()
        p[1, 2] = bad
        got = run(pos=p)
        assert got[3] == 5 and bool((got[0][1, 2] == 7).all() and (got[1][1, 2] == 7).all())
        assert bool((got[2][3, 0] == 7).all())
        for k in range(2):
            same = (got[k] == good[k]).flatten(2).all(dim=2).cpu()
            assert int((~same).sum()) == 1 and not bool(same[1, 2])
    assert run(pos=None)[3] == 5  # position 62 and on, in a table of 50
    for lens, new in (([129, 66, 66], [4] * 3), ([66, 66, 66], [5, 4, 4]),
                      ([66, 66, 66], [-1, 4, 4]), ([3, 66, 66], [4, 4, 4]),
                      ([-1, 66, 66], [0, 4, 4])):
        got = run(lens=lens, new=new)
        assert got[3] == 5 and bool((got[0][0] == 7).all() and (got[1][0] == 7).all())
        assert bool((got[2][:2] == 7).all())
        assert torch.equal(got[0][1:], good[0][1:]) and torch.equal(got[2][2:], good[2][2:])
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[2, 0] = bad
        got = run(table=t)
        assert got[3] == 5 and torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])
        assert bool((got[2][4] == 7).all())
        assert torch.equal(got[2][5], good[2][5]) and torch.equal(got[2][:4], good[2][:4])


# ---------------------------------------------------------------- together
def chain_inputs(B, T, H, lens, seed):
    g = torch.Generator().manual_seed(seed)
    table, used = tables(lens, seed)
    d = good_dims(batch=B, q_len=T, num_heads=H, num_pages=used, max_pages_per_seq=table.shape[1])
    rand = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()  # noqa: E731
    return d, dict(q=rand(B, T, H, 192), kv=rand(B, T, 576), w_uk=rand(H, 128, 512) / 11,
                   w_uv=rand(H, 512, 128) / 22, kvw=rand(512), table=table.cuda(),
                   lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                   cos_sin=cos_sin_table(table.shape[1] * 64).cuda(),
                   kv4=torch.zeros(used, 64, 336, dtype=torch.uint8, device="cuda"),
                   kvs=torch.ones(used, device="cuda"), prompt=rand(B, max(lens), 576))


def decode_step(d, m, x, out, lse, rows, q):
    """What a layer does with its new tokens, over the 4-bit cache."""
    binding.norm_rope(d, x["lens"], x["cos_sin"], q=x["q"], q_out=q, kv=x["kv"],
                      kv_weight=x["kvw"], rows=rows)
    binding.append_fp4kv(d, rows, x["kv4"], x["kvs"], x["table"], x["lens"])
    m.run_fp4kv(q, x["kv4"], x["kvs"], x["table"], x["lens"], x["w_uk"], x["w_uv"], 192 ** -0.5,
                out, lse)


@gpu
@pytest.mark.parametrize("B,T,H", [(3, 1, 16), (4, 4, 128)])
def test_a_decode_step_eager_captured_and_on_another_stream(B, T, H):
    lens = [64 * i + 17 * i * i + 40 for i in range(B)]
    d, x = chain_inputs(B, T, H, lens, 81)
    binding.append_fp4kv(d, x["prompt"], x["kv4"], x["kvs"], x["table"], x["lens"], x["lens"])
    start = x["kv4"].clone(), x["kvs"].clone()
    m = binding.MlaDecode(d, fp8_kv=True)
    results = []
    bufs = [(torch.empty(B, T, H, 128, dtype=BF, device="cuda"),
             torch.empty(B, T, H, device="cuda"), torch.empty_like(x["kv"]),
             torch.empty_like(x["q"])) for _ in range(3)]

    def step(k):
        x["kv4"].copy_(start[0])
        x["kvs"].copy_(start[1])
        m.plan(x["lens"])
        decode_step(d, m, x, *bufs[k])

    step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(1)
    for b in bufs[1]:
        b.fill_(7)
    graph.replay()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(2)
    torch.cuda.synchronize()
    assert m.check() == 0
    for b in bufs[1:]:
        results.append([torch.equal(p, q) for p, q in zip(bufs[0], b)])
    assert all(all(r) for r in results), results
    # Against the formulas, from the bytes that the cache holds now.
    v = ref.decode(x["kv4"].cpu()) * x["kvs"].cpu().double()[:, None, None]
    q = bufs[0][3].cpu().double()
    for b in range(B):
        rows = v[x["table"][b].cpu().long()[:(lens[b] + 63) // 64]].reshape(-1, 576)
        for t in range(T):
            c = rows[:lens[b] - T + t + 1]
            lat = torch.bmm(q[b, t][:, None, :128], x["w_uk"].cpu().double())[:, 0]
            s = (lat @ c[:, :512].T + q[b, t][:, 128:] @ c[:, 512:].T) * 192 ** -0.5
            lse = torch.logsumexp(s, dim=1)
            o = torch.exp(s - lse[:, None]) @ c[:, :512]
            o = torch.bmm(o[:, None], x["w_uv"].cpu().double())[:, 0]
            assert float((bufs[0][0][b, t].cpu().double() - o).abs().max()) <= 5e-2
            assert float((bufs[0][1][b, t].cpu().double() - lse).abs().max()) <= 1e-3


@gpu
@pytest.mark.parametrize("B,T,H", [(2, 1, 16), (3, 2, 128), (128, 1, 128), (300, 4, 64),
                                   (512, 8, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_queries_are_rotated_before_the_absorb_step_reads_them(B, T, H, in_place):
    # The absorb step reads q without waiting for the kernel in front of it.  Layers of
    # their own queries go through one q_out, nothing between its writer and the step.
    layers, lens = 4, [T + (29 * i) % 150 for i in range(B)]
    d, x = chain_inputs(B, T, H, lens, 83)
    cache = torch.zeros(d.num_pages, 64, 576, dtype=BF, device="cuda")
    prompt = torch.tensor(lens, dtype=torch.int32).cuda()
    binding.norm_rope(d, prompt, x["cos_sin"], kv=x["prompt"], cache=cache,
                      block_table=x["table"], new_lens=prompt)
    queries = [x["q"].roll(7 * i, -1) for i in range(layers)]
    latents = [x["kv"].roll(7 * i, -1) for i in range(layers)]
    q_buf = torch.empty_like(x["q"])
    m = binding.MlaDecode(d)
    outs = [[(torch.empty(B, T, H, 128, dtype=BF, device="cuda"),
              torch.empty(B, T, H, device="cuda"),
              torch.empty(B * T * H, 576, dtype=BF, device="cuda")) for _ in range(layers)]
            for _ in range(3)]

    def steps(results, between=lambda: None):
        m.plan(x["lens"])
        between()
        for q, kv, (out, lse, lat) in zip(queries, latents, results):
            # In place: on a buffer that the queries were copied to just before.
            src = q_buf.copy_(q) if in_place else q
            binding.norm_rope(d, x["lens"], x["cos_sin"], q=src, q_out=q_buf, kv=kv,
                              kv_weight=x["kvw"], cache=cache, block_table=x["table"])
            between()
            m.run(q_buf, cache, x["table"], x["lens"], x["w_uk"], x["w_uv"], 192 ** -0.5, out, lse)
            between()
            src = q_buf.copy_(-q) if in_place else -q
            binding.norm_rope(d, x["lens"], x["cos_sin"], q=src, q_out=q_buf)
            between()
            m.absorb(q_buf, x["w_uk"])
            between()
            lat.copy_(m.q_lat())

    steps(outs[0], torch.cuda.synchronize)
    assert m.check() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps(outs[2])
    for _ in range(3):
        for results in outs[1:]:
            for t in (t for r in results for t in r):
                t.fill_(7)
        steps(outs[1])
        graph.replay()
        assert m.check() == 0
        for results in outs[1:]:
            for got, want in zip(results, outs[0]):
                assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
@pytest.mark.parametrize("B,T,H", [(1, 1, 16), (8, 2, 32), (128, 1, 128), (200, 8, 64)])
def test_norms_and_absorb_steps_in_turn_on_one_buffer(B, T, H):
    # Nothing but the two kernels, each layer's absorb step into a workspace of its own: what
    # the SMs hold of the buffer is the layer's before.
    layers = 6
    d = good_dims(batch=B, q_len=T, num_heads=H)
    g = torch.Generator(device="cuda").manual_seed(85)
    rand = lambda *n: torch.randn(*n, generator=g, device="cuda").to(BF)  # noqa: E731
    queries, w_uk = [rand(B, T, H, 192) for _ in range(layers)], rand(H, 128, 512) / 11
    lens, cs = torch.full((B,), T, dtype=torch.int32, device="cuda"), cos_sin_table(T).cuda()
    q_buf, ms = torch.empty_like(queries[0]), [binding.MlaDecode(d) for _ in range(layers)]

    def steps(between=lambda: None):
        for m, q in zip(ms, queries):
            binding.norm_rope(d, lens, cs, q=q, q_out=q_buf)
            between()
            m.absorb(q_buf, w_uk)
            between()

    for m in ms:
        m.plan(lens)
    torch.cuda.synchronize()
    steps(torch.cuda.synchronize)
    want = [m.q_lat().clone() for m in ms]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            steps()
    for k in range(40):
        for m in ms:
            m.q_lat().zero_()
        graph.replay() if k % 2 else steps()
        assert all(torch.equal(m.q_lat(), w) for m, w in zip(ms, want)), k
        assert all(m.check() == 0 for m in ms)


@gpu
@pytest.mark.parametrize("H", [16, 128])
def test_queries_of_prompts_are_rotated_before_the_absorb_step_reads_them(H):
    # Enough tokens for a list of them; the absorb step takes them eight at a time.
    B, n, layers = 4, 4096, 3
    d = good_dims(batch=B, num_heads=H, num_pages=1, max_pages_per_seq=64)
    m = binding.MlaDecode(good_dims(batch=B * n // 8, q_len=8, num_heads=H))
    g = torch.Generator(device="cuda").manual_seed(84)
    queries = [torch.randn(B, n, H, 192, generator=g, device="cuda").to(BF) for _ in range(layers)]
    w_uk = (torch.randn(H, 128, 512, generator=g, device="cuda") / 11).to(BF)
    q_buf, cs = torch.empty_like(queries[0]), cos_sin_table(n).cuda()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")

    def steps(between=lambda: None):
        got = []
        for q in queries:
            binding.norm_rope(d, lens, cs, q=q, q_out=q_buf, new_lens=lens)
            between()
            m.absorb(q_buf.view(-1, 8, H, 192), w_uk)
            between()
            got.append(m.q_lat().clone())
            between()
        return got

    m.plan(torch.full((B * n // 8,), 8, dtype=torch.int32, device="cuda"))
    want = steps(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(steps(), want))
    assert m.check() == 0


@gpu
def test_block_sparse_decode_over_the_4_bit_cache():
    # Keys, scores, selection and attention over what an append wrote; with as many
    # pages as there are the sparse step is the dense one.
    B, T, H, lens = 2, 2, 32, [700, 130]
    d, x = chain_inputs(B, T, H, lens, 91)
    binding.append_fp4kv(d, x["prompt"], x["kv4"], x["kvs"], x["table"], x["lens"], x["lens"])
    keys = torch.zeros(d.num_pages, 576, dtype=BF, device="cuda")
    binding.page_keys_fp4kv(d, x["kv4"], x["kvs"], x["table"], x["lens"], max(lens), keys,
                            x["lens"])
    assert bool(keys.isfinite().all() and keys.abs().sum() > 0)
    results = {}
    for top_k in (d.max_pages_per_seq, 4):
        ds = good_dims(batch=B * T, q_len=1, num_heads=H, num_pages=d.num_pages,
                       max_pages_per_seq=top_k)
        m = binding.MlaDecode(ds, fp8_kv=True)
        m.absorb(x["q"], x["w_uk"])
        scores = torch.empty(B, T, d.max_pages_per_seq, device="cuda")
        binding.score_pages(d, m.q_lat().view(B, T, H, 576), keys, x["table"], x["lens"], scores)
        table = torch.empty(B * T, top_k, dtype=torch.int32, device="cuda")
        sel = torch.empty(B * T, dtype=torch.int32, device="cuda")
        binding.select_pages(d, scores, x["table"], x["lens"], top_k, 1, 1, table, sel)
        m.plan(sel)
        lse = torch.empty(B, T, H, device="cuda")
        out = torch.empty(B, T, H, 128, dtype=BF, device="cuda")
        m.attend_fp4kv(x["kv4"], x["kvs"], table, sel, 192 ** -0.5, lse)
        m.combine(192 ** -0.5, lse)
        m.up_project(x["w_uv"], out)
        assert m.check() == 0
        results[top_k] = out, lse
    dense = binding.MlaDecode(d, fp8_kv=True)
    out, lse = torch.empty_like(out), torch.empty_like(lse)
    dense.plan(x["lens"])
    dense.run_fp4kv(x["q"], x["kv4"], x["kvs"], x["table"], x["lens"], x["w_uk"], x["w_uv"],
                    192 ** -0.5, out, lse)
    full = results[d.max_pages_per_seq]
    assert float((full[0].float() - out.float()).abs().max()) <= 2e-2
    assert float((full[1] - lse).abs().max()) <= 1e-3
    # Fewer pages: a smaller sum of weights, never a larger one.
    assert bool((results[4][1] <= lse + 1e-3).all())
    assert torch.allclose(results[4][1][1], lse[1], atol=1e-3)  # three pages: all of them
