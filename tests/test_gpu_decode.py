"""The operators of one decoding step against their formulas in 64 bits.

Tolerances count the roundings of the definition, element by element:
 - a rounding to a type is off by at most eps / 2 of the value (plus half the
   type's smallest subnormal);
 - a 32-bit addition or multiplication, the tensor cores' included (which may
   truncate), by at most U = 2^-23 of the largest partial sum, which the sum
   of the terms' magnitudes bounds.
"""
import math

import numpy as np
import pytest

from audio_encoder_b200 import binding
from conftest import weights

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -23
BF16, F16 = torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25, torch.float32: 2.0 ** -150, E4M3: 2.0 ** -10}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.fixture(scope="module")
def enc():
    e = binding.Encoder(weights(1), 1, max_samples=16000, max_clips=1)
    yield e
    e.close()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def within(got, ref, tol, what=""):
    got = got.double()
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((got - ref).abs().max()), float(((got - ref).abs() / tol).max()))


# ------------------------------------------------------ 4-bit products

def unpack(codes):
    q = torch.stack((codes & 15, codes >> 4), 2).flatten(1).double() - 8
    return q


def gemv_case(M, N, K, seed, bias=True):
    g = gen(seed)
    x = randn((M, K), g, BF16)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand((K // 128, N), generator=g, device="cuda") + 0.5) / (7 * math.sqrt(K))
    b = randn((N,), g) if bias else None
    return x, codes, scales, b


def gemv_ref(x, codes, scales, b):
    """The product in 64 bits and the bound on a 32-bit sum's error: a group's
    sum of (q + 8) x less 8 times its sum of x, 127 additions each and one
    more, whose partial sums sum (q + 8) |x| + 8 sum |x| bounds; two
    multiplications, and the sum over groups (warps and all) and the bias."""
    K = x.shape[1]
    s = scales.double().repeat_interleave(128, 0).t()
    y = x.double() @ (unpack(codes) * s).t()
    size = x.double().abs() @ ((unpack(codes) + 16) * s).t()
    if b is not None:
        y, size = y + b.double(), size + b.double().abs()
    return y, size * U * (128 + 3 + K // 128 + 16)


GELU_SLOPE = 1.13  # the largest slope of x Phi(x)


def gelu64(y):
    return y * torch.special.ndtr(y)


SHAPES = [(1, 1, 128), (1, 17, 128), (3, 31, 384), (8, 1280, 1280), (9, 1281, 1280), (13, 5120, 1280), (16, 1279, 896),
          (17, 250, 2048), (25, 2047, 640), (32, 2048, 1152), (1, 40000, 256), (5, 2048, 8192), (2, 3, 65536),
          (32, 33, 16384), (32, 5000, 4096), (7, 131071, 128), (12, 9999, 2176)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("epi", [0, 1, 2, 5])
def test_gemv_q4_is_the_product_with_q_times_s(enc, M, N, K, epi):
    x, codes, scales, b = gemv_case(M, N, K, M * 7 + N + K + epi, bias=N % 2 == 1 or epi == 1)
    y, tol = gemv_ref(x, codes, scales, b)
    if epi == 2:
        base = randn((M, N), gen(5))
        out = base.clone()
        got = enc.gemv_q4(x, codes, scales, b, out, 2)
        assert got is out
        ref = y + base.double()
        tol = tol + ref.abs() * U
    else:
        got = enc.gemv_q4(x, codes, scales, b, epilogue=epi)
        ref = gelu64(y) if epi == 1 else y
    if epi == 1:  # the library's erf: 5.5e-7 per unit of x
        tol = tol * GELU_SLOPE + 6e-7 * y.abs().clamp(min=1)
    if epi in (0, 1):
        tol = tol + (ref.abs() + tol) * half_step(BF16) + TINY[BF16]
    enc.synchronize()
    assert got.dtype == (BF16 if epi in (0, 1) else torch.float32)
    within(got, ref, tol)


def test_gemv_q4_counts_every_code(enc):
    # each code value at each place of a group, one row of x picking one k
    N, K = 16, 256
    codes = torch.zeros(N, K, dtype=torch.uint8)
    for n in range(N):
        codes[n] = (torch.arange(K) * 7 + n) % 16
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).cuda()
    scales = torch.stack((torch.full((N,), 0.5), torch.full((N,), 2.0))).cuda()
    want = (codes.double() - 8) * torch.tensor([0.5, 2.0]).double().repeat_interleave(128)
    for k0 in range(0, K, 32):
        x = torch.zeros(32, K, dtype=BF16)
        x[torch.arange(32), k0 + torch.arange(32)] = 1.0
        got = enc.gemv_q4(x.cuda(), packed, scales, epilogue=5)
        assert torch.equal(got.double().cpu(), want[:, k0:k0 + 32].t())


@pytest.mark.parametrize("N,K", [(333, 1280), (7000, 512), (70000, 384), (50, 16384), (4100, 2176)])
def test_gemv_q4_rows_do_not_depend_on_the_others(enc, N, K):
    x, codes, scales, b = gemv_case(32, N, K, 3)
    alone = {m: enc.gemv_q4(x[:m].contiguous(), codes, scales, b, epilogue=5) for m in (1, 8, 9, 16, 17, 32)}
    for m, y in alone.items():
        assert torch.equal(y, alone[32][:m]), m


def test_gemv_q4_passes_on_nan_and_infinity(enc):
    x, codes, scales, b = gemv_case(4, 64, 512, 4)
    x[1, 200] = float("nan")
    x[2, 300] = float("inf")
    y = enc.gemv_q4(x, codes, scales, b, epilogue=5)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    ref, tol = gemv_ref(x[[0, 3]], codes, scales, b)
    within(y[[0, 3]], ref, tol)


@pytest.mark.parametrize("rows", [1, 8, 32])
def test_gemv_q4_large_and_small_values(enc, rows):
    # rows of very different sizes, each to its own precision
    x, codes, scales, b = gemv_case(rows, 96, 16384 if rows == 32 else 512, 6, bias=False)
    for top in (1e20, 1e30):
        size = torch.logspace(-20, math.log10(top), rows).cuda() if rows > 1 else torch.tensor([top]).cuda()
        xs = (x.float() * size[:, None]).to(BF16)
        y = enc.gemv_q4(xs, codes, scales, None, epilogue=5)
        within(y, *gemv_ref(xs, codes, scales, None))
        assert torch.isfinite(y).all()
        # and within a row, from group to group
        xs = (x.float() * torch.logspace(-5, math.log10(top), x.shape[1]).cuda()).to(BF16)
        within(enc.gemv_q4(xs, codes, scales, None, epilogue=5), *gemv_ref(xs, codes, scales, None))
    xs = (x.float() * 1e-25).to(BF16)
    ref, tol = gemv_ref(xs, codes, scales, None)
    # what is held is 2^-43 of the sums, in steps of 2^-149
    within(enc.gemv_q4(xs, codes, scales, None, epilogue=5), ref, tol + 2.0 ** (-149 + 43) * x.shape[1])


def test_gemv_q4_no_rows_and_refusals(enc):
    x, codes, scales, b = gemv_case(4, 48, 256, 5)
    assert enc.gemv_q4(x[:0], codes, scales, b).shape == (0, 48)
    for bad in [dict(x=x.float()), dict(x=x[:, :128]), dict(codes=codes[:, :64]), dict(scales=scales.t().contiguous()),
                dict(b=b[:40]), dict(epi=3), dict(epi=2), dict(x=x.repeat(9, 1)), dict(out=torch.empty(4, 48, device="cuda")),
                dict(x=x.cpu()), dict(x=torch.zeros(4, 192, dtype=BF16, device="cuda"), codes=codes[:, :96].contiguous())]:
        a = {**dict(x=x, codes=codes, scales=scales, b=b, out=None, epi=0), **bad}
        with pytest.raises((ValueError, binding.MossEncError)):
            enc.gemv_q4(a["x"], a["codes"], a["scales"], a["b"], a["out"], a["epi"])
    # a row that starts off a 16-byte boundary
    off = torch.zeros(4 * 256 + 1, dtype=BF16, device="cuda")[1:].view(4, 256)
    with pytest.raises(binding.MossEncError):
        enc.gemv_q4(off, codes, scales, b)
    within(enc.gemv_q4(x, codes, scales, b, epilogue=5), *gemv_ref(x, codes, scales, b))


# ------------------------------------------------------ caches

def make_cache(n_seqs, capacity, page, heads, dim, dtype, g, layout="token", fill="random", spare=2, k_scale=0.0625,
               v_scale=0.03125):
    """A cache whose sequences' pages lie anywhere in the pool, with a few
    pages nobody owns."""
    per = max(1, -(-capacity // page))
    pages = n_seqs * per + spare
    shape = (pages, page, heads, dim) if layout == "token" else (pages, heads, page, dim)
    ks, vs = (k_scale, v_scale) if dtype == E4M3 else (1.0, 1.0)

    def pool(s):
        if fill == "nan":
            return torch.full(shape, float("nan"), device="cuda").to(dtype)
        return randn(shape, g, dtype, 1.0 / s)

    k, v = pool(ks), pool(vs)
    if layout != "token":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    table = torch.randperm(pages, generator=g, device="cuda")[:n_seqs * per].to(torch.int32).view(n_seqs, per)
    return binding.KVCache(k, v, table, ks, vs)


def read(cache, s, n):
    """Keys and values of positions 0 .. n-1 of sequence s, in 64 bits."""
    page = cache.k.shape[1]
    p = torch.arange(n, device="cuda")
    at = cache.page_table[s].long()[p // page]
    byte = torch.uint8 if cache.dtype == E4M3 else cache.dtype
    k, v = (t.view(byte)[at, p % page].view(cache.dtype).double() for t in (cache.k, cache.v))
    return k * cache.desc.k_scale, v * cache.desc.v_scale


# ------------------------------------------------------ append

def e4m3_64(x):
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def turned(x, pos, inv_freq, interleaved):
    """x's leading dims turned, in 64 bits, and the magnitude of the pair."""
    y = x.double().clone()
    size = y.abs()
    r = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    if r:
        angle = (pos.double()[:, None] * inv_freq)[:, None, :]
        i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
        a, b = x[..., i].double(), x[..., j].double()
        y[..., i] = a * torch.cos(angle) - b * torch.sin(angle)
        y[..., j] = b * torch.cos(angle) + a * torch.sin(angle)
        size[..., i] = size[..., j] = a.abs() + b.abs()
    return y, size, r


# sine and cosine: the fraction of a turn is rounded to 32 bits (2^-26 turns,
# 9.4e-8 rad) and its sine taken to 2 ulp (1.2e-7); then a product and a sum
TURN = 9.4e-8 + 1.2e-7 + 2 * U


def check_rows(got, x, pos, inv_freq, interleaved, dtype, scale=1.0):
    ref, size, r = turned(x, pos, inv_freq, interleaved)
    tol = size * TURN
    if dtype == E4M3:
        ref, tol = ref / scale, tol / scale
        clear = ref.abs() + tol < 448
        tol = tol + torch.where(clear, (ref.abs() + tol) * half_step(E4M3) + TINY[E4M3], 448 * half_step(E4M3) + tol)
        within(got, ref.clamp(-448, 448), tol)
        plain = e4m3_64(x.double()[..., r:] / scale)
    else:
        tol = tol + (ref.abs() + tol) * half_step(dtype) + TINY[dtype]
        within(got, ref, tol)
        plain = x.double()[..., r:]
    assert torch.equal(got[..., r:].double(), plain)  # what does not turn is only stored


APPENDS = [
    # seqs, longest, page, hq, hkv, dim, rows' type, cache's, rotary, interleaved, layout
    (1, 1, 16, 1, 1, 64, BF16, BF16, 64, False, "token"),
    (3, 40, 16, 4, 2, 64, BF16, BF16, 32, True, "token"),
    (5, 100, 32, 0, 3, 128, F16, F16, 128, False, "head"),
    (2, 375, 64, 20, 20, 64, F16, F16, 64, True, "head"),
    (4, 65, 16, 16, 8, 128, BF16, E4M3, 64, False, "token"),
    (4, 65, 256, 5, 5, 256, F16, E4M3, 256, True, "head"),
    (2, 17, 16, 8, 1, 256, BF16, BF16, 16, False, "token"),
    (3, 33, 16, 6, 2, 128, BF16, BF16, 0, False, "token"),
    (1, 700, 128, 64, 4, 128, BF16, BF16, 128, False, "token"),
    # enough rows for several a CTA, an odd number of them
    (13, 900, 64, 4, 2, 64, F16, F16, 64, True, "token"),
    (13, 901, 16, 3, 3, 128, BF16, E4M3, 64, False, "head"),
    (6, 2500, 256, 24, 4, 256, BF16, BF16, 256, False, "token"),
    # few, wide rows
    (1, 7, 16, 60, 10, 256, F16, E4M3, 16, False, "token"),
    (3, 90, 32, 64, 16, 256, BF16, BF16, 128, True, "head"),
]


@pytest.mark.parametrize("seqs,longest,page,hq,hkv,dim,dt,ct,rotary,inter,layout", APPENDS)
def test_kv_append_prompt_then_token(enc, seqs, longest, page, hq, hkv, dim, dt, ct, rotary, inter, layout):
    g = gen(seqs + longest + dim + rotary)
    cache = make_cache(seqs, longest + 1, page, hkv, dim, ct, g, layout)
    inv = 1e6 ** (-torch.arange(rotary // 2, device="cuda", dtype=torch.float64) * 2 / rotary) if rotary else None
    n = np.random.default_rng(1).integers(0, longest + 1, seqs)
    n[0] = longest
    # the prompt's rows in any order, a few rows of padding among them
    seq = np.concatenate([np.repeat(np.arange(seqs), n), [-1, -1, -5]])
    pos = np.concatenate([np.arange(c) for c in n] + [[0, 3, 1 << 30]])
    order = np.random.default_rng(2).permutation(len(seq))
    for seq, pos in [(seq[order], pos[order]), (np.arange(seqs), n)]:
        rows = len(seq)
        st = torch.from_numpy(seq.astype(np.int32)).cuda()
        pt = torch.from_numpy(pos.astype(np.int32)).cuda()
        fused = randn((rows, (hq + 2 * hkv) * dim + 8), g, dt, 3.0)
        q = fused[:, :hq * dim].view(rows, hq, dim) if hq else None
        k = fused[:, hq * dim:(hq + hkv) * dim].view(rows, hkv, dim)
        v = fused[:, (hq + hkv) * dim:(hq + 2 * hkv) * dim].view(rows, hkv, dim)
        before = cache.k.clone(), cache.v.clone()
        marker = torch.full((rows, hq, dim), 7.5, dtype=dt, device="cuda") if hq else None
        got = enc.kv_append(cache, k, v, pt, None if rows == seqs and len(n) == rows and (seq == np.arange(seqs)).all() else st,
                            q=q, q_out=marker, inv_freq=inv, interleaved=inter)
        enc.synchronize()
        live = torch.from_numpy(np.flatnonzero(seq >= 0)).cuda()
        page_at = cache.page_table.long()[st.long()[live], pt.long()[live] // page]
        byte = torch.uint8 if ct == E4M3 else ct
        at = (page_at, pt.long()[live] % page)
        check_rows(cache.k.view(byte)[at].view(ct), k[live], pt[live], inv, inter, ct, cache.desc.k_scale)
        check_rows(cache.v.view(byte)[at].view(ct), v[live], pt[live], None, inter, ct, cache.desc.v_scale)
        if hq:
            assert got is marker
            check_rows(got[live], q[live], pt[live], inv, inter, dt)
            pad = torch.from_numpy(np.flatnonzero(seq < 0)).cuda()
            assert (got[pad] == 7.5).all()  # rows of padding are left as they were
        # every other place of the pool is left as it was
        for now, was in zip((cache.k, cache.v), before):
            same = torch.ones(now.shape[:2], dtype=torch.bool, device="cuda")
            same[at] = False
            assert torch.equal(now.view(byte)[same], was.view(byte)[same])


def test_kv_append_far_positions(enc):
    # positions up to 2^30: the angle is taken in 64 bits
    dim, page = 128, 1 << 20
    g = gen(9)
    per = 1 << 10
    k = randn((2, 64, 1, dim), g, BF16)
    # a table whose far entries name page 1, and a page of 2^20 positions would
    # be large: rows of the page lie on top of one another (token stride 128)
    pool = torch.zeros(2 * (1 << 20) * dim, dtype=BF16, device="cuda").view(2, 1 << 20, 1, dim)
    table = torch.zeros(1, per, dtype=torch.int32, device="cuda")
    table[0, per - 1] = 1
    cache = binding.KVCache(pool, pool.clone(), table)
    pos = torch.tensor([5, (1 << 30) - 1, (1 << 30) - 77, (1 << 30) - (1 << 19)], dtype=torch.int32, device="cuda")
    x = randn((4, 1, dim), g, BF16)
    inv = 1e6 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)
    q = enc.kv_append(cache, x, x, pos, torch.zeros(4, dtype=torch.int32, device="cuda"), q=x, inv_freq=inv)
    enc.synchronize()
    # pos * inv_freq itself is rounded to 64 bits: 2^30 rad to 1.2e-7
    ref, size, _ = turned(x, pos, inv, False)
    tol = size * (TURN + 3e-7)
    within(q, ref, tol + (ref.abs() + tol) * half_step(BF16))
    at = torch.tensor([0, 1, 1, 1], device="cuda")
    assert torch.equal(cache.k[at, pos.long() % page], q)


def test_kv_append_in_place_queries_and_special_values(enc):
    g = gen(11)
    cache = make_cache(2, 40, 16, 2, 64, E4M3, g)
    k = randn((2, 2, 64), g, BF16, 100.0)
    k[0, 0, 0], k[0, 0, 1], k[0, 0, 2], k[1, 1, 5] = float("inf"), float("-inf"), float("nan"), 0.0
    pos = torch.tensor([3, 39], dtype=torch.int32, device="cuda")
    q = randn((2, 4, 64), g, BF16)
    was = q.clone()
    inv = 1e4 ** (-torch.arange(16, device="cuda", dtype=torch.float64) / 16)
    out = enc.kv_append(cache, k, k, pos, q=q, q_out=q, inv_freq=inv, interleaved=True)
    assert out is q
    check_rows(q, was, pos, inv, True, BF16)
    page = cache.page_table[torch.arange(2, device="cuda"), pos.long() // 16].long()
    got = cache.v.view(torch.uint8)[page, pos.long() % 16].view(E4M3).float()
    assert got[0, 0, 0] == 448 and got[0, 0, 1] == -448 and torch.isnan(got[0, 0, 2]) and got[1, 1, 5] == 0
    live = torch.isfinite(k.float())
    assert torch.equal(got[live].double(), e4m3_64(k.double() / cache.desc.v_scale)[live])
    enc.synchronize()


@pytest.mark.parametrize("k_scale,v_scale", [(0.1, 3.0), (129 / 21, 133 / 21), (1025 / 17, 1025 / 31), (1 / 192, 1031 / 23 / 1024),
                                             (0.25, 4.0)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_kv_append_rounds_the_quotient_by_the_scale_once(enc, dt, k_scale, v_scale):
    # every finite value of the type, as keys and as values; with 129 / 21 and the
    # like 32 bits put quotients on the middle between two e4m3 values that are
    # only near it
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(dt)
    x = torch.where(torch.isfinite(bits.float()), bits, torch.zeros((), dtype=dt, device="cuda")).view(512, 2, 64)
    cache = make_cache(1, 512, 16, 2, 64, E4M3, gen(71), k_scale=k_scale, v_scale=v_scale)
    pos = torch.arange(512, dtype=torch.int32, device="cuda")
    enc.kv_append(cache, x, x.flip(0), pos, torch.zeros_like(pos))
    enc.synchronize()
    at = cache.page_table[0].long()[pos.long() // 16], pos.long() % 16
    for pool, rows, scale in ((cache.k, x, cache.desc.k_scale), (cache.v, x.flip(0), cache.desc.v_scale)):
        got = pool.view(torch.uint8)[at].view(E4M3).double()
        bad = got != e4m3_64(rows.double() / scale)
        assert not bad.any(), (int(bad.sum()), rows[bad][:4], got[bad][:4])


def test_kv_append_reports_places_outside_the_cache(enc):
    g = gen(12)
    cache = make_cache(2, 32, 16, 2, 64, BF16, g)
    k = randn((4, 2, 64), g, BF16)
    was = cache.k.clone(), cache.v.clone()
    good = cache.page_table.clone()
    for seq, pos, table in [(2, 0, None), (0, 32, None), (1, -1, None), (1, 20, -3), (1, 20, cache.k.shape[0]), (0, 1 << 30, None)]:
        cache.page_table.copy_(good)
        if table is not None:
            cache.page_table[1, 1] = table
        q = torch.full((4, 2, 64), 1.0, dtype=BF16, device="cuda")
        st = torch.tensor([-1, seq, -1, -1], dtype=torch.int32, device="cuda")
        pt = torch.tensor([0, pos, 0, 0], dtype=torch.int32, device="cuda")
        enc.kv_append(cache, k, k, pt, st, q=q, q_out=q)
        with pytest.raises(binding.MossEncError) as e:
            enc.synchronize()
        assert e.value.status == 1
        assert torch.equal(cache.k, was[0]) and torch.equal(cache.v, was[1]) and (q == 1).all()
        enc.synchronize()  # reported once
    # and the handle still works
    cache.page_table.copy_(good)
    enc.kv_append(cache, k[:2], k[:2], torch.tensor([31, 0], dtype=torch.int32, device="cuda"))
    enc.synchronize()
    assert torch.equal(cache.k[good[0, 1].long(), 15], k[0])


def test_synchronize_reports_a_page_error_behind_a_timeout(enc):
    cache = make_cache(2, 32, 16, 2, 64, BF16, gen(73))
    k = randn((2, 2, 64), gen(74), BF16)
    enc.selftest_timeout(20)
    enc.kv_append(cache, k, k, torch.tensor([5, 32], dtype=torch.int32, device="cuda"))
    got = []
    for _ in range(2):
        with pytest.raises(binding.MossEncError) as e:
            enc.synchronize()
        got.append(e.value.status)
    assert got == [5, 1]
    enc.synchronize()


def test_page_errors_in_a_row_on_a_stream_of_its_own_are_all_reported():
    # the error word is cleared in the order of the handle's stream, which the
    # default stream does not wait for
    e = binding.Encoder(weights(1), 1, max_samples=16000, max_clips=1)
    cache = make_cache(2, 32, 16, 2, 64, BF16, gen(77))
    k = randn((2, 2, 64), gen(78), BF16)
    bad, good = (torch.tensor([5, p], dtype=torch.int32, device="cuda") for p in (32, 31))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    e.set_stream(side)
    for i in range(200):
        e.kv_append(cache, k, k, bad if i % 3 else good)
        if i % 3:
            with pytest.raises(binding.MossEncError):
                e.synchronize()
        else:
            e.synchronize()
    e.close()


def test_kv_append_nothing_and_refusals(enc):
    g = gen(13)
    cache = make_cache(2, 32, 16, 2, 64, BF16, g)
    k = randn((2, 2, 64), g, BF16)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert enc.kv_append(cache, k[:0], k[:0], pos[:0]) is None
    inv = torch.ones(32, device="cuda", dtype=torch.float64)
    for kw in [dict(k=k.half()), dict(k=k.float(), v=k.float()), dict(k=k[:, :1]), dict(pos=pos.long()), dict(pos=pos[:1]),
               dict(inv=inv.float()), dict(inv=inv[:5]), dict(inv=inv.repeat(2)), dict(seqs=pos.long()), dict(q_out=k),
               dict(q=k.transpose(0, 1)), dict(q=k, q_out=k.half()), dict(k=k.cpu()), dict(q=k.half())]:
        a = {**dict(k=k, v=k, pos=pos, seqs=None, q=None, q_out=None, inv=inv), **kw}
        with pytest.raises((ValueError, binding.MossEncError)):
            enc.kv_append(cache, a["k"], a["v"], a["pos"], a["seqs"], q=a["q"], q_out=a["q_out"], inv_freq=a["inv"])
    three = randn((3, 2, 64), g, BF16)
    with pytest.raises(binding.MossEncError):  # more rows than sequences, and no seqs
        enc.kv_append(cache, three, three, torch.zeros(3, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------ attention

def attn_ref(cache, q, lengths, scale):
    """out, lse in 64 bits and the bounds on their errors."""
    S, hq, dim = q.shape
    G = hq // cache.n_kv_heads
    half = half_step(F16 if cache.dtype in (F16, E4M3) else BF16)
    tiny = 2.0 ** -25 if cache.dtype in (F16, E4M3) else 0.0
    out = torch.zeros(S, hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((S, hq), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for s, n in enumerate(lengths):
        if n == 0:
            continue
        k, v = read(cache, s, n)
        qs = q[s].double().view(-1, G, dim)
        score = torch.einsum("hgd,nhd->hgn", qs, k) * scale
        size = torch.einsum("hgd,nhd->hgn", qs.abs(), k.abs()) * abs(scale)
        p = torch.softmax(score, 2)
        out[s] = torch.einsum("hgn,nhd->hgd", p, v).reshape(hq, dim)
        lse[s] = torch.logsumexp(score, 2).reshape(hq)
        # a score: dim additions, the scale's two roundings; its difference to
        # the maximum in units of log 2, one rounding; 2^x to 2^-22
        d = (size * U * (dim + 4) + score.abs() * 4 * U).amax(2) + 2 * 2.0 ** -22
        # each probability is rounded to 16 bits (to half a subnormal in f16,
        # relative to the largest, whose own is 1); a chain of products and
        # rescalings per position and join
        l_top = torch.exp(torch.logsumexp(score, 2) - score.amax(2))
        pv = torch.einsum("hgn,nhd->hgd", p, v.abs())
        sums = (n + 64) * 2 * U
        t = pv * (half + 2 * d[..., None] + 2 * sums)
        t = t + tiny * v.abs().sum(0).repeat_interleave(G, 0).view(-1, G, dim) / l_top[..., None]
        t = t.reshape(hq, dim)
        tol[s] = t + (out[s].abs() + t) * half_step(q.dtype) + TINY[q.dtype]
        tol_lse[s] = (2 * d + sums).reshape(hq) + lse[s].abs() * 2 * U
    return out, lse, tol, tol_lse


def check_attn(enc, cache, q, lengths, scale=None, **kw):
    lt = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = enc.paged_attn(cache, q, lt, scale, return_lse=True, **kw)
    enc.synchronize()
    ref, rlse, tol, tlse = attn_ref(cache, q, lengths, q.shape[2] ** -0.5 if scale is None else scale)
    within(out, ref, tol, "out")
    empty = torch.tensor([n == 0 for n in lengths], device="cuda")
    assert (out[empty] == 0).all() and (lse[empty] == -math.inf).all()
    within(lse[~empty], rlse[~empty], tlse[~empty], "lse")
    return out, lse


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 127, 128, 129, 375, 1000, 0]


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (6, 2), (8, 1), (9, 1), (16, 1), (40, 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dt,ct", [(BF16, BF16), (F16, F16), (BF16, E4M3), (F16, E4M3)])
def test_paged_attn_heads_and_types(enc, hq, hkv, dim, dt, ct):
    g = gen(hq + dim)
    cache = make_cache(len(LENGTHS), max(LENGTHS), 16, hkv, dim, ct, g)
    check_attn(enc, cache, randn((len(LENGTHS), hq, dim), g, dt, 2.0), LENGTHS)


@pytest.mark.parametrize("page", [16, 32, 64, 256, 2048])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_paged_attn_pages_and_layouts(enc, page, layout):
    g = gen(page)
    for ct in (BF16, E4M3):
        cache = make_cache(len(LENGTHS), max(LENGTHS), page, 2, 128, ct, g, layout)
        check_attn(enc, cache, randn((len(LENGTHS), 8, 128), g, BF16, 2.0), LENGTHS)


@pytest.mark.parametrize("ct", [BF16, F16, E4M3])
@pytest.mark.parametrize("lengths", [[1500], [9000], [45000], [20000, 3], [4097, 0, 4096, 4095, 1, 12345], [130000],
                                     [0] * 70 + [9000, 0, 2500] + [1100] * 50, [3] * 1100 + [20000] + [0, 5] * 40,
                                     [0] * 33 + [30000]])
def test_paged_attn_long(enc, ct, lengths):
    g = gen(sum(lengths))
    cache = make_cache(len(lengths), max(lengths), 64, 2, 128, ct, g)
    q = randn((len(lengths), 10, 128), g, F16 if ct == F16 else BF16, 2.0)
    check_attn(enc, cache, q, lengths)


@pytest.mark.parametrize("ct", [BF16, F16, E4M3])
@pytest.mark.parametrize("hq,hkv,dim", [(3, 1, 256), (20, 2, 256), (32, 2, 128), (40, 2, 64), (24, 2, 64), (4, 2, 64), (17, 1, 128)])
@pytest.mark.parametrize("lengths", [[70000, 0, 3], [66000, 0, 12345, 1, 700]])
def test_paged_attn_split_over_the_card(enc, hq, hkv, dim, ct, lengths):
    # the split and its join at every head width, with one and two groups of
    # eight query heads a pass and several passes a key head
    g = gen(hq + dim)
    cache = make_cache(len(lengths), max(lengths), 64, hkv, dim, ct, g)
    assert enc.paged_attn_workspace(cache, hq) > 0  # not a CTA or a cluster per key head
    check_attn(enc, cache, randn((len(lengths), hq, dim), g, F16 if ct == F16 else BF16, 2.0), lengths)


@pytest.mark.parametrize("seqs", [1, 40, 300, 1500])
def test_paged_attn_many_sequences(enc, seqs):
    g = gen(seqs)
    lengths = np.random.default_rng(seqs).integers(0, 200, seqs).tolist()
    cache = make_cache(seqs, 200, 16, 2, 64, BF16, g)
    check_attn(enc, cache, randn((seqs, 6, 64), g, BF16, 2.0), lengths)


@pytest.mark.parametrize("hq,hkv,dim,ct", [(50, 10, 256, F16), (48, 16, 128, BF16), (20, 20, 64, BF16), (36, 4, 128, E4M3),
                                           (40, 2, 64, E4M3)])
@pytest.mark.parametrize("longest", [1, 17, 60, 200])
def test_paged_attn_many_short_sequences(enc, hq, hkv, dim, ct, longest):
    g = gen(hq + longest)
    seqs = 133
    lengths = np.random.default_rng(longest).integers(0, longest + 1, seqs).tolist()
    cache = make_cache(seqs, longest, 16, hkv, dim, ct, g, "head" if longest == 60 else "token")
    q = randn((seqs, hq, dim), g, F16 if ct == F16 else BF16, 2.0)
    check_attn(enc, cache, q, lengths)
    check_attn(enc, cache, q, lengths, max_len=1)  # a bound below the lengths only sizes the launch


def test_paged_attn_sharp_and_flat_scores(enc):
    g = gen(31)
    n = [777, 128, 4000]
    for ct, dt in ((BF16, BF16), (F16, F16), (E4M3, BF16)):
        cache = make_cache(3, 4000, 16, 2, 128, ct, g)
        q = randn((3, 4, 128), g, dt, 20.0)  # scores of hundreds: one position takes all
        check_attn(enc, cache, q, n)
        check_attn(enc, cache, q, n, scale=0.0)
        check_attn(enc, cache, q, n, scale=-0.05)
        # rising scores: every position is the largest so far
        for s in range(3):
            page = cache.page_table[s].long()
            ramp = (torch.arange(n[s], device="cuda").float() / n[s]).view(-1, 1, 1)
            p = torch.arange(n[s], device="cuda")
            key = (q[s].float().view(2, 2, 128)[:, 0][None] * ramp / 4 / cache.desc.k_scale).clamp(-448, 448).to(ct)
            byte = torch.uint8 if ct == E4M3 else ct
            cache.k.view(byte)[page[p // 16], p % 16] = key.view(byte)
        check_attn(enc, cache, q, n)


@pytest.mark.parametrize("dt,ct", [(F16, F16), (BF16, E4M3), (F16, E4M3)])
@pytest.mark.parametrize("lengths,max_len", [([16], 0), ([300, 0, 40], 0), ([5000], 0), ([131072], 0), ([9000, 16] * 80, 16)])
def test_paged_attn_keeps_small_probabilities(enc, dt, ct, lengths, max_len):
    # every 16th position scores 18 above the others and its value is zero, so
    # the outputs are the others' alone: probabilities of 2^-26 of the largest
    g = gen(70)
    cache = make_cache(len(lengths), max(lengths), 16, 2, 64, ct, g)
    byte = torch.uint8 if ct == E4M3 else ct
    key, value = torch.zeros(2, 16, 2, 64, device="cuda")
    key[0, :, 3] = 18.0
    value[1:] = torch.linspace(2.0, 8.0, 64, device="cuda")
    cache.k.view(byte)[:] = (key / cache.desc.k_scale).to(ct).view(byte)
    cache.v.view(byte)[:] = (value / cache.desc.v_scale).to(ct).view(byte)
    q = torch.zeros(len(lengths), 4, 64, dtype=dt, device="cuda")
    q[..., 3] = 1.0
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = enc.paged_attn(cache, q, n, 1.0, return_lse=True, max_len=max_len)
    enc.synchronize()
    ref, rlse, _, tlse = attn_ref(cache, q, lengths, 1.0)
    # as attn_ref's bound, with the probabilities' rounding relative to each:
    # a score to 18 * 2^-23 and the like, 2^-11 a probability
    tol = ref.abs() * (half_step(F16) + 2 * (18 * U * 72 + 2.0 ** -21) + 4 * U * (n.double()[:, None, None] + 64))
    within(out, ref, tol + (ref.abs() + tol) * half_step(dt) + TINY[dt], "out")
    live = n > 0
    within(lse[live], rlse[live], tlse[live], "lse")


@pytest.mark.parametrize("dt,ct", [(BF16, BF16), (F16, F16), (BF16, E4M3), (F16, E4M3)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_paged_attn_probabilities_are_not_held_in_16_bits(enc, dt, ct, dim):
    # values of +w and -w in turn: the outputs are small differences of the
    # probabilities, which the outputs' own rounding does not hide
    g = gen(80 + dim)
    lengths = [2, 3, 8, 15, 16, 17, 33, 40]
    cache = make_cache(len(lengths), 40, 16, 2, dim, ct, g)
    w = randn((1, 1, 2, dim), g, ct, 1 / cache.desc.v_scale).float()
    sign = 1.0 - 2.0 * (torch.arange(16, device="cuda") % 2).view(1, 16, 1, 1)
    byte = torch.uint8 if ct == E4M3 else ct
    cache.v.view(byte)[:] = (w * sign).expand(cache.v.shape).to(ct).view(byte)
    q = randn((len(lengths), 6, dim), g, dt)
    scale = 0.2 * dim ** -0.5
    out = enc.paged_attn(cache, q, torch.tensor(lengths, dtype=torch.int32, device="cuda"), scale)
    enc.synchronize()
    half = half_step(F16 if ct in (F16, E4M3) else BF16)
    for s, n in enumerate(lengths):
        k, v = read(cache, s, n)
        qs = q[s].double().view(2, 3, dim)
        score = torch.einsum("hgd,nhd->hgn", qs, k) * scale
        size = torch.einsum("hgd,nhd->hgn", qs.abs(), k.abs()) * scale
        p = torch.softmax(score, 2)
        ref = torch.einsum("hgn,nhd->hgd", p, v)
        pv = torch.einsum("hgn,nhd->hgd", p, v.abs())
        # as attn_ref's bound, but a probability's rounding is that of what a
        # rounding to 16 bits leaves of it
        d = (size * U * (dim + 4) + score.abs() * 4 * U).amax(2) + 2 * 2.0 ** -22
        tol = pv * (half * half + 2 * d[..., None] + 4 * U * (n + 64))
        within(out[s].view(2, 3, dim), ref, tol + (ref.abs() + tol) * half_step(dt) + TINY[dt])


@pytest.mark.parametrize("dt,ct", [(BF16, BF16), (F16, F16), (BF16, E4M3), (F16, E4M3)])
def test_paged_attn_very_large_scores_stay_finite(enc, dt, ct):
    # every second position has the largest score, the others one far below:
    # the outputs are the means of the former's values, whatever the score.
    # Around 2^23 (5.81e6 log2(e)) 32 bits no longer tell a score less 15 from it
    g = gen(76)
    n = [1, 2, 15, 100, 3000]
    cache = make_cache(5, 3000, 16, 2, 64, ct, g)
    byte = torch.uint8 if ct == E4M3 else ct
    key = torch.zeros(16, 2, 64, device="cuda")
    key[0::2, :, 3], key[1::2, :, 3] = 8.0, -8.0
    key[:, :, 4] = -16.0
    cache.k.view(byte)[:] = (key / cache.desc.k_scale).to(ct).view(byte)
    cache.v.view(byte)[:] = randn(cache.v.shape, g, ct, 1 / cache.desc.v_scale).view(byte)
    lt = torch.tensor(n, dtype=torch.int32, device="cuda")
    for top in (1e3, 5.7e6, 5.8145e6, 5.815e6, 5.9e6, 1.17e7, 1.2e7, 2.4e7, 5e7, 3e9, 1e30):
        for below_zero in (0.0, 1.0):  # scores of top and -top, or of -top and -3 top
            q = torch.zeros(5, 4, 64, dtype=dt, device="cuda")
            q[..., 3], q[..., 4] = 1.0, below_zero
            out, lse = enc.paged_attn(cache, q, lt, top / 8, return_lse=True)
            enc.synchronize()
            assert torch.isfinite(lse).all()
            for s, count in enumerate(n):
                v = read(cache, s, count)[1][0::2].repeat_interleave(2, 1)
                ref = v.mean(0)
                tol = v.abs().mean(0) * (half_step(ct if ct in (BF16, F16) else F16) + (count + 64) * 4 * U)
                within(out[s], ref, tol + (ref.abs() + tol) * half_step(dt) + TINY[dt])


def test_paged_attn_extreme_queries_over_an_e4m3_cache(enc):
    # bf16 queries outside f16's range, one head each; the products stay finite
    g = gen(33)
    cache = make_cache(3, 300, 16, 1, 128, E4M3, g)
    q = randn((3, 4, 128), g, BF16)
    size = torch.tensor([1e6, 1e-7, 1e-30, 3e4], device="cuda").view(1, 4, 1)
    check_attn(enc, cache, (q.float() * size).to(BF16), [300, 1, 130], scale=1e-5)


def test_paged_attn_ignores_what_lies_past_the_lengths(enc):
    # NaN in every place that no sequence has written: pages nobody owns, the
    # rest of the last page, table entries past it that name no page
    g = gen(35)
    lengths = [0, 1, 15, 16, 17, 100, 130, 257]
    for ct in (BF16, F16, E4M3):
        cache = make_cache(len(lengths), 300, 32, 2, 128, ct, g, fill="nan")
        byte = torch.uint8 if ct == E4M3 else ct
        for s, n in enumerate(lengths):
            p = torch.arange(n, device="cuda")
            at = (cache.page_table[s].long()[p // 32], p % 32)
            for t, scale in ((cache.k, cache.desc.k_scale), (cache.v, cache.desc.v_scale)):
                t.view(byte)[at] = randn((n, 2, 128), g, ct, 1.0 / scale).view(byte)
            cache.page_table[s, -(-n // 32):] = -(1 << 30) if s % 2 else (1 << 30)
        out, _ = check_attn(enc, cache, randn((len(lengths), 6, 128), g, F16 if ct == F16 else BF16), lengths)
        assert torch.isfinite(out).all()


def test_paged_attn_nan_in_a_live_place_reaches_its_rows_alone(enc):
    g = gen(36)
    cache = make_cache(2, 100, 16, 2, 64, BF16, g)
    cache.v[cache.page_table[0, 3].long(), 2, 1, 7] = float("nan")
    cache.k[cache.page_table[1, 0].long(), 5, 0, 9] = float("nan")
    q = randn((2, 4, 64), g, BF16)
    out = enc.paged_attn(cache, q, torch.tensor([100, 100], dtype=torch.int32, device="cuda"))
    enc.synchronize()
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[0, 2:, 7] = True
    want[1, :2] = True
    assert torch.equal(bad, want)


def test_paged_attn_live_scores_of_minus_infinity(enc):
    # a row that its keys mask throughout is as one without positions
    g = gen(75)
    lengths = [1, 40, 700, 20000, 130]
    for ct, dt in ((BF16, BF16), (F16, F16)):
        for seqs, max_len in ((1, 0), (5, 0), (5, 16), (5, 1 << 20)):
            cache = make_cache(seqs, 20000 if seqs > 1 else 1000, 16, 2, 64, ct, g)
            cache.k[..., 5] = -math.inf
            q = randn((seqs, 4, 64), g, dt).abs()
            n = torch.tensor(lengths[:seqs], dtype=torch.int32, device="cuda")
            out, lse = enc.paged_attn(cache, q, n, return_lse=True, max_len=max_len)
            enc.synchronize()
            assert (out == 0).all() and (lse == -math.inf).all()


def test_paged_attn_infinite_values_in_live_places(enc):
    # a value of +-inf makes its dim +-inf, and no other
    g = gen(81)
    for ct, dt in ((BF16, BF16), (F16, F16)):
        for seqs, longest, max_len in ((2, 1, 0), (2, 100, 0), (2, 2000, 0), (2, 20000, 0), (2, 20000, 16)):
            cache = make_cache(seqs, longest, 16, 2, 64, ct, g)
            cache.v[cache.page_table[0, 0].long(), 0, 1, 5] = math.inf
            cache.v[cache.page_table[1, 0].long(), 0, 0, 60] = -math.inf
            n = torch.full((seqs,), longest, dtype=torch.int32, device="cuda")
            for size in (0.0, 1.0):  # equal probabilities, or any
                out = enc.paged_attn(cache, randn((seqs, 4, 64), g, dt, size), n, max_len=max_len).float()
                enc.synchronize()
                want = torch.zeros_like(out)
                want[0, 2:, 5], want[1, :2, 60] = math.inf, -math.inf
                assert torch.equal(torch.where(torch.isfinite(out), 0.0, out), want)


def test_paged_attn_a_score_of_infinity_makes_its_row_nan(enc):
    g = gen(79)
    for ct, dt in ((BF16, BF16), (F16, F16)):
        for seqs, longest, max_len in ((1, 100, 0), (2, 2000, 0), (2, 20000, 0), (2, 20000, 16)):
            cache = make_cache(seqs, longest, 16, 2, 64, ct, g)
            cache.k[cache.page_table[0, 2].long(), 7, 1, 5] = math.inf
            q = randn((seqs, 4, 64), g, dt).abs()
            n = torch.full((seqs,), longest, dtype=torch.int32, device="cuda")
            out, lse = enc.paged_attn(cache, q, n, return_lse=True, max_len=max_len)
            enc.synchronize()
            want = torch.zeros(seqs, 4, dtype=torch.bool, device="cuda")
            want[0, 2:] = True
            assert torch.equal(torch.isnan(out).all(2), want) and torch.equal(torch.isnan(out).any(2), want)
            assert torch.equal(torch.isnan(lse), want)


def test_paged_attn_strided_queries_and_given_outputs(enc):
    g = gen(37)
    cache = make_cache(5, 64, 16, 2, 64, BF16, g)
    fused = randn((5, 8 * 64 + 24), g, BF16)
    q = fused[:, 16:16 + 8 * 64].view(5, 8, 64)
    out = torch.full((5, 8, 64), 9.0, dtype=BF16, device="cuda")
    lse = torch.empty(5, 8, device="cuda")
    got = check_attn(enc, cache, q, [64, 3, 0, 1, 20], out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    alone = enc.paged_attn(cache, q, torch.tensor([64, 3, 0, 1, 20], dtype=torch.int32, device="cuda"))
    assert torch.equal(alone, out)


def test_paged_attn_is_the_same_every_time(enc):
    g = gen(38)
    lengths = torch.tensor([30000, 5, 7000], dtype=torch.int32, device="cuda")
    cache = make_cache(3, 30000, 64, 4, 128, BF16, g)
    q = randn((3, 8, 128), g, BF16, 2.0)
    first = enc.paged_attn(cache, q, lengths, return_lse=True)
    for _ in range(20):
        again = enc.paged_attn(cache, q, lengths, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_paged_attn_bound_on_the_lengths(enc):
    # a bound sizes the launch; a wrong one costs time, not results
    g = gen(39)
    lengths = [100, 3000, 0, 17]
    cache = make_cache(4, 4000, 16, 2, 128, BF16, g)
    q = randn((4, 4, 128), g, BF16, 2.0)
    for bound in (0, 1, 100, 1000, 3000, 1 << 30):
        check_attn(enc, cache, q, lengths, max_len=bound)


def test_paged_attn_refuses_a_workspace_that_is_too_small(enc):
    g = gen(64)
    cache = make_cache(2, 60000, 16, 2, 64, BF16, g)
    q = randn((2, 4, 64), g, BF16)
    n = torch.tensor([60000, 6], dtype=torch.int32, device="cuda")
    need = enc.paged_attn_workspace(cache, 4)
    assert need > 0
    big = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    for bad in (big[:need - 1], big[8:8 + need], big[::2], big.view(torch.int8)):
        with pytest.raises((ValueError, binding.MossEncError)):
            enc.paged_attn(cache, q, n, workspace=bad)
    check_attn(enc, cache, q, [60000, 6], workspace=big)
    n_short = make_cache(2, 100, 16, 2, 64, BF16, g)
    assert enc.paged_attn_workspace(n_short, 4) == 0 and enc.paged_attn_workspace(cache, 4, max_len=100) == 0


def test_paged_workspace_of_refused_heads(enc):
    cache = make_cache(2, 64, 16, 1, 64, BF16, gen(72))
    assert enc.paged_attn_workspace(cache, 65535) >= 0
    for heads in (65536, 0, -1, 1 << 30):
        with pytest.raises(binding.MossEncError):
            enc.paged_attn_workspace(cache, heads)


def test_paged_attn_reports_lengths_and_pages_outside_the_cache(enc):
    g = gen(40)
    cache = make_cache(2, 64, 16, 1, 64, BF16, g)
    q = randn((2, 2, 64), g, BF16)
    good = cache.page_table.clone()
    for lengths, page in [([64, 65], None), ([-1, 64], None), ([64, 64], -1), ([64, 64], cache.k.shape[0]), ([1 << 30, 1], None)]:
        cache.page_table.copy_(good)
        if page is not None:
            cache.page_table[1, 2] = page
        enc.paged_attn(cache, q, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
        with pytest.raises(binding.MossEncError) as e:
            enc.synchronize()
        assert e.value.status == 1
        enc.synchronize()
    cache.page_table.copy_(good)
    check_attn(enc, cache, q, [64, 64])


def test_paged_attn_no_sequences_and_refusals(enc):
    g = gen(41)
    cache = make_cache(2, 64, 16, 2, 64, BF16, g)
    q = randn((2, 4, 64), g, BF16)
    n = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    none = binding.KVCache(cache.k, cache.v, cache.page_table[:0])
    assert enc.paged_attn(none, q[:0], n[:0]).shape == (0, 4, 64)
    for kw in [dict(q=q.half()), dict(q=q[:1]), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(n=n.long()), dict(n=n[:1]),
               dict(out=q.float()), dict(out=q[:, :2]), dict(lse=torch.empty(2, 4, dtype=F16, device="cuda")), dict(max_len=-1),
               dict(scale=float("nan")), dict(q=q.cpu())]:
        a = {**dict(q=q, n=n, out=None, lse=None, max_len=0, scale=None), **kw}
        with pytest.raises((ValueError, binding.MossEncError)):
            enc.paged_attn(cache, a["q"], a["n"], a["scale"], out=a["out"], lse=a["lse"], max_len=a["max_len"])
    check_attn(enc, cache, q, [5, 6])


def test_paged_calls_past_32_bits(enc):
    # three pages 1.3e9 elements apart: byte and element offsets pass 2^32
    far = 1_300_000_000
    buf = torch.zeros(2 * far + 4096, dtype=BF16, device="cuda")
    k = buf.as_strided((3, 16, 2, 64), (far, 128, 64, 1))
    v = buf.as_strided((3, 16, 2, 64), (far, 128, 64, 1), 2048)
    g = gen(42)
    table = torch.tensor([[2, 1, 0]], dtype=torch.int32, device="cuda")
    cache = binding.KVCache(k, v, table)
    rows = randn((48, 2, 64), g, BF16)
    enc.kv_append(cache, rows, rows * 2, torch.arange(48, dtype=torch.int32, device="cuda"),
                  torch.zeros(48, dtype=torch.int32, device="cuda"))
    enc.synchronize()
    got_k, got_v = read(cache, 0, 48)
    assert torch.equal(got_k, rows.double()) and torch.equal(got_v, rows.double() * 2)
    check_attn(enc, cache, randn((1, 4, 64), g, BF16), [41])
    del k, v, cache, buf
    torch.cuda.empty_cache()


# ------------------------------------------------------ together

def step_setup(g, seqs, capacity, ct=BF16):
    hq, hkv, dim, width = 8, 2, 64, 512
    cache = make_cache(seqs, capacity, 16, hkv, dim, ct, g)
    qkv = gemv_case(1, (hq + 2 * hkv) * dim, width, 50)[1:]
    proj = gemv_case(1, width, hq * dim, 51)[1:]
    inv = 1e4 ** (-torch.arange(dim // 2, device="cuda", dtype=torch.float64) * 2 / dim)
    return cache, qkv, proj, inv, (hq, hkv, dim, width)


def step(enc, cache, qkv, proj, inv, dims, x, resid, lengths, workspace=None):
    """One layer's attention side: products, append, attention, product onto
    the residual.  lengths count the new token."""
    hq, hkv, dim, _ = dims
    rows = x.shape[0]
    y = enc.gemv_q4(x, *qkv)
    q = y[:, :hq * dim].view(rows, hq, dim)
    k = y[:, hq * dim:(hq + hkv) * dim].view(rows, hkv, dim)
    v = y[:, (hq + hkv) * dim:].view(rows, hkv, dim)
    turned_q = enc.kv_append(cache, k, v, lengths - 1, q=q, inv_freq=inv)
    o = enc.paged_attn(cache, turned_q, lengths, workspace=workspace)
    enc.gemv_q4(o.view(rows, hq * dim), *proj, out=resid, epilogue=2)
    return y, o


@pytest.mark.parametrize("ct", [BF16, E4M3])
def test_decoding_steps(enc, ct):
    g = gen(60)
    seqs = 5
    cache, qkv, proj, inv, dims = step_setup(g, seqs, 400, ct)
    hq, hkv, dim, width = dims
    lengths = torch.tensor([1, 16, 33, 200, 380], dtype=torch.int32, device="cuda")
    for _ in range(6):
        x = randn((seqs, width), g, BF16)
        resid = randn((seqs, width), g)
        was = resid.clone()
        y, o = step(enc, cache, qkv, proj, inv, dims, x, resid, lengths)
        enc.synchronize()
        ref, tol = gemv_ref(x, *qkv)
        within(y, ref, tol + (ref.abs() + tol) * half_step(BF16) + TINY[BF16])
        pos = lengths - 1
        q, k, v = y[:, :hq * dim], y[:, hq * dim:(hq + hkv) * dim], y[:, (hq + hkv) * dim:]
        for s in range(seqs):
            got_k, got_v = read(cache, s, int(lengths[s]))
            check_rows((got_k[-1:] / cache.desc.k_scale).to(ct), k[s:s + 1].view(1, hkv, dim), pos[s:s + 1], inv, False, ct, cache.desc.k_scale)
            check_rows((got_v[-1:] / cache.desc.v_scale).to(ct), v[s:s + 1].view(1, hkv, dim), pos[s:s + 1], None, False, ct, cache.desc.v_scale)
        again = torch.empty(seqs, hq, dim, dtype=BF16, device="cuda")
        enc.kv_append(cache, k.reshape(seqs, hkv, dim), v.reshape(seqs, hkv, dim), pos, q=q.reshape(seqs, hq, dim), q_out=again, inv_freq=inv)
        ref, _, tol, _ = attn_ref(cache, again, lengths.tolist(), dim ** -0.5)
        within(o, ref, tol)
        ref, tol = gemv_ref(o.view(seqs, -1), *proj)
        within(resid, ref + was.double(), tol + (ref + was.double()).abs() * U)
        lengths = lengths + 1


def test_decoding_step_on_another_stream_and_in_graphs():
    # two captured steps over two caches, each with its own workspace, replayed
    # side by side on two streams with new inputs, against the eager step
    g = gen(61)
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    e = binding.Encoder(weights(1), 1, max_samples=16000, max_clips=1)
    sets = []
    for stream, longest in ((s0, 90000), (s1, 50000)):
        cache, qkv, proj, inv, dims = step_setup(g, 3, longest)
        n = torch.tensor([longest - 50, 700, 1], dtype=torch.int32, device="cuda")
        x = randn((3, dims[3]), g, BF16)
        resid = torch.zeros(3, dims[3], device="cuda")
        work = torch.empty(max(16, e.paged_attn_workspace(cache, dims[0])), dtype=torch.uint8, device="cuda")
        e.set_stream(stream)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            step(e, cache, qkv, proj, inv, dims, x, resid, n, work)  # eager once
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(e, cache, qkv, proj, inv, dims, x, resid, n, work)
        sets.append((stream, graph, cache, qkv, proj, inv, dims, x, resid, n))
    torch.cuda.synchronize()
    for round_ in range(4):
        news = []
        for stream, graph, cache, qkv, proj, inv, dims, x, resid, n in sets:
            x.copy_(randn(x.shape, g, BF16))
            n += 1
            resid.zero_()
        torch.cuda.synchronize()
        for stream, graph, *_ in sets:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for stream, graph, cache, qkv, proj, inv, dims, x, resid, n in sets:
            news.append(resid.clone())
        e.set_stream(torch.cuda.current_stream())
        for (stream, graph, cache, qkv, proj, inv, dims, x, resid, n), got in zip(sets, news):
            resid.zero_()
            step(e, cache, qkv, proj, inv, dims, x, resid, n)
            torch.cuda.synchronize()
            assert torch.equal(resid, got)
    e.synchronize()
    del sets, graph
    e.close()


def test_decode_calls_on_a_stream_that_is_not_current():
    # the handle's stream is not torch's: what the calls allocate belongs to
    # the handle's, and work before and after is ordered by the caller
    g = gen(62)
    e = binding.Encoder(weights(1), 1, max_samples=16000, max_clips=1)
    cache, qkv, proj, inv, dims = step_setup(g, 3, 9000)
    n = torch.tensor([8000, 700, 1], dtype=torch.int32, device="cuda")
    x = randn((3, dims[3]), g, BF16)
    want = torch.zeros(3, dims[3], device="cuda")
    step(e, cache, qkv, proj, inv, dims, x, want, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    e.set_stream(side)
    for _ in range(5):
        got = torch.zeros(3, dims[3], device="cuda")
        pos = n - 1
        torch.cuda.synchronize()
        y = e.gemv_q4(x, *qkv)
        hq, hkv, dim, _ = dims
        q = e.kv_append(cache, y[:, hq * dim:(hq + hkv) * dim].view(3, hkv, dim), y[:, (hq + hkv) * dim:].view(3, hkv, dim),
                        pos, q=y[:, :hq * dim].view(3, hq, dim), inv_freq=inv)
        o = e.paged_attn(cache, q, n)
        e.gemv_q4(o.view(3, -1), *proj, out=got, epilogue=2)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]  # the current stream reuses what is free
        e.synchronize()
        assert torch.equal(got, want)
        del junk
    e.close()


def test_decode_calls_on_another_stream_may_be_given_temporaries():
    # the handle's stream is busy while the caller's goes on: what the calls
    # were given is freed at once, and the next tensors of its size are NaN
    g = gen(65)
    e = binding.Encoder(weights(1), 1, max_samples=16000, max_clips=1)
    cache, qkv, proj, inv, dims = step_setup(g, 3, 9000)
    hq, hkv, dim, width = dims
    n = torch.tensor([8000, 700, 1], dtype=torch.int32, device="cuda")
    x = randn((3, width), g, BF16)

    def ready(*made):  # on the current stream, before the handle's goes on
        e.stream.wait_stream(torch.cuda.current_stream())
        return made

    def calls():
        y = e.gemv_q4(*ready(x.clone()), *qkv)
        q, k, v = (t.view(3, -1, dim) for t in y.split([hq * dim, hkv * dim, hkv * dim], 1))
        q = e.kv_append(cache, k, v, *ready(n - 1, torch.arange(3, dtype=torch.int32, device="cuda"), q, None, inv.clone()))
        o, lse = e.paged_attn(cache, q, *ready(n.clone()), return_lse=True)
        return y, q, o, lse, e.gemv_q4(o.flatten(1), *ready(*(t.clone() for t in proj)), epilogue=5)

    want = calls()
    torch.cuda.synchronize()
    sizes = [(t.shape, t.dtype) for t in (x, n, n.long(), inv, *proj)]
    side = torch.cuda.Stream()
    e.set_stream(side)
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
        got = calls()
        junk = [torch.empty(s, dtype=t, device="cuda").view(torch.uint8).fill_(255) for s, t in sizes for _ in range(6)]
        e.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
    e.close()


def test_decode_calls_are_counted_and_profiled(enc):
    g = gen(63)
    cache, qkv, proj, inv, dims = step_setup(g, 3, 100)
    n = torch.tensor([80, 70, 1], dtype=torch.int32, device="cuda")
    x, resid = randn((3, dims[3]), g, BF16), torch.zeros(3, dims[3], device="cuda")
    enc.synchronize()
    before = enc.launch_count()
    enc.profile_enable(64)
    step(enc, cache, qkv, proj, inv, dims, x, resid, n)
    stats = enc.profile_read()
    enc.profile_enable(0)
    assert stats["gemv_q4"]["launches"] == 2 and stats["kv_append"]["launches"] == 1
    assert stats["paged_attn"]["launches"] >= 1 and enc.launch_count() - before >= 4
