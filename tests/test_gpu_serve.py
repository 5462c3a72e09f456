"""Serving operators on the GPU against the float64 oracle.

Tolerances (half a unit in the last place u: bf16 2^-8, float32 2^-24, e4m3
2^-4 relative, e4m3 subnormals 2^-10 of the scale):
  * rotation: u |y| for the one rounding, plus 2^-18 of the head's largest
    element for the float32 arithmetic before it (a norm over 128 dims is under
    24 roundings of 2^-24; the fast cos and sin of bf16 heads are off by at
    most 2^-20 absolute after the angle's own 2^-22) and 2^-19 for float32;
  * append: half a code step of the exact value, widened by 2^-16 of the
    head's largest element for the same float32 arithmetic;
  * cache attention: u |o| for the bf16 output plus 2^-10 of the largest |v|
    of the keys: probabilities enter the product as float16 (2^-11 relative,
    2^-25 absolute against the largest, so 2^-11 + n 2^-25 of sum p|v|/sum p
    with n <= 2^12 keys here), and 2^-11 is left for ex2.approx (2^-22) and
    float32 sums;
  * packed prompts: u |o| for the output, u times the row's sum p|v| / sum p for
    probabilities that enter the product as bf16, and 2^-12 of the largest |v|
    for ex2.approx and float32 sums;
  * log-sum-exp: 2^-17 (1 + the largest sum |q_d k_d| scale): float32 sums of
    128 products and one exp2/log2 each way.
"""
import math

import numpy as np
import pytest
import torch

from content_routed_block_ssa_b200 import ssa
from oracle import serve_oracle as S

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def rng_of(*key):
    return np.random.default_rng([sum(map(ord, str(k))) for k in key])


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(dtype) if dtype is not None else t).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def ok():
    torch.cuda.synchronize()
    assert ssa.ssa_device_error() == 0


# ---------------------------------------------------------------- rotation

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
FUZZ = {"bf16": 2.0 ** -18, "f32": 2.0 ** -19}


def check_rope(got, x, w, f, pos, layout, m, norm, eps, dtype):
    ref = S.norm(x, w, eps) if norm else np.array(x)
    big = np.abs(ref).max(-1, keepdims=True) * max(abs(m), 1.0)
    ref = S.rotate(ref, f, pos, layout, m)
    assert (np.abs(f64(got) - ref) <= U[dtype] * np.abs(ref) + FUZZ[dtype] * big).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,layout", [(128, 128, "half"), (128, 128, "pairs"), (128, 96, "half"), (64, 16, "pairs"),
                                          (64, 64, "half"), (64, 48, "half"), (128, 32, "pairs"), (128, 0, "half")])
@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (3, 7, 2), (37, 32, 8)])
def test_rope(dtype, d, rot, layout, T, hq, hkv):
    r = rng_of(dtype, d, rot, layout, T)
    # a joint projection with a gap behind it: strided tokens
    x = dev(r.normal(size=(T, hq + 2 * hkv + 1, d)) * r.choice([0.1, 1, 30], size=(T, 1, 1)), TD[dtype])
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    qw, kw = dev(r.normal(size=d), torch.float32), dev(1 + r.normal(size=d), torch.float32)
    f, _ = ssa.rope_frequencies(max(rot, 2), 10000.0)
    f = f[:rot // 2]
    pos = r.integers(-5, 1 << 20, size=T)
    qo, ko = torch.full_like(q, 7.0).contiguous(), torch.full_like(k, 7.0).contiguous()
    p = ssa.make_rope_params(T, hq, hkv, d, rot, layout, dtype, True, 1e-5, 1.25, q_stride=x.stride(0), k_stride=x.stride(0))
    before = x.clone()
    ssa.ssa_qk_rope(p, q, k, qw, kw, f.cuda(), dev(pos, torch.int32), qo, ko)
    ok()
    assert torch.equal(x, before)
    check_rope(qo, f64(q), f64(qw), f.numpy(), pos, layout, 1.25, True, 1e-5, dtype)
    check_rope(ko, f64(k), f64(kw), f.numpy(), pos, layout, 1.25, True, 1e-5, dtype)
    # in place, without the norm
    p = ssa.make_rope_params(T, hq, hkv, d, rot, layout, dtype, False, q_stride=x.stride(0), k_stride=x.stride(0),
                             q_out_stride=x.stride(0), k_out_stride=x.stride(0))
    ssa.ssa_qk_rope(p, q, k, qw, kw, f.cuda(), dev(pos, torch.int32), q, k)
    ok()
    check_rope(q, f64(before[:, :hq]), None, f.numpy(), pos, layout, 1.0, False, 0, dtype)
    check_rope(k, f64(before[:, hq:hq + hkv]), None, f.numpy(), pos, layout, 1.0, False, 0, dtype)
    assert torch.equal(x[:, hq + hkv:], before[:, hq + hkv:])      # values and gap untouched


def test_rope_many_tokens_and_far_positions():
    """More tokens than one wave of warps, positions up to 2^31 - 1: a
    float32 angle would be off by many turns."""
    T, d = 3001, 64
    r = rng_of("far")
    q, k = dev(r.normal(size=(T, 2, d)), torch.float32), dev(r.normal(size=(T, 1, d)), torch.float32)
    f, m = ssa.rope_frequencies(d, 500000.0, "blend", 32.0, 8192.0)
    pos = r.integers(-(1 << 31), 1 << 31, size=T)
    pos[:3] = [(1 << 31) - 1, -(1 << 31), 0]
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    p = ssa.make_rope_params(T, 2, 1, d, dtype="f32", norm=False, mscale=m)
    ssa.ssa_qk_rope(p, q, k, None, None, f.cuda(), dev(pos, torch.int32), qo, ko)
    ok()
    # 2^-53 relative in the frequency is 2^-22 turns of 2^31 positions at one
    # radian each: allow 2 pi 2^-23 of the pair besides the float32 part
    ref = S.rotate(f64(q), f.numpy(), pos, "half", m)
    big = np.abs(f64(q)).max(-1, keepdims=True) * m
    assert (np.abs(f64(qo) - ref) <= U["f32"] * np.abs(ref) + (FUZZ["f32"] + 2.0 ** -20) * big).all()


def turns(freq, pos):
    """pos * freq / (2 pi) modulo one in exact arithmetic (freq is a float64)."""
    from fractions import Fraction
    two_pi = Fraction(62831853071795864769252867665590057683943387987502, 10 ** 49)
    return float(Fraction(float(freq)) * int(pos) / two_pi % 1)


@pytest.mark.parametrize("T", [40, 15000])   # straight, and streamed
@pytest.mark.parametrize("fast", [3.0, 1000.0, 1e6])
def test_rope_positions_lose_nothing(T, fast):
    """Frequencies of up to `fast` radians at positions up to 2^31: the angle's
    error does not grow with either (the float32 part is FUZZ, as above)."""
    d = 64
    r = rng_of("turns", fast)
    x = dev(r.normal(size=(T, 1, d)), torch.float32)
    f = torch.from_numpy(np.exp(r.uniform(np.log(fast) - 3, np.log(fast), size=d // 2)))
    pos = r.integers(-(1 << 31), 1 << 31, size=T)
    pos[:4] = [(1 << 31) - 1, -(1 << 31), 0, 1]
    q, k = torch.empty_like(x), torch.empty_like(x)
    p = ssa.make_rope_params(T, 1, 1, d, dtype="f32", norm=False)
    ssa.ssa_qk_rope(p, x, x, None, None, f.cuda(), dev(pos, torch.int32), q, k)
    ok()
    assert torch.equal(q, k)
    n = np.arange(40) if T == 40 else np.concatenate([[0, 1, 2, 3], r.integers(0, T, 60)])
    a = np.array([[2 * math.pi * turns(g, t) for g in f] for t in pos[n]])
    v = f64(x)[n, 0]
    u, w = v[:, :d // 2], v[:, d // 2:]
    ref = np.concatenate([u * np.cos(a) - w * np.sin(a), w * np.cos(a) + u * np.sin(a)], 1)
    big = np.abs(v).max(-1, keepdims=True)
    assert (np.abs(f64(q)[n, 0] - ref) <= U["f32"] * np.abs(ref) + FUZZ["f32"] * big).all()


def test_appended_keys_turn_by_their_far_positions():
    """The same for keys appended next to position 2^31."""
    d, page, n = 64, 128, 100
    r = rng_of("turnsapp")
    width = (1 << 31) // page - 1
    have = width * page - n
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, have // page:] = 0
    x = dev(r.normal(size=(n, 1, d)), torch.float32)
    f = torch.from_numpy(np.exp(r.uniform(11, 14, size=d // 2)))
    kc, vc = (torch.zeros(1, 1, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((1, 1), 2.0 ** -40, device="cuda") for _ in range(2))
    p = ssa.make_append_params(n, 1, width, 1, page, 1, d, dtype="f32", norm=False)
    ssa.ssa_cache_append(p, x, x, None, f.cuda(), dev([0, n], torch.int32), dev([have], torch.int32), table, kc, vc, ks, vs)
    ok()
    a = np.array([[2 * math.pi * turns(g, have + t) for g in f] for t in range(n)])
    v = f64(x)[:, 0]
    u, w = v[:, :d // 2], v[:, d // 2:]
    ref = np.concatenate([u * np.cos(a) - w * np.sin(a), w * np.cos(a) + u * np.sin(a)], 1)
    s = float(ks)
    got = S.e4m3_values()[kc.cpu().numpy()[0, 0, page - n:]] * s
    assert (np.abs(got - ref) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * s + 2.0 ** -16 * np.abs(v).max(-1, keepdims=True)).all()


@pytest.mark.parametrize("dtype,d,rot,layout,hq,hkv,T", [
    ("bf16", 128, 128, "half", 32, 8, 2600), ("bf16", 64, 32, "pairs", 33, 1, 3000), ("f32", 128, 96, "half", 9, 3, 3001),
    ("f32", 64, 64, "pairs", 5, 17, 2500), ("bf16", 128, 0, "half", 1, 1, 4000),
    # runs of pieces that end inside a token, and whole tokens per warp
    ("bf16", 128, 128, "half", 17, 3, 1800), ("bf16", 128, 0, "half", 1, 1, 6000),
    ("bf16", 128, 128, "half", 2, 1, 14300), ("f32", 64, 48, "pairs", 9, 1, 14500)])
def test_rope_of_many_tokens(dtype, d, rot, layout, hq, hkv, T):
    """Enough tokens for the streaming kernel, ragged numbers of heads per
    piece, in place too: sampled tokens against the oracle, every token
    against the same tokens in small calls (two roundings apart at most)."""
    r = rng_of("stream", dtype, d, hq)
    x = dev(r.normal(size=(T, hq + hkv + 1, d)), TD[dtype])
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    qw, kw = dev(r.normal(size=d), torch.float32), dev(1 + r.normal(size=d), torch.float32)
    f = ssa.rope_frequencies(max(rot, 2))[0][:rot // 2]
    pos = r.integers(-100, 1 << 20, size=T)
    pd, fd = dev(pos, torch.int32), f.cuda()
    small = []
    for i in range(0, T, 100):
        n = min(100, T - i)
        p = ssa.make_rope_params(n, hq, hkv, d, rot, layout, dtype, True, 1e-6, 1.1, q_stride=x.stride(0), k_stride=x.stride(0))
        o = torch.empty(n, hq, d, device="cuda", dtype=TD[dtype]), torch.empty(n, hkv, d, device="cuda", dtype=TD[dtype])
        ssa.ssa_qk_rope(p, q[i:i + n], k[i:i + n], qw, kw, fd, pd[i:i + n], *o)
        small.append(o)
    small = [torch.cat(s) for s in zip(*small)]
    before = x.clone()
    s = x.stride(0)
    p = ssa.make_rope_params(T, hq, hkv, d, rot, layout, dtype, True, 1e-6, 1.1, s, s, s, s)
    ssa.ssa_qk_rope(p, q, k, qw, kw, fd, pd, q, k)
    ok()
    assert torch.equal(x[:, hq + hkv:], before[:, hq + hkv:])
    at = np.unique(np.concatenate([r.integers(0, T, 60), [0, T - 1]]))
    for got, was, w, sm in ((q, before[:, :hq], qw, small[0]), (k, before[:, hq:hq + hkv], kw, small[1])):
        check_rope(got[at], f64(was[at]), f64(w), f.numpy(), pos[at], layout, 1.1, True, 1e-6, dtype)
        a, b = got.double(), sm.double()
        big = b.abs().amax(-1, keepdim=True)
        assert ((a - b).abs() <= 2 * U[dtype] * b.abs() + 2 * FUZZ[dtype] * big).all()


def test_rope_leaves_unrotated_infinities_and_keeps_heads_apart():
    x = torch.ones(2, 3, 128, device="cuda")
    x[0, 0, 100] = math.inf
    x[1, 1, 3] = math.nan
    f = ssa.rope_frequencies(64)[0].cuda()
    p = ssa.make_rope_params(2, 2, 1, 128, 64, dtype="f32", norm=False, q_stride=384, k_stride=384)
    q, k = torch.empty(2, 2, 128, device="cuda"), torch.empty(2, 1, 128, device="cuda")
    ssa.ssa_qk_rope(p, x[:, :2], x[:, 2:], None, None, f, torch.tensor([5, 9], dtype=torch.int32, device="cuda"), q, k)
    ok()
    assert q[0, 0, 100] == math.inf and torch.isfinite(q[0, 0, :100]).all() and torch.isfinite(q[0, 1]).all()
    assert q[1, 1].isnan().nonzero().flatten().tolist() == [3, 35] and torch.isfinite(k).all()


# ---------------------------------------------------------------- append

def pool(r, n_pages, h, page, d):
    codes = r.integers(0, 256, size=(2, n_pages, h, page, d)).astype(np.uint8)
    codes[(codes & 127) == 127] = 0
    scale = 2.0 ** r.integers(-9, -5, size=(2, n_pages, h))
    return codes, scale


def run_append(p, K, V, w, f, cu, have, table, codes, scale):
    kc, vc = dev(codes[0]), dev(codes[1])
    ks, vs = dev(scale[0], torch.float32), dev(scale[1], torch.float32)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (p, K, V, w, f, dev(cu, torch.int32), dev(have, torch.int32), dev(table, torch.int32), kc, vc, ks, vs)
    ssa.ssa_cache_append(*args, bad)
    ok()
    one = [t.clone() for t in (kc, vc, ks, vs)]
    ssa.ssa_cache_append(*args)                     # the same tokens again: the same bytes
    ok()
    assert all(torch.equal(a, b) for a, b in zip(one, (kc, vc, ks, vs)))
    return (kc, vc, ks, vs), int(bad)


def check_codes(got_c, got_s, ref_c, ref_s, x, cu, have, table, page, old_c):
    """Scales equal; codes equal but where the exact value is too near a
    border between codes for float32 to tell; nothing else changed."""
    got_c, got_s = got_c.cpu().numpy(), f64(got_s)
    assert np.array_equal(got_s, ref_s)
    differ = np.argwhere(got_c != ref_c)
    where = {}
    for s in range(len(have)):
        for o, row in enumerate(range(cu[s], cu[s + 1])):
            pos = have[s] + o
            if have[s] >= 0 and pos // page < table.shape[1] and 0 <= table[s, pos // page] < len(ref_c):
                where[(table[s, pos // page], pos % page)] = row
    val = S.e4m3_values()
    for pid, h, sl, i in differ:
        row = where[(pid, sl)]                      # only appended slots may differ
        step = max(2.0 ** -4 * abs(x[row, h, i]), 2.0 ** -10 * ref_s[pid, h])
        off = abs(val[got_c[pid, h, sl, i]] * ref_s[pid, h] - x[row, h, i])
        assert off <= step * (1 + 2.0 ** -8) + 2.0 ** -16 * np.abs(x[row, h]).max()
    assert len(differ) <= 1 + 1e-3 * sum(cu[s + 1] - cu[s] for s in range(len(have))) * ref_c.shape[1] * ref_c.shape[3]


def append_case(r, n_seq, page, news, haves):
    cu = np.concatenate([[0], np.cumsum(news)])
    pages = [(h + n + page - 1) // page for h, n in zip(haves, news)]
    width = max(max(pages), 1)
    ids = r.permutation(sum(pages) + 2)
    table, at = np.full((n_seq, width), -1), 0
    for s, n in enumerate(pages):
        table[s, :n] = ids[at:at + n]
        at += n
    return cu, table, len(ids)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,rot,layout", [(128, 64, 128, "half"), (64, 128, 48, "pairs"), (128, 128, 64, "half"),
                                               (64, 64, 0, "half")])
@pytest.mark.parametrize("news,haves", [
    ([1], [0]), ([1, 1, 1, 1], [0, 63, 64, 130]),             # decode: fresh page, last slot, page border
    ([3, 0, 17, 1, 5], [62, 5, 120, 0, 127]),                 # ragged, an empty sequence, pages that end inside
    ([200], [0]), ([131, 1, 70], [30, 64, 1]),                # prompts over several pages
    ([0, 0], [3, 0]),
])
def test_append(dtype, d, page, rot, layout, news, haves):
    r = rng_of(dtype, d, page, rot, news, haves)
    h = 3
    cu, table, n_pages = append_case(r, len(news), page, news, haves)
    T = int(cu[-1]) + 4                                       # tokens behind the last sequence are not used
    x = dev(r.normal(size=(T, 2 * h, d)) * 2.0 ** r.integers(-3, 4, size=(T, 1, 1)), TD[dtype])
    x[cu[-1]:] = math.nan
    K, V = x[:, :h], x[:, h:]
    w = dev(1 + 0.2 * r.normal(size=d), torch.float32)
    f, _ = ssa.rope_frequencies(max(rot, 2))
    f = f[:rot // 2]
    codes, scale = pool(r, n_pages, h, page, d)
    p = ssa.make_append_params(T, len(news), table.shape[1], n_pages, page, h, d, rot, layout, dtype, True, 1e-6, 1.0,
                               k_stride=x.stride(0), v_stride=x.stride(0))
    (kc, vc, ks, vs), bad = run_append(p, K, V, w, f.cuda(), cu, haves, table, codes, scale)
    assert bad == 0
    pos = np.concatenate([np.arange(hv, hv + n) for hv, n in zip(haves, news)] + [np.zeros(4, int)])
    kx = f64(K)
    kx[cu[-1]:] = 0
    kx = S.rotate(S.norm(kx, f64(w), 1e-6), f.numpy(), pos, layout)
    for got, gs, xx, j in ((kc, ks, kx, 0), (vc, vs, f64(V), 1)):
        rc, rs, _ = S.append(xx, cu, haves, table, page, codes[j], scale[j])
        check_codes(got, gs, rc, rs, xx, cu, haves, table, page, codes[j])


@pytest.mark.parametrize("few", [True, False])
def test_append_plain_values_are_bit_exact_and_survive_growth(few):
    """No norm, no rotation: the codes are the rounding of the inputs, bit
    for bit, through a growing scale, infinities, NaN and zeros."""
    r = rng_of("grow")
    page, d, h = 64, 128, 2
    n = 40 if not few else 8
    codes, scale = pool(r, 3, h, page, d)
    scale[:] = 2.0 ** -12
    x = r.normal(size=(n, h, d)).astype(np.float32)
    x[0, 0, :4] = [np.inf, -np.inf, np.nan, 0.0]
    x[n - 1, 1] = 1e30                                        # far above the page's old scale
    x[1, 1, 0] = 3e-39                                        # a float32 subnormal
    K = dev(x)
    V = torch.zeros_like(K)
    cu, have, table = np.array([0, n]), np.array([20]), np.array([[2]])
    if few:                                                   # many sequences without tokens: the decode kernel
        cu, have, table = np.array([0] * 4 + [n]), np.array([5, 5, 5, 20]), np.array([[0], [0], [1], [2]])
    p = ssa.make_append_params(n, len(have), 1, 3, page, h, d, 0, "half", "f32", False)
    (kc, vc, ks, vs), bad = run_append(p, K, V, None, None, cu, have, table, codes, scale)
    rc, rs, _ = S.append(x.astype(np.float64), cu, have, table, page, codes[0], scale[0])
    got = kc.cpu().numpy()
    nan = (rc & 127) == 127
    assert np.array_equal(got[~nan], rc[~nan]) and ((got[nan] & 127) == 127).all()
    assert np.array_equal(f64(ks), rs) and bad == 0
    assert rs[2, 1] == 2.0 ** S.exponent([1e30])
    rv, rvs, _ = S.append(np.zeros((n, h, d)), cu, have, table, page, codes[1], scale[1])
    assert np.array_equal(vc.cpu().numpy(), rv) and np.array_equal(f64(vs), rvs) and (rvs[2] == 2.0 ** -12).all()


def test_append_fresh_page_of_zeros_and_tiny_values():
    K = torch.zeros(2, 1, 64, device="cuda")
    V = torch.full((2, 1, 64), 1e-20, device="cuda")
    codes, scale = pool(rng_of("z"), 1, 1, 64, 64)
    p = ssa.make_append_params(2, 1, 1, 1, 64, 1, 64, 0, "half", "f32", False)
    (kc, vc, ks, vs), _ = run_append(p, K, V, None, None, np.array([0, 2]), np.array([0]), np.array([[0]]), codes, scale)
    assert ks.item() == vs.item() == 2.0 ** -40
    assert not (kc[0, 0, :2] & 127).any() and not (vc[0, 0, :2] & 127).any()
    assert np.array_equal(kc[0, 0, 2:].cpu().numpy(), codes[0][0, 0, 2:])   # the rest of the page as it was


@pytest.mark.parametrize("n", [2, 150])
def test_append_leaves_out_what_does_not_fit(n):
    """Pages outside the pool, negative lengths, tokens past the table and
    decreasing offsets are left out and counted; nothing else is written."""
    r = rng_of("bad", n)
    page, d, h = 64, 64, 2
    x = dev(r.normal(size=(5 * n, 2 * h, d)), torch.bfloat16)
    cu = np.array([0, n, 2 * n, 3 * n, 4 * n, 5 * n])
    have = np.array([0, -1, 3 * page - 1, 10, 2 * page])      # the third has one slot left in the table
    table = np.array([[7, 7, 7], [0, 1, 2], [-1, -1, 5], [-9, 1 << 30, 6], [0, 1, 2]])
    codes, scale = pool(r, 7, h, page, d)
    p = ssa.make_append_params(5 * n, 5, 3, 7, page, h, d, 0, "half", "bf16", False, k_stride=x.stride(0),
                               v_stride=x.stride(0))
    (kc, vc, ks, vs), bad = run_append(p, x[:, :h], x[:, h:], None, None, cu, have, table, codes, scale)
    for got, gs, xx, j in ((kc, ks, f64(x[:, :h]), 0), (vc, vs, f64(x[:, h:]), 1)):
        rc, rs, rb = S.append(xx, cu, have, table, page, codes[j], scale[j])
        assert np.array_equal(got.cpu().numpy(), rc) and np.array_equal(f64(gs), rs) and rb == bad
    # offsets that decrease or leave the rows: nothing out of bounds is read
    for odd in ([0, 4 * n, n, 1 << 30, -5, 5 * n], [-3, -2, -1, 9 * n, 9 * n, 9 * n], [5 * n] * 6):
        run_append(p, x[:, :h], x[:, h:], None, None, np.array(odd), have, table, codes, scale)


def test_append_many_sequences():
    """More sequences than one 32-way search step covers, some without tokens."""
    r = rng_of("many")
    page, d, h, n_seq = 64, 64, 1, 1100
    news = r.integers(0, 4, size=n_seq)
    news[500] = 90
    haves = r.integers(0, 130, size=n_seq)
    cu, table, n_pages = append_case(r, n_seq, page, news, haves)
    x = r.normal(size=(int(cu[-1]), h, d)).astype(np.float32)
    codes, scale = pool(r, n_pages, h, page, d)
    p = ssa.make_append_params(int(cu[-1]), n_seq, table.shape[1], n_pages, page, h, d, 0, "half", "f32", False)
    (kc, vc, ks, vs), bad = run_append(p, dev(x), dev(-x), None, None, cu, haves, table, codes, scale)
    rc, rs, _ = S.append(x.astype(np.float64), cu, haves, table, page, codes[0], scale[0])
    assert np.array_equal(kc.cpu().numpy(), rc) and np.array_equal(f64(ks), rs) and bad == 0


# ---------------------------------------------------------------- attention over the cache

def cache_case(r, lens, n_q, h_kv, G, d, page, topk=0):
    n = len(lens)
    pages = [max((L + page - 1) // page, 0) for L in lens]
    width = max(max(pages), 1) + 1
    ids = r.permutation(sum(pages) + 1)
    table, at = np.full((n, width), -1), 0
    for s, c in enumerate(pages):
        table[s, :c] = ids[at:at + c]
        at += c
    codes, scale = pool(r, len(ids), h_kv, page, d)
    codes = S.to_e4m3(100 * r.normal(size=codes.shape))
    scale = 2.0 ** r.integers(-9, -4, size=scale.shape)
    q = dev(r.normal(size=(n, n_q, h_kv * G, d)), torch.bfloat16)
    idx = None
    if topk:
        idx = np.full((n, n_q, h_kv, topk), -1)
        for s in range(n):
            for i in range(n_q):
                nvis = max(lens[s] - n_q + i + 1, 0) // page
                for h in range(h_kv):
                    c = np.sort(r.permutation(nvis)[:topk])
                    idx[s, i, h, :len(c)] = c
    return table, codes, scale, q, idx


def run_cache(q, lens, table, codes, scale, page, idx=None, window=0, sm_scale=None, bad=None, stream=None):
    n, n_q, h_q, d = q.shape
    _, n_pages, h_kv = scale.shape
    p = ssa.make_cache_attn_params(n, n_q, table.shape[1], n_pages, page, h_q, h_kv, d,
                                   0 if idx is None else idx.shape[-1], window, sm_scale)
    ws = ssa.byte_buffer(ssa.ssa_cache_attn_workspace_size(p))
    ws.fill_(255)                                             # NaN: nothing of it may count
    o = torch.full_like(q, math.nan)
    lse = torch.full((n, n_q, h_q), math.nan, device="cuda")
    ssa.ssa_cache_attn(p, q, dev(table, torch.int32), dev(lens, torch.int32), dev(codes[0]), dev(codes[1]),
                       dev(scale[0], torch.float32), dev(scale[1], torch.float32),
                       None if idx is None else dev(idx, torch.int32), o, lse, bad, ws, stream)
    ok()
    return o, lse, p


def check_cache(o, lse, q, lens, table, codes, scale, page, idx=None, window=0, sm_scale=None):
    d = q.shape[-1]
    sm = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    ro, rl = S.cache_attention(f64(q), table, lens, page, codes[0], codes[1], scale[0], scale[1], sm, idx, window)
    o, lse = f64(o), f64(lse)
    vmax = 448.0 * scale[1].max() if codes[1].size else 1.0
    qmax = np.abs(f64(q)).sum(-1).max() * 448.0 * scale[0].max() * sm
    assert (np.abs(o - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * vmax).all()
    empty = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), empty) and (o[empty] == 0).all()
    assert (np.abs(lse[~empty] - rl[~empty]) <= 2.0 ** -17 * (1 + qmax)).all()


@pytest.mark.parametrize("d,page", [(128, 64), (64, 128), (128, 128), (64, 64)])
@pytest.mark.parametrize("h_kv,G,n_q", [(2, 4, 1), (1, 8, 3), (3, 1, 1), (2, 3, 5), (1, 16, 2), (1, 2, 37)])
@pytest.mark.parametrize("lens", [[1], [0, 31, 32, 33, 64], [700, 1, 129], [40, -7, 2]])
def test_cache_attention(d, page, h_kv, G, n_q, lens):
    r = rng_of(d, page, h_kv, G, n_q, lens)
    table, codes, scale, q, _ = cache_case(r, lens, n_q, h_kv, G, d, page)
    o, lse, _ = run_cache(q, lens, table, codes, scale, page)
    check_cache(o, lse, q, lens, table, codes, scale, page)


@pytest.mark.parametrize("d,page", [(128, 64), (64, 128)])
def test_cache_attention_split_over_a_long_axis(d, page):
    r = rng_of("long", d)
    lens = [3000, 4096, 1500]
    table, codes, scale, q, _ = cache_case(r, lens, 1, 2, 4, d, page)
    o, lse, p = run_cache(q, lens, table, codes, scale, page)
    assert ssa.ssa_cache_attn_workspace_size(p) > 0            # several splits, joined
    check_cache(o, lse, q, lens, table, codes, scale, page)
    # a table far wider than the lengths: most splits are empty
    wide = np.full((3, 4096), -1)
    wide[:, :table.shape[1]] = table
    o2, lse2, _ = run_cache(q, lens, wide, codes, scale, page)
    check_cache(o2, lse2, q, lens, table, codes, scale, page)


@pytest.mark.parametrize("d,page,window", [(128, 64, 64), (64, 128, 200), (128, 128, 1), (64, 64, 333)])
@pytest.mark.parametrize("h_kv,G,n_q,topk", [(2, 4, 1, 8), (1, 8, 3, 32), (2, 1, 2, 1)])
def test_cache_attention_over_selected_blocks(d, page, window, h_kv, G, n_q, topk):
    r = rng_of("sel", d, page, window, h_kv, n_q, topk)
    lens = [2500, 64, 1, 0, 129, 640]
    table, codes, scale, q, idx = cache_case(r, lens, n_q, h_kv, G, d, page, topk)
    o, lse, _ = run_cache(q, lens, table, codes, scale, page, idx, window)
    check_cache(o, lse, q, lens, table, codes, scale, page, idx, window)
    # out-of-order, repeated, invisible and negative entries are skipped and counted
    idx[0, 0, 0, :] = -1
    row = [5, 5, 3, 1 << 29, -4, 9, 2400 // page + 5][:topk]
    idx[0, 0, 0, :len(row)] = row
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse, _ = run_cache(q, lens, table, codes, scale, page, idx, window, bad=bad)
    check_cache(o, lse, q, lens, table, codes, scale, page, idx, window)
    _, skipped = S.used_blocks(idx[0, 0, 0], 2500 - n_q, page)
    assert int(bad) == skipped


@pytest.mark.parametrize("d,page", [(128, 64), (64, 128)])
def test_cache_attention_many_rows_over_a_split_axis(d, page):
    """More rows per kv-head than one unit holds, and a split axis; sixteen
    query heads per kv-head over selected blocks."""
    r = rng_of("rows", d)
    lens = [2100, 3, 1777]
    table, codes, scale, q, _ = cache_case(r, lens, 5, 1, 8, d, page)
    o, lse, p = run_cache(q, lens, table, codes, scale, page)
    assert ssa.ssa_cache_attn_workspace_size(p) > 0
    check_cache(o, lse, q, lens, table, codes, scale, page)
    table, codes, scale, q, idx = cache_case(r, lens, 2, 1, 16, d, page, 8)
    o, lse, _ = run_cache(q, lens, table, codes, scale, page, idx, 150)
    check_cache(o, lse, q, lens, table, codes, scale, page, idx, 150)


def test_cache_pool_past_32_bit_offsets():
    """A pool of more than 2^32 bytes: appended to and attended at its end."""
    page, d, h = 128, 128, 8
    n_pages = (1 << 32) // (page * d * h) + 40
    kc = torch.zeros(n_pages, h, page, d, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = torch.ones(n_pages, h, device="cuda"), torch.ones(n_pages, h, device="cuda")
    r = rng_of("far")
    table = np.array([[n_pages - 1, 3, n_pages - 17]])
    T = 300
    x = dev(r.normal(size=(T, 2 * h, d)), torch.bfloat16)
    p = ssa.make_append_params(T, 1, 3, n_pages, page, h, d, 0, norm=False, k_stride=x.stride(0), v_stride=x.stride(0))
    td = dev(table, torch.int32)
    ssa.ssa_cache_append(p, x[:, :h], x[:, h:], None, None, dev([0, T], torch.int32), dev([0], torch.int32), td, kc, vc, ks, vs)
    q = dev(r.normal(size=(1, 1, 16, d)), torch.bfloat16)
    pa = ssa.make_cache_attn_params(1, 1, 3, n_pages, page, 16, h, d)
    o, lse = torch.empty_like(q), torch.empty(1, 1, 16, device="cuda")
    ws = ssa.byte_buffer(ssa.ssa_cache_attn_workspace_size(pa))
    # the codes may come as float8, the same memory
    ssa.ssa_cache_attn(pa, q, td, dev([T], torch.int32), kc.view(E4M3), vc.view(E4M3), ks, vs, None, o, lse, ws=ws)
    ok()
    at = td[0].long()
    codes, scale = np.stack([kc[at].cpu().numpy(), vc[at].cpu().numpy()]), np.stack([f64(ks[at]), f64(vs[at])])
    check_cache(o, lse, q, [T], np.array([[0, 1, 2]]), codes, scale, page)
    rc, rs, _ = S.append(f64(x[:, :h]), [0, T], [0], [[0, 1, 2]], page, np.zeros_like(codes[0]), np.ones_like(scale[0]))
    assert np.array_equal(codes[0], rc) and np.array_equal(scale[0], rs)
    used = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
    used[at] = True
    assert not kc[~used].any() and (ks[~used] == 1).all()


def test_tokens_far_apart():
    """Tokens 2^27 elements apart: offsets past 2^31 elements in every operator
    that takes strided tokens, also with a gap before the first sequence."""
    T, h, d, step = 40, 2, 64, 1 << 27
    buf = torch.empty(T * step, dtype=torch.bfloat16, device="cuda")
    r = rng_of("apart")
    x = buf.as_strided((T, 4 * h, d), (step, d, 1))
    x.copy_(dev(r.normal(size=(T, 4 * h, d)), torch.bfloat16))
    near = x.contiguous()
    q, k, v, o = (x[:, i * h:(i + 1) * h] for i in range(4))
    nq, nk, nv, _ = (near[:, i * h:(i + 1) * h] for i in range(4))
    qs = [3, 20, 40]
    pp = ssa.make_prompt_params(2, T, T, h, h, d, step, step, step, step)
    st = dev(qs, torch.int32)
    ssa.ssa_prompt_attn(pp, q, k, v, st, st, o)
    ok()
    on, _ = run_prompt(nq, nk, nv, qs, qs)
    assert torch.equal(o[3:], on[3:]) and torch.equal(o[:3], near[:3, 3 * h:]) and (on[:3] == 7).all()
    f, pos = ssa.rope_frequencies(d)[0].cuda(), dev(np.arange(T), torch.int32)
    want = torch.empty(T, h, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, h, d, dtype=torch.bfloat16, device="cuda")
    s = near.stride(0)
    ssa.ssa_qk_rope(ssa.make_rope_params(T, h, h, d, q_stride=s, k_stride=s), nq, nk, None, None, f, pos, *want)
    for n in (2, 40):                                           # the decode kernel and the page kernel
        table, codes, scale = np.array([[2, 0], [1, 3]]), *pool(r, 4, h, 64, d)
        two = []
        for a, b, sa in ((k, v, step), (nk, nv, s)):
            ap = ssa.make_append_params(n, 2, 2, 4, 64, h, d, k_stride=sa, v_stride=sa)
            (kc, vc, ks, vs), bad = run_append(ap, a[T - n:], b[T - n:], None, f, np.array([1, n - n // 2, n]), np.array([60, 0]), table, codes, scale)
            two.append((kc, vc, ks, vs))
        assert all(torch.equal(a, b) for a, b in zip(*two))
    ssa.ssa_qk_rope(ssa.make_rope_params(T, h, h, d, q_stride=step, k_stride=step, q_out_stride=step, k_out_stride=step),
                    q, k, None, None, f, pos, q, k)
    ok()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_cache_attention_equals_the_layer_on_the_same_keys():
    """With values that the codes hold exactly, decode over the cache is the
    layer's decode (route, then attend) over dense keys: same selection, same
    output to the rounding of the two paths."""
    from content_routed_block_ssa_b200.workload import Workload, make_inputs, problem_dict
    w = Workload("serve", 77, 3, 2048, 8, 2, 128, "bf16", 64, "diag", 8, 128, 4, "per_seq", decode=True)
    Q, K, V, _ = make_inputs(w, "cpu")
    b, n, h, d = K.shape
    kc, vc = S.to_e4m3(K.float().numpy() * 16), S.to_e4m3(V.float().numpy() * 16)
    val = S.e4m3_values() / 16
    K, V = dev(val[kc], torch.bfloat16), dev(val[vc], torch.bfloat16)
    p = ssa.make_params(**problem_dict(w))
    Q = Q.cuda()
    tab = torch.empty(ssa.summary_shapes(p)[2], dtype=torch.bfloat16, device="cuda")
    ssa.ssa_block_summary(p, K, None, None, tab)
    idx = torch.empty(ssa.idx_shape(p), dtype=torch.int32, device="cuda")
    ssa.ssa_route_topk(p, Q, None, None, tab, idx)
    O, lse = torch.empty_like(Q), torch.empty(b, 1, w.h_q, device="cuda")
    ssa.ssa_sparse_attn(p, Q, K, V, idx, O, lse)
    nb = n // 64
    paged = lambda c: c.reshape(b, nb, 64, h, d).transpose(0, 1, 3, 2, 4).reshape(b * nb, h, 64, d)  # noqa: E731
    table = np.arange(b * nb).reshape(b, nb)
    scale = np.full((2, b * nb, h), 1 / 16)
    o, l2, _ = run_cache(Q, [n] * b, table, np.stack([paged(kc), paged(vc)]), scale, 64, idx.cpu().numpy(), w.window)
    check_cache(o, l2, Q, [n] * b, table, np.stack([paged(kc), paged(vc)]), scale, 64, idx.cpu().numpy(), w.window)
    assert (o.float() - O.float()).abs().max() <= 2 * 2.0 ** -8 * O.float().abs().max() + 2.0 ** -9 * V.float().abs().max()
    assert (l2 - lse).abs().max() <= 1e-4 * lse.abs().max()


def test_cache_attention_ignores_what_it_does_not_attend():
    """NaN codes behind a sequence's end, in other pages and in later new
    tokens have no part in a row; a NaN key or value that it attends does."""
    r = rng_of("nan")
    d, page, n_q, lens = 128, 64, 4, [100, 70]
    table, codes, scale, q, _ = cache_case(r, lens, n_q, 2, 4, d, page)
    clean_o, clean_l, _ = run_cache(q, lens, table, codes, scale, page)
    dirty = codes.copy()
    for s, L in enumerate(lens):
        dirty[:, table[s, L // page], :, L % page:] = 127                    # behind the end
    unused = sorted(set(range(codes.shape[1])) - set(table.flatten()))
    dirty[:, unused] = 255
    o, lse, _ = run_cache(q, lens, table, dirty, scale, page)
    assert torch.equal(o, clean_o) and torch.equal(lse, clean_l)
    dirty = codes.copy()
    dirty[1, table[0, 98 // page], 1, 98 % page, 17] = 127                   # one value of new token 2
    o, lse, _ = run_cache(q, lens, table, dirty, scale, page)
    assert torch.equal(lse, clean_l)
    nan = o.isnan()
    want = torch.zeros_like(nan)
    want[0, 2:, 4:, 17] = True                                               # tokens 2, 3 of kv-head 1's group
    assert torch.equal(nan, want) and torch.equal(o[~nan], clean_o[~nan])
    dirty = codes.copy()
    dirty[0, table[0, 98 // page], 1, 98 % page, 17] = 127                   # the same of a key
    o, lse, _ = run_cache(q, lens, table, dirty, scale, page)
    assert torch.equal(lse.isnan(), want.any(-1)) and torch.equal(o.isnan(), want.any(-1, keepdim=True).expand_as(o))
    assert torch.equal(o[~o.isnan()], clean_o[~o.isnan()])


def test_cache_attention_pages_outside_the_pool_are_left_out():
    r = rng_of("badpage")
    d, page, lens = 64, 64, [400, 1000]
    table, codes, scale, q, _ = cache_case(r, lens, 1, 2, 2, d, page)
    table[0, 2], table[0, 3], table[1, 5] = -3, 1 << 30, codes.shape[1]
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse, _ = run_cache(q, lens, table, codes, scale, page, bad=bad)
    check_cache(o, lse, q, lens, table, codes, scale, page)
    assert int(bad) == 3 * 2                                  # pages, for each of two kv-heads
    table[:] = -1                                             # nothing left: every row is empty
    o, lse, _ = run_cache(q, lens, table, codes, scale, page)
    assert not o.any() and (lse == -math.inf).all()
    # lengths beyond the table are cut to it
    table, codes, scale, q, _ = cache_case(r, [128], 1, 2, 2, d, page)
    o, lse, _ = run_cache(q, [1 << 30], table[:, :2], codes, scale, page)
    check_cache(o, lse, q, [128], table[:, :2], codes, scale, page)


def test_cache_attention_scales_and_queries_of_very_different_size():
    """Pages whose value scales differ by 2^40, rows whose elements differ by
    2^20: the running reference keeps every product in range."""
    r = rng_of("range")
    d, page, lens = 128, 64, [320]
    table, codes, scale, q, _ = cache_case(r, lens, 1, 1, 8, d, page)
    scale[1, table[0, 1]] = 2.0 ** 30
    scale[1, table[0, 3]] = 2.0 ** -40
    scale[0, table[0, 2]] = 2.0 ** -12
    q[..., ::7] *= 2.0 ** -20
    o, lse, _ = run_cache(q, lens, table, codes, scale, page)
    check_cache(o, lse, q, lens, table, codes, scale, page)
    # the same with the large page out of reach: the tiny page's rows count in full
    scale[1, table[0, 1]] = 2.0 ** -40
    o, lse, _ = run_cache(q * 64, lens, table, codes, scale, page)
    check_cache(o, lse, q * 64, lens, table, codes, scale, page)
    o, lse, _ = run_cache(q * 0, lens, table, codes, scale, page)
    check_cache(o, lse, q * 0, lens, table, codes, scale, page)


# Per row and dim, against the row's own sum p|v| / sum p.  float16 keeps a
# probability to 2^-11 of itself where p times the page's scale is above 2^-29
# of the row's largest such product, which these cases stay within; 2^-11 more
# is left for ex2.approx (2^-22) and float32 sums (n 2^-24).

def check_cache_rows(o, lse, q, lens, table, codes, scale, page, idx=None, window=0, sm_scale=None):
    args = (scale[0], scale[1], 1 / math.sqrt(q.shape[-1]) if sm_scale is None else sm_scale, idx, window)
    ro, rl = S.cache_attention(f64(q), table, lens, page, codes[0], codes[1], *args)
    ra, _ = S.cache_attention(f64(q), table, lens, page, codes[0], codes[1] & 0x7F, *args)
    assert (np.abs(f64(o) - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * ra).all()
    assert (np.abs(f64(lse) - rl) <= 2.0 ** -17 * (1 + np.abs(rl))).all()


@pytest.mark.parametrize("d,page", [(128, 64), (64, 128)])
@pytest.mark.parametrize("h_kv,G,n_q,topk", [(2, 4, 1, 0), (1, 8, 3, 0), (1, 4, 2, 4), (1, 12, 1, 4)])
@pytest.mark.parametrize("nats", [4, 17, 18, 20])
def test_cache_attention_beside_a_key_that_dominates(d, page, h_kv, G, n_q, topk, nats):
    """One key far above the others with a value of zero: all of a row's output
    comes from the others."""
    r = rng_of("sink", d, h_kv, G, n_q)
    lens, sink = [1000], 37
    table, codes, scale, q, idx = cache_case(r, lens, n_q, h_kv, G, d, page, topk)
    if topk:
        idx[..., :] = [0, 2, 4, 5]                             # the dominating key's block among them
    codes[0] = 0
    codes[0, table[0, 0], :, sink, 0] = S.to_e4m3(1.0)
    codes[1] = S.to_e4m3(100 + 50 * r.normal(size=codes[1].shape))
    codes[1, table[0, 0], :, sink] = 0
    scale[0], scale[1] = 1.0, 2.0 ** -7
    q.zero_()
    q[..., 0] = nats
    o, lse, _ = run_cache(q, lens, table, codes, scale, page, idx, 64 if topk else 0, 1.0)
    check_cache_rows(o, lse, q, lens, table, codes, scale, page, idx, 64 if topk else 0, 1.0)


@pytest.mark.parametrize("d,page,G", [(128, 64, 4), (64, 128, 16)])
@pytest.mark.parametrize("n_seq", [1, 600])
def test_cache_attention_of_128k_keys_beside_a_key_that_dominates(d, page, G, n_seq):
    """The same over an axis of many splits, or (sequences that share their
    pages) of few long ones, and every one of its keys counted."""
    r = rng_of("sink128k", d)
    n = (1 << 17) + 77
    pages = -(-n // page)
    table, scale = r.permutation(pages)[None], np.ones((2, pages, 1))
    scale[1] = 4.0
    codes = np.zeros((2, pages, 1, page, d), np.uint8)
    v = S.to_e4m3(100 + 50 * r.normal(size=(n, d)))
    at = table[0, np.arange(n) // page], 0, np.arange(n) % page
    codes[1][at] = v
    sink = 70001
    codes[0][table[0, sink // page], 0, sink % page, 0] = S.to_e4m3(1.0)
    codes[1][table[0, sink // page], 0, sink % page] = 0
    q = torch.zeros(n_seq, 1, G, d, device="cuda", dtype=torch.bfloat16)
    val = 4.0 * S.e4m3_values()[codes[1][at]]
    for nats in (17, 18, 0):
        q[..., 0] = nats
        o, lse, _ = run_cache(q, [n] * n_seq, np.repeat(table, n_seq, 0), codes, scale, page, sm_scale=1.0)
        total = n - 1 + math.exp(nats)
        ro, ra = val.sum(0) / total, np.abs(val).sum(0) / total
        assert (np.abs(f64(o) - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * ra).all()
        # at 0 nats the sum is a whole number times a power of two, exact but for ex2.approx's common factor
        # (2^-22), and 2^30 in all: log2f is off by one unit of 2^-19 at most, adding the reference by half
        # of one, times ln 2, and that product by 2^-21: 0.64 of 2^-18, and one key is 2^-17
        assert (np.abs(f64(lse) - math.log(total)) <= (2.0 ** -18 if nats == 0 else 2.0 ** -17 * (1 + nats))).all()


@pytest.mark.parametrize("d,page", [(128, 64), (64, 128), (128, 128), (64, 64)])
@pytest.mark.parametrize("h_kv,G,n_q,topk", [(2, 4, 1, 0), (1, 8, 3, 0), (2, 4, 2, 16), (1, 12, 1, 16)])
def test_cache_attention_counts_every_key(d, page, h_kv, G, n_q, topk):
    """Equal logits and a value of 1 in dim j % d alone: dim c counts the
    attended keys j = c (mod d), and the log-sum-exp all of them."""
    r = rng_of("count", d, page, h_kv, G, n_q)
    lens = [3000, 4096, 1501]
    table, codes, scale, q, idx = cache_case(r, lens, n_q, h_kv, G, d, page, topk)
    window = 150 if topk else 0
    codes[1] = 0
    for s, L in enumerate(lens):
        j = np.arange(L)
        codes[1, table[s, j // page], :, j % page, j % d] = S.to_e4m3(1.0)
    scale[1] = 1.0
    q.zero_()
    o, lse, p = run_cache(q, lens, table, codes, scale, page, idx, window)
    assert topk or ssa.ssa_cache_attn_workspace_size(p) > 0
    o, lse = f64(o), f64(lse)
    for s, L in enumerate(lens):
        for i in range(n_q):
            pos = L - n_q + i
            for h in range(h_kv * G):
                keys = np.arange(pos + 1)
                if topk:
                    used, _ = S.used_blocks(idx[s, i, h // G], pos, page)
                    keys = keys[np.isin(keys // page, used) | (keys > pos - window)]
                n = len(keys)
                want = np.bincount(keys % d, minlength=d) / n
                # one key more or less is at least 1/64 of a dim's count
                assert (np.abs(o[s, i, h] - want) <= (2.0 ** -8 + 2.0 ** -10) * want).all()
                assert abs(lse[s, i, h] - math.log(n)) <= 2.0 ** -16          # one key is 2^-12


def test_cache_attention_beside_a_page_of_far_larger_values():
    """A page whose value scale is 2^26 times the others' and whose codes are
    zero in half of the dims: there the other pages' values count in full."""
    r = rng_of("bigpage")
    d, page, lens = 128, 128, [500] * 40                       # one split: a warp meets the page and others
    table, codes, scale, q, _ = cache_case(r, lens, 1, 2, 4, d, page)
    scale[1] = 2.0 ** -8
    scale[1, table[:, 2]] = 2.0 ** 18
    codes[1, table[:, 2], :, :, ::2] = 0
    for factor in (0.0, 1.0):
        o, lse, _ = run_cache(q * factor, lens, table, codes, scale, page, sm_scale=2.0 ** -12)
        check_cache_rows(o, lse, q * factor, lens, table, codes, scale, page, sm_scale=2.0 ** -12)


@pytest.mark.parametrize("low", [0.0, 2.0 ** -126, 2.0 ** -40])
def test_cache_attention_over_pages_of_zeros(low):
    """Pages of zero codes, with scales of zero too (a pool as it was allocated):
    their keys count in the softmax like any other."""
    r = rng_of("zeros", low)
    d, page, lens = 128, 64, [1000, 3, 700]
    table, codes, scale, q, _ = cache_case(r, lens, 1, 2, 4, d, page)
    codes[:], scale[:] = 0, low
    o, lse, _ = run_cache(q, lens, table, codes, scale, page)
    assert not o.any()
    assert (np.abs(f64(lse)[:, 0] - np.log(lens)[:, None]) <= 2.0 ** -16).all()
    codes[1, table[0, 5], :, 7] = S.to_e4m3(np.arange(-64, 64) * 1.0)       # one page holds something
    scale[1, table[0, 5]] = 2.0 ** -3
    o, lse, _ = run_cache(q, lens, table, codes, scale, page)
    assert (np.abs(f64(lse)[:, 0] - np.log(lens)[:, None]) <= 2.0 ** -16).all()
    want = S.e4m3_values()[codes[1, table[0, 5], 0, 7]] / 8 / 1000
    assert not o[1:].any() and (np.abs(f64(o)[0] - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want)).all()


@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** 18, 2.0 ** 22, 2.0 ** 24, 2.0 ** 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_cache_attention_of_logits_past_float32_steps(size, sign):
    """Logits whose float32 steps are 1 and more: the largest key takes the row."""
    r = rng_of("huge", size)
    d, page, lens = 64, 64, [900]
    table, codes, scale, q, _ = cache_case(r, lens, 1, 1, 4, d, page)
    scale[0], scale[1] = 1.0, 2.0 ** -7
    codes[0] = 0
    rank = r.permutation(900)
    j = np.arange(900)
    codes[0, table[0, j // page], 0, j % page, 0] = np.where(rank < 800, 0x38 + rank % 40, 0x38 + 50)   # 1 .. 30, 80
    best = 417
    codes[0, table[0, best // page], 0, best % page, 0] = S.to_e4m3(112.0) if sign > 0 else S.to_e4m3(0.5)
    q.zero_()
    q[..., 0] = sign * size
    o, lse, _ = run_cache(q, lens, table, codes, scale, page, sm_scale=1.0)
    want = S.e4m3_values()[codes[1, table[0, best // page], 0, best % page]] * scale[1, 0, 0]
    assert (np.abs(f64(o) - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want)).all()
    logit = sign * size * (112.0 if sign > 0 else 0.5)
    assert (np.abs(f64(lse) - logit) <= 2.0 ** -17 * abs(logit)).all()


# ---------------------------------------------------------------- packed prompts

def run_prompt(q, k, v, qs, ks, sm_scale=None, lse=True, stream=None):
    T, h_q, d = q.shape
    p = ssa.make_prompt_params(len(qs) - 1, T, k.shape[0], h_q, k.shape[1], d, q.stride(0), k.stride(0), v.stride(0),
                               h_q * d + 8, sm_scale)
    buf = torch.full((T, h_q * d + 8), 7.0, device="cuda", dtype=torch.bfloat16)   # strided, with a gap
    o = buf[:, :h_q * d].view(T, h_q, d)
    out_l = torch.full((T, h_q), 7.0, device="cuda") if lse else None
    ssa.ssa_prompt_attn(p, q, k, v, dev(qs, torch.int32), dev(ks, torch.int32), o, out_l, stream)
    ok()
    assert (buf[:, h_q * d:] == 7.0).all()
    return o, out_l


def check_prompt(o, lse, q, k, v, qs, ks, sm_scale=None):
    d = q.shape[-1]
    sm = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    q, k, v, o, lse = f64(q), f64(k), f64(v), f64(o), f64(lse)
    ro, rl = S.prompt_attention(q, k, v, qs, ks, sm)
    ra, _ = S.prompt_attention(q, k, np.abs(v), qs, ks, sm)
    out = np.isnan(ro)                                        # rows outside every sequence: as they were
    assert (o[out] == 7.0).all() and (lse[np.isnan(rl)] == 7.0).all()
    rows = ~out.any(-1)
    vmax = max(np.abs(v[ks[0]:ks[-1]]).max(initial=0), 1e-30)
    assert (np.abs(o - ro) <= 2.0 ** -8 * (np.abs(ro) + ra) + 2.0 ** -12 * vmax)[rows].all()
    empty = rows & np.isinf(rl)
    assert np.array_equal(np.isinf(lse) & rows, empty) and (o[empty] == 0).all()
    rows &= ~empty
    big = sm * np.abs(q).sum(-1).max(initial=0) * np.abs(k[ks[0]:ks[-1]]).max(initial=0)
    assert (np.abs(lse[rows] - rl[rows]) <= 2.0 ** -17 * (1 + big)).all()


def prompt_case(r, lens, kv_lens, h_kv, G, d, pad=3):
    qs, ks = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(kv_lens)])
    T, N = int(qs[-1]) + pad, int(ks[-1]) + pad
    x = dev(r.normal(size=(T, h_kv * G + 1, d)), torch.bfloat16)
    y = dev(r.normal(size=(N, 2 * h_kv, d)) * r.choice([0.5, 1, 4], size=(N, 1, 1)), torch.bfloat16)
    return x[:, :h_kv * G], y[:, :h_kv], y[:, h_kv:], qs, ks


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("h_kv,G", [(2, 4), (1, 8), (2, 1), (1, 3), (1, 16), (2, 2), (1, 7)])
@pytest.mark.parametrize("lens", [[1], [1, 1, 1], [127], [128, 129], [5, 0, 200, 1, 64], [300]])
def test_prompt(d, h_kv, G, lens):
    r = rng_of(d, h_kv, G, lens)
    q, k, v, qs, ks = prompt_case(r, lens, lens, h_kv, G, d)
    o, lse = run_prompt(q, k, v, qs, ks)
    check_prompt(o, lse, q, k, v, qs, ks)


@pytest.mark.parametrize("d,h_kv,G", [(128, 70, 4), (64, 60, 7), (128, 160, 1), (64, 40, 16)])
@pytest.mark.parametrize("lens,kv_lens", [([1, 0, 200, 7], [1, 0, 200, 7]), ([130, 3], [260, 0])])
def test_prompt_of_many_heads(d, h_kv, G, lens, kv_lens):
    """Enough blocks for two tensor-core tiles each."""
    r = rng_of("heads", d, h_kv, lens)
    if len(lens) * h_kv < 2 * 148:
        lens, kv_lens = lens * 6, kv_lens * 6
    q, k, v, qs, ks = prompt_case(r, lens, kv_lens, h_kv, G, d)
    v[int(ks[-1]):] = math.nan
    o, lse = run_prompt(q, k, v, qs, ks)
    pick = [0, h_kv // 2, h_kv - 1]                            # the oracle on three kv-heads
    hd = [g * G + i for g in pick for i in range(G)]
    check_prompt(o[:, hd], lse[:, hd], q[:, hd], k[:, pick], v[:, pick], qs, ks)


@pytest.mark.parametrize("d,h_kv,G", [(128, 1, 4), (64, 2, 2)])
@pytest.mark.parametrize("lens,kv_lens", [([1, 1, 1], [1, 128, 400]), ([40, 7], [300, 129]),       # keys before the prompt
                                          ([50, 9, 300], [20, 0, 130]), ([3], [0]), ([200], [1])])  # rows without keys
def test_prompt_with_other_key_lengths(d, h_kv, G, lens, kv_lens):
    r = rng_of("kv", d, lens, kv_lens)
    q, k, v, qs, ks = prompt_case(r, lens, kv_lens, h_kv, G, d)
    o, lse = run_prompt(q, k, v, qs, ks)
    check_prompt(o, lse, q, k, v, qs, ks)


def test_prompt_large_logits_move_the_reference():
    """Logits that grow along the keys by far more than the 2^8 at which the
    running reference moves, and rows that one key dominates."""
    r = rng_of("grow")
    q, k, v, qs, ks = prompt_case(r, [700], [700], 1, 4, 128)
    k *= torch.linspace(0.1, 20, k.shape[0], device="cuda", dtype=torch.bfloat16)[:, None, None]
    o, lse = run_prompt(q, k, v, qs, ks, 1.0)
    check_prompt(o, lse, q, k, v, qs, ks, 1.0)


def test_prompt_ignores_what_a_row_does_not_attend():
    """Infinities and NaN behind a sequence, in its neighbour or at later keys
    have no part in a row; where a row attends them they show."""
    r = rng_of("pnan")
    lens = [150, 77, 260]
    q, k, v, qs, ks = prompt_case(r, lens, lens, 1, 4, 128)
    clean, clean_l = run_prompt(q, k, v, qs, ks)
    k2, v2 = k.clone(), v.clone()
    k2[ks[-1]:], v2[ks[-1]:] = math.nan, math.inf              # rows behind the last sequence
    o, lse = run_prompt(q, k2, v2, qs, ks)
    assert torch.equal(o, clean) and torch.equal(lse, clean_l)
    bad = qs[1] + 40                                           # a value inside the second sequence
    v2 = v.clone()
    v2[bad, 0, 5], v2[bad + 1, 0, 9] = math.inf, math.nan
    o, lse = run_prompt(q, k, v2, qs, ks)
    assert torch.equal(lse, clean_l)
    want = torch.zeros_like(o, dtype=torch.bool)
    want[bad:qs[2], :, 5] = True
    want[bad + 1:qs[2], :, 9] = True
    want[qs[-1]:] = False
    assert torch.equal(~torch.isfinite(o), want)
    keep = ~want
    keep[qs[1]:qs[2]] = False                                  # its own tile is evaluated another way
    assert torch.equal(o[keep], clean[keep])
    rows = slice(int(qs[1]), int(bad))
    assert (o[rows].float() - clean[rows].float()).abs().max() <= 2.0 ** -6 * v.float().abs().max()
    k2 = k.clone()
    k2[bad, 0, 5] = math.nan                                   # a key: every later row of the sequence
    o, lse = run_prompt(q, k2, v, qs, ks)
    want = torch.zeros_like(lse, dtype=torch.bool)
    want[bad:qs[2]] = True
    assert torch.equal(lse.isnan(), want) and torch.equal(o.isnan(), want[..., None].expand_as(o))
    assert torch.equal(o[~o.isnan()], clean[~o.isnan()])


@pytest.mark.parametrize("d,h_kv,G", [(128, 1, 4), (64, 1, 8), (128, 40, 4), (64, 60, 4), (64, 40, 7), (128, 20, 16)])
@pytest.mark.parametrize("more", [0, 300])   # keys before the prompt
def test_prompt_of_values_that_are_not_finite(d, h_kv, G, more):
    """Infinities and NaN among a sequence's values, in one-tile and two-tile
    blocks: rows behind them show them in their own dims, all others are the
    oracle's as closely as ever."""
    r = rng_of("podd", d, h_kv, G, more)
    lens = [700, 150, 5]
    q, k, v, qs, ks = prompt_case(r, lens, [n + more for n in lens], h_kv, G, d)
    pick = sorted({0, h_kv // 2, h_kv - 1})
    v = v.clone()
    odd = [math.inf, -math.inf, math.nan]
    at = [0, 1, 63, 64, 130, 333, 334, 511, 639, 640, 698, 699, 700, 849]   # of the first two sequences' rows
    for i, row in enumerate(at):
        s = int(row >= 700)
        key = row - 700 * s + (int(ks[s + 1] - ks[s]) - lens[s] if i % 2 else 0) + int(ks[s])
        v[key, pick[i % len(pick)], (7 * i) % d] = odd[i % 3]
    o, lse = run_prompt(q, k, v, qs, ks)
    hd = [g * G + i for g in pick for i in range(G)]
    qn, kn, vn, o, lse = f64(q[:, hd]), f64(k[:, pick]), f64(v[:, pick]), f64(o[:, hd]), f64(lse[:, hd])
    with np.errstate(invalid="ignore"):
        ro, rl = S.prompt_attention(qn, kn, vn, qs, ks, 1 / math.sqrt(d))
    fin = np.nan_to_num(vn, nan=0, posinf=0, neginf=0)
    ra, _ = S.prompt_attention(qn, kn, np.abs(fin), qs, ks, 1 / math.sqrt(d))
    rows = int(qs[-1])
    ro, ra, o, rl, lse = ro[:rows], ra[:rows], o[:rows], rl[:rows], lse[:rows]
    assert np.array_equal(np.isnan(o), np.isnan(ro)) and np.array_equal(o[np.isinf(ro)], ro[np.isinf(ro)])
    ok_ = np.isfinite(ro)
    assert 0 < (~ok_).sum() < ok_.sum() and np.array_equal(np.isfinite(o), ok_)
    assert (np.abs(o[ok_] - ro[ok_]) <= (2.0 ** -8 * (np.abs(ro) + ra) + 2.0 ** -12 * np.abs(fin).max())[ok_]).all()
    big = np.abs(qn).sum(-1).max() * np.abs(kn).max() / math.sqrt(d)
    assert (np.abs(lse - rl) <= 2.0 ** -17 * (1 + big)).all()


def test_prompt_one_odd_value_costs_little():
    """One value that is not finite near the end of a long prompt: its own
    tile's last keys are summed another way, not the whole prompt before them."""
    r = rng_of("pcost")
    T, d = 8192, 128
    q, k, v = (dev(r.normal(size=(T, h, d)), torch.bfloat16) for h in (8, 1, 1))
    p = ssa.make_prompt_params(1, T, T, 8, 1, d)
    st, o = dev([0, T], torch.int32), torch.empty_like(q)

    def time():
        best = math.inf
        for _ in range(4):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            ssa.ssa_prompt_attn(p, q, k, v, st, st, o)
            b.record()
            ok()
            best = min(best, a.elapsed_time(b))
        return best

    clean = time()
    v[T - 40, 0, 3] = math.inf
    assert time() < 4 * clean
    assert torch.isinf(o[T - 40:, :, 3]).all() and torch.isfinite(o[:T - 40]).all()


def test_prompt_without_any_keys():
    q = torch.ones(5, 8, 64, device="cuda", dtype=torch.bfloat16)
    kv = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    o, lse = run_prompt(q, kv, kv, [0, 4], [0, 0])
    assert not o[:4].any() and (lse[:4] == -math.inf).all() and (o[4] == 7).all() and (lse[4] == 7).all()


def test_prompt_offsets_that_do_not_fit():
    """Decreasing or out-of-range offsets read and write nothing outside the
    operands; rows that no sequence covers stay as they were."""
    r = rng_of("poff")
    q, k, v, qs, ks = prompt_case(r, [100, 100], [100, 100], 2, 4, 64, pad=0)
    for odd in ([0, 1 << 30, -7], [-5, 300, 100], [200, 200, 200], [50, 20, 10]):
        o, lse = run_prompt(q, k, v, odd, odd)
    assert (o == 7.0).all() and (lse == 7.0).all()             # the last: no rows
    o, lse = run_prompt(q, k, v, [0, 100, 300], [0, 100, 300])  # cut to what is there
    check_prompt(o, lse, q, k, v, qs, ks)
    o, _ = run_prompt(q, k, v, qs, ks, lse=False)
    assert torch.equal(o, run_prompt(q, k, v, qs, ks)[0])


@pytest.mark.parametrize("lens,h_kv,G,d", [([3000], 1, 8, 128), ([700, 1500, 33], 4, 4, 128), ([2049], 2, 2, 64),
                                            ([3000, 1000], 8, 4, 128), ([2600], 4, 16, 64),
                                            ([1500], 60, 1, 64)])
def test_prompt_long(lens, h_kv, G, d):
    """Many steps and more units than SMs, against float64 on sampled rows."""
    r = rng_of("plong", lens)
    q, k, v, qs, ks = prompt_case(r, lens, lens, h_kv, G, d, pad=0)
    o, lse = run_prompt(q, k, v, qs, ks)
    q, k, v, o, lse = map(f64, (q, k, v, o, lse))
    for row in np.unique(np.concatenate([r.integers(0, len(o), 150), qs[1:] - 1, qs[:-1]])):
        s = int(np.searchsorted(qs, row, side="right")) - 1
        for h in range(h_kv * G):
            a = (q[row, h], k[qs[s]:row + 1, h // G])
            vv = v[qs[s]:row + 1, h // G]
            ro, rl = S.attend(*a, vv, 1 / math.sqrt(d))
            ra, _ = S.attend(*a, np.abs(vv), 1 / math.sqrt(d))
            assert (np.abs(o[row, h] - ro) <= 2.0 ** -8 * (np.abs(ro) + ra) + 2.0 ** -12 * np.abs(vv).max()).all()
            assert abs(lse[row, h] - rl) <= 2.0 ** -17 * (1 + np.abs(a[0]).sum() * np.abs(a[1]).max() / math.sqrt(d))


# ---------------------------------------------------------------- together

def test_a_serving_loop_matches_attention_over_everything():
    """Prompt, then decode steps: rotate, append, attend; each step's output
    against the oracle over the cache as it stands, and the cache against the
    exact keys to its rounding."""
    r = rng_of("loop")
    n_seq, h_q, h_kv, d, page, width = 3, 8, 2, 128, 64, 6
    f, m = ssa.rope_frequencies(d, 10000.0, "blend", 4.0, 128.0)
    fd = f.cuda()
    qw, kw = dev(1 + 0.1 * r.normal(size=d), torch.float32), dev(1 + 0.1 * r.normal(size=d), torch.float32)
    table = r.permutation(n_seq * width).reshape(n_seq, width)
    td = dev(table, torch.int32)
    codes, scale = pool(r, n_seq * width, h_kv, page, d)
    kc, vc, ks, vs = dev(codes[0]), dev(codes[1]), dev(scale[0], torch.float32), dev(scale[1], torch.float32)
    have = np.zeros(n_seq, int)
    keys = [[] for _ in range(n_seq)]
    for step in range(6):
        news = [5, 130, 64] if step == 0 else [1] * n_seq
        n_q = 1
        cu = np.concatenate([[0], np.cumsum(news)])
        T = int(cu[-1])
        x = dev(r.normal(size=(T, h_q + 2 * h_kv, d)), torch.bfloat16)
        q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(have, news)])
        qo, ko = torch.empty(T, h_q, d, device="cuda", dtype=torch.bfloat16), torch.empty(T, h_kv, d, device="cuda", dtype=torch.bfloat16)
        rp = ssa.make_rope_params(T, h_q, h_kv, d, mscale=m, q_stride=x.stride(0), k_stride=x.stride(0))
        ssa.ssa_qk_rope(rp, q, k, qw, kw, fd, dev(pos, torch.int32), qo, ko)
        ap = ssa.make_append_params(T, n_seq, width, n_seq * width, page, h_kv, d, mscale=m, k_stride=x.stride(0),
                                    v_stride=x.stride(0))
        ssa.ssa_cache_append(ap, k, v, kw, fd, dev(cu, torch.int32), dev(have, torch.int32), td, kc, vc, ks, vs)
        exact = S.rotate(S.norm(f64(k), f64(kw)), f.numpy(), pos, "half", m)
        for s in range(n_seq):
            keys[s] += list(exact[cu[s]:cu[s + 1]])
        have = have + news
        last = qo[dev(cu[1:] - 1)].view(n_seq, n_q, h_q, d).contiguous()
        cs = np.stack([kc.cpu().numpy(), vc.cpu().numpy()])
        sc = np.stack([f64(ks), f64(vs)])
        o, lse, _ = run_cache(last, have, table, cs, sc, page)
        check_cache(o, lse, last, have, table, cs, sc, page)
    val = S.e4m3_values()
    for s in range(n_seq):
        for j, x in enumerate(keys[s]):
            pid, sl = table[s, j // page], j % page
            got = val[cs[0, pid, :, sl]] * sc[0, pid][:, None]
            # a key stored before its page's scale grew was rounded twice, the second time only where subnormal
            assert (np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * sc[0, pid][:, None] + 2.0 ** -16 * np.abs(x).max()).all()


def test_operators_run_on_a_side_stream_and_replay_from_a_graph():
    r = rng_of("graph")
    lens, page, d = [500, 1300], 64, 128
    table, codes, scale, q, idx = cache_case(r, lens, 1, 2, 4, d, page, 4)
    ref, ref_l, p = run_cache(q, lens, table, codes, scale, page)
    td, ld = dev(table, torch.int32), dev(lens, torch.int32)
    kc, vc, ks, vs = dev(codes[0]), dev(codes[1]), dev(scale[0], torch.float32), dev(scale[1], torch.float32)
    ws = ssa.byte_buffer(ssa.ssa_cache_attn_workspace_size(p))
    o, lse = torch.zeros_like(q), torch.zeros(2, 1, 8, device="cuda")
    x = dev(r.normal(size=(2, 4, d)), torch.bfloat16)
    f = ssa.rope_frequencies(d)[0].cuda()
    cu, have = dev([0, 1, 2], torch.int32), dev(np.array(lens) - 1, torch.int32)
    rp = ssa.make_rope_params(2, 2, 2, d, q_stride=x.stride(0), k_stride=x.stride(0))
    ap = ssa.make_append_params(2, 2, td.shape[1], kc.shape[0], page, 2, d, k_stride=x.stride(0), v_stride=x.stride(0))
    qo, ko = torch.empty(2, 2, d, device="cuda", dtype=torch.bfloat16), torch.empty(2, 2, d, device="cuda", dtype=torch.bfloat16)

    def step(stream=None):
        ssa.ssa_qk_rope(rp, x[:, :2], x[:, 2:], None, None, f, have, qo, ko, stream)
        ssa.ssa_cache_append(ap, x[:, :2], x[:, 2:], None, f, cu, have, td, kc, vc, ks, vs, None, stream)
        ssa.ssa_cache_attn(p, q, td, ld, kc, vc, ks, vs, None, o, lse, ws=ws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    ok()
    first, first_l, rot = o.clone(), lse.clone(), qo.clone()
    cs, sc = np.stack([kc.cpu().numpy(), vc.cpu().numpy()]), np.stack([f64(ks), f64(vs)])
    check_cache(first, first_l, q, lens, table, cs, sc, page)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    o.zero_(), lse.zero_(), qo.zero_(), ws.fill_(255)
    x.copy_(x.flip(0))
    g.replay()
    ok()
    assert not torch.equal(qo, rot) and not torch.equal(o, first)      # the new inputs are used
    cs, sc = np.stack([kc.cpu().numpy(), vc.cpu().numpy()]), np.stack([f64(ks), f64(vs)])
    check_cache(o, lse, q, lens, table, cs, sc, page)
    again = o.clone()
    g.replay()
    ok()
    assert torch.equal(o, again)                                       # and the same bytes each time


def test_prompt_then_decode_agree():
    """The last row of a prompt equals a decode step over the cache that the
    same prompt filled, when the codes hold the keys and values exactly; and the
    prompt operator replays from a graph."""
    r = rng_of("agree")
    lens, h_kv, G, d, page = [200, 65], 2, 4, 64, 64
    q, k, v, qs, ks = prompt_case(r, lens, lens, h_kv, G, d, pad=0)
    val = S.e4m3_values()
    k.copy_(dev(val[S.to_e4m3(f64(k) * 16)] / 16)), v.copy_(dev(val[S.to_e4m3(f64(v) * 16)] / 16))
    o, lse = run_prompt(q, k, v, qs, ks)
    table = np.arange(8).reshape(2, 4)
    codes, scale = pool(r, 8, h_kv, page, d)
    p = ssa.make_append_params(int(qs[-1]), 2, 4, 8, page, h_kv, d, 0, norm=False, k_stride=k.stride(0), v_stride=v.stride(0))
    kc, vc, kss, vss = dev(codes[0]), dev(codes[1]), dev(scale[0], torch.float32), dev(scale[1], torch.float32)
    ssa.ssa_cache_append(p, k, v, None, None, dev(qs, torch.int32), dev([0, 0], torch.int32), dev(table, torch.int32), kc, vc, kss, vss)
    last = q[dev(qs[1:] - 1)].view(2, 1, h_kv * G, d).contiguous()
    cs, sc = np.stack([kc.cpu().numpy(), vc.cpu().numpy()]), np.stack([f64(kss), f64(vss)])
    o2, l2, _ = run_cache(last, lens, table, cs, sc, page)
    at = dev(qs[1:] - 1)
    assert (o2[:, 0].float() - o[at].float()).abs().max() <= 2.0 ** -6 * v.float().abs().max()
    assert (l2[:, 0] - lse[at]).abs().max() <= 1e-3
    pp = ssa.make_prompt_params(2, q.shape[0], k.shape[0], h_kv * G, h_kv, d, q.stride(0), k.stride(0), v.stride(0))
    out, ol = torch.zeros(q.shape, device="cuda", dtype=torch.bfloat16), torch.zeros_like(lse)
    st = dev(qs, torch.int32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssa.ssa_prompt_attn(pp, q, k, v, st, st, out, ol)
    for _ in range(2):
        out.zero_(), ol.zero_()
        g.replay()
        ok()
        assert torch.equal(out, o) and torch.equal(ol, lse)


FIRST_CALL = """
import torch
from content_routed_block_ssa_b200 import ssa
dev = dict(device="cuda")
q = torch.randn(4, 8, 64, **dev).bfloat16()
k = torch.randn(4, 2, 64, **dev).bfloat16()
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, **dev)
o, qo, ko = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k)
kc, vc = torch.zeros(2, 2, 64, 64, dtype=torch.uint8, **dev), torch.zeros(2, 2, 64, 64, dtype=torch.uint8, **dev)
ks, vs = torch.zeros(2, 2, **dev), torch.zeros(2, 2, **dev)
f, cu, pos, table, have = ssa.rope_frequencies(64)[0].cuda(), i32(0, 4), i32(0, 1, 2, 3), i32(0, 1).view(1, 2), i32(0)
oc, ln = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16, **dev), i32(4)
def step():
    ssa.ssa_qk_rope(ssa.make_rope_params(4, 8, 2, 64), q, k, None, None, f, pos, qo, ko)
    ssa.ssa_cache_append(ssa.make_append_params(4, 1, 2, 2, 64, 2, 64), k, k, None, f, cu, have, table, kc, vc, ks, vs)
    ssa.ssa_cache_attn(ssa.make_cache_attn_params(1, 1, 2, 2, 64, 8, 2, 64), qo[3:].view(1, 1, 8, 64), table, ln, kc, vc, ks, vs, None, oc)
    ssa.ssa_prompt_attn(ssa.make_prompt_params(1, 4, 4, 8, 2, 64), qo, ko, k, cu, cu, o)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
a, b = o.clone(), oc.clone()
step()
torch.cuda.synchronize()
assert a.any() and b.any() and torch.equal(a, o) and torch.equal(b, oc) and ssa.ssa_device_error() == 0
print("captured first")
"""


def test_the_first_call_may_be_captured():
    import subprocess
    import sys
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_two_calls_at_once_with_a_workspace_each():
    r = rng_of("two")
    lens, page = [3000, 2500], 64
    table, codes, scale, q, _ = cache_case(r, lens, 1, 2, 4, 128, page)
    ref, ref_l, p = run_cache(q, lens, table, codes, scale, page)
    args = (p, q, dev(table, torch.int32), dev(lens, torch.int32), dev(codes[0]), dev(codes[1]),
            dev(scale[0], torch.float32), dev(scale[1], torch.float32), None)
    n = ssa.ssa_cache_attn_workspace_size(p)
    outs = [(torch.zeros_like(q), torch.zeros_like(ref_l), ssa.byte_buffer(n), torch.cuda.Stream()) for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, l, ws, st in outs:
            ssa.ssa_cache_attn(*args, o, l, None, ws, st)
    ok()
    assert all(torch.equal(o, ref) and torch.equal(l, ref_l) for o, l, _, _ in outs)


def test_results_do_not_depend_on_the_run():
    r = rng_of("same")
    lens = [2000, 77, 1024]
    table, codes, scale, q, _ = cache_case(r, lens, 2, 2, 4, 128, 64)
    a, al, _ = run_cache(q, lens, table, codes, scale, 64)
    b, bl, _ = run_cache(q, lens, table, codes, scale, 64)
    assert torch.equal(a, b) and torch.equal(al, bl)
