"""Host-side checks of the serving operators: struct layouts, refusals before
any launch, the frequency schedules, and pins of their float64 oracle."""
import ctypes as C
import math
import os
import re

import numpy as np
import pytest
import torch

from content_routed_block_ssa_b200 import ssa
from oracle import serve_oracle as S

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ssa.h")
D = 256   # a non-null, 16-byte-aligned stand-in address: validation fails first


@pytest.mark.parametrize("name", ["ssa_rope_params", "ssa_append_params", "ssa_cache_attn_params", "ssa_prompt_params"])
def test_struct_layouts_match_the_header(name):
    text = open(HEADER).read()
    body = text[:text.index("} %s;" % name)]
    body = re.sub(r"/\*.*?\*/", "", body[body.rindex("typedef struct {"):], flags=re.S)
    fields = []
    for names in re.findall(r"\b(?:int32_t|int64_t|float)\s+([\w\s,]+);", body):
        fields += [f.strip() for f in names.split(",")]
    assert fields == [f for f, _ in getattr(ssa, name)._fields_]


def rope(**kw):
    return ssa.make_rope_params(**{**dict(n_tokens=4, h_q=4, h_kv=2, d=128), **kw})


def call_rope(p, **kw):
    a = {**dict(Q=D, K=D, qw=None, kw=None, f=D, pos=D, qo=D, ko=D), **kw}
    return ssa.lib.ssa_qk_rope(C.byref(p), a["Q"], a["K"], a["qw"], a["kw"], a["f"], a["pos"], a["qo"], a["ko"], None)


INVALID, UNSUPPORTED = ssa.SSA_ERR_INVALID_ARG, ssa.SSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(n_tokens=-1), INVALID), (dict(h_q=0), INVALID), (dict(h_kv=0), INVALID), (dict(d=0), INVALID),
    (dict(rot=-16), INVALID), (dict(rot=144), INVALID), (dict(layout=2), INVALID), (dict(dtype=5), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(mscale=float("inf")), INVALID),
    (dict(q_stride=4 * 128 - 8), INVALID), (dict(k_stride=2 * 128 + 4), INVALID), (dict(q_out_stride=0), INVALID),
    (dict(k_out_stride=-512), INVALID), (dict(d=96, rot=0), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
    (dict(dtype="f32", q_stride=4 * 128 + 2), INVALID),
])
def test_rope_refusals(kw, code):
    before = ssa.ssa_launch_count()
    assert call_rope(rope(**kw)) == code
    assert ssa.ssa_launch_count() == before


def test_rope_pointers():
    p = rope()
    for kw in (dict(Q=None), dict(K=None), dict(qo=None), dict(ko=None), dict(f=None), dict(pos=None), dict(Q=D + 8),
               dict(qw=D + 4), dict(f=D + 8), dict(pos=D + 2)):
        assert call_rope(p, **kw) == INVALID, kw
    assert call_rope(rope(q_out_stride=1024)) == INVALID   # in place with another stride
    assert ssa.lib.ssa_qk_rope(None, D, D, None, None, D, D, D, D, None) == INVALID
    assert call_rope(rope(n_tokens=0), Q=None) == ssa.SSA_OK


def append(**kw):
    return ssa.make_append_params(**{**dict(n_tokens=4, n_seq=2, max_pages=3, n_pages=9, page=64, h_kv=2, d=128), **kw})


def call_append(p, **kw):
    a = {**dict(K=D, V=D, w=None, f=D, cu=D, have=D, table=D, kc=D, vc=D, ks=D, vs=D, bad=None), **kw}
    return ssa.lib.ssa_cache_append(C.byref(p), a["K"], a["V"], a["w"], a["f"], a["cu"], a["have"], a["table"],
                                    a["kc"], a["vc"], a["ks"], a["vs"], a["bad"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_tokens=-1), INVALID), (dict(n_seq=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(n_pages=-1), INVALID),
    (dict(page=0), INVALID), (dict(h_kv=0), INVALID), (dict(k_stride=128), INVALID), (dict(v_stride=257), INVALID),
    (dict(page=32), UNSUPPORTED), (dict(d=80), UNSUPPORTED), (dict(rot=8), UNSUPPORTED),
    (dict(max_pages=1 << 26), UNSUPPORTED),   # positions past 32 bits
])
def test_append_refusals(kw, code):
    before = ssa.ssa_launch_count()
    assert call_append(append(**kw)) == code
    assert ssa.ssa_launch_count() == before


@pytest.mark.parametrize("kw", [dict(n_seq=1 << 24, h_kv=128), dict(n_seq=1 << 24, h_kv=65535),
                                dict(n_tokens=2 ** 31 - 1, h_kv=64), dict(n_tokens=2 ** 31 - 1, n_seq=1 << 24, page=128, h_kv=50)])
def test_append_refuses_more_pages_of_heads_than_it_counts(kw):
    before = ssa.ssa_launch_count()
    assert call_append(append(**kw)) == UNSUPPORTED
    assert ssa.ssa_launch_count() == before


def test_append_pointers():
    p = append()
    for n in ("K", "V", "f", "cu", "have", "table", "kc", "vc", "ks", "vs"):
        assert call_append(p, **{n: None}) == INVALID, n
    for n in ("K", "V", "w", "f", "kc", "vc"):
        assert call_append(p, **{n: D + 8}) == INVALID, n
    for n in ("cu", "have", "table", "ks", "vs", "bad"):
        assert call_append(p, **{n: D + 2}) == INVALID, n
    p.reserved = 1
    assert call_append(p) == INVALID
    assert call_append(append(n_tokens=0), K=None) == ssa.SSA_OK
    assert call_append(append(n_seq=0), K=None) == ssa.SSA_OK


def cache(**kw):
    return ssa.make_cache_attn_params(**{**dict(n_seq=2, n_q=1, max_pages=3, n_pages=9, page=64, h_q=8, h_kv=2,
                                                d=128), **kw})


def call_cache(p, **kw):
    a = {**dict(Q=D, table=D, len=D, kc=D, vc=D, ks=D, vs=D, idx=D if p.topk else None, O=D, lse=None, bad=None, ws=D,
                n=1 << 40), **kw}
    return ssa.lib.ssa_cache_attn(C.byref(p), a["Q"], a["table"], a["len"], a["kc"], a["vc"], a["ks"], a["vs"],
                                  a["idx"], a["O"], a["lse"], a["bad"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=-1), INVALID), (dict(n_q=-1), INVALID), (dict(h_q=0), INVALID), (dict(h_q=9), INVALID),
    (dict(topk=-1), INVALID), (dict(topk=4), INVALID), (dict(window=64), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(topk=33, window=64), UNSUPPORTED),
    (dict(topk=4, window=4033), UNSUPPORTED), (dict(h_q=34), UNSUPPORTED), (dict(page=16), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(n_seq=1 << 20, n_q=1 << 10), UNSUPPORTED),
])
def test_cache_attn_refusals(kw, code):
    before = ssa.ssa_launch_count()
    p = cache(**kw)
    assert call_cache(p) == code
    assert ssa.ssa_cache_attn_workspace_size(p) == 0
    assert ssa.ssa_launch_count() == before


@pytest.mark.parametrize("kw", [dict(n_seq=2 ** 31 - 1, n_q=2 ** 31 - 1, h_q=4, h_kv=4),   # past 64 bits together
                                dict(n_seq=2 ** 31 - 1, n_q=2 ** 31 - 1, h_q=16, h_kv=1, topk=4, window=64),
                                dict(n_seq=1 << 30, n_q=1 << 30, h_q=16, h_kv=16), dict(n_seq=2 ** 31 - 1),
                                dict(n_seq=1, n_q=2 ** 31 - 1), dict(n_seq=1 << 29, n_q=1, h_q=4, h_kv=4)])
def test_cache_attn_refuses_more_rows_than_it_counts(kw):
    before = ssa.ssa_launch_count()
    p = cache(**kw)
    assert ssa.ssa_cache_attn_workspace_size(p) == 0
    assert call_cache(p) == UNSUPPORTED
    assert ssa.ssa_launch_count() == before


def test_cache_attn_pointers_and_workspace():
    p = cache()
    for n in ("Q", "table", "len", "kc", "vc", "ks", "vs", "O"):
        assert call_cache(p, **{n: None}) == INVALID, n
    assert call_cache(p, idx=D) == INVALID                      # blocks without topk
    assert call_cache(cache(topk=4, window=64), idx=None) == INVALID
    for n in ("Q", "kc", "vc", "O"):
        assert call_cache(p, **{n: D + 8}) == INVALID, n
    long = cache(max_pages=4096)                                 # few rows, a long axis: split
    need = ssa.ssa_cache_attn_workspace_size(long)
    assert need > 0 and need % (128 * 4 + 8) == 0
    assert call_cache(long, ws=None, n=0) == ssa.SSA_ERR_WORKSPACE
    assert call_cache(long, n=need - 1) == ssa.SSA_ERR_WORKSPACE
    assert call_cache(long, ws=D + 8, n=need) == ssa.SSA_ERR_WORKSPACE
    p.reserved = 1
    assert call_cache(p) == INVALID
    assert call_cache(cache(n_seq=0), Q=None) == ssa.SSA_OK
    assert call_cache(cache(n_q=0), Q=None) == ssa.SSA_OK


def prompt(**kw):
    return ssa.make_prompt_params(**{**dict(n_seq=2, n_q=9, n_kv=9, h_q=8, h_kv=2, d=128), **kw})


def call_prompt(p, **kw):
    a = {**dict(Q=D, K=D, V=D, qs=D, ks=D, O=D, lse=None), **kw}
    return ssa.lib.ssa_prompt_attn(C.byref(p), a["Q"], a["K"], a["V"], a["qs"], a["ks"], a["O"], a["lse"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=-1), INVALID), (dict(n_q=-1), INVALID), (dict(n_kv=-1), INVALID), (dict(h_q=7), INVALID),
    (dict(h_kv=0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q_stride=1020), INVALID), (dict(k_stride=255), INVALID), (dict(v_stride=260), INVALID),
    (dict(o_stride=512), INVALID), (dict(d=192), UNSUPPORTED), (dict(h_q=34), UNSUPPORTED),
    (dict(q_stride=1 << 39), UNSUPPORTED),
])
def test_prompt_refusals(kw, code):
    before = ssa.ssa_launch_count()
    assert call_prompt(prompt(**kw)) == code
    assert ssa.ssa_launch_count() == before


def test_prompt_pointers():
    p = prompt()
    for n in ("Q", "K", "V", "qs", "ks", "O"):
        assert call_prompt(p, **{n: None}) == INVALID, n
    for n in ("Q", "K", "V", "O"):
        assert call_prompt(p, **{n: D + 8}) == INVALID, n
    for n in ("qs", "ks", "lse"):
        assert call_prompt(p, **{n: D + 2}) == INVALID, n
    p.reserved = 3
    assert call_prompt(p) == INVALID
    assert call_prompt(prompt(n_q=0), Q=None) == ssa.SSA_OK
    assert call_prompt(prompt(n_seq=0), Q=None) == ssa.SSA_OK


def test_binding_refuses_other_types_shapes_and_devices():
    p = rope(n_tokens=2)
    q, k = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    f, pos = torch.zeros(64, dtype=torch.float64), torch.zeros(2, dtype=torch.int32)
    before = ssa.ssa_launch_count()
    for a, why in (((q.float(), k, None, None, f, pos, q, k), "Q: expected torch.bfloat16"),
                   ((q[:1], k, None, None, f, pos, q, k), "Q: expected shape"),
                   ((q.transpose(0, 1).contiguous().transpose(0, 1), k, None, None, f, pos, q, k), "Q: expected strides"),
                   ((q, k, None, None, f, pos, q, k), "Q: expected a tensor on the current CUDA device")):
        with pytest.raises(ValueError, match=re.escape(why)):
            ssa.ssa_qk_rope(p, *a)
    assert ssa.ssa_launch_count() == before


# ---------------------------------------------------------------- frequencies

def test_frequency_schedules():
    f, m = ssa.rope_frequencies(128, 10000.0)
    ref = 10000.0 ** (-np.arange(64) / 64.0)
    assert m == 1.0 and np.allclose(f.numpy(), ref, rtol=1e-14)
    f4, m = ssa.rope_frequencies(128, 10000.0, "linear", 4.0)
    assert m == 1.0 and np.allclose(f4.numpy(), ref / 4, rtol=1e-14)
    fb, _ = ssa.rope_frequencies(128, 10000.0, "base", 8.0)
    assert np.allclose(fb.numpy(), (10000.0 * 8 ** (128 / 126)) ** (-np.arange(64) / 64.0), rtol=1e-13)
    # the slowest pair of the larger base turns as slowly as interpolation's
    assert math.isclose(fb[-1].item(), ref[-1] / 8, rel_tol=1e-12)


def test_blended_frequencies_keep_fast_pairs_and_divide_slow_ones():
    base, L, s = 1e6, 32768.0, 4.0
    f, m = ssa.rope_frequencies(128, base, "blend", s, L, 32.0, 1.0)
    plain = base ** (-np.arange(64) / 64.0)
    turns = L * plain / (2 * math.pi)
    r = f.numpy() / plain
    assert math.isclose(m, 0.1 * math.log(s) + 1.0, rel_tol=1e-6)
    x = lambda t: 128 * math.log(L / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    lo, hi = math.floor(x(32.0)), math.ceil(x(1.0))
    for i in range(64):
        if i <= lo:
            assert math.isclose(r[i], 1.0, rel_tol=1e-12) and (turns[i] > 32 or i == lo)
        elif i >= hi:
            assert math.isclose(r[i], 1 / s, rel_tol=1e-12) and turns[i] <= 1.0
        else:
            t = (i - lo) / (hi - lo)
            assert math.isclose(r[i], 1 - t + t / s, rel_tol=1e-12)
    assert 0 < lo < hi < 63
    same, one = ssa.rope_frequencies(128, base, "blend", 1.0, L)
    assert one == 1.0 and np.allclose(same.numpy(), plain, rtol=1e-14)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=3), dict(base=1.0), dict(base=float("nan")), dict(factor=0.5),
                                dict(schedule=9), dict(schedule="base", rot=2), dict(schedule="blend"),
                                dict(schedule="blend", trained_len=100.0, fast=1.0, slow=2.0),
                                dict(schedule="blend", trained_len=100.0, slow=0.0)])
def test_frequency_refusals(kw):
    with pytest.raises(ssa.SSAError):
        ssa.rope_frequencies(**{**dict(rot=64), **kw})


# ---------------------------------------------------------------- oracle pins

def test_oracle_e4m3_matches_torch_on_every_code_and_between():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(codes, S.e4m3_values().astype(np.float32), equal_nan=True)
    v = S.e4m3_values()[:127]
    x = np.concatenate([v, (v[1:] + v[:-1]) / 2, v * 1.01, v * 0.99])
    x = np.concatenate([x, -x])
    x = x[np.abs(x) <= 448.0]
    ours = S.to_e4m3(x)
    theirs = torch.tensor(x, dtype=torch.float64).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ours & 127, theirs & 127) and np.array_equal((ours >> 7)[x != 0], (theirs >> 7)[x != 0])
    assert list(S.to_e4m3([np.inf, -np.inf, 1e30, np.nan])) == [126, 254, 126, 127]


def test_oracle_exponent_and_append_on_a_hand_case():
    assert S.exponent([0.0]) == -40 and S.exponent([448.0]) == 0 and S.exponent([448.5]) == 1
    assert S.exponent([0.875]) == -9 and S.exponent([1.0]) == -8 and S.exponent([np.inf, 7.0]) == -6
    codes, scale = np.zeros((2, 1, 64, 64), np.uint8), np.full((2, 1), 99.0)
    x = np.zeros((3, 1, 64))
    x[0], x[1], x[2] = 1.0, 0.5, 448.0
    c1, s1, bad = S.append(x[:2], [0, 2], [0], [[1]], 64, codes, scale)
    assert bad == 0 and s1[1, 0] == 2.0 ** -8 and s1[0, 0] == 99.0       # 1 = 256 * 2^-8
    assert (c1[1, 0, 0] == S.to_e4m3(256.0)).all() and (c1[1, 0, 1] == S.to_e4m3(128.0)).all() and not c1[0].any()
    c2, s2, _ = S.append(x[2:], [0, 1], [2], [[1]], 64, c1, s1)           # the scale grows to 1
    assert s2[1, 0] == 1.0 and (S.e4m3_values()[c2[1, 0, :3, 0]] == [1.0, 0.5, 448.0]).all()
    _, _, bad = S.append(x, [0, 3], [63], [[1]], 64, codes, scale)        # two tokens past the table
    assert bad == 2


def test_oracle_rotation_is_a_rotation_and_relative():
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(1, 1, 64)), rng.normal(size=(1, 1, 64))
    f = 10000.0 ** (-np.arange(24) / 24.0)
    for layout in ("half", "pairs"):
        a = S.rotate(q, f, [1000], layout) * S.rotate(k, f, [990], layout)
        b = S.rotate(q, f, [13], layout) * S.rotate(k, f, [3], layout)
        assert np.isclose(a.sum(), b.sum())                               # depends on the distance alone
        assert np.allclose(S.rotate(q, f, [5], layout)[..., 48:], q[..., 48:])
        assert np.isclose(np.linalg.norm(S.rotate(q, f, [77], layout)), np.linalg.norm(q))
    one = np.zeros((1, 1, 64))
    one[..., 0] = 1.0
    assert np.isclose(S.rotate(one, f, [1], "half")[0, 0, 24], np.sin(1.0))
    assert np.isclose(S.rotate(one, f, [1], "pairs")[0, 0, 1], np.sin(1.0))
    x = rng.normal(size=(2, 3, 64))
    y = S.norm(x, eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0)


def test_oracle_attention_on_known_cases():
    k = np.array([[0.0, 1.0], [0.0, -1.0]])
    v = np.array([[1.0, 0.0], [0.0, 3.0]])
    o, lse = S.attend(np.array([5.0, 0.0]), k, v, 1.0)
    assert np.allclose(o, [0.5, 1.5]) and np.isclose(lse, math.log(2.0))
    o, lse = S.attend(np.zeros(2), k[:0], v[:0], 1.0)
    assert (o == 0).all() and lse == -np.inf
    assert S.used_blocks([3, 1, 1, 4, -1, 9, -5], 10 * 64 + 63, 64) == ([3, 4, 9], 3)
    assert S.used_blocks([0, 2], 2 * 64 + 62, 64) == ([0], 1)             # the query's own block is not whole
    # a page that holds every key: the paged form equals the plain one
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 120, size=(2, 1, 64, 64)).astype(np.uint8)
    sc = np.array([[0.5], [2.0]])
    q = rng.normal(size=(1, 1, 2, 64))
    o, lse = S.cache_attention(q, np.array([[1, 0]]), [70], 64, codes, codes, sc, sc, 0.1)
    keys = np.concatenate([S.e4m3_values()[codes[1, 0]] * 2.0, S.e4m3_values()[codes[0, 0, :6]] * 0.5])
    ref, rl = S.attend(q[0, 0, 1], keys, keys, 0.1)
    assert np.allclose(o[0, 0, 1], ref) and np.isclose(lse[0, 0, 1], rl)
    # selecting every whole block with a window over the rest is the same set
    idx = np.array([[[[0, -1]]]])
    o2, _ = S.cache_attention(q, np.array([[1, 0]]), [70], 64, codes, codes, sc, sc, 0.1, idx, 6)
    assert np.allclose(o2, o)
    # packed prompts: each row sees its own prefix
    k, v = rng.normal(size=(5, 1, 4)), rng.normal(size=(5, 1, 4))
    o, _ = S.prompt_attention(k, k, v, [0, 2, 4], [0, 2, 4], 1.0)
    assert np.allclose(o[0, 0], v[0, 0]) and np.allclose(o[2, 0], v[2, 0]) and np.isnan(o[4]).all()
    o, _ = S.prompt_attention(k, k, v, [0, 3], [0, 2], 1.0)
    assert (o[0] == 0).all() and np.allclose(o[1, 0], v[0, 0])
