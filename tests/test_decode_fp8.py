"""The decode-step operators over a cache in 8 bits (gpt_kv_append_fp8, gpt_decode_attention_fp8) and the drawing of
tokens (gpt_sample_token).

Refusals are checked through the C ABI and the binding without a GPU; on a GPU each operator is compared with its
definition in float64 (numpy).  Tolerances are worst-case bounds of the arithmetic: u = 2^-24 per fp32 operation, half a
step of bf16 (2^-8 of the value), fp16 (2^-11) or e4m3 (2^-4 of the value, 2^-10 below 2^-6) for a rounding to these.
Scales, tokens and counts are equal."""

import ctypes
import math
import os
import re
import subprocess
import sys

import numpy as np
import pytest

from persistent_gpt_step_gb300 import binding as B

torch = pytest.importorskip("torch")

from test_decode_ops import (DT, FAKE, U, _append, _attend, _cache, _check, _i, _np, _pages, _rng, _t, _turned,  # noqa: E402
                             _turn_tolerance, cuda, gpu, lib)  # noqa: F401

F8 = torch.float8_e4m3fn


# ----------------------------------------------------------------- refusals (no GPU needed)

def _cache8(**kw):
    c = B.gpt_fp8_cache(pages=_cache(), k_scale=FAKE, v_scale=FAKE + 4096, scale_page=4, scale_head=1)
    for k, v in kw.items():
        setattr(c.pages if hasattr(c.pages, k) else c, k, v)
    return c


def _append8(**kw):
    a = B.gpt_kv_append_fp8_args()
    for f, _ in B.gpt_kv_append_args._fields_:
        if hasattr(a, f):
            setattr(a, f, getattr(_append(), f))
    a.before = FAKE
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _sample(**kw):
    a = B.gpt_sample_token_args(logits=FAKE, uniform=FAKE, token=FAKE, logprob=FAKE, kept=FAKE, logits_stride=100, rows=2, vocab=100)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,code,word", [
    (dict(dtype=5), -1, "dtype"), (dict(n_pages=0), -1, "sizes"), (dict(head_dim=136), -8, "head_dim"), (dict(head_dim=72), -8, "head_dim"),
    (dict(k=None), -1, "NULL"), (dict(v=FAKE + 8), -1, "16 bytes"), (dict(slot_stride=264), -1, "16 bytes"),
    (dict(table_stride=7), -1, "table_stride"), (dict(k_scale=None), -1, "k_scale"), (dict(v_scale=FAKE + 2), -1, "4-byte"),
    (dict(scale_page=-1), -1, "negative"), (dict(max_pages=1 << 28, table_stride=1 << 28), -8, "32 bits")])
def test_bad_caches_are_refused(lib, change, code, word):
    c = _cache8(**change)
    for fn, a in ((lib.gpt_kv_append_fp8, _append8()), (lib.gpt_decode_attention_fp8, _attend())):
        assert fn(ctypes.byref(c), ctypes.byref(a), None) == code
        assert word in lib.gpt_last_error(None).decode()
    assert lib.gpt_decode_attention_fp8_workspace(ctypes.byref(c), 8) == 0


@pytest.mark.parametrize("change,word", [
    (dict(n_tokens=-1), "negative"), (dict(n_head=-1), "negative"), (dict(rope_dims=63), "rope_dims"), (dict(rope_dims=66), "rope_dims"),
    (dict(rope_base=0.5), "rope_base"), (dict(rope_base=math.nan), "rope_base"), (dict(k=None), "NULL"), (dict(before=None), "NULL"),
    (dict(n_tokens=4), "sequences"), (dict(k_row=250), "16 bytes"), (dict(v=FAKE + 2), "16 bytes"), (dict(q=None), "n_head"),
    (dict(q_out=None), "n_head"), (dict(n_head=0), "n_head"), (dict(qo_head=60), "16 bytes"), (dict(q_row=-512), "16 bytes"),
    (dict(qo_row=0), "smaller"), (dict(q_row=1024, q_out=FAKE), "strides")])
def test_append_refusals(lib, change, word):
    assert lib.gpt_kv_append_fp8(ctypes.byref(_cache8()), ctypes.byref(_append8(**change)), None) == -1
    assert word in lib.gpt_last_error(None).decode()
    assert lib.gpt_kv_append_fp8(None, ctypes.byref(_append8()), None) == -1
    assert lib.gpt_kv_append_fp8(ctypes.byref(_cache8()), None, None) == -1
    assert lib.gpt_kv_append_fp8(ctypes.byref(_cache8(n_seq=0)), ctypes.byref(_append8()), None) == -1


@pytest.mark.parametrize("change,word", [
    (dict(page_stride=0), "smaller"), (dict(slot_stride=48), "smaller"), (dict(head_stride=0), "smaller"), (dict(scale_page=0), "scales"),
    (dict(scale_page=3), "scales"), (dict(scale_head=0), "scales"), (dict(v_scale=FAKE), "k_scale")])
def test_append_into_overlapping_memory_is_refused(lib, change, word):
    assert lib.gpt_kv_append_fp8(ctypes.byref(_cache8(**change)), ctypes.byref(_append8()), None) == -1
    assert word in lib.gpt_last_error(None).decode()


@pytest.mark.parametrize("change,word", [
    (dict(n_head=6), "multiple"), (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(lens=None), "NULL"), (dict(q=FAKE + 4), "16 bytes"),
    (dict(out_row=508), "16 bytes"), (dict(out_row=0), "smaller"), (dict(scale=math.nan), "scale"), (dict(out=FAKE), "q"),
    (dict(workspace=None), "workspace"), (dict(workspace_bytes=64), "workspace")])
def test_attention_refusals(lib, change, word):
    c = _cache8(max_pages=10000, table_stride=10000) if word == "workspace" else _cache8()
    if word == "workspace":
        assert lib.gpt_decode_attention_fp8_workspace(ctypes.byref(c), 8) > 64
    assert lib.gpt_decode_attention_fp8(ctypes.byref(c), ctypes.byref(_attend(**change)), None) == -1
    assert word in lib.gpt_last_error(None).decode()
    assert lib.gpt_decode_attention_fp8(None, ctypes.byref(_attend()), None) == -1
    assert lib.gpt_decode_attention_fp8(ctypes.byref(_cache8()), None, None) == -1


@pytest.mark.parametrize("change,code,word", [
    (dict(dtype=7), -1, "dtype"), (dict(rows=-1), -1, "negative"), (dict(vocab=0), -1, "vocab"), (dict(vocab=(1 << 30) + 1), -8, "vocab"),
    (dict(token=None, logprob=None, kept=None), -1, "NULL"), (dict(logits=None), -1, "NULL"), (dict(uniform=None), -1, "NULL"),
    (dict(logits_stride=99), -1, "stride"), (dict(logits_stride=-1), -1, "stride"), (dict(logits=FAKE + 2), -1, "boundaries"),
    (dict(logits=FAKE + 1, dtype=1), -1, "boundaries")])
def test_sample_refusals(lib, change, code, word):
    assert lib.gpt_sample_token(ctypes.byref(_sample(**change)), None) == code
    assert word in lib.gpt_last_error(None).decode()
    assert lib.gpt_sample_token(None, None) == -1


def test_head_and_token_counts_beyond_32_bits_of_work_are_refused(lib):
    heads = 1 << 17
    assert lib.gpt_kv_append_fp8(ctypes.byref(_cache8()), ctypes.byref(_append8(n_head=heads)), None) == -8
    assert lib.gpt_kv_append_fp8(ctypes.byref(_cache8()), ctypes.byref(_append8(n_tokens=(1 << 30) + 1, starts=FAKE)), None) == -8
    assert lib.gpt_kv_append_fp8(ctypes.byref(_cache8(n_kv_head=1 << 14, page_stride=1 << 30, slot_stride=1 << 20, scale_page=1 << 14)),
                                 ctypes.byref(_append8(n_tokens=1 << 29, starts=FAKE)), None) == -8
    assert lib.gpt_decode_attention_fp8(ctypes.byref(_cache8()), ctypes.byref(_attend(n_head=heads)), None) == -8


def test_sequence_counts_at_the_end_of_32_bits_are_refused(lib):
    for n in (2 ** 31 - 1, 2 ** 31 - 4096):
        for rc in (lib.gpt_kv_append_fp8(ctypes.byref(_cache8(n_seq=n)), ctypes.byref(_append8()), None),
                   lib.gpt_decode_attention_fp8(ctypes.byref(_cache8(n_seq=n)), ctypes.byref(_attend()), None),
                   lib.gpt_kv_append(ctypes.byref(_cache(n_seq=n)), ctypes.byref(_append()), None),
                   lib.gpt_decode_attention(ctypes.byref(_cache(n_seq=n)), ctypes.byref(_attend()), None)):
            assert rc == -8 and "n_seq" in lib.gpt_last_error(None).decode()
        assert lib.gpt_decode_attention_fp8_workspace(ctypes.byref(_cache8(n_seq=n)), 8) == 0


def test_nothing_to_do_is_no_error(lib):
    assert lib.gpt_kv_append_fp8(ctypes.byref(_cache8()), ctypes.byref(_append8(n_tokens=0)), None) == 0
    assert lib.gpt_decode_attention_fp8(ctypes.byref(_cache8(n_seq=0)), ctypes.byref(_attend()), None) == 0
    assert lib.gpt_sample_token(ctypes.byref(_sample(rows=0)), None) == 0


def test_calls_without_a_gpu_fail_cleanly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for rc in (lib.gpt_kv_append_fp8(ctypes.byref(_cache8()), ctypes.byref(_append8()), None),
               lib.gpt_decode_attention_fp8(ctypes.byref(_cache8()), ctypes.byref(_attend()), None),
               lib.gpt_sample_token(ctypes.byref(_sample()), None)):
        assert rc == -2 and lib.gpt_last_error(None)


def test_structs_match_the_header():
    text = open(os.path.join(os.path.dirname(B.HERE), "include", "gpt.h")).read()
    kinds = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t, "float": ctypes.c_float, "double": ctypes.c_double,
             "gpt_paged_cache": B.gpt_paged_cache}
    for cls in (B.gpt_fp8_cache, B.gpt_kv_append_fp8_args, B.gpt_sample_token_args):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (cls.__name__, cls.__name__), text, re.S).group(1)
        fields = []
        for decl in filter(None, (d.strip() for d in re.sub(r"/\*.*?\*/", "", body, flags=re.S).split(";"))):
            m = re.match(r"((?:const\s+)?\w+)\s*(.*)", decl, re.S)
            fields += [(m.group(1).split()[-1], f.strip()) for f in m.group(2).split(",")]
        want = [(f.lstrip("* "), ctypes.c_void_p if f.startswith("*") else kinds[t]) for t, f in fields]
        assert want == list(cls._fields_), cls.__name__


def test_binding_refuses_tensors_off_the_gpu():
    x, cache, scale = torch.zeros(2, 4, 64), torch.zeros(8, 16, 4, 64).to(F8), torch.zeros(8, 4)
    table, one = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: B.kv_append_fp8(x, x, cache, cache, scale, scale, table, one),
                 lambda: B.decode_attention_fp8(x, cache, cache, scale, scale, table, one),
                 lambda: B.sample_token(torch.zeros(2, 100), torch.zeros(2))):
        with pytest.raises(B.GptError) as e:
            call()
        assert e.value.name == "INVALID_ARG" and "CUDA" in str(e.value)


# ----------------------------------------------------------------- definitions

def _number(bits):
    """The e4m3 numbers of uint8 codes, in float64."""
    bits = np.asarray(bits).astype(np.int64)
    e, f = bits >> 3 & 15, bits & 7
    x = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    x = np.where(bits & 127 == 127, np.nan, x)
    return np.where(bits & 128, -x, x)


def _nearest(x):
    """float64 to the nearest e4m3 number, ties to even; NaN where it is not finite."""
    with np.errstate(all="ignore"):
        e = np.maximum(np.frexp(np.where(np.isfinite(x), x, 0))[1], -5)
        step = 2.0 ** (e - 4.0)
        return np.where(np.isfinite(x), np.rint(x / step) * step, np.nan)


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


def _scale_for(rows):
    """The scale of new rows [rows, heads, dim]."""
    top = np.where(np.isfinite(rows), np.abs(rows), 0).max(axis=(0, 2))
    return np.where(top >= 2.0 ** -119, 2.0 ** (np.frexp(np.maximum(top, 2.0 ** -119))[1] - 8.0), 2.0 ** -126)


def _pool8(rng, n_pages, page, heads, dim, order):
    """A cache of random numbers (no NaN) over memory in the given order of dimensions, and random scales."""
    shape = {"slot": (n_pages, page, heads, dim), "head": (n_pages, heads, page, dim), "gaps": (n_pages, page + 1, heads + 1, dim + 16)}[order]
    pools, scales = [], []
    for _ in range(2):
        bits = rng.integers(0, 256, shape).astype(np.uint8)
        bits = np.where(bits & 127 == 127, 0x33, bits).astype(np.uint8)
        x = torch.from_numpy(bits).cuda().view(F8)
        pools.append(x.transpose(1, 2) if order == "head" else x[:, :page, :heads, :dim] if order == "gaps" else x)
        s = torch.from_numpy(2.0 ** rng.integers(-9, 0, (n_pages, heads)).astype(np.float32)).cuda()
        scales.append(s.t().contiguous().t() if order == "head" else s)
    return (*pools, *scales)


# ----------------------------------------------------------------- kv_append_fp8

def _expect_append(raw, turned, codes, scales, table, page, starts, before, reach):
    """The definition: (numbers, scales, written) after the call."""
    numbers, scales = _number(codes), scales.astype(np.float64).copy()
    written = np.zeros(numbers.shape[:2], dtype=bool)
    for s, b in enumerate(before):
        row, end = starts[s], starts[s + 1]
        if b < 0:
            continue
        while row < end and b < reach:
            p, slot = table[s, b // page], b % page
            n = min(page - slot, end - row)
            if 0 <= p < len(numbers):
                scale = _scale_for(raw[row:row + n])
                if slot > 0:
                    scale = np.maximum(scale, scales[p])
                    moved = scale != scales[p]
                    numbers[p, :slot, moved] = _nearest(numbers[p, :slot, moved] * (scales[p] / scale)[moved, None, None])
                scales[p] = scale
                with np.errstate(all="ignore"):
                    numbers[p, slot:slot + n] = turned[row:row + n] / scale[:, None]
                written[p, slot:slot + n] = True
            row, b = row + n, b + n
    return numbers, scales, written


def _run_append(rng, counts, before, heads, kv, dim, rope, page, order, kind, tail=3, spread=3.0, plain=False, change=None, base=10000.0):
    """One call; everything that it wrote and everything else is compared."""
    n_seq, n = len(counts), sum(counts) + tail
    starts = [1 + sum(counts[:i]) for i in range(n_seq + 1)] if not plain else list(range(n_seq + 1))
    n += 0 if plain else 1
    lens = [max(b, 0) + c for b, c in zip(before, counts)]
    table, n_pages = _pages(rng, lens, page)
    kc, vc, ks, vs = _pool8(rng, n_pages, page, kv, dim, order)
    size = np.exp2(rng.uniform(-spread, spread, (n, 1)))  # tokens of different size: scales that grow
    qkv = _t(rng.standard_normal((n, (heads + 2 * kv) * dim)) * size, kind)
    q, k, v = (x.unflatten(1, (-1, dim)) if x.shape[1] else None for x in qkv.split([heads * dim, kv * dim, kv * dim], dim=1))
    if change:
        change(k, v)
    was = [_codes(x) for x in (kc, vc)] + [_np(x) for x in (ks, vs)]
    qo = torch.full((n, heads + 1, dim), 5.0, dtype=DT[kind], device="cuda")[:, :heads] if heads else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = B.kv_append_fp8(k, v, kc, vc, ks, vs, _i(table), _i(before), starts=None if plain else _i(starts), q=q, rope_dims=rope,
                          rope_base=base, q_out=qo, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    pos = np.zeros(n, dtype=np.int64)
    used = np.zeros(n, dtype=bool)
    for s, b in enumerate(before):
        if b >= 0:
            pos[starts[s]:starts[s + 1]] = b + np.arange(starts[s + 1] - starts[s])
            used[starts[s]:starts[s + 1]] = True
    reach = table.shape[1] * page
    for raw, cache, scale, at, turn in ((_np(k), kc, ks, 0, rope), (_np(v), vc, vs, 1, 0)):
        with np.errstate(all="ignore"):
            turned = _turned(raw, pos, turn, base)
        want, ws, written = _expect_append(raw, turned, was[at], was[2 + at], table, page, starts, before, reach)
        assert np.array_equal(_np(scale), ws)
        have = _number(_codes(cache))
        assert np.array_equal(np.isnan(have), ~np.isfinite(want))
        keep = ~written
        assert np.array_equal(have[keep], want[keep])
        x, y = have[written], want[written]
        fine = np.isfinite(y)
        if turn == 0:
            assert np.array_equal(x[fine], _nearest(y)[fine])
        else:  # the rotation's error in numbers, then one rounding
            r = _turn_tolerance(raw, turned, rope, "fp32", 2.0 ** -24)
            off = _expect_append(raw, r, was[at], was[2 + at], table, page, starts, before, reach)[0][written] + 4 * U * np.abs(y)
            off = np.abs(x - y) - off - np.maximum((np.abs(y) + off) * 2.0 ** -4, 2.0 ** -10)
            assert (off[fine] <= 0).all(), float(off[fine].max())
    if heads:
        assert got is qo
        want = _turned(_np(q), pos, rope, base)
        tol = _turn_tolerance(_np(q), want, rope, kind, 2.0 ** -24)
        want[~used], tol[~used] = 5.0, 0
        _check(qo, want, tol)
    return kc, vc, ks, vs


APPENDS = [  # new tokens of each sequence, tokens before, heads, kv heads, dim, rope, page, order of the cache
    ([1], [0], 8, 8, 64, 64, 16, "slot"), ([1], [37], 2, 1, 16, 2, 1, "slot"), ([3, 0, 20, 1], [5, 9, 0, 31], 12, 4, 64, 32, 24, "head"),
    ([64, 64, 17], [0, 64, 60], 4, 4, 128, 128, 16, "gaps"), ([40, 25], [3, 100], 14, 2, 96, 24, 7, "slot"),
    ([9], [2], 0, 3, 80, 80, 64, "head"), ([300, 5], [100, 0], 8, 1, 128, 0, 128, "slot"), ([200, 1, 1, 90], [0, 7, 8, 63], 6, 6, 32, 10, 33, "head"),
    # rows that a block takes in several windows
    ([700], [11], 2, 1, 128, 64, 512, "slot"), ([1500, 3], [0, 1000], 1, 1, 16, 16, 4000, "slot"),
    # more rows than the small strips are for
    ([4200, 1, 130], [0, 40, 8], 3, 1, 64, 64, 64, "slot"), ([2200, 2300], [5, 63], 4, 2, 96, 96, 32, "gaps")]


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("counts,before,heads,kv,dim,rope,page,order", APPENDS)
def test_append(cuda, kind, counts, before, heads, kv, dim, rope, page, order):
    """Ragged sequences continued in pages begun before: numbers and scales are the definition's, everything else in
    the cache and the query rows of no sequence is what it was."""
    _run_append(_rng(kind, sum(counts), heads, dim), counts, before, heads, kv, dim, rope, page, order, kind)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n,heads,kv,dim,page", [(1, 8, 8, 64, 16), (37, 4, 2, 128, 16), (300, 8, 1, 96, 24), (700, 1, 3, 32, 5), (5000, 2, 1, 64, 16)])
def test_append_one_token_each(cuda, kind, n, heads, kv, dim, page):
    """Without starts: row s is sequence s's, sequences of a negative count left out."""
    rng = _rng(kind, n, dim)
    before = rng.integers(0, 60, n)
    before[rng.random(n) < 0.1] = -1
    _run_append(rng, [1] * n, before.tolist(), heads, kv, dim, dim, page, "slot", kind, tail=0, plain=True)


@gpu
@pytest.mark.parametrize("n_seq", [1023, 1024, 1025, 2047, 2048, 5000])
def test_append_many_sequences(cuda, n_seq):
    """More sequences than a block keeps the starts of."""
    rng = _rng(n_seq)
    counts = rng.integers(0, 4, n_seq)
    before = rng.integers(0, 20, n_seq)
    before[rng.random(n_seq) < 0.05] = -5
    _run_append(rng, counts.tolist(), before.tolist(), 2, 1, 32, 32, 8, "slot", "bf16")


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_append_values_at_the_ends_of_their_range(cuda, kind):
    """Zeros, subnormal, largest and not finite elements; a scale that was 0."""
    def change(k, v):
        big = torch.finfo(k.dtype).max
        k[1:4], v[1:4] = 0, 0
        k[4, 0, :4] = torch.tensor([1e-39, -1e-42, 0, 2.0 ** -126], device="cuda")
        k[4, 0, 4:] = 0
        k[5, 0], v[5, 0] = big, -big
        k[6, 0, 3], v[6, 0, 5] = math.nan, math.inf
        v[7, 0, 2], v[7, 1] = -math.inf, math.nan
        v[8, 0] = 2.0 ** -130
    for counts, before in (([3, 1, 1, 1, 1, 1], [4, 0, 0, 3, 5, 6]), ([3, 4, 2], [16, 1, 30])):
        _run_append(_rng(kind, len(counts)), counts, before, 2, 2, 64, 0, 16, "slot", kind, change=change)
        _run_append(_rng(kind, len(counts)), counts, before, 0, 2, 64, 0, 16, "slot", kind, change=change)
    rng = _rng(kind)
    table, n_pages = _pages(rng, [16], 16)
    kc, vc, ks, vs = _pool8(rng, n_pages, 16, 1, 32, "slot")
    ks.zero_(), vs.zero_()
    x = torch.ones(1, 1, 32, device="cuda", dtype=DT[kind])
    B.kv_append_fp8(x, x, kc, vc, ks, vs, _i(table), _i([5]))
    page = int(table[0, 0])
    assert float(ks[page, 0]) == 2.0 ** -7 and bool((kc.float()[page, :5] == 0).all()) and bool((kc.float()[page, 5] == 128).all())


@gpu
def test_append_token_by_token_is_near_append_at_once(cuda):
    """Pages filled a token at a time and in one call stand for the same values to two roundings."""
    rng = _rng(5)
    n, page, kv, dim = 70, 16, 2, 64
    table, n_pages = _pages(rng, [n], page)
    x = _t(rng.standard_normal((n, 2 * kv, dim)) * np.exp2(rng.uniform(-4, 4, (n, 1, 1))), "bf16")
    k, v = x[:, :kv], x[:, kv:]
    one, all_ = _pool8(rng, n_pages, page, kv, dim, "slot"), _pool8(rng, n_pages, page, kv, dim, "slot")
    for i in range(n):
        B.kv_append_fp8(k[i:i + 1], v[i:i + 1], *one, _i(table), _i([i]), rope_dims=dim)
    B.kv_append_fp8(k, v, *all_, _i(table), _i([0]), starts=_i([0, n]), rope_dims=dim)
    at = np.arange(n)
    for c in range(2):
        got = [(_number(_codes(p[c])) * _np(p[2 + c])[:, None, :, None])[table[0, at // page], at % page] for p in (one, all_)]
        assert np.array_equal(_np(one[2 + c])[table[0, :5]], _np(all_[2 + c])[table[0, :5]])
        step = np.repeat(_np(one[2 + c])[table[0, at // page]][:, :, None], dim, axis=2) * 2.0 ** -9
        off = np.abs(got[0] - got[1]) - np.maximum(np.abs(got[1]) * 2.0 ** -3, step)  # a subnormal number rounded more than once: a step
        assert (off <= 0).all()


@gpu
@pytest.mark.parametrize("what,bit", [("pos", 2), ("page", 4), ("page_low", 4), ("starts", 1), ("end", 1), ("low", 1)])
def test_append_bad_indices_are_skipped_and_reported(cuda, what, bit):
    """What a bad index touches is left as it was; the other sequences are written."""
    rng = _rng(what)
    page, kv, dim, counts, before = 8, 2, 32, [5, 9, 6], [6, 4, 10]
    table, n_pages = _pages(rng, [11, 13, 16], page)
    starts = [0, 5, 14, 20]
    bad = {1}
    if what == "pos":
        before[1] = table.shape[1] * page
    elif what in ("page", "page_low"):
        table[1, :2] = n_pages if what == "page" else -1
    elif what == "starts":
        starts, bad = [0, 5, 30, 20], {1, 2}  # (sequence 2 has no row: 30 is past row 20)
    elif what == "end":
        starts, bad = [0, 5, 14, 30], {2}
    else:
        starts, bad = [-3, 5, 14, 20], {0}
    kc, vc, ks, vs = _pool8(rng, n_pages, page, kv, dim, "slot")
    was = [x.clone() for x in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs)]
    x = _t(rng.standard_normal((20, 3 * kv, dim)), "bf16")
    qo = torch.full((20, kv, dim), 7.0, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.kv_append_fp8(x[:, :kv], x[:, kv:2 * kv], kc, vc, ks, vs, _i(table), _i(before), starts=_i(starts), q=x[:, 2 * kv:], q_out=qo, status=status)
    torch.cuda.synchronize()
    assert int(status) == bit
    for s in range(3):
        rows = slice(sum(counts[:s]), sum(counts[:s + 1]))
        if s in bad:
            assert bool((qo[rows] == 7.0).all())
            pages = [p for p in table[s] if 0 <= p < n_pages]
            for have, old in zip((kc.view(torch.uint8), vc.view(torch.uint8), ks, vs), was):
                assert torch.equal(have[pages], old[pages])
        else:
            assert torch.equal(qo[rows], x[rows, 2 * kv:])
            at = before[s] + np.arange(counts[s])
            got = (_number(_codes(vc)) * _np(vs)[:, None, :, None])[table[s, at // page], at % page]
            want = _np(x[rows, kv:2 * kv])
            assert (np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10 * _np(vs).max())).all()


@gpu
@pytest.mark.parametrize("plain", [False, True])
@pytest.mark.parametrize("pos,turn", [(0, 0.0), (60000, 2.0 ** -32), ((1 << 24) - 2100, 2.0 ** -25)])
def test_append_angles(cuda, pos, turn, plain):
    """Queries (1, 0) become cosine and sine: off by the angle (a turn's part), one step of 2^-24, a rounding."""
    dim, n = 128, 2000
    kc, vc = (torch.zeros(1, 16, 1, dim, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
    ks, vs = torch.ones(1, 1, device="cuda"), torch.ones(1, 1, device="cuda")
    table = torch.zeros(1, 1 << 20, dtype=torch.int32, device="cuda").expand(n if plain else 1, -1)  # (every position in one page)
    x = torch.zeros(n, 1, dim, device="cuda")
    q = torch.zeros(n, 1, dim, device="cuda")
    q[..., ::2] = 1.0
    at = pos + np.arange(n)
    got = B.kv_append_fp8(x, x, kc, vc, ks, vs, table, _i(at if plain else [pos]), starts=None if plain else _i([0, n]), q=q, rope_dims=dim)
    want = _turned(_np(q), at, dim, 10000.0)
    _check(got, want, 2 * math.pi * turn + 2.0 ** -24 + 2.0 ** -25)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("many", [None, 1, 12])
def test_append_to_pages_of_any_scale(cuda, kind, many):
    """Pages begun by other code, with scales that are no powers of two: elements at (and near) the middle between two numbers
    of their page's scale, and numbers whose product with the old scale over the new one is near the middle, are
    rounded as the exact quotients.  many: rows of each sequence; None: one each, without starts."""
    rng = _rng(kind, str(many))
    n_seq, kv, dim, page, slot = 300, 2, 32, 16, 3
    n = many or 1
    bits = 19 if kind == "fp32" else 3  # 5 bits of the middle and these are the element's
    mant = 1 + rng.integers(1, 1 << bits, (n_seq, kv)) / 2.0 ** bits
    scale = mant * 2.0 ** rng.integers(-3, 4, (n_seq, kv))
    grown = np.arange(n_seq) % 3 == 0  # the others keep their scales
    middle = (2 * rng.integers(8, 16, (n_seq, n, kv, dim)) + 1) * 2.0 ** rng.integers(-6, 3, (n_seq, n, kv, dim))
    x = middle * scale[:, None, :, None] * rng.choice([-1.0, 1.0], middle.shape)
    x += np.where(rng.random(x.shape) < 0.3, x * 2.0 ** -23, 0)
    x[grown] *= 2.0 ** 10
    number = rng.integers(9, 16, (n_seq, kv))  # n m is within n / 2 of a middle of 5 bits, m the old scale's 24 bits
    m = (2 * rng.integers(8, 16, (n_seq, kv)) + 1) * 2.0 ** 23 / number
    m = np.rint(np.where(m < 2 ** 24, m, m / 2))
    scale[grown] = (m * 2.0 ** -24)[grown]
    scale = scale.astype(np.float32)
    kc, vc, ks, vs = _pool8(rng, n_seq, page, kv, dim, "slot")
    ks.copy_(torch.from_numpy(scale)), vs.copy_(torch.from_numpy(scale))
    for c in (kc, vc):
        c[:, 0] = torch.from_numpy(number[:, :, None] * np.ones(dim)).cuda().float().to(F8)
    was = [_codes(c) for c in (kc, vc)]
    rows = _t(x.reshape(n_seq * n, kv, dim), kind)
    table, before, starts = np.arange(n_seq)[:, None], [slot] * n_seq, [n * s for s in range(n_seq + 1)]
    B.kv_append_fp8(rows, rows, kc, vc, ks, vs, _i(table), _i(before), starts=_i(starts) if many else None)
    for c, s, old in ((kc, ks, was[0]), (vc, vs, was[1])):
        want, ws, written = _expect_append(_np(rows), _np(rows), old, scale, table, page, starts, before, page)
        assert np.array_equal(_np(s), ws) and bool((ws[grown] != scale[grown]).all()) and bool((ws[~grown] == scale[~grown]).all())
        have = _number(_codes(c))
        assert np.array_equal(have[~written], want[~written])
        assert np.array_equal(have[written], _nearest(want[written]))


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("many", [None, 2, 12])
def test_append_rotated_to_pages_of_any_scale(cuda, kind, many):
    rng = _rng(kind, str(many), 1)
    n_seq, kv, dim, page, slot, n = 60, 2, 64, 16, 3, many or 1
    kc, vc, ks, vs = _pool8(rng, n_seq, page, kv, dim, "slot")
    scale = rng.uniform(0.01, 0.04, (n_seq, kv)).astype(np.float32)
    scale[0] = 1.5 * 2.0 ** 127
    ks.copy_(torch.from_numpy(scale)), vs.copy_(torch.from_numpy(scale))
    was, rows = _codes(kc), _t(rng.standard_normal((n_seq * n, kv, dim)), kind)
    rows[:n] *= 2.0 ** 124
    table, before, starts = np.arange(n_seq)[:, None], [slot] * n_seq, [n * s for s in range(n_seq + 1)]
    B.kv_append_fp8(rows, rows, kc, vc, ks, vs, _i(table), _i(before), starts=_i(starts) if many else None, rope_dims=dim)
    pos = slot + np.arange(n_seq * n) % n
    turned = _turned(_np(rows), pos, dim, 10000.0)
    want, ws, written = _expect_append(_np(rows), turned, was, scale, table, page, starts, before, page)
    assert np.array_equal(_np(ks), ws)
    have, off = _number(_codes(kc)), _turn_tolerance(_np(rows), turned, dim, "fp32", 2.0 ** -24)
    off = _expect_append(_np(rows), off, was, scale, table, page, starts, before, page)[0]
    assert np.array_equal(have[~written], want[~written])
    x, y, off = have[written], want[written], off[written]
    assert (np.abs(x - y) <= off + np.maximum((np.abs(y) + off) * 2.0 ** -4, 2.0 ** -10)).all()


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_append_starts_that_decrease_stay_inside_their_pages(cuda, kind):
    """Row 5 is found in sequence 3, at the last slot of a page, rows 6 to 8 in sequence 5, which begins at row 5 too: they
    are not the slots after that page's last one.  Sequences that nothing overlaps are written."""
    rng = _rng(kind)
    page, kv, dim, heads = 16, 2, 32, 2
    starts, before = [0, 2, 4, 5, 6, 5, 9, 12], [0, 3, 0, 15, 0, 0, 14]
    table = np.array([[0, 9], [1, 9], [2, 9], [7, 9], [3, 9], [4, 9], [5, 6]])  # 7: the last of the pool
    pools = [torch.full((9, page, kv, dim), 0x33, dtype=torch.uint8, device="cuda") for _ in range(2)]
    kc, vc = (x[:8].view(F8) for x in pools)
    ks, vs = torch.full((8, kv), 0.5, device="cuda"), torch.full((8, kv), 0.5, device="cuda")
    x = _t(rng.standard_normal((12, 2 * kv + heads, dim)), kind)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.kv_append_fp8(x[:, :kv], x[:, kv:2 * kv], kc, vc, ks, vs, _i(table), _i(before), starts=_i(starts), q=x[:, 2 * kv:], status=status)
    torch.cuda.synchronize()
    assert int(status) == B.STATUS_BAD_SEQ
    for pool in pools:
        assert bool((pool[8] == 0x33).all()) and bool((pool[3] == 0x33).all())  # behind the pool; the sequence whose pair decreases
    for s in (0, 1, 2, 6):
        rows, at = np.arange(starts[s], starts[s + 1]), before[s] + np.arange(starts[s + 1] - starts[s])
        got = (_number(_codes(vc)) * _np(vs)[:, None, :, None])[table[s, at // page], at % page]
        want = _np(x)[rows, kv:2 * kv]
        assert (np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10 * _np(vs).max())).all()


# ----------------------------------------------------------------- decode_attention_fp8

def _fill8(rng, lens, table, page, cache, spread=1):
    """Random keys and values with a scale for each page and head at the sequences' positions, NaN elsewhere; returns what they
    stand for, per sequence, in float64."""
    kc, vc, ks, vs = cache
    n_pages, _, heads, dim = kc.shape
    out = []
    numbers = []
    for c, s in ((kc, ks), (vc, vs)):
        scale = 2.0 ** rng.integers(-spread, spread + 1, (n_pages, heads)) * rng.uniform(1, 2, (n_pages, heads)) / 64
        s.copy_(torch.from_numpy(scale.astype(np.float32)))
        x = torch.from_numpy(np.clip(rng.standard_normal((n_pages, page, heads, dim)) * 64, -440, 440).astype(np.float32)).cuda().to(F8)
        inside = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
        for i, n in enumerate(lens):
            at = np.arange(n)
            inside[torch.from_numpy(table[i, at // page].astype(np.int64)).cuda(), torch.from_numpy(at % page).cuda()] = True
        x = torch.where(inside[:, :, None, None], x.view(torch.uint8), 0x7f).to(torch.uint8)
        c.view(torch.uint8).copy_(x)
        numbers.append(_number(x.cpu().numpy()) * _np(s)[:, None, :, None])
    for i, n in enumerate(lens):
        at = np.arange(n)
        out.append([x[table[i, at // page], at % page] for x in numbers])
    return out


def _attention8(q, keys, values, scale, kind):
    """Definition and bounds for one sequence: (out, lse, bound of out without its last rounding, of lse)."""
    heads, dim = q.shape
    n, kv = keys.shape[:2]
    g = heads // kv
    if n == 0:
        return np.zeros((heads, dim)), np.full(heads, -np.inf), np.zeros((heads, dim)), np.zeros(heads)
    K, V = np.repeat(keys, g, axis=1), np.repeat(values, g, axis=1)
    z = np.einsum("hd,nhd->hn", q, K) * scale
    a = np.einsum("hd,nhd->hn", np.abs(q), np.abs(K)) * abs(scale)
    small = np.abs(q).max(axis=1)[:, None] * np.abs(K).sum(axis=2).T * abs(scale)
    m = z.max(axis=1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(axis=1, keepdims=True)
    w = p / l
    out = np.einsum("hn,nhd->hd", w, V)
    spread = np.einsum("hn,nhd->hd", w, np.abs(V))
    # a score: sums of dim products, cut, not rounded (2 u), its factors; fp32 queries in two fp16 parts (2^-23), elements below
    # 2^-25 of 2^14 lost.  A weight: that, 2^-20 for the exponentials, its rounding to fp16 (2^-11; two parts: 2^-22).
    dz = ((2 * dim + 8) * U + (2.0 ** -23 if kind == "fp32" else 0)) * a.max(axis=1) + 2.0 ** -39 * small.max(axis=1) + 3 * U * np.abs(z - m).max(axis=1)
    dz = dz + 2.0 ** -20
    dw = dz + (2.0 ** -22 if kind == "fp32" else 2.0 ** -11)
    tol = spread * (2 * dw + 2 * (n + 8) * U)[:, None] + 2.0 ** -32 * n * np.abs(V).max(axis=(0, 2))[:, None]
    return out, (m + np.log(l))[:, 0], tol, dz + (n + 8) * U + 4 * U * np.abs(m[:, 0])


def _check_attention(got, lse, q, parts, scale, kind, least=0.0):
    """``least``: half a step of subnormal results."""
    for s, (k, v) in enumerate(parts):
        want, wl, tol, tl = _attention8(_np(q)[s], k, v, scale, kind)
        if kind == "bf16":
            tol = tol + (np.abs(want) + tol) * 2.0 ** -8
        _check(got[s], want, tol + least)
        if len(k):
            _check(lse[s], wl, tl)
        else:
            assert bool((lse[s] == -math.inf).all())


def _run_attention8(rng, lens, heads, kv, dim, page, kind, order="slot", scale=None, strided=False, reach=0, spread=1):
    table, n_pages = _pages(rng, lens, page, width=-(-reach // page))
    cache = _pool8(rng, n_pages, page, kv, dim, order)
    parts = _fill8(rng, lens, table, page, cache, spread)
    q = _t(rng.standard_normal((len(lens), heads, dim)), kind)
    out = None
    if strided:
        wide = torch.full((len(lens), heads + 2, dim + 16), 3.0, dtype=DT[kind], device="cuda")
        out = wide[:, :heads, :dim]
        q = torch.cat([q, q.new_zeros(len(lens), 1, dim)], dim=1)[:, :heads]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = B.decode_attention_fp8(q, *cache, _i(table), _i(lens), scale=scale, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    _check_attention(got, lse, q, parts, dim ** -0.5 if scale is None else scale, kind)
    if strided:
        assert bool((wide[:, heads:] == 3.0).all()) and bool((wide[..., dim:] == 3.0).all())
    return got, lse


ATTENDS = [  # lengths, heads, kv heads, dim, page, order
    ([1], 8, 8, 64, 16, "slot"), ([0], 4, 4, 64, 16, "slot"), ([513], 12, 12, 64, 16, "slot"),
    ([0, 1, 15, 16, 17, 300, 0], 16, 16, 64, 16, "head"), ([257, 1, 64, 1000], 32, 8, 128, 16, "slot"),
    ([129, 700], 7, 1, 80, 24, "gaps"), ([33, 200, 128], 12, 4, 96, 7, "head"), ([5, 2000], 64, 2, 32, 64, "slot"),
    ([31, 32, 33], 3, 3, 16, 1, "slot"), ([400], 17, 1, 64, 128, "slot"), ([63, 65], 24, 2, 112, 40, "gaps"),
    ([4097], 8, 8, 64, 32, "head"), ([3001, 2], 16, 1, 128, 16, "head"), ([100, 1000], 5, 1, 128, 8, "slot"), ([77, 300], 9, 1, 48, 12, "slot")]


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,heads,kv,dim,page,order", ATTENDS)
def test_attention(cuda, kind, lens, heads, kv, dim, page, order, reach):
    """Everything that no sequence's length covers is NaN, and table entries past it name no page."""
    _run_attention8(_rng(kind, dim, len(lens), heads), lens, heads, kv, dim, page, kind, order, reach=reach)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("page", [16, 8, 5])
def test_attention_scales_far_apart(cuda, kind, page):
    """Neighbouring pages' scales differ by up to 2^24."""
    _run_attention8(_rng(kind, page), [100, 37, 611], 8, 2, 64, page, kind, spread=12)
    _run_attention8(_rng(kind, page), [100, 37, 611], 8, 2, 128, page, kind, spread=12, reach=400000)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("page", [16, 8, 5])
@pytest.mark.parametrize("heads,dim", [(4, 64), (3, 128), (8, 64), (7, 128), (16, 64), (17, 96)])
def test_attention_weight_in_pages_of_small_scales(cuda, kind, heads, dim, page, reach):
    """One page has the weight, the others a larger value scale: what is lost is 2^-32 of the largest product of a weight and
    a scale, not of the largest weight times the largest scale.  Scores are one exact product: off by the roundings of its
    factors, 4 u of itself."""
    rng = _rng(kind, heads, dim, page)
    cases = [(gap, up, at) for gap, up in ((80, 10), (80, 20), (80, 28), (80, 33), (80, 40), (80, 90), (20, 28), (20, 40), (0, 40), (0, -40))
             for at in (0, 2, 5)]
    lens = [5 * page + 1 + i % page for i in range(len(cases))]
    table, n_pages = _pages(rng, lens, page, width=-(-reach // page))
    kc, vc, ks, vs = cache = _pool8(rng, n_pages, page, 1, dim, "slot")
    _fill8(rng, lens, table, page, cache)
    ks.fill_(2.0 ** -6), vs.fill_(1.0)
    first = torch.full((n_pages, page), -320.0, device="cuda")
    for s, (gap, up, at) in enumerate(cases):
        pages = table[s, :6]
        vs[torch.from_numpy(pages).cuda().long()] = 2.0 ** up * float(rng.uniform(1, 2))
        vs[int(pages[at])] = float(rng.uniform(1, 2))
        first[torch.from_numpy(pages).cuda().long()] = -4.0 * gap  # (gap 80: -320 / 64 * 8 = -40)
        first[int(pages[at])] = 4.0 * gap
    kc[:, :, 0, 0] = (first * torch.from_numpy(rng.choice([1.0, 0.9375], (n_pages, page))).cuda().float()).to(F8)
    q = torch.zeros(len(cases), heads, dim, device="cuda", dtype=DT[kind])
    q[:, :, 0] = 8.0
    out, lse = B.decode_attention_fp8(q, *cache, _i(table), _i(lens), scale=1.0)
    for s, n in enumerate(lens):
        at = np.arange(n)
        where = table[s, at // page], at % page
        z = 8 * _number(_codes(kc))[where][:, 0, 0] / 64
        numbers, scale = _number(_codes(vc))[where][:, 0], _np(vs)[where[0], 0]
        w = np.exp(z - z.max())
        total, w = w.sum(), w / w.sum()
        want = (w * scale) @ numbers
        dw = 4 * U * 1.5 * np.abs(z).max() + 2.0 ** -20 + 2.0 ** -22
        tol = (w * scale) @ np.abs(numbers) * (2 * dw + 2 * (n + 8) * U) + 2.0 ** -32 * n * 448 * (w * scale).max()
        step = 2.0 ** (np.floor(np.log2(np.abs(want) + tol)) - 8) if kind == "bf16" else 0
        _check(out[s], np.tile(want, (heads, 1)), np.tile(tol + step, (heads, 1)))
        _check(lse[s], np.full(heads, z.max() + np.log(total)), dw + (n + 8) * U + 4 * U * abs(z).max())


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -126, 2.0 ** -140, 2.0 ** 118])
def test_attention_value_scales_at_the_ends(cuda, kind, size):
    """Pages whose value scales are 0, subnormal or near the largest, beside ordinary ones and alone."""
    rng = _rng(kind, str(size))
    lens, heads, kv, dim, page = [64, 40, 64], 4, 1, 64, 16
    table, n_pages = _pages(rng, lens, page)
    cache = _pool8(rng, n_pages, page, kv, dim, "slot")
    parts = _fill8(rng, lens, table, page, cache)
    vs = cache[3]
    for s, pages in ((0, [0, 1, 2, 3]), (1, [1]), (2, [0, 3])):
        for i in pages:
            p = int(table[s, i])
            at = slice(16 * i, min(16 * i + 16, lens[s]))
            parts[s][1][at] *= float(np.float32(size)) / float(vs[p, 0])
            vs[p] = size
    q = _t(rng.standard_normal((3, heads, dim)), kind)
    out, lse = B.decode_attention_fp8(q, *cache, _i(table), _i(lens))
    # (half a step of subnormal results, 2^-150, in bf16 2^-134)
    _check_attention(out, lse, q, parts, dim ** -0.5, kind, 2.0 ** -134 if kind == "bf16" else 2.0 ** -150)


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("page", [16, 8, 5])
@pytest.mark.parametrize("heads,dim", [(4, 64), (3, 128), (8, 64), (7, 128), (16, 64), (17, 96)])
def test_attention_rounds_bf16_results_once(cuda, heads, dim, page, reach):
    """Results in bf16 are those in fp32 and one rounding: half a step of the binade.  (Small scores, so that
    their own errors do not hide what the weights lose.)"""
    rng = _rng(heads, dim, page)
    lens, scale = [1, 2, 3, 5, 9, 30, 70], 2.0 ** -8
    table, n_pages = _pages(rng, lens, page, width=-(-reach // page))
    cache = _pool8(rng, n_pages, page, 1, dim, "slot")
    parts = _fill8(rng, lens, table, page, cache)
    q = _t(rng.standard_normal((len(lens), heads, dim)), "bf16")
    out, _ = B.decode_attention_fp8(q, *cache, _i(table), _i(lens), scale=scale)
    for s, (k, v) in enumerate(parts):
        want, _, tol, _ = _attention8(_np(q)[s], k, v, scale, "fp32")
        _check(out[s], want, tol + 2.0 ** (np.floor(np.log2(np.abs(want) + tol)) - 8))


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_attention_strided_and_scaled(cuda, kind):
    _run_attention8(_rng(kind), [70, 0, 9], 6, 2, 64, 16, kind, "gaps", scale=0.3, strided=True)
    _run_attention8(_rng(kind), [70, 3], 6, 2, 64, 16, kind, scale=0.0)


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("page", [16, 8, 5])
def test_attention_every_length_near_a_split(cuda, kind, page, reach):
    _run_attention8(_rng(kind, page, 1), list(range(0, 70)) + [127, 128, 129, 255, 256, 257], 4, 2, 64, page, kind, reach=reach)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n_seq", [19, 37, 50, 76, 152, 153, 304, 305, 609, 2433])
def test_attention_rows_per_block(cuda, kind, n_seq):
    rng = _rng(kind, n_seq)
    _run_attention8(rng, rng.integers(0, 60, n_seq).tolist(), 2, 1, 64, 16, kind)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n_seq,kv", [(700, 1), (300, 4), (2000, 2)])
def test_attention_many_sequences(cuda, kind, n_seq, kv):
    rng = _rng(kind, n_seq, kv)
    _run_attention8(rng, rng.integers(0, 130, n_seq).tolist(), 2 * kv, kv, 32, 16, kind, reach=100000)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -60, 1.0, 2.0 ** 60, 2.0 ** 118])
def test_attention_query_and_scale_sizes(cuda, kind, size):
    """Queries and key scales of any size whose scores are ordinary; value scales of any size."""
    rng = _rng(kind, str(size))
    lens, heads, kv, dim, page = [90, 41], 4, 2, 64, 16
    table, n_pages = _pages(rng, lens, page)
    cache = _pool8(rng, n_pages, page, kv, dim, "slot")
    parts = _fill8(rng, lens, table, page, cache)
    cache[2].mul_(1 / size)
    cache[3].mul_(size)
    q = _t(rng.standard_normal((2, heads, dim)), "fp32")
    q = (q * size).to(DT[kind])
    out, lse = B.decode_attention_fp8(q, *cache, _i(table), _i(lens))
    # results below 2^-126 are multiples of 2^-149, in bf16 of 2^-133: half of that, in parts of the size
    _check_attention(out.double() / size, lse, q.double() / size, parts, dim ** -0.5, kind, (2.0 ** -134 if kind == "bf16" else 2.0 ** -150) / size)


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("page", [16, 5])
def test_attention_nan_values(cuda, kind, page, reach):
    """A NaN belongs in the result of its dim at any key that counts, however small the key's weight; elsewhere nothing changes."""
    rng = _rng(kind, page)
    lens, heads, kv, dim = [300, 40], 4, 2, 64
    table, n_pages = _pages(rng, lens, page, width=-(-reach // page))
    cache = _pool8(rng, n_pages, page, kv, dim, "slot")
    parts = _fill8(rng, lens, table, page, cache)
    q = _t(rng.standard_normal((2, heads, dim)), kind)
    z = np.einsum("hd,nhd->hn", _np(q)[0], np.repeat(parts[0][0], 2, axis=1))
    j = int(z[:2].max(axis=0).argmin())  # the least weight of key head 0
    cache[1].view(torch.uint8)[int(table[0, j // page]), j % page, 0, 7] = 0xff
    out, lse2 = B.decode_attention_fp8(q, *cache, _i(table), _i(lens))
    nan = torch.isnan(out)
    assert bool(nan[0, :2, 7].all()) and int(nan.sum()) == 2
    step = 2.0 ** -8 if kind == "bf16" else 0
    for s, (k, v) in enumerate(parts):
        want, wl, tol, tl = _attention8(_np(q)[s], k, v, dim ** -0.5, kind)
        _check(lse2[s], wl, tl)  # (heads with a NaN are computed once more, in another order)
        off = np.abs(_np(out)[s] - want) - tol - (np.abs(want) + tol) * step
        assert (off[~nan[s].cpu().numpy()] <= 0).all()


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_attention_bad_pages_and_lengths(cuda, kind):
    rng = _rng(kind)
    lens, page, heads, kv, dim = [100, 60, 30, 20], 16, 4, 2, 64
    table, n_pages = _pages(rng, lens, page)
    cache = _pool8(rng, n_pages, page, kv, dim, "slot")
    parts = _fill8(rng, lens, table, page, cache)
    q = _t(rng.standard_normal((4, heads, dim)), kind)
    broken = table.copy()
    broken[0, 2], broken[1, 0] = n_pages, -7
    given = [100, 60, -4, 20]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = B.decode_attention_fp8(q, *cache, _i(broken), _i(given), status=status)
    assert int(status) == B.STATUS_BAD_PAGE | B.STATUS_BAD_POS
    keep0 = np.r_[0:32, 48:100]
    want = [[x[keep0] for x in parts[0]], [x[16:] for x in parts[1]], [x[:0] for x in parts[2]], parts[3]]
    _check_attention(out, lse, q, want, dim ** -0.5, kind)


@gpu
def test_attention_shared_scales_pages_and_repeats(cuda):
    """One table row and one scale for all; the same bits every time."""
    rng = _rng(3)
    page, kv, dim, n = 16, 2, 64, 200
    table, n_pages = _pages(rng, [n], page)
    kc, vc, _, _ = _pool8(rng, n_pages, page, kv, dim, "slot")
    scale = [torch.full((1, 1), x, device="cuda").expand(n_pages, kv) for x in (0.01, 0.02)]
    shared = _i(table).expand(5, -1)
    q = _t(rng.standard_normal((5, 4, dim)), "bf16")
    lens = [n, 3, 100, 0, 200]
    got = [B.decode_attention_fp8(q, kc, vc, *scale, shared, _i(lens)) for _ in range(3)]
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    at = np.arange(n)
    k, v = (_number(_codes(c))[table[0, at // page], at % page] * float(s[0, 0]) for c, s in zip((kc, vc), scale))
    _check_attention(*got[0], q, [(k[:m], v[:m]) for m in lens], dim ** -0.5, "bf16")


@gpu
@pytest.mark.parametrize("step", [(1 << 31) + 4096, (1 << 33) + 4096])
def test_offsets_past_32_bits(cuda, step):
    """Pages whose offsets in bytes do not fit 32 bits, written and read."""
    kv, dim, page, heads = 1, 64, 16, 2
    pools = [torch.empty(step + page * kv * dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    kc, vc = (x.as_strided((2, page, kv, dim), (step, kv * dim, dim, 1)).view(F8) for x in pools)
    ks, vs = torch.zeros(2, kv, device="cuda"), torch.zeros(2, kv, device="cuda")
    rng = _rng(step % 1000)
    x = _t(rng.standard_normal((20, 2 * kv, dim)), "bf16")
    table = np.array([[1, 0]])
    B.kv_append_fp8(x[:, :kv], x[:, kv:], kc, vc, ks, vs, _i(table), _i([0]), starts=_i([0, 20]))
    q = _t(rng.standard_normal((1, heads, dim)), "bf16")
    out, lse = B.decode_attention_fp8(q, kc, vc, ks, vs, _i(table), _i([20]))
    at = np.arange(20)
    k, v = ((_number(_codes(c.contiguous())) * _np(s)[:, None, :, None])[table[0, at // page], at % page] for c, s in ((kc, ks), (vc, vs)))
    want = _np(x[:, kv:])
    assert (np.abs(v - want) <= np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10)).all()
    _check_attention(out, lse, q, [(k, v)], dim ** -0.5, "bf16")


# ----------------------------------------------------------------- sample_token

def _draw(z, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Definition for one row: (token, logprob, kept, how near a limit or the number is to a border, in parts of the sum)."""
    z = np.asarray(z, dtype=np.float64)
    ids = np.nonzero(z > -np.inf)[0]
    if len(ids) == 0:
        return -1, -np.inf, 0, 1.0
    ids = ids[np.lexsort((ids, -z[ids]))]
    if not t > 0:
        return int(ids[0]), 0.0, 1, 1.0
    m = z[ids[0]]
    with np.errstate(all="ignore"):
        w = np.where(z[ids] == m, 1.0, np.exp((z[ids] - m) / np.float64(t)) if np.isfinite(m) else 0.0)
    n, near = len(ids), 1.0
    if top_k >= 1:
        n = min(n, top_k)
    if top_p < 1:
        sums = np.cumsum(w[:n])
        goal = np.float64(top_p) * sums[-1]
        near = min(near, np.abs(sums - goal).min() / sums[-1]) if top_p > 0 else near
        n = 1 + int((sums[:-1] < goal).sum()) if top_p > 0 else 1
    if min_p > 0:
        near = min(near, np.abs(np.log(np.maximum(w[:n], 1e-300)) - np.log(np.float64(min_p))).min())
        n = max(1, min(n, int((w >= np.float64(min_p)).sum())))
    order = np.argsort(ids[:n])
    kept, w = ids[:n][order], w[:n][order]
    sums = np.cumsum(w)
    u = 0.0 if not u >= 0 else float(u)
    if u >= 1:
        at = int(np.nonzero(w > 0)[0][-1])
    else:
        at = int((sums <= u * sums[-1]).sum())
        near = min(near, np.abs(sums - u * sums[-1])[w > 0].min() / sums[-1])
    return int(kept[at]), float(np.log(w[at] / sums[-1])), n, near


def _run_sample(z, u, kind="fp32", t=None, k=None, p=None, mp=None, exact=False):
    """Rows drawn and compared; rows whose numbers lie within 2^-33 of a border (64-bit sums of many weights, each side's) may differ, unless
    ``exact``: inputs whose sums have no rounding."""
    zt = _t(z, kind) if not isinstance(z, torch.Tensor) else z
    f = lambda x: None if x is None else _t(np.broadcast_to(np.asarray(x, dtype=np.float32), len(zt)).copy())  # noqa: E731
    kt = None if k is None else _i(np.broadcast_to(np.asarray(k), len(zt)).copy())
    ut, tt, pt, mt = f(u), f(t), f(p), f(mp)
    token, logprob, kept = B.sample_token(zt, ut, temperature=tt, top_k=kt, top_p=pt, min_p=mt)
    torch.cuda.synchronize()
    zn, sure = _np(zt), 0
    val = lambda x, i, d: d if x is None else x[i].item()  # noqa: E731
    for i in range(len(zn)):
        want, lp, n, near = _draw(zn[i], val(ut, i, 0.0), val(tt, i, 1.0), val(kt, i, 0), val(pt, i, 1.0), val(mt, i, 0.0))
        if not exact and near < 2.0 ** -33:
            continue
        sure += 1
        assert int(token[i]) == want and int(kept[i]) == n, (i, int(token[i]), want, int(kept[i]), n, near)
        if math.isinf(lp):
            assert float(logprob[i]) == lp
        else:
            # Weight, sum and quotient rounded to fp32 (3 * 2^-24), the logarithm to 2^-23 of itself: below 2^-21.  Without
            # limits the sum is of fp32 numbers, good to 2^-21, and in other units (a power of two to 2^-21, a product's 2^-24):
            # 2^-20 + 4 * 2^-24 + 2^-23, below 2^-19.
            free = not 1 <= val(kt, i, 0) < zn.shape[1] and not val(pt, i, 1.0) < 1 and not val(mt, i, 0.0) > 0
            assert abs(float(logprob[i]) - lp) <= 2.0 ** (-19 if free else -21) * max(1.0, abs(lp)), (i, float(logprob[i]), lp)
    assert sure >= 0.9 * len(zn) - 1
    return token, logprob, kept


def _logits(rng, rows, vocab, tail=1.5):
    return 2.5 * rng.standard_normal((rows, vocab)) + rng.exponential(tail, (rows, vocab))


FILTERS = {"none": {}, "k": dict(k=40), "k1": dict(k=1), "big_k": dict(k=3000), "p": dict(p=0.9), "small_p": dict(p=0.1), "min": dict(mp=0.05),
           "all": dict(k=50, p=0.95, mp=0.02), "k_p": dict(k=5000, p=0.97), "wide_p": dict(p=0.9999)}


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 256), (3, 12288), (5, 50304), (7, 4999), (2, 1), (9, 33), (3, 131072), (2, 200001)])
@pytest.mark.parametrize("which", list(FILTERS))
def test_sample(cuda, kind, rows, vocab, which):
    rng = _rng(kind, rows, vocab, which)
    _run_sample(_logits(rng, rows, vocab), rng.random(rows), kind, t=rng.uniform(0.5, 1.5, rows), **FILTERS[which])


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(200, 300), (41, 6000), (700, 1000), (160, 20000)])
def test_sample_mixed_rows(cuda, kind, rows, vocab):
    """Every row with settings of its own, some of them off."""
    rng = _rng(kind, rows, vocab)
    pick = lambda on, off: np.where(rng.random(rows) < 0.5, on, off)  # noqa: E731
    _run_sample(_logits(rng, rows, vocab), rng.random(rows), kind, t=pick(rng.uniform(0.3, 2.0, rows), 0.0 if vocab == 300 else 1.0),
                k=pick(rng.integers(1, vocab, rows), 0), p=pick(rng.random(rows), 1.0), mp=pick(rng.random(rows) ** 3, 0.0))


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 7, 64, 1000, 8192, 50304])
def test_sample_equal_logits(cuda, kind, vocab):
    """All weights the same: limits cut by id, borders are met exactly."""
    u = np.array([0.0, 0.25, 0.5, 0.75, 0.999, 0.5, 0.5, 0.5])
    k = np.array([0, 0, 0, 0, 0, 8, 8, 3])
    p = np.array([1, 1, 1, 1, 0.5, 0.5, 1, 0.25])
    for c in (0.0, -7.25, 300.0):
        _run_sample(np.full((8, vocab), c), u, kind, t=2.0, k=k, p=p, mp=1.0, exact=True)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_sample_few_values(cuda, kind):
    """Logits of a few values, thousands of each: limits that end among equal ones."""
    rng = _rng(kind)
    z = rng.integers(-3, 3, (24, 9000)).astype(float)
    _run_sample(z, rng.random(24), kind, t=0.7, k=np.arange(24) * 250, p=np.linspace(0.05, 1.2, 24))
    _run_sample(z, rng.random(24), kind, k=np.arange(24) * 400 + 1, mp=np.linspace(0, 1.1, 24))
    _run_sample(z, rng.random(24), kind, p=np.linspace(0.001, 0.999, 24))


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [4096, 20011, 131072])
def test_sample_counts_near_list_sizes(cuda, kind, vocab):
    """top_k around the lengths at which lists are treated in other ways, logits all apart and of a few values."""
    rng = _rng(kind, vocab)
    k = np.array([1, 2, 255, 256, 257, 511, 1023, 1024, 1025, 2047, 4095, vocab - 1])
    for z in (_logits(rng, len(k), vocab), rng.integers(-4, 4, (len(k), vocab)).astype(float)):
        _run_sample(z, rng.random(len(k)), kind, t=1.3, k=k)
        _run_sample(z, rng.random(len(k)), kind, t=0.8, k=k, p=0.9, mp=0.001)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab,t,p,mp", [(131072, 2.0, 0.9, None), (131072, 5.0, 0.6, None), (50304, 2.0, 0.97, 1e-6), (50304, 2.0, 0.97, 0.01), (9999, 1.5, 0.9, None),
                                          (20000, 50.0, 0.5, None), (20000, 3.0, 0.99999, None), (700, 2.0, 0.95, 1e-3)])
def test_sample_wide_nucleus(cuda, kind, vocab, t, p, mp):
    """top_p that keeps thousands: numbers across [0, 1) give tokens of every part of the row."""
    rng = _rng(kind, vocab, t, p)
    z = np.repeat(_logits(rng, 2, vocab), 33, axis=0)
    _run_sample(z, np.tile((np.arange(33) + rng.random(33)) / 33, 2), kind, t=t, p=p, mp=mp)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_sample_one_value_beside_thousands(cuda, kind):
    """One token far above, all others at or near one value: a bin with most of the row in it."""
    rng = _rng(kind)
    z = np.full((12, 30000), -2.0)
    z[4:8] += 2.0 ** -7 * rng.integers(0, 2, (4, 30000))
    z[8:] += 1e-3 * rng.random((4, 30000))
    z[np.arange(12), rng.integers(0, 30000, 12)] = 6.0
    for p in (0.05, 0.5, 0.999):
        _run_sample(z, rng.random(12), kind, p=p)
    _run_sample(z, rng.random(12), kind, k=5000)
    _run_sample(z, rng.random(12), kind, k=5000, p=0.7)
    _run_sample(z, rng.random(12), kind, mp=1e-5)


@gpu
def test_sample_edge_rows(cuda):
    inf, nan = math.inf, math.nan
    z = np.zeros((14, 40))
    z[0] = -inf
    z[1] = nan
    z[2], z[2, 7] = -inf, -3.0
    z[3, 5], z[3, 6] = nan, 2.0
    z[4, 9] = z[4, 30] = inf
    z[5, 3] = -inf
    z[6, :] = -3e38
    z[6, 8] = 3e38
    z[7] = np.arange(40) * 3e36
    z[8, 11] = 1.0
    z[9, 0] = -0.0
    z[10:] = np.linspace(-1, 1, 40)
    u = np.array([0.5] * 10 + [0.0, 1.0, -1.0, nan])
    token, logprob, kept = _run_sample(z, u, t=[1, 1, 1, 1, 1, 1, 1, 1, 0, 0, 1, 1, 1, 1], exact=True)
    assert token[:2].tolist() == [-1, -1] and kept[:2].tolist() == [0, 0] and int(token[2]) == 7
    assert token[8:].tolist() == [11, 0, 0, 39, 0, 0]
    for t in (-1.0, nan, 0.0):
        assert _run_sample(z, u, t=t, exact=True)[0].tolist()[2:9] == [7, 6, 9, 0, 8, 39, 11]
    for t in (1e-40, 1e-20, 1e20, inf):
        _run_sample(z[:, :32], u, t=t, exact=True)
    _run_sample(z, u, p=[0.0, -1, nan, 1, 2, 0, -1, 1e-30, 1e-45, 0.5, nan, 0, 1, inf], exact=True)
    _run_sample(z, u, k=[0, -5, 1, 2, 1, 1 << 30, 40, 39, 1, 3, -1, 41, 40, 2], exact=True)
    _run_sample(z, u, mp=[0, -1, nan, 0.2, 1, 2, inf, 1e-30, 0.9, 1, 1, 0, -inf, 0.5], exact=True)


@gpu
def test_sample_reaches_every_token(cuda):
    """Numbers across [0, 1) give tokens in order of id, each as often as its weight says."""
    w = np.array([1, 3, 0, 2, 8, 1, 1])
    z = np.where(w > 0, np.log(np.maximum(w, 1)), -np.inf)
    u = (np.arange(16) + 0.5) / 16
    token, _, kept = _run_sample(np.tile(z, (16, 1)), u)
    assert token.tolist() == [i for i, n in enumerate(w) for _ in range(n)] and kept.tolist() == [6] * 16


@gpu
@pytest.mark.parametrize("kind,offset,width", [("fp32", 1, 1003), ("bf16", 1, 1001), ("bf16", 3, 1003), ("fp32", 0, 1000), ("bf16", 8, 1008)])
def test_sample_strides(cuda, kind, offset, width):
    rng = _rng(kind, offset)
    pool = _t(np.full(7 * width + offset, 50.0), kind)
    z = pool[offset:].view(7, width)[:, :997]
    z.copy_(_t(_logits(rng, 7, 997), kind))
    _run_sample(z, rng.random(7), kind, t=0.8, k=[0, 5, 100, 0, 1, 7, 900], p=0.9)
    one = z[:1].expand(7, 997)
    _run_sample(one, rng.random(7), kind, t=0.8, p=[0.5, 0.6, 0.7, 0.8, 0.9, 1, 1])


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 54, 1821, 13395])
def test_sample_number_zero_in_rows_off_boundaries(cuda, kind, vocab):
    """Rows that begin anywhere between boundaries of eight logits; the number 0 lies at a border, and half the tokens
    of some rows are not there."""
    rng = _rng(kind, vocab)
    z = _logits(rng, 24, vocab)
    z[8:16, 1::2] = -np.inf
    u = np.where(np.arange(24) % 3 < 2, 0.0, 0.7)
    _run_sample(z, u, kind)
    for k in (vocab // 2, (vocab + 1) // 2 + 2, vocab - 1):
        _run_sample(z, u, kind, t=3.0, k=max(k, 1))
        _run_sample(z, u, kind, t=3.0, k=max(k, 1), p=0.9999)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab,filters", [(300, {}), (131072, {}), (40, dict(k=39)), (40, dict(mp=1e-16)), (600, dict(k=599)), (5000, dict(k=4999)),
                                           (5000, dict(mp=1e-16)), (131072, dict(mp=1e-16))])
def test_sample_logprob_of_hardly_any_weight(cuda, kind, vocab, filters):
    """The number 0 draws the first token that has a weight, here one of a few units (2^-48 of the largest and more): its
    log probability is its logit's.  Bounds as in _run_sample; the weight's log2, up to 64, by three roundings of fp32."""
    rng = _rng(kind, vocab, str(filters))
    rows, t = 24, 0.7
    z = rng.uniform(-1.0, 0.0, (rows, vocab))
    z[:, 5] = 0.0
    z[:, 0] = -t * math.log(2.0) * rng.uniform(40.0, 48.5, rows)
    z[:, 1] = -80.0  # (no weight, and not among the first top_k)
    zt = _t(z, kind)
    f = lambda x: _t(np.full(rows, x))  # noqa: E731
    token, logprob, kept = B.sample_token(zt, f(0.0), temperature=f(t), top_k=_i([filters["k"]] * rows) if "k" in filters else None,
                                          min_p=f(filters["mp"]) if "mp" in filters else None)
    z, small = _np(zt), 0
    for i in range(rows):
        at = int(token[i])
        assert at in (0, 2)  # (a weight of less than half a unit is none)
        small += at == 0
        want = z[i] / np.float64(np.float32(t))
        want = want[at] - np.log(np.exp(want).sum())
        assert abs(float(logprob[i]) - want) <= 2.0 ** (-21 if filters else -19) * max(1.0, abs(want)), (i, at, float(logprob[i]), want)
    assert small > rows // 2


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 50, 5000, 131072])
def test_sample_logprob_of_all_the_weight(cuda, kind, vocab):
    """Rows of one token, or of one far above all others: no probability above 1."""
    rng = _rng(kind, vocab)
    z = np.full((96, vocab), -np.inf)
    z[1::2] = -200.0
    z[np.arange(96), rng.integers(0, vocab, 96)] = rng.uniform(-9, 9, 96)
    t, u = rng.uniform(0.3, 3.0, 96), 0.1 + 0.8 * rng.random(96)
    for filters in ({}, dict(k=30), dict(p=0.9), dict(mp=0.5)):
        _, logprob, _ = _run_sample(z, u, kind, t=t, **filters)
        assert bool((logprob <= 0).all())


@gpu
def test_sample_rows_past_32_bits(cuda):
    rng = _rng(9)
    wide = torch.empty(3, (1 << 31) + 64, dtype=torch.bfloat16, device="cuda")
    z = wide[:, :500]
    z.copy_(_t(_logits(rng, 3, 500), "bf16"))
    _run_sample(z, rng.random(3), "bf16", k=40)


@gpu
def test_sample_repeats(cuda):
    """The same bits every time, alone and in a larger batch."""
    rng = _rng(11)
    z, u = _t(_logits(rng, 64, 30011)), _t(rng.random(64))
    k, p = _i(rng.integers(0, 400, 64)), _t(rng.random(64))
    first = B.sample_token(z, u, top_k=k, top_p=p)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, B.sample_token(z, u, top_k=k, top_p=p)))
    for i in range(0, 64, 9):
        one = B.sample_token(z[i:i + 1], u[i:i + 1], top_k=k[i:i + 1], top_p=p[i:i + 1])
        assert all(torch.equal(a[i:i + 1], b) for a, b in zip(first, one))


@gpu
@pytest.mark.parametrize("rows,vocab", [(64, 30011), (400, 20000)])
def test_sample_repeats_without_limits(cuda, rows, vocab):
    """The same bits every time; alone, in other numbers of blocks, the same tokens and counts, and log probabilities within
    both sides' bounds."""
    rng = _rng(rows)
    z, u = _t(_logits(rng, rows, vocab)), _t(rng.random(rows))
    first = B.sample_token(z, u)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, B.sample_token(z, u)))
    for i in range(0, rows, rows // 8):
        token, logprob, kept = B.sample_token(z[i:i + 1], u[i:i + 1])
        assert int(token) == int(first[0][i]) and int(kept) == int(first[2][i])
        assert abs(float(logprob) - float(first[1][i])) <= 2.0 ** -18 * max(1.0, abs(float(logprob)))


# ----------------------------------------------------------------- together

@gpu
def test_binding_refuses_wrong_tensors(cuda):
    kc = torch.zeros(8, 16, 2, 64, device="cuda").to(F8)
    s = torch.ones(8, 2, device="cuda")
    s2 = torch.ones(8, 2, device="cuda")
    x = torch.zeros(3, 2, 64, device="cuda")
    table, one = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    u = torch.zeros(3, device="cuda")
    z = torch.zeros(3, 100, device="cuda")
    half = torch.zeros(3, 2, 64, device="cuda", dtype=torch.float16)
    for call, word in ((lambda: B.kv_append_fp8(x, x, kc.float(), kc, s, s2, table, one), "float8"),
                       (lambda: B.kv_append_fp8(x, x.bfloat16(), kc, kc, s, s2, table, one), "v must be"),
                       (lambda: B.kv_append_fp8(half, half, kc, kc, s, s2, table, one), "k must be"),
                       (lambda: B.kv_append_fp8(x, x, kc, kc, s, s2[:, :1], table, one), "v_scale"),
                       (lambda: B.kv_append_fp8(x, x, kc, kc, s.double(), s2, table, one), "k_scale"),
                       (lambda: B.kv_append_fp8(x, x, kc, kc, s, s2, table, one.long()), "before"),
                       (lambda: B.kv_append_fp8(x, x, kc, kc, s, s2, table, one, starts=one), "starts"),
                       (lambda: B.kv_append_fp8(x, x, kc, kc, s, s2, table, one, q_out=x), "q_out"),
                       (lambda: B.kv_append_fp8(x, x, kc, kc, s, s, table, one), "v_scale"),
                       (lambda: B.kv_append_fp8(x.requires_grad_(), x, kc, kc, s, s2, table, one), "gradient"),
                       (lambda: B.decode_attention_fp8(half, kc, kc, s, s, table, one), "q must be"),
                       (lambda: B.decode_attention_fp8(u[:, None, None].expand(3, 3, 64), kc, kc, s, s, table, one), "contiguous"),
                       (lambda: B.decode_attention_fp8(z.view(3, 1, 100), kc, kc, s, s, table, one), "shape"),
                       (lambda: B.sample_token(z[0], u), "rows"), (lambda: B.sample_token(z.half(), u), "logits"),
                       (lambda: B.sample_token(z, u[:2]), "uniform"), (lambda: B.sample_token(z, u, top_k=u), "top_k"),
                       (lambda: B.sample_token(z, u, temperature=one), "temperature"), (lambda: B.sample_token(z, u.cpu()), "uniform")):
        with pytest.raises(B.GptError) as e:
            call()
        assert e.value.name == "INVALID_ARG" and word in str(e.value), word


@gpu
def test_written_tensors_move_their_versions(cuda):
    kc, vc = (torch.zeros(8, 16, 2, 64, device="cuda").to(F8) for _ in range(2))
    ks, vs = torch.ones(8, 2, device="cuda"), torch.ones(8, 2, device="cuda")
    x = torch.zeros(3, 2, 64, device="cuda")
    table, one = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), _i([-1, -1, 0])
    before = [t._version for t in (kc, vc, ks, vs)]
    B.kv_append_fp8(x, x, kc, vc, ks, vs, table, one)
    assert [t._version for t in (kc, vc, ks, vs)] == [v + 1 for v in before]


@gpu
def test_empty_batches(cuda):
    kc = torch.zeros(8, 16, 2, 64, device="cuda").to(F8)
    s, s2 = torch.ones(8, 2, device="cuda"), torch.ones(8, 2, device="cuda")
    x = torch.zeros(0, 2, 64, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    table = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert B.kv_append_fp8(x, x, kc, kc, s, s2, table, none, q=x).shape == (0, 2, 64)
    assert B.decode_attention_fp8(x, kc, kc, s, s2, table, none)[0].shape == (0, 2, 64)
    assert [t.shape for t in B.sample_token(torch.zeros(0, 10, device="cuda"), torch.zeros(0, device="cuda"))] == [(0,)] * 3


class _Step:
    """Prompts, then decode steps of one layer over a cache in 8 bits: append, attention, penalties, a drawn token."""

    def __init__(self, seed, prompts, steps, page=8, heads=6, kv=2, dim=32, vocab=777):
        rng = np.random.default_rng(seed)
        w = lambda *s: (rng.standard_normal(s) / np.sqrt(s[-1])).astype(np.float32)  # noqa: E731
        self.heads, self.kv, self.dim, self.vocab, self.page, self.steps = heads, kv, dim, vocab, page, steps
        self.w = [_t(x) for x in (w(vocab, 64) * 8, w((heads + 2 * kv) * dim, 64), w(64, heads * dim), w(vocab, 64) * 8)]
        self.prompts = [rng.integers(0, vocab, n).tolist() for n in prompts]
        table, n_pages = _pages(rng, [n + steps for n in prompts], page)
        self.table = _i(table)
        self.cache = _pool8(rng, n_pages, page, kv, dim, "slot")
        width = max(prompts) + steps
        self.hist = _i([p + [0] * (width - len(p)) for p in self.prompts])
        self.hl, self.pl = _i(prompts), _i(prompts)
        n = len(prompts)
        self.u = _t(rng.random((steps, n)))
        self.at = torch.zeros(1, dtype=torch.long, device="cuda")
        self.rep = torch.full((n,), 1.3, device="cuda")
        self.t, self.k, self.p = _t(rng.uniform(0.5, 1.2, n)), _i(rng.integers(5, 100, n)), _t(rng.uniform(0.6, 1.0, n))
        ids = [t for p in self.prompts for t in p[:-1]] + [0, 0]  # two rows of padding
        _, k, v = self.split(_i(ids))
        starts = np.cumsum([0] + [n - 1 for n in prompts])
        B.kv_append_fp8(k, v, *self.cache, self.table, _i([0] * n), starts=_i(starts), rope_dims=dim)
        self.token = _i([p[-1] for p in self.prompts])

    def split(self, x):
        d = self.dim
        return [y.unflatten(1, (-1, d)) for y in (self.w[0][x.long()] @ self.w[1].t()).split([self.heads * d, self.kv * d, self.kv * d], dim=1)]

    def step(self):
        """On device state only (capturable)."""
        q, k, v = self.split(self.token)
        q = B.kv_append_fp8(k, v, *self.cache, self.table, self.hl - 1, q=q, rope_dims=self.dim)
        self.q = q
        self.o, _ = B.decode_attention_fp8(q, *self.cache, self.table, self.hl)
        x = self.w[0][self.token.long()] + self.o.flatten(1) @ self.w[2].t()
        _, self.z, _ = B.next_token(x @ self.w[3].t(), history=self.hist, history_lens=self.hl, prompt_lens=self.pl, repetition=self.rep)
        self.uniform = self.u.index_select(0, self.at).squeeze(0)
        token, self.logprob, self.kept = B.sample_token(self.z, self.uniform, temperature=self.t, top_k=self.k, top_p=self.p)
        self.hist.scatter_(1, self.hl[:, None].long(), token[:, None])
        self.token.copy_(token)
        self.at += 1
        self.hl += 1

    def check(self):
        """The last step: attention over what the cache stands for, and the draw."""
        n = (self.hl - 1).tolist()
        table = self.table.cpu().numpy()
        kc, vc, ks, vs = self.cache
        k, v = (_number(_codes(c)) * _np(s)[:, None, :, None] for c, s in ((kc, ks), (vc, vs)))
        parts = [[x[table[s, np.arange(m) // self.page], np.arange(m) % self.page] for x in (k, v)] for s, m in enumerate(n)]
        for s, (keys, values) in enumerate(parts):
            want, _, tol, _ = _attention8(_np(self.q)[s], keys, values, self.dim ** -0.5, "fp32")
            _check(self.o[s], want, tol)
            token, lp, kept, near = _draw(_np(self.z)[s], float(self.uniform[s]), float(self.t[s]), int(self.k[s]), float(self.p[s]))
            assert near < 2.0 ** -33 or (int(self.token[s]), int(self.kept[s])) == (token, kept)


PROMPTS = [5, 1, 17, 8, 9]


@gpu
def test_decode_loop(cuda):
    m = _Step(1, PROMPTS, 12)
    for _ in range(12):
        m.step()
        m.check()


@gpu
def test_decode_loop_captured(cuda):
    """Two models' steps captured into two graphs on side streams and replayed in turns give what eager loops give."""
    eager = [_Step(s, PROMPTS, 10) for s in (2, 3)]
    for m in eager:
        for _ in range(10):
            m.step()
    models, graphs = [_Step(s, PROMPTS, 10) for s in (2, 3)], []
    for m in models:
        m.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.step()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in models]
    torch.cuda.synchronize()
    for _ in range(9):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for m, e in zip(models, eager):
        assert torch.equal(m.hist, e.hist) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(m.cache, e.cache))
        m.check()


@gpu
def test_given_streams_and_threads(cuda):
    """Calls on streams of their own, from threads at once, give what calls one after another give."""
    import threading
    rng = _rng(21)
    lens, page = [2000, 300, 7], 16
    table, n_pages = _pages(rng, lens, page, width=4000)  # a table so wide that there is a workspace
    cache = _pool8(rng, n_pages, page, 2, 64, "slot")
    _fill8(rng, lens, table, page, cache)
    q, z, u = (_t(rng.standard_normal(s)) for s in ((3, 4, 64), (3, 5000), (3,)))
    x = _t(rng.standard_normal((3, 2, 64)))
    t, n, low = _i(table), _i(lens), _i([3, 4, 5])
    u = u.abs().clamp(max=0.99)

    def call(stream=None):
        own = [c.clone() for c in cache]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        B.kv_append_fp8(x, x, *own, t, low, rope_dims=64, stream=stream)
        out = B.decode_attention_fp8(q, *own, t, n, stream=stream), B.sample_token(z, u, top_p=u, stream=stream)
        (stream or torch.cuda.current_stream()).synchronize()
        return [y.clone() for o in out for y in o]

    want = call()
    got = [None] * 6

    def work(i):
        torch.cuda.set_device(0)
        got[i] = call(torch.cuda.Stream())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))


FIRST_CALLS = """
import torch
from persistent_gpt_step_gb300 import binding as B
i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
kc, vc = (torch.zeros(40, 16, 2, 64, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
ks, vs = torch.zeros(40, 2, device="cuda"), torch.zeros(40, 2, device="cuda")
q, z = torch.randn(2, 4, 64, device="cuda"), torch.randn(2, 300, device="cuda")
k = torch.full((2, 2, 64), 3.5, device="cuda")
u = torch.zeros(2, device="cuda")
table, pos, lens = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20), i(0, 0), i(1, 1)
far = torch.zeros(2, 9000, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    B.kv_append_fp8(k, k, kc, vc, ks, vs, table, pos)
    near = B.decode_attention_fp8(q, kc, vc, ks, vs, table, lens)[0]
    wide = B.decode_attention_fp8(q, kc, vc, ks, vs, far, lens)[0]
    token = B.sample_token(z, u, temperature=u)[0]
g.replay()
torch.cuda.synchronize()
want = k.repeat_interleave(2, 1)
for got in (near, wide[:1]):  # one key: its weight in two fp16 parts (2^-22) over itself, and three roundings
    assert bool(((got - want[:len(got)]).abs() <= want[:len(got)] * (2.0 ** -22 + 3 * 2.0 ** -24)).all())
assert torch.equal(token, z.argmax(1).int())
"""


@gpu
def test_first_calls_of_a_process_are_captured(cuda):
    """No call has to run eagerly before it can be captured."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
