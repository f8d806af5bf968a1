"""The operators of a batched decode step (gpt_kv_append, gpt_decode_attention, gpt_next_token).

Refusals are checked through the C ABI and the binding without a GPU; on a GPU each operator is compared
with its definition in float64 (numpy).  Tolerances are worst-case bounds of the arithmetic: u = 2^-24 per
fp32 operation, half a step of bf16 (2^-8 of the value) for the one rounding of a bf16 result."""

import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest

from persistent_gpt_step_gb300 import binding as B
from persistent_gpt_step_gb300 import build as build_mod

torch = pytest.importorskip("torch")

gpu = pytest.mark.gpu
U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


@pytest.fixture
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.backends.cuda.matmul.allow_tf32 = False


# ----------------------------------------------------------------- refusals (no GPU needed)

FAKE = 0x10000  # never dereferenced: every call below is refused before a launch


def _cache(**kw):
    c = B.gpt_paged_cache(k=FAKE, v=FAKE, page_table=FAKE, page_stride=16 * 4 * 64, slot_stride=4 * 64, head_stride=64,
                          table_stride=8, n_pages=32, page_size=16, n_seq=3, max_pages=8, n_kv_head=4, head_dim=64,
                          dtype=B.DTYPE_BF16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _append(**kw):
    a = B.gpt_kv_append_args(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, q_row=512, q_head=64, k_row=256, k_head=64, v_row=256,
                             v_head=64, qo_row=512, qo_head=64, positions=FAKE, rope_base=10000.0, n_tokens=3, n_head=8,
                             rope_dims=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _attend(**kw):
    a = B.gpt_decode_attention_args(q=FAKE, out=FAKE + 4096, lens=FAKE, q_row=512, q_head=64, out_row=512, out_head=64,
                                    workspace=FAKE, workspace_bytes=1 << 40, scale=0.125, n_head=8)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _token(**kw):
    a = B.gpt_next_token_args(logits=FAKE, out=FAKE, token=FAKE, lse=FAKE, logits_stride=100, out_stride=100, rows=2,
                              vocab=100, dtype=B.DTYPE_FP32)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_CACHES = [(dict(dtype=5), -1, "dtype"), (dict(n_pages=0), -1, "sizes"), (dict(page_size=0), -1, "sizes"),
              (dict(n_seq=-1), -1, "sizes"), (dict(max_pages=0), -1, "sizes"), (dict(n_kv_head=0), -1, "sizes"),
              (dict(head_dim=136), -8, "head_dim"), (dict(head_dim=60), -8, "head_dim"), (dict(k=None), -1, "NULL"),
              (dict(page_table=None), -1, "NULL"), (dict(v=FAKE + 8), -1, "16 bytes"),
              (dict(slot_stride=252), -1, "16 bytes"), (dict(head_stride=-64), -1, "16 bytes"),
              (dict(table_stride=7), -1, "table_stride"), (dict(max_pages=1 << 28, table_stride=1 << 28), -8, "32 bits")]


@pytest.mark.parametrize("change,code,word", BAD_CACHES)
def test_bad_caches_are_refused(lib, change, code, word):
    c = _cache(**change)
    for fn, a in ((lib.gpt_kv_append, _append()), (lib.gpt_decode_attention, _attend())):
        assert fn(ctypes.byref(c), ctypes.byref(a), None) == code
        assert word in lib.gpt_last_error(None).decode()
    assert lib.gpt_decode_attention_workspace(ctypes.byref(c), 8) == 0


@pytest.mark.parametrize("change,word", [
    (dict(n_tokens=-1), "negative"), (dict(n_head=-1), "negative"), (dict(rope_dims=63), "rope_dims"),
    (dict(rope_dims=66), "rope_dims"), (dict(rope_dims=-2), "rope_dims"), (dict(rope_base=0.5), "rope_base"),
    (dict(rope_base=math.inf), "rope_base"), (dict(rope_base=math.nan), "rope_base"), (dict(k=None), "NULL"),
    (dict(positions=None), "NULL"), (dict(n_tokens=4), "sequences"), (dict(k_row=250), "16 bytes"),
    (dict(v=FAKE + 2), "16 bytes"), (dict(q=None), "n_head"), (dict(q_out=None), "n_head"), (dict(n_head=0), "n_head"),
    (dict(qo_head=60), "16 bytes"), (dict(q_row=-512), "16 bytes"), (dict(qo_row=0), "smaller"), (dict(qo_head=56), "smaller")])
def test_append_refusals(lib, change, word):
    assert lib.gpt_kv_append(ctypes.byref(_cache()), ctypes.byref(_append(**change)), None) == -1
    assert word in lib.gpt_last_error(None).decode()
    assert lib.gpt_kv_append(None, ctypes.byref(_append()), None) == -1
    assert lib.gpt_kv_append(ctypes.byref(_cache()), None, None) == -1
    assert lib.gpt_kv_append(ctypes.byref(_cache(n_seq=0)), ctypes.byref(_append(seq=FAKE)), None) == -1


@pytest.mark.parametrize("change,word", [
    (dict(n_head=6), "multiple"), (dict(n_head=0), "multiple"), (dict(q=None), "NULL"), (dict(out=None), "NULL"),
    (dict(lens=None), "NULL"), (dict(q=FAKE + 4), "16 bytes"), (dict(out_row=508), "16 bytes"), (dict(out_row=0), "smaller"),
    (dict(out_head=0), "smaller"), (dict(scale=3e38), "scale"),
    (dict(scale=math.nan), "scale"), (dict(scale=math.inf), "scale"), (dict(out=FAKE), "q"), (dict(workspace=None), "workspace"),
    (dict(workspace=FAKE + 8), "workspace"), (dict(workspace_bytes=64), "workspace")])
def test_attention_refusals(lib, change, word):
    if word == "workspace":  # a table that reaches far enough for one to be needed
        c = _cache(max_pages=10000, table_stride=10000)
        assert lib.gpt_decode_attention_workspace(ctypes.byref(c), 8) > 64
        assert lib.gpt_decode_attention(ctypes.byref(c), ctypes.byref(_attend(**change)), None) == -1
        assert word in lib.gpt_last_error(None).decode()
        return
    assert lib.gpt_decode_attention(ctypes.byref(_cache()), ctypes.byref(_attend(**change)), None) == -1
    assert word in lib.gpt_last_error(None).decode()
    assert lib.gpt_decode_attention(None, ctypes.byref(_attend()), None) == -1
    assert lib.gpt_decode_attention(ctypes.byref(_cache()), None, None) == -1


@pytest.mark.parametrize("change,word", [
    (dict(dtype=7), "dtype"), (dict(rows=-1), "negative"), (dict(vocab=0), "vocab"), (dict(max_history=-1), "negative"),
    (dict(out=None, token=None, lse=None), "NULL"), (dict(logits=None), "NULL"), (dict(logits_stride=99), "stride"),
    (dict(out_stride=99), "stride"), (dict(history=FAKE, max_history=9, history_stride=8), "stride"),
    (dict(allowed=FAKE, allowed_stride=3), "stride"), (dict(history_lens=FAKE), "history"),
    (dict(prompt_lens=FAKE), "history"), (dict(bias_ids=FAKE), "together"), (dict(bias_values=FAKE), "together"),
    (dict(out=FAKE, dtype=1), "in place"), (dict(out=FAKE, out_stride=104), "in place"),
    (dict(logits=FAKE + 2), "boundaries"), (dict(logits=FAKE + 1, dtype=1), "boundaries"), (dict(out=FAKE + 4098), "boundaries")])
def test_next_token_refusals(lib, change, word):
    change = {"out": FAKE + 4096, **change}
    assert lib.gpt_next_token(ctypes.byref(_token(**change)), None) == -1
    assert word in lib.gpt_last_error(None).decode()
    assert lib.gpt_next_token(None, None) == -1


@pytest.mark.parametrize("change", [dict(page_stride=0), dict(slot_stride=56), dict(head_stride=0)])
def test_append_into_overlapping_slots_is_refused(lib, change):
    assert lib.gpt_kv_append(ctypes.byref(_cache(**change)), ctypes.byref(_append()), None) == -1
    assert "smaller" in lib.gpt_last_error(None).decode()


def test_head_counts_beyond_32_bits_of_work_are_refused(lib):
    heads = 1 << 17
    assert lib.gpt_kv_append(ctypes.byref(_cache()), ctypes.byref(_append(n_head=heads)), None) == -8
    assert lib.gpt_decode_attention(ctypes.byref(_cache()), ctypes.byref(_attend(n_head=heads)), None) == -8
    for fn, a in ((lib.gpt_kv_append, _append()), (lib.gpt_decode_attention, _attend(n_head=heads))):
        assert fn(ctypes.byref(_cache(n_kv_head=heads)), ctypes.byref(a), None) == -8


def test_nothing_to_do_is_no_error(lib):
    c = ctypes.byref(_cache())
    assert lib.gpt_kv_append(c, ctypes.byref(_append(n_tokens=0)), None) == 0
    assert lib.gpt_decode_attention(ctypes.byref(_cache(n_seq=0)), ctypes.byref(_attend()), None) == 0
    assert lib.gpt_next_token(ctypes.byref(_token(rows=0, out=FAKE + 4096)), None) == 0


def test_calls_without_a_gpu_fail_cleanly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    c = ctypes.byref(_cache())
    for rc in (lib.gpt_kv_append(c, ctypes.byref(_append()), None), lib.gpt_decode_attention(c, ctypes.byref(_attend()), None),
               lib.gpt_next_token(ctypes.byref(_token(out=FAKE + 4096)), None)):
        assert rc == -2 and lib.gpt_last_error(None)


def test_structs_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(B.HERE), "include", "gpt.h")).read()
    for name, cls in (("gpt_paged_cache", B.gpt_paged_cache), ("gpt_kv_append_args", B.gpt_kv_append_args),
                      ("gpt_decode_attention_args", B.gpt_decode_attention_args),
                      ("gpt_next_token_args", B.gpt_next_token_args)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = []
        for decl in filter(None, (d.strip() for d in body.split(";"))):
            m = re.match(r"((?:const\s+)?\w+)\s*(.*)", decl, re.S)
            fields += [(m.group(1).split()[-1], f.strip()) for f in m.group(2).split(",")]
        size = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t, "float": ctypes.c_float,
                "double": ctypes.c_double}
        want = [(f.lstrip("* "), ctypes.c_void_p if f.startswith("*") else size[t]) for t, f in fields]
        assert want == list(cls._fields_), name


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(2, 4, 64)
    cache = torch.zeros(8, 16, 4, 64)
    table = torch.zeros(2, 4, dtype=torch.int32)
    one = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: B.kv_append(x, x, cache, cache, table, one), lambda: B.decode_attention(x, cache, cache, table, one),
                 lambda: B.next_token(torch.zeros(2, 100))):
        with pytest.raises(B.GptError) as e:
            call()
        assert e.value.name == "INVALID_ARG" and "CUDA" in str(e.value)


# ----------------------------------------------------------------- inputs and definitions

def _rng(*key):
    return np.random.default_rng([_key(k) for k in key])


def _key(k):
    return k if isinstance(k, int) else sum(ord(c) * 31 ** i for i, c in enumerate(str(k))) % (1 << 31)


def _t(x, kind="fp32"):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(DT[kind])


def _i(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _pages(rng, lens, page, spare=3, width=None):
    """A table whose sequences' pages come from a shuffled pool; unused entries name pages outside it."""
    used = [-(-n // page) for n in lens]
    n_pages = sum(used) + spare
    ids = rng.permutation(n_pages)
    table = np.full((len(lens), max(width or 0, max(used + [1]))), n_pages + 7, dtype=np.int32)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = ids[at:at + n]
        at += n
    return table, n_pages


def _pool(n_pages, page, heads, dim, kind, order, fill):
    """An empty cache pair [pages, page, heads, dim] over memory in the given order of dimensions."""
    shape = {"slot": (n_pages, page, heads, dim), "head": (n_pages, heads, page, dim), "gaps": (n_pages, page + 1, heads + 1, dim + 16)}
    pools = [torch.full(shape[order], fill, dtype=DT[kind], device="cuda") for _ in range(2)]
    if order == "head":
        return [x.transpose(1, 2) for x in pools]
    if order == "gaps":
        return [x[:, :page, :heads, :dim] for x in pools]
    return pools


def _turned(x, pos, rope, base):
    """float64 rotation of [tokens, heads, dim]."""
    y = np.array(x, dtype=np.float64)
    for i in range(rope // 2):
        t = pos.astype(np.float64) * float(base) ** (-2.0 * i / rope)
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        a, b = x[..., 2 * i], x[..., 2 * i + 1]
        y[..., 2 * i], y[..., 2 * i + 1] = a * c - b * s, a * s + b * c
    return y


def _turn_tolerance(x, want, rope, kind, turn):
    """Angle off by `turn` turns, sine and cosine by two steps (2^-22), three roundings; then one rounding to bf16."""
    r = np.array(np.abs(x), dtype=np.float64)
    for i in range(rope // 2):
        r[..., 2 * i] = r[..., 2 * i + 1] = np.hypot(x[..., 2 * i], x[..., 2 * i + 1])
    tol = r * (2 * math.pi * turn + 2 * 2.0 ** -22 + 3 * U)
    tol[..., rope:] = 0
    return tol + (np.abs(want) + tol) * (2.0 ** -8 if kind == "bf16" else 0) * (np.arange(x.shape[-1]) < rope)


def _check(got, want, tol):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    off = np.abs(got - want) - tol
    assert not np.isnan(got).any()
    assert (off <= 0).all(), (float(off.max()), np.unravel_index(int(off.argmax()), off.shape))


# ----------------------------------------------------------------- kv_append

APPENDS = [  # tokens, heads, kv heads, dim, rope, page, order of the cache
    (1, 8, 8, 64, 64, 16, "slot"), (1, 1, 1, 8, 2, 1, "slot"), (37, 12, 4, 64, 32, 24, "head"),
    (130, 4, 4, 128, 128, 16, "gaps"), (65, 14, 2, 96, 24, 7, "slot"), (9, 0, 3, 80, 80, 64, "head"),
    (33, 32, 1, 128, 0, 16, "slot"), (515, 6, 6, 16, 10, 33, "head"),
    # more tokens than blocks run at once: of many heads one, of few heads two to eight in a block
    (611, 12, 12, 64, 64, 16, "slot"), (1301, 8, 4, 64, 48, 16, "gaps"), (2437, 4, 1, 80, 80, 24, "slot"),
    (4869, 2, 1, 96, 6, 7, "head"), (4871, 0, 1, 8, 8, 16, "slot")]


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n,heads,kv,dim,rope,page,order", APPENDS)
def test_append(cuda, kind, n, heads, kv, dim, rope, page, order):
    """Ragged sequences with padding tokens: the written slots hold the definition's values, every other
    element of the cache and of the padded query rows is what it was."""
    rng = _rng(n, heads, kv, dim, kind)
    n_seq = min(n, 5)
    seq = np.sort(rng.integers(0, n_seq, n))
    pos = np.zeros(n, dtype=np.int64)
    lens = []
    for s in range(n_seq):
        first = int(rng.integers(0, 40))
        rows = np.nonzero(seq == s)[0]
        pos[rows] = first + np.arange(len(rows))
        lens.append(first + len(rows))
    table, n_pages = _pages(rng, lens, page)
    pad = rng.random(n) < 0.2 if n > 1 else np.zeros(1, dtype=bool)
    order_of_tokens = rng.permutation(n)
    seq, pos, pad = seq[order_of_tokens], pos[order_of_tokens], pad[order_of_tokens]
    kc, vc = _pool(n_pages, page, kv, dim, kind, order, 77.0)
    qkv = _t(rng.standard_normal((n, (heads + 2 * kv) * dim)), kind)
    q, k, v = (x.unflatten(1, (-1, dim)) if x.shape[1] else None for x in qkv.split([heads * dim, kv * dim, kv * dim], dim=1))
    qo = torch.full((n, heads + 1, dim), 5.0, dtype=DT[kind], device="cuda")[:, :heads] if heads else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = B.kv_append(k, v, kc, vc, _i(table), _i(pos), seq=_i(np.where(pad, -1 - seq, seq)), q=q, rope_dims=rope, rope_base=10000.0,
                      q_out=qo, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    want_k = np.full((n_pages, page, kv, dim), 77.0)
    want_v, tol_k = want_k.copy(), np.zeros_like(want_k)
    tk = _turned(_np(k), pos, rope, 10000.0)
    ok = _turn_tolerance(_np(k), tk, rope, kind, 2.0 ** -24)
    for i in np.nonzero(~pad)[0]:
        at = table[seq[i], pos[i] // page], pos[i] % page
        want_k[at], want_v[at], tol_k[at] = tk[i], _np(v)[i], ok[i]
    _check(kc, want_k, tol_k)
    _check(vc, want_v, 0)
    if heads:
        assert got is qo
        want = _turned(_np(q), pos, rope, 10000.0)
        tol = _turn_tolerance(_np(q), want, rope, kind, 2.0 ** -24)
        want[pad], tol[pad] = 5.0, 0
        _check(got, want, tol)
    else:
        assert got is None


@gpu
@pytest.mark.parametrize("pos,turn", [(131071, 2.0 ** -24), ((1 << 24) - 1, 2.0 ** -24), ((1 << 24) + 5, 2.0 ** -20), ((1 << 31) - 129, 2.0 ** -20)])
def test_append_far_positions(cuda, pos, turn):
    """Angles stay exact at far positions (an fp32 angle would be off by radians)."""
    page, dim = 1 << 14, 64
    rng = _rng(pos % 1000)
    max_pages = (1 << 31) // page - 1
    if pos // page >= max_pages:
        pos = max_pages * page - 1
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    table[0, pos // page] = 1
    kc, vc = _pool(2, page, 1, dim, "fp32", "slot", 0.0)
    k, q = _t(rng.standard_normal((1, 1, dim))), _t(rng.standard_normal((1, 2, dim)))
    got = B.kv_append(k, k, kc, vc, table, _i([pos]), q=q, rope_dims=dim, rope_base=500000.0)
    p = np.array([pos])
    for x, y in ((q, _np(got)), (k, _np(kc[1, pos % page])[None])):
        want = _turned(_np(x), p, dim, 500000.0)
        _check(y, want, _turn_tolerance(_np(x), want, dim, "fp32", turn))


@gpu
@pytest.mark.parametrize("pos,turn", [((1 << 24) - 1, 2.0 ** -23), ((1 << 31) - 4200, 2.0 ** -18)])
@pytest.mark.parametrize("base", [1.0, 1.0003, 4.0])
def test_append_slow_rates_at_far_positions(cuda, base, pos, turn):
    """Rates that hardly fall off leave every pair with millions of turns: the bounds of the header hold for all of them."""
    page, dim = 1 << 14, 128
    rng = _rng(int(base * 1000), pos % 1000)
    table = torch.full((1, (1 << 31) // page - 1), -1, dtype=torch.int32, device="cuda")
    pos = min(pos, table.shape[1] * page - 1)
    table[0, pos // page] = 0
    kc, vc = _pool(1, page, 1, dim, "fp32", "slot", 0.0)
    k = _t(rng.standard_normal((1, 1, dim)))
    B.kv_append(k, k, kc, vc, table, _i([pos]), rope_dims=dim, rope_base=base)
    want = _turned(_np(k), np.array([pos]), dim, base)
    _check(_np(kc[0, pos % page])[None], want, _turn_tolerance(_np(k), want, dim, "fp32", turn))


@gpu
def test_append_in_place_queries_and_no_seq(cuda):
    rng = _rng(5)
    n, dim = 6, 64
    q, k, v = (_t(rng.standard_normal((n, 4, dim)), "bf16") for _ in range(3))
    table, n_pages = _pages(rng, [20] * n, 16)
    pos = rng.integers(0, 20, n)
    kc, vc = _pool(n_pages, 16, 4, dim, "bf16", "slot", 0.0)
    want = _turned(_np(q), pos, 64, 10000.0)
    tol = _turn_tolerance(_np(q), want, 64, "bf16", 2.0 ** -24)
    assert B.kv_append(k, v, kc, vc, _i(table), _i(pos), q=q, rope_dims=64, q_out=q) is q
    _check(q, want, tol)
    for i in range(n):
        assert torch.equal(vc[int(table[i, pos[i] // 16]), int(pos[i] % 16)], v[i])


@gpu
@pytest.mark.parametrize("what,bit", [("seq", 1), ("low", 2), ("high", 2), ("page", 4), ("page_low", 4)])
def test_append_bad_indices_are_skipped_and_reported(cuda, what, bit):
    """A bad token changes nothing and leaves the others' writes alone (the checks are also shown by the
    kernel's index arithmetic: page and slot are only used when all of them hold)."""
    rng = _rng(what)
    n, dim, page = 4, 32, 8
    table, n_pages = _pages(rng, [16] * n, page)
    seq, pos = np.arange(n), np.array([3, 9, 0, 15])
    if what == "seq":
        seq[1] = n
    elif what == "low":
        pos[1] = -1
    elif what == "high":
        pos[1] = 16
    else:
        table[1, 1] = n_pages if what == "page" else -1
    kc, vc = _pool(n_pages, page, 2, dim, "fp32", "slot", 9.0)
    q, k, v = (_t(rng.standard_normal((n, 2, dim))) for _ in range(3))
    qo = torch.full_like(q, 4.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.kv_append(k, v, kc, vc, _i(table), _i(pos), seq=_i(seq), q=q, rope_dims=0, q_out=qo, status=status)
    assert int(status) == bit
    want = torch.full_like(vc, 9.0)
    for i in (0, 2, 3):
        want[int(table[i, pos[i] // page]), int(pos[i] % page)] = v[i]
    assert torch.equal(vc, want)
    assert bool((qo[1] == 4.0).all()) and torch.equal(qo[[0, 2, 3]], q[[0, 2, 3]])
    B.kv_append(k, v, kc, vc, _i(table), _i(pos), seq=_i(seq))  # without a status word
    assert torch.equal(vc, want)


@gpu
def test_append_bad_tokens_beside_others_in_a_block(cuda):
    """Every way to be bad or padding, next to good tokens: those are written, nothing else is."""
    rng = _rng(16)
    n, dim, page = 5001, 32, 8
    lens = np.full(10, 600)
    table, n_pages = _pages(rng, lens, page)
    seq, pos = np.arange(n) % 10, np.arange(n) // 10
    kinds = rng.integers(0, 8, n)
    bad_seq, bad_pos = seq.copy(), pos.copy()
    bad_seq[kinds == 0], bad_seq[kinds == 1] = -5, 10
    bad_pos[kinds == 2], bad_pos[kinds == 3] = -1, 10 ** 9
    table[3, 7] = n_pages
    good = (kinds > 3) & ~((seq == 3) & (pos // page == 7))
    kc, vc = _pool(n_pages, page, 1, dim, "bf16", "slot", 9.0)
    q, k, v = (_t(rng.standard_normal((n, 1, dim)), "bf16") for _ in range(3))
    qo = torch.full_like(q, 4.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.kv_append(k, v, kc, vc, _i(table), _i(bad_pos), seq=_i(bad_seq), q=q, rope_dims=0, q_out=qo, status=status)
    assert int(status) == 7
    for pool, x in ((kc, k), (vc, v)):
        want = torch.full_like(pool, 9.0)
        want[_i(table[seq[good], pos[good] // page]).long(), _i(pos[good] % page).long()] = x[torch.from_numpy(good).cuda()]
        assert torch.equal(pool, want)
    want = torch.where(torch.from_numpy(good).cuda()[:, None, None], q, torch.full_like(q, 4.0))
    assert torch.equal(qo, want)


# ----------------------------------------------------------------- decode_attention

def _fill(rng, lens, table, kc, vc, page):
    """Normal keys and values at the sequences' positions only; returns them per sequence in float64."""
    out = []
    heads, dim = kc.shape[2:]
    for s, n in enumerate(lens):
        at = np.arange(n)
        where = (torch.from_numpy(table[s, at // page].astype(np.int64)).cuda(), torch.from_numpy(at % page).cuda())
        kv = [_t(rng.standard_normal((n, heads, dim))).to(kc.dtype) for _ in range(2)]
        kc[where], vc[where] = kv
        out.append([_np(x) for x in kv])
    return out


def _attention(q, keys, values, scale):
    """Definition and bounds for one sequence: (out, lse, bound of out without its last rounding, of lse)."""
    heads, dim = q.shape
    n, kv = keys.shape[:2]
    g = heads // kv
    if n == 0:
        return np.zeros((heads, dim)), np.full(heads, -np.inf), np.zeros((heads, dim)), np.zeros(heads)
    K, V = np.repeat(keys, g, axis=1), np.repeat(values, g, axis=1)
    z = np.einsum("hd,nhd->hn", q, K) * scale
    a = np.einsum("hd,nhd->hn", np.abs(q), np.abs(K)) * abs(scale)
    m = z.max(axis=1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(axis=1, keepdims=True)
    w = p / l
    out = np.einsum("hn,nhd->hd", w, V)
    spread = np.einsum("hn,nhd->hd", w, np.abs(V))
    # a score: dim products and sums, the scale and its change of base; a weight: that, and 2^-20 of itself for the
    # exponentials (its own and the rescalings) and for the two parts it may be multiplied in (2^-16 each)
    dz = (dim + 4) * U * a.max(axis=1) + 2.0 ** -20 + 3 * U * np.abs(z - m).max(axis=1)
    dw = dz + 2.0 ** -16
    return out, (m + np.log(l))[:, 0], spread * (2 * dw + (n + 8) * U)[:, None], dz + (n + 8) * U + 4 * U * np.abs(m[:, 0])


def _run_attention(rng, lens, heads, kv, dim, page, kind, order="slot", scale=None, fill=math.nan, strided=False, reach=0):
    """``reach``: positions that the table has room for, if more than the lengths need; the kernel is chosen by it."""
    table, n_pages = _pages(rng, lens, page, width=-(-reach // page))
    kc, vc = _pool(n_pages, page, kv, dim, kind, order, fill)
    parts = _fill(rng, lens, table, kc, vc, page)
    q = _t(rng.standard_normal((len(lens), heads, dim)), kind)
    out = None
    if strided:
        wide = torch.full((len(lens), heads + 2, dim + 16), 3.0, dtype=DT[kind], device="cuda")
        out = wide[:, :heads, :dim]
        q = torch.cat([q, q.new_zeros(len(lens), 1, dim)], dim=1)[:, :heads]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = B.decode_attention(q, kc, vc, _i(table), _i(lens), scale=scale, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for s, (k, v) in enumerate(parts):
        want, wl, tol, tl = _attention(_np(q)[s], k, v, dim ** -0.5 if scale is None else scale)
        if kind == "bf16":
            tol = tol + (np.abs(want) + tol) * 2.0 ** -8
        _check(got[s], want, tol)
        if len(k):
            _check(lse[s], wl, tl)
        else:
            assert bool((lse[s] == -math.inf).all())
    if strided:
        assert bool((wide[:, heads:] == 3.0).all()) and bool((wide[..., dim:] == 3.0).all())
    return got, lse


ATTENDS = [  # lengths, heads, kv heads, dim, page, order
    ([1], 8, 8, 64, 16, "slot"), ([0], 4, 4, 64, 16, "slot"), ([513], 12, 12, 64, 16, "slot"),
    ([0, 1, 15, 16, 17, 300, 0], 16, 16, 64, 16, "head"), ([257, 1, 64, 1000], 32, 8, 128, 16, "slot"),
    ([129, 700], 7, 1, 80, 24, "gaps"), ([33, 200, 128], 12, 4, 96, 7, "head"), ([5, 2000], 64, 2, 32, 64, "slot"),
    ([31, 32, 33], 3, 3, 8, 1, "slot"), ([400], 17, 1, 64, 128, "slot"), ([63, 65], 24, 2, 112, 40, "gaps"),
    ([4097], 8, 8, 64, 32, "head"), ([3001, 2], 16, 1, 128, 16, "head")]


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,heads,kv,dim,page,order", ATTENDS)
def test_attention(cuda, kind, lens, heads, kv, dim, page, order, reach):
    """Everything that no sequence's length covers is NaN, and table entries past it name no page."""
    _run_attention(_rng(kind, dim, len(lens), heads), lens, heads, kv, dim, page, kind, order, reach=reach)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("offset,gap", [(1, 0), (0, 1), (1, 1), (2, 2)])
def test_attention_cache_on_16_byte_boundaries(cuda, kind, offset, gap):
    """Bases and strides that are odd multiples of 16 bytes."""
    rng = _rng(kind, offset, gap)
    e, page, heads, dim = 16 // (2 if kind == "bf16" else 4), 16, 2, 64
    lens = [100, 33]
    table, n_pages = _pages(rng, lens, page)
    row = dim + gap * e
    pools = [torch.full((offset * e + n_pages * page * heads * row,), math.nan, dtype=DT[kind], device="cuda") for _ in range(2)]
    kc, vc = (x[offset * e:].view(n_pages, page, heads, row)[..., :dim] for x in pools)
    parts = _fill(rng, lens, table, kc, vc, page)
    q = _t(rng.standard_normal((2, 4, dim)), kind)
    out, lse = B.decode_attention(q, kc, vc, _i(table), _i(lens))
    for s, (k, v) in enumerate(parts):
        want, wl, tol, tl = _attention(_np(q)[s], k, v, dim ** -0.5)
        _check(out[s], want, tol + ((np.abs(want) + tol) * 2.0 ** -8 if kind == "bf16" else 0))
        _check(lse[s], wl, tl)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_attention_strided_and_scaled(cuda, kind):
    _run_attention(_rng(kind), [70, 0, 9], 6, 2, 64, 16, kind, "gaps", scale=0.3, strided=True)
    _run_attention(_rng(kind), [70, 3], 6, 2, 64, 16, kind, scale=0.0)
    for reach in (0, 400000):
        _run_attention(_rng(kind), [70, 3], 6, 2, 64, 16, kind, scale=-0.7, fill=math.inf, reach=reach)


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("page", [16, 8, 5])
def test_attention_every_length_near_a_split(cuda, kind, page, reach):
    """Lengths around every power of two and tile: one launch, a sequence each."""
    lens = sorted({max(0, (1 << e) + d) for e in range(0, 12) for d in (-1, 0, 1)})
    _run_attention(_rng(kind, 3), lens, 4, 2, 64, page, kind, reach=reach)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n_seq", [19, 37, 43, 50, 60, 76, 101, 152, 153, 304, 305, 609, 913, 2433])
def test_attention_rows_per_block(cuda, kind, n_seq):
    """Rows from a few to many: every number of blocks to a row and of rows to a block, whole waves and one row more."""
    rng = _rng(kind, n_seq)
    lens = rng.integers(0, 300 if n_seq > 300 else 1200, n_seq).tolist()
    _run_attention(rng, lens, 2, 1, 64, 16, kind)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n_seq,kv", [(700, 1), (300, 4), (2000, 2)])
def test_attention_many_sequences(cuda, kind, n_seq, kv):
    """More sequences than are looked at at a time, most of them short or empty, a few long."""
    rng = _rng(kind, n_seq)
    lens = np.where(rng.random(n_seq) < 0.3, 0, (rng.random(n_seq) ** 6 * 900).astype(np.int64) + 1)
    lens[[0, n_seq // 2, n_seq - 1]] = [0, 1500, 7]
    _run_attention(rng, lens.tolist(), 2 * kv, kv, 32, 16, kind)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("reach", [10000, 400000])
@pytest.mark.parametrize("where", [0, 1, 127, 128, 4095, 5000, 9999])
def test_attention_finds_one_key(cuda, kind, where, reach):
    """One key of 10,000 carries nearly all of the weight, wherever it stands; far smaller and far larger
    scores before and after it (the running maximum jumps by more than exp's range)."""
    rng = _rng(where)
    n, page, dim = 10000, 16, 64
    table, n_pages = _pages(rng, [n], page, width=reach // page)
    kc, vc = _pool(n_pages, page, 2, dim, kind, "slot", math.nan)
    k = rng.standard_normal((n, 2, dim)) * 0.01
    k[: where // 2, :, 0] -= 300.0
    k[where, :, 0] = 200.0
    v = rng.standard_normal((n, 2, dim))
    at = np.arange(n)
    idx = (torch.from_numpy(table[0, at // page].astype(np.int64)).cuda(), torch.from_numpy(at % page).cuda())
    kc[idx], vc[idx] = _t(k, kind), _t(v, kind)
    q = torch.zeros(1, 8, dim, dtype=DT[kind], device="cuda")
    q[..., 0] = 8.0
    out, lse = B.decode_attention(q, kc, vc, _i(table), _i([n]))
    want = np.repeat(_np(vc[idx][where])[None], 4, axis=1)  # its score is 200 above the rest's: no other weight survives fp32
    _check(out, want.reshape(1, 8, dim), 2.0 ** -20 * np.abs(want.reshape(1, 8, dim)) + 1e-30)
    _check(lse, np.full((1, 8), 200.0), 200 * 70 * U)


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
def test_attention_infinite_scores_are_absent_keys(cuda, reach):
    rng = _rng(9)
    table, n_pages = _pages(rng, [40, 3], 16, width=reach // 16)
    kc, vc = _pool(n_pages, 16, 1, 64, "fp32", "slot", math.nan)
    parts = _fill(rng, [40, 3], table, kc, vc, 16)
    q = _t(np.abs(rng.standard_normal((2, 1, 64))) + 0.1)
    for s, j in [(0, 7), (0, 39), (1, 0), (1, 1), (1, 2)]:
        kc[int(table[s, j // 16]), j % 16, 0, 3] = -math.inf
    out, lse = B.decode_attention(q, kc, vc, _i(table), _i([40, 3]))
    keep = [j for j in range(40) if j not in (7, 39)]
    want, wl, tol, tl = _attention(_np(q)[0], parts[0][0][keep], parts[0][1][keep], 0.125)
    _check(out[0], want, tol)
    _check(lse[0], wl, tl)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_attention_bad_pages_and_lengths(cuda, kind):
    """Keys of a bad page are absent; a length past the table is cut to it, a negative one is zero."""
    rng = _rng(kind, 2)
    page, dim = 16, 64
    lens = [100, 80, 64, 33]
    table, n_pages = _pages(rng, lens, page, width=7)
    kc, vc = _pool(n_pages, page, 2, dim, kind, "slot", math.nan)
    parts = _fill(rng, lens, table, kc, vc, page)
    q = _t(rng.standard_normal((4, 4, dim)), kind)
    bad = table.copy()
    bad[0, 1], bad[0, 6], bad[1, :] = -1, n_pages, 1 << 30
    bad[2, 4:] = bad[2, :3]  # 64 keys and then, cut at the table's reach, 48 of them again
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = B.decode_attention(q, kc, vc, _i(bad), _i([100, 80, 5000, -3]), status=status)
    assert int(status) == B.STATUS_BAD_PAGE | B.STATUS_BAD_POS
    keep = {0: [j for j in range(96) if j // 16 != 1], 1: [], 2: list(range(64)) + list(range(48)), 3: []}
    for s, rows in keep.items():
        want, wl, tol, tl = _attention(_np(q)[s], parts[s][0][rows], parts[s][1][rows], 0.125)
        _check(out[s], want, tol + ((np.abs(want) + tol) * 2.0 ** -8 if kind == "bf16" else 0))
        if rows:
            _check(lse[s], wl, tl)
        else:
            assert bool((out[s] == 0).all()) and bool((lse[s] == -math.inf).all())


@gpu
@pytest.mark.parametrize("step", [(1 << 31) + 4096, (1 << 33) + 4096])
def test_attention_offsets_past_32_bits(cuda, step):
    """Pages 2^32 bytes and more apart in one pool (of more than 2^36 bytes, the second time); `step`: elements between pages."""
    rng = _rng(4)
    page, dim, n_pages = 16, 128, 5
    pool = torch.empty((n_pages - 1) * step + 2 * page * dim, dtype=torch.bfloat16, device="cuda")
    kc, vc = (x.as_strided((n_pages, page, 1, dim), (step, dim, dim, 1), at) for x, at in ((pool, 0), (pool, page * dim)))
    kc.fill_(math.nan), vc.fill_(math.nan)
    table = np.array([[4, 0, 3]], dtype=np.int32)
    parts = _fill(rng, [41], table, kc, vc, page)
    q = _t(rng.standard_normal((1, 4, dim)), "bf16")
    new = _t(rng.standard_normal((1, 1, dim)), "bf16")
    B.kv_append(new, new, kc, vc, _i(table), _i([40]))
    assert torch.equal(kc[3, 8], new[0]) and torch.equal(vc[3, 8], new[0])
    for x in parts[0]:
        x[40] = _np(new)[0]
    out, lse = B.decode_attention(q, kc, vc, _i(table), _i([41]))
    want, wl, tol, tl = _attention(_np(q)[0], *parts[0], dim ** -0.5)
    _check(out[0], want, tol + (np.abs(want) + tol) * 2.0 ** -8)
    _check(lse[0], wl, tl)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_attention_shared_pages_and_repeats(cuda, kind):
    """Sequences that share pages and the same call twice give the same bits."""
    rng = _rng(kind, 8)
    table, n_pages = _pages(rng, [3000], 16)
    kc, vc = _pool(n_pages, 16, 4, 64, kind, "slot", math.nan)
    _fill(rng, [3000], table, kc, vc, 16)
    q = _t(rng.standard_normal((1, 16, 64)), kind).expand(3, 16, 64)
    many = _i(np.repeat(table, 3, axis=0))
    out, lse = B.decode_attention(q, kc, vc, many, _i([3000, 3000, 3000]))
    again, lse2 = B.decode_attention(q, kc, vc, many, _i([3000, 3000, 3000]))
    assert torch.equal(out, again) and torch.equal(lse, lse2)


# ----------------------------------------------------------------- next_token

def _next(z, hist=None, hl=None, pl=None, rep=None, pres=None, freq=None, ids=None, vals=None, allowed=None):
    """The definition, each step rounded to fp32 on its own, row by row; (token, out, lse in float64)."""
    f = np.float32
    z = np.array(z, dtype=f)
    rows, vocab = z.shape
    with np.errstate(all="ignore"):
        for b in range(rows):
            if hist is not None:
                n, first = (len(hist[b]) if hl is None else hl[b]), (0 if pl is None else pl[b])
                h = [t for t in hist[b][:n] if 0 <= t < vocab]
                made = np.bincount([t for t in hist[b][first:n] if 0 <= t < vocab], minlength=vocab)
                for t in sorted(set(h)):
                    if rep is not None:
                        z[b, t] = z[b, t] / f(rep[b]) if z[b, t] > 0 else z[b, t] * f(rep[b])
                    c = made[t]
                    if c:
                        z[b, t] = f(z[b, t] - f(f(freq[b] if freq is not None else 0) * f(c))) - f(pres[b] if pres is not None else 0)
            if ids is not None:
                total = {}
                for t, x in zip(ids[b], vals[b]):
                    if 0 <= t < vocab:
                        total[t] = f(total.get(t, f(0)) + f(x))
                for t, x in total.items():
                    z[b, t] = z[b, t] + x
            if allowed is not None:
                bits = (allowed[b][np.arange(vocab) // 32].astype(np.int64) >> (np.arange(vocab) % 32)) & 1
                z[b, bits == 0] = -np.inf
        token = []
        for b in range(rows):
            m = np.nanmax(np.where(np.isnan(z[b]), -np.inf, z[b]))
            token.append(-1 if m == -np.inf else int(np.nonzero(z[b] == m)[0][0]))
        d = z.astype(np.float64)
        m = np.where(np.isfinite(d.max(axis=1)), d.max(axis=1), 0)
        lse = m + np.log(np.exp(d - m[:, None]).sum(axis=1))
    return np.array(token), z, lse


def _check_next(got, want):
    token, out, lse = got
    t, z, l = want
    np.testing.assert_array_equal(out.cpu().numpy(), z)
    np.testing.assert_array_equal(token.cpu().numpy(), t)
    lse = lse.double().cpu().numpy()
    same = (lse == l) | (np.isnan(lse) & np.isnan(l))
    # exponentials 2^-20; at most vocab/256 + 64 additions one after another; the result's own rounding
    tol = 2.0 ** -20 + (z.shape[1] / 256 + 64) * U + 4 * U * np.abs(np.where(np.isfinite(l), l, 0))
    with np.errstate(invalid="ignore"):
        assert (same | (np.abs(lse - l) <= tol)).all(), (lse, l)


def _token_inputs(rng, rows, vocab, most, kind):
    z = _np(_t(rng.standard_normal((rows, vocab)) * 3, kind)).astype(np.float32)
    hist = (rng.random((rows, most)) ** 4 * vocab).astype(np.int32)
    n_bias = min(vocab, 7)
    return dict(z=z, hist=hist, hl=rng.integers(0, most + 1, rows), pl=rng.integers(0, most + 1, rows),
                rep=(1 + rng.random(rows)).astype(np.float32), pres=rng.standard_normal(rows).astype(np.float32),
                freq=rng.random(rows).astype(np.float32), ids=np.stack([rng.permutation(vocab)[:n_bias] for _ in range(rows)]),
                vals=rng.standard_normal((rows, n_bias)).astype(np.float32),
                allowed=rng.integers(-(1 << 31), 1 << 31, (rows, -(-vocab // 32))).astype(np.int32))


def _run_next(x, kind, **kw):
    names = dict(hist="history", hl="history_lens", pl="prompt_lens", rep="repetition", pres="presence", freq="frequency",
                 ids="bias_ids", vals="bias_values", allowed="allowed")
    args = {names[k]: (_t(v) if k in ("rep", "pres", "freq", "vals") else _i(v)) for k, v in x.items() if k != "z"}
    return B.next_token(_t(x["z"], kind), **args, **kw)


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab,most", [(1, 256, 1), (3, 12288, 1000), (5, 50304, 300), (7, 4999, 2049), (2, 1, 5),
                                             (4, 33, 64), (9, 131, 17), (2, 131072, 40), (1, 300001, 9), (40, 8191, 33)])
def test_next_token(cuda, kind, rows, vocab, most):
    x = _token_inputs(_rng(kind, rows, vocab), rows, vocab, most, kind)
    _check_next(_run_next(x, kind), _next(**x))


@gpu
@pytest.mark.parametrize("rows,vocab,most,n_bias", [(2, 50304, 30000, 40), (1, 131072, 9000, 5000), (3, 4096, 4096, 3000),
                                                    (1, 65, 5000, 65)])
def test_next_token_many_marked_ids(cuda, rows, vocab, most, n_bias):
    """Long histories and bias lists spread evenly over the vocabulary: more marked ids than a block's table has places."""
    rng = _rng(rows, vocab, most)
    x = _token_inputs(rng, rows, vocab, most, "fp32")
    x["hist"] = rng.integers(0, vocab, (rows, most)).astype(np.int32)
    x["hl"] = np.array([most - i for i in range(rows)])
    x["ids"] = rng.integers(0, vocab, (rows, n_bias))
    x["vals"] = rng.standard_normal((rows, n_bias)).astype(np.float32)
    _check_next(_run_next(x, "fp32"), _next(**x))


@gpu
@pytest.mark.parametrize("keep", [[], ["hist"], ["hist", "rep"], ["hist", "hl", "freq"], ["hist", "pl", "pres"], ["ids", "vals"],
                                  ["allowed"], ["rep", "pres"], ["hist", "hl", "allowed", "rep"]])
def test_next_token_parts(cuda, keep):
    """Every argument but the logits may be absent."""
    x = _token_inputs(_rng(*keep, 1), 3, 1000, 50, "fp32")
    x = {k: v for k, v in x.items() if k in ["z"] + keep}
    _check_next(_run_next(x, "fp32"), _next(**x))


@gpu
def test_next_token_edge_rows(cuda):
    """Rows that the mask empties, infinities and NaN in masked and in open places, ties, repeated bias ids,
    ids outside the vocabulary."""
    rng = _rng(77)
    vocab = 5000
    x = _token_inputs(rng, 10, vocab, 20, "fp32")
    x["allowed"][:] = -1
    x["allowed"][0] = 0                                       # nothing left
    x["z"][1] = -np.inf                                       # nothing there
    x["allowed"][2, 0] = ~np.int32(6)
    x["z"][2, 1], x["z"][2, 2] = np.nan, np.inf               # masked
    x["z"][3, 4000] = np.inf
    x["z"][4, 17] = np.nan
    x["z"][5] = np.finfo(np.float32).min                      # the type's lowest value everywhere
    x["z"][6, [4998, 4097, 4096, 31]] = 50.0                  # ties: the lowest id
    x["hl"][6] = 0
    x["ids"][6] = -1
    x["ids"][7] = [3, 3, vocab - 1, 3, vocab - 1, -5, 3]
    x["z"][8] = np.nan
    x["allowed"][9] = 0
    x["allowed"][9, vocab // 32] = 1 << (vocab - 1) % 32      # one token left: the last
    want = _next(**x)
    assert want[0][0] == -1 and want[0][1] == -1 and want[0][3] == 4000 and want[0][6] == 31 and want[0][9] == vocab - 1
    assert want[0][8] == -1 and want[2][0] == -np.inf and want[2][3] == np.inf and np.isnan(want[2][[4, 8]]).all()
    _check_next(_run_next(x, "fp32"), want)


@gpu
def test_next_token_bad_ids(cuda):
    x = _token_inputs(_rng(6), 3, 500, 30, "fp32")
    x["hist"][0, 3], x["hist"][1, 0], x["hist"][1, 29] = -1, 500, 1 << 30
    x["hl"][:] = [30, 29, 30]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check_next(_run_next(x, "fp32", status=status), _next(**x))
    assert int(status) == B.STATUS_BAD_TOKEN
    status.zero_()
    x["hist"] = np.abs(x["hist"]) % 500
    x["ids"][2, 4] = 500
    _check_next(_run_next(x, "fp32", status=status), _next(**x))
    assert int(status) == B.STATUS_BAD_TOKEN
    status.zero_()
    x["ids"][2, 4] = 0
    x["hl"][:] = [31, -1, 30]                                 # cut to the history's width, and to nothing
    got = _run_next(x, "fp32", status=status)
    x["hl"][:] = [30, 0, 30]
    _check_next(got, _next(**x))
    assert int(status) == B.STATUS_BAD_POS


@gpu
@pytest.mark.parametrize("kind,offset,width", [("fp32", 1, 1003), ("bf16", 1, 1001), ("bf16", 3, 1003), ("fp32", 0, 1000), ("bf16", 8, 1008)])
def test_next_token_strides_and_in_place(cuda, kind, offset, width):
    """Rows at any alignment; what lies between and behind the rows stays as it was."""
    x = _token_inputs(_rng(width, kind), 6, 990, 30, kind)
    pool = torch.full((6, width + 2), 7.0, dtype=DT[kind], device="cuda").flatten()[offset:offset + 6 * width].view(6, width)
    logits = pool[:, :990]
    logits.copy_(_t(x["z"], kind))
    names = dict(history=_i(x["hist"]), repetition=_t(x["rep"]), allowed=torch.cat([_i(x["allowed"]), _i(x["allowed"])], 1)[:, :31])
    ref = _next(x["z"], hist=x["hist"], rep=x["rep"], allowed=x["allowed"])
    dest = torch.full((6 * 1100 + 5,), 8.0, device="cuda")
    out = dest[5:].view(6, 1100)[:, :990]
    _check_next(B.next_token(logits, out=out, **names), ref)
    assert bool((dest[5:].view(6, 1100)[:, 990:] == 8.0).all()) and bool((dest[:5] == 8.0).all())
    assert bool((pool[:, 990:] == 7.0).all())
    if kind == "fp32":
        got = B.next_token(logits, out=logits, **names)
        assert got[1] is logits
        _check_next(got, ref)
        assert bool((pool[:, 990:] == 7.0).all())


# ----------------------------------------------------------------- refusals of the binding, streams, graphs

@gpu
def test_binding_refuses_wrong_tensors(cuda):
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    i32 = torch.int32
    cache, table, one = z(8, 16, 4, 64), z(2, 4, t=i32), z(2, t=i32)
    q, k = z(2, 8, 64), z(2, 4, 64)
    bad = [
        lambda: B.kv_append(k.double(), k, cache, cache, table, one), lambda: B.kv_append(k, k[:1], cache, cache, table, one),
        lambda: B.kv_append(k, k, cache, cache.transpose(1, 2).contiguous().transpose(1, 2), table, one),
        lambda: B.kv_append(k, k, cache[0], cache[0], table, one), lambda: B.kv_append(k, k, cache, cache, table[0], one),
        lambda: B.kv_append(k, k, cache, cache, table.long(), one), lambda: B.kv_append(k, k, cache, cache, table, one[:1]),
        lambda: B.kv_append(k, k, cache, cache, table, one, q_out=q), lambda: B.kv_append(k, k, cache, cache, table, one, q=q.bfloat16()),
        lambda: B.kv_append(k, k, cache, cache, table, one, rope_dims=65), lambda: B.kv_append(k, k.cpu(), cache, cache, table, one),
        lambda: B.kv_append(k.transpose(0, 1), k, cache, cache, table, one),
        lambda: B.kv_append(k, k, cache.half(), cache.half(), table, one),
        lambda: B.kv_append(z(2, 4, 65)[..., 1:], k, cache, cache, table, one),
        lambda: B.decode_attention(q[0], cache, cache, table, one), lambda: B.decode_attention(q[:1], cache, cache, table, one),
        lambda: B.decode_attention(q[:, :6], cache, cache, table, one), lambda: B.decode_attention(q, cache, cache, table, one.long()),
        lambda: B.decode_attention(q, cache, cache, table, one, scale=math.nan),
        lambda: B.decode_attention(q, cache, cache, table, one, out=z(2, 8, 32)),
        lambda: B.next_token(z(4)), lambda: B.next_token(z(4, 9).half()), lambda: B.next_token(z(4, 9), history=z(3, 5, t=i32)),
        lambda: B.next_token(z(4, 9), history=z(4, 5)), lambda: B.next_token(z(4, 9), history_lens=z(4, t=i32)),
        lambda: B.next_token(z(4, 9), bias_ids=z(4, 2, t=i32)), lambda: B.next_token(z(4, 9), allowed=z(4, 2, t=i32)),
        lambda: B.next_token(z(4, 9), repetition=z(3)), lambda: B.next_token(z(4, 9), out=z(4, 9, t=torch.bfloat16)),
        lambda: B.next_token(z(9, 4).t())]
    for call in bad:
        with pytest.raises(B.GptError):
            call()
    torch.cuda.synchronize()


@gpu
def test_empty_batches(cuda):
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    i32 = torch.int32
    cache = z(8, 16, 4, 64)
    assert B.kv_append(z(0, 4, 64), z(0, 4, 64), cache, cache, z(2, 4, t=i32), z(0, t=i32), q=z(0, 8, 64)).shape == (0, 8, 64)
    out, lse = B.decode_attention(z(0, 8, 64), cache, cache, z(0, 4, t=i32), z(0, t=i32))
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    assert B.next_token(z(0, 50))[0].shape == (0,)
    x = _token_inputs(_rng(3), 2, 50, 4, "fp32")
    token, _, _ = B.next_token(_t(x["z"]), history=z(2, 0, t=i32), history_lens=z(2, t=i32), bias_ids=z(2, 0, t=i32), bias_values=z(2, 0))
    assert token.tolist() == x["z"].argmax(axis=1).tolist()


@gpu
def test_broadcast_inputs(cuda):
    """Inputs expanded over rows, sequences and heads (stride 0)."""
    rng = _rng(21)
    x = _token_inputs(rng, 4, 700, 30, "fp32")
    for k in ("z", "hist", "ids", "vals", "allowed"):
        x[k] = np.repeat(x[k][:1], 4, axis=0)
    want = _next(**x)
    wide = {k: (_t(x[k][:1]) if k in ("z", "vals") else _i(x[k][:1])).expand(4, -1) for k in ("z", "hist", "ids", "vals", "allowed")}
    got = B.next_token(wide["z"], history=wide["hist"], history_lens=_i(x["hl"]), prompt_lens=_i(x["pl"]), repetition=_t(x["rep"]),
                       presence=_t(x["pres"]), frequency=_t(x["freq"]), bias_ids=wide["ids"], bias_values=wide["vals"], allowed=wide["allowed"])
    _check_next(got, want)
    table, n_pages = _pages(rng, [77], 16)
    kc, vc = _pool(n_pages, 16, 1, 64, "bf16", "slot", math.nan)
    (k, v), = _fill(rng, [77], table, kc, vc, 16)
    q = _t(rng.standard_normal((3, 1, 64)), "bf16").expand(3, 6, 64)
    out, lse = B.decode_attention(q, kc.expand(-1, -1, 2, -1), vc.expand(-1, -1, 2, -1), _i(table).expand(3, -1), _i([77, 30, 1]))
    for s, n in enumerate((77, 30, 1)):
        w, wl, tol, tl = _attention(_np(q)[s], k[:n], v[:n], 0.125)
        _check(out[s], w, tol + (np.abs(w) + tol) * 2.0 ** -8)
        _check(lse[s], wl, tl)
    new = _t(rng.standard_normal((2, 1, 64)), "bf16").expand(2, 3, 64)
    kc, vc = _pool(4, 16, 3, 64, "bf16", "slot", 0.0)
    assert B.kv_append(new, new, kc, vc, _i([[1, 2]]), _i([3, 20]), seq=_i([0, 0])) is None
    assert torch.equal(kc[1, 3], new[0]) and torch.equal(vc[2, 4], new[1])


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
def test_captured_behind_a_join_and_copies(cuda, reach):
    """Captured where the stream has just joined another and copied, replayed with other inputs, beside eager calls."""
    rng = _rng(31)
    table, n_pages = _pages(rng, [300, 40, 0], 16, width=reach // 16)
    kc, vc = _pool(n_pages, 16, 2, 64, "bf16", "slot", math.nan)
    _fill(rng, [300, 40, 0], table, kc, vc, 16)
    tab, lens = _i(table), _i([300, 40, 0])
    qs = [_t(rng.standard_normal((3, 8, 64)), "bf16") for _ in range(3)]
    zs = [_t(rng.standard_normal((3, 999))) for _ in range(3)]
    want = [(*B.decode_attention(q, kc, vc, tab, lens), *B.next_token(z)) for q, z in zip(qs, zs)]
    q, z, side = torch.zeros_like(qs[0]), torch.zeros_like(zs[0]), torch.cuda.Stream()
    q_in, z_in = torch.zeros_like(q), torch.zeros_like(z)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            z.copy_(z_in)
            token = B.next_token(z)
        q.copy_(q_in)
        main.wait_stream(side)
        att = B.decode_attention(q, kc, vc, tab, lens)
        again = B.decode_attention(q, kc, vc, tab, lens)
    for i in (1, 2, 0):
        q_in.copy_(qs[i])
        z_in.copy_(zs[i])
        g.replay()
        eager = B.decode_attention(qs[i], kc, vc, tab, lens)
        torch.cuda.synchronize()
        for a, b in zip((*att, *token), want[i]):
            assert torch.equal(a, b)
        for other in (again, eager):
            assert torch.equal(other[0], want[i][0]) and torch.equal(other[1], want[i][1])


@gpu
def test_calls_from_threads_on_their_own_streams(cuda):
    """Four threads, a stream each, calling at once."""
    import threading
    rng = _rng(41)
    lens = [2000, 1, 555, 90]
    table, n_pages = _pages(rng, lens, 16, width=30000)
    kc, vc = _pool(n_pages, 16, 2, 128, "bf16", "slot", math.nan)
    _fill(rng, lens, table, kc, vc, 16)
    tab, ln = _i(table), _i(lens)
    qs = [_t(rng.standard_normal((4, 8, 128)), "bf16") for _ in range(4)]
    x = _token_inputs(rng, 4, 3000, 64, "fp32")
    z, hist, rep = _t(x["z"]), _i(x["hist"]), _t(x["rep"])
    want = [B.decode_attention(q, kc, vc, tab, ln) for q in qs]
    token = B.next_token(z, history=hist, repetition=rep)
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(50):
                out, lse = B.decode_attention(qs[i], kc, vc, tab, ln)
                t = B.next_token(z, history=hist, repetition=rep)
                st.synchronize()
                if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]) and all(torch.equal(a, b) for a, b in zip(t, token))):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


class _Layer:
    """One attention layer and an LM head with random fp32 weights: the operators as a decode loop uses them."""

    def __init__(self, seed, n_seq, prompts, steps, page=8, heads=6, kv=2, dim=32, vocab=777):
        rng = np.random.default_rng(seed)
        w = lambda *s: (rng.standard_normal(s) / np.sqrt(s[-1])).astype(np.float32)  # noqa: E731
        self.heads, self.kv, self.dim, self.vocab, self.page, self.steps = heads, kv, dim, vocab, page, steps
        self.emb, self.wqkv, self.wo, self.lm = w(vocab, 64) * 8, w((heads + 2 * kv) * dim, 64), w(64, heads * dim), w(vocab, 64) * 8
        self.prompts = [rng.integers(0, vocab, n).tolist() for n in prompts]
        table, n_pages = _pages(rng, [n + steps for n in prompts], page)
        self.table_np, self.table = table, _i(table)
        self.kc, self.vc = _pool(n_pages, page, kv, dim, "fp32", "slot", math.nan)
        width = max(prompts) + steps
        self.hist = _i([p + [0] * (width - len(p)) for p in self.prompts])
        self.hl, self.pl = _i(prompts), _i(prompts)
        self.rep, self.freq = torch.full((n_seq,), 1.3, device="cuda"), torch.full((n_seq,), 0.1, device="cuda")
        self.W = [_t(x) for x in (self.emb, self.wqkv, self.wo, self.lm)]

    def split(self, x):
        d = self.dim
        qkv = (self.W[0][x.long()] @ self.W[1].t())
        return [y.unflatten(1, (-1, d)) for y in qkv.split([self.heads * d, self.kv * d, self.kv * d], dim=1)]

    def prefill(self):
        """All prompt tokens but the last of every sequence, as one ragged batch with two padding rows."""
        ids = [t for p in self.prompts for t in p[:-1]] + [0, 0]
        seq = [s for s, p in enumerate(self.prompts) for _ in p[:-1]] + [-1, -1]
        pos = [i for p in self.prompts for i in range(len(p) - 1)] + [0, 1 << 20]
        _, k, v = self.split(_i(ids))
        B.kv_append(k, v, self.kc, self.vc, self.table, _i(pos), seq=_i(seq), rope_dims=self.dim)
        self.token = _i([p[-1] for p in self.prompts])

    def step(self):
        """One decode step on device state only (capturable)."""
        q, k, v = self.split(self.token)
        q = B.kv_append(k, v, self.kc, self.vc, self.table, self.hl - 1, q=q, rope_dims=self.dim)
        o, _ = B.decode_attention(q, self.kc, self.vc, self.table, self.hl)
        x = self.W[0][self.token.long()] + o.flatten(1) @ self.W[2].t()
        token, self.out, _ = B.next_token(x @ self.W[3].t(), history=self.hist, history_lens=self.hl, prompt_lens=self.pl,
                                          repetition=self.rep, frequency=self.freq)
        self.hist.scatter_(1, self.hl[:, None].long(), token[:, None])
        self.token.copy_(token)
        self.hl += 1

    def check(self):
        """Every generated token is a maximum of the float64 logits, given the tokens before it."""
        hist = self.hist.cpu().numpy()
        d, (E, Wq, Wo, L) = self.dim, (x.astype(np.float64) for x in (self.emb, self.wqkv, self.wo, self.lm))
        E, Wq, Wo, L = (np.asarray(x) for x in (E, Wq, Wo, L))
        for s, p in enumerate(self.prompts):
            seq = hist[s, :len(p) + self.steps].tolist()
            qkv = E[seq] @ Wq.T
            q, k, v = (x.reshape(len(seq), -1, d) for x in np.split(qkv, [self.heads * d, (self.heads + self.kv) * d], axis=1))
            at = np.arange(len(seq))
            q, k = _turned(q, at, d, 10000.0), _turned(k, at, d, 10000.0)
            for n in range(len(p), len(seq)):
                o = _attention(q[n - 1], k[:n], v[:n], d ** -0.5)[0]
                z = L @ (E[seq[n - 1]] + Wo @ o.reshape(-1))
                for t in set(seq[:n]):
                    z[t] = z[t] / 1.3 if z[t] > 0 else z[t] * 1.3
                    z[t] -= 0.1 * seq[len(p):n].count(t)
                assert z[seq[n]] >= z.max() - 1e-3, (s, n)


PROMPTS = [5, 1, 17, 8, 9]


@gpu
def test_decode_loop(cuda):
    m = _Layer(1, 5, PROMPTS, 12)
    m.prefill()
    for _ in range(12):
        m.step()
    m.check()


@gpu
def test_decode_loop_captured(cuda):
    """Two models' steps captured into two graphs on side streams and replayed in turns, with eager calls
    between, give the tokens of eager loops."""
    eager = [_Layer(s, 5, PROMPTS, 10) for s in (2, 3)]
    for m in eager:
        m.prefill()
        for _ in range(10):
            m.step()
    models, graphs = [_Layer(s, 5, PROMPTS, 10) for s in (2, 3)], []
    for m in models:
        m.prefill()
        m.step()  # eager warm-up
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.step()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in models]
    torch.cuda.synchronize()
    for _ in range(9):  # a captured step has not run: nine are left
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for m, e in zip(models, eager):
        assert torch.equal(m.hist, e.hist)
        m.check()


@gpu
def test_given_stream(cuda):
    """A stream passed to the calls orders them behind that stream's work."""
    st = torch.cuda.Stream()
    rng = _rng(12)
    table, n_pages = _pages(rng, [600, 40], 16)
    kc, vc = _pool(n_pages, 16, 2, 64, "bf16", "slot", 0.0)
    _fill(rng, [600, 40], table, kc, vc, 16)
    tab, lens, q = _i(table), _i([600, 40]), _t(rng.standard_normal((2, 8, 64)), "bf16")
    x = _token_inputs(rng, 2, 4000, 9, "fp32")
    z = _t(x["z"])
    want, _ = B.decode_attention(q, kc, vc, tab, lens)
    tok = B.next_token(z)[0]
    late_q, late_z = torch.zeros_like(q), torch.zeros_like(z)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        big = torch.zeros(1 << 28, device="cuda")
        for _ in range(5):
            big += 1
        late_q.copy_(q)
        late_z.copy_(z)
    out, _ = B.decode_attention(late_q, kc, vc, tab, lens, stream=st)
    tok2 = B.next_token(late_z, stream=st)[0]
    qo = B.kv_append(late_q[:, :2], late_q[:, :2], kc, vc, tab, _i([0, 0]), q=late_q, stream=st)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(tok, tok2) and torch.equal(qo, q)


@gpu
@pytest.mark.parametrize("rows,vocab,pad", [(1, 140000, 3), (305, 20011, 0)])
def test_next_token_in_place_on_long_rows(cuda, rows, vocab, pad):
    """Rows of several loads a thread and ranges a block, read and written over; what lies between rows stays."""
    x = _token_inputs(_rng(rows, vocab), rows, vocab, 2500, "fp32")
    wide = torch.full((rows, vocab + pad), 5.0, device="cuda")
    z = wide[:, :vocab]
    z.copy_(_t(x["z"]))
    got = B.next_token(z, history=_i(x["hist"]), history_lens=_i(x["hl"]), prompt_lens=_i(x["pl"]), repetition=_t(x["rep"]),
                       presence=_t(x["pres"]), frequency=_t(x["freq"]), bias_ids=_i(x["ids"]), bias_values=_t(x["vals"]),
                       allowed=_i(x["allowed"]), out=z)
    assert got[1] is z
    _check_next(got, _next(**x))
    assert bool((wide[:, vocab:] == 5.0).all())


@gpu
def test_append_and_next_token_offsets_past_32_bits(cuda):
    """Pages, token rows, logits and histories 2^31 elements and more apart."""
    step = (1 << 31) + 64
    rng = _rng(15)
    kc, vc = (torch.zeros(step + 4096, dtype=torch.bfloat16, device="cuda").as_strided((2, 4, 2, 64), (step, 128, 64, 1))
              for _ in range(2))
    x = torch.zeros(step + 4096, dtype=torch.bfloat16, device="cuda").as_strided((2, 2, 64), (step, 64, 1))
    x.copy_(_t(rng.standard_normal((2, 2, 64)), "bf16"))
    B.kv_append(x, x, kc, vc, _i([[0, 1], [1, 0]]), _i([3, 1]))
    want = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    want[0, 3], want[1, 1] = x[0], x[1]
    assert torch.equal(kc, want) and torch.equal(vc, want)
    x = _token_inputs(rng, 2, 1000, 40, "fp32")
    z, out = (torch.full((step + 2000,), 2.0, device="cuda").as_strided((2, 1000), (step, 1)) for _ in range(2))
    z.copy_(_t(x["z"]))
    hist = torch.zeros(step + 100, dtype=torch.int32, device="cuda").as_strided((2, 40), (step, 1))
    hist.copy_(_i(x["hist"]))
    got = B.next_token(z, history=hist, history_lens=_i(x["hl"]), repetition=_t(x["rep"]), out=out)
    _check_next(got, _next(x["z"], hist=x["hist"], hl=x["hl"], rep=x["rep"]))


@gpu
def test_default_stream_given_from_another(cuda):
    side = torch.cuda.Stream()
    z = _t(_rng(13).standard_normal((3, 500)))
    want = B.next_token(z)[0]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = B.next_token(z, stream=torch.cuda.default_stream())[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)


FIRST_CALLS = """
import torch
from persistent_gpt_step_gb300 import binding as B
i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
kc, vc = (torch.zeros(40, 16, 2, 64, device="cuda") for _ in range(2))
q, k, z = (torch.randn(s, device="cuda") for s in ((2, 4, 64), (2, 2, 64), (2, 300)))
table, pos, lens = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20), i(0, 0), i(1, 1)
far = torch.zeros(2, 9000, dtype=torch.int32, device="cuda")  # room for so many keys that the other kernel is taken
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    B.kv_append(k, k, kc, vc, table, pos)
    near = B.decode_attention(q, kc, vc, table, lens)[0]
    wide = B.decode_attention(q, kc, vc, far[:, :9000], lens)[0]
    token = B.next_token(z)[0]
g.replay()
torch.cuda.synchronize()
want = k.repeat_interleave(2, 1)
assert torch.equal(near, want) and torch.equal(wide[0], want[0]) and torch.equal(token, z.argmax(1).int())
"""


@gpu
def test_first_calls_of_a_process_are_captured(cuda):
    """No call has to run eagerly before it can be captured."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@gpu
@pytest.mark.parametrize("name", ["tiny", "small_gated"])
def test_serve_bench_times_the_operators(cuda, name):
    from persistent_gpt_step_gb300 import inputs, serve_bench
    got = serve_bench.decode_bench(inputs.CONFIGS[name], 3, 40, reps=2)
    assert all(v > 0 for v in got.values())
    assert set(got) == {"kv_append_us", "decode_attention_us", "next_token_us", "step_us", "cache_gb_per_s"}


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("kv,n_seq", [(1, 90), (2, 45), (4, 25), (8, 12)])
def test_attention_short_rows_in_a_wide_table(cuda, kind, kv, n_seq):
    """Rows of a few keys cut by the parts of the line, in teams of one, two and four warps: a warp's piece is there
    however soon it is done, and again in every repeat of the call."""
    def once():
        rng = _rng(kind, kv, n_seq)
        return _run_attention(rng, rng.integers(1, 200, n_seq).tolist(), 2 * kv, kv, 64, 16, kind, reach=400000)
    got, lse = once()
    for _ in range(4):
        again, lse2 = once()
        assert torch.equal(got, again) and torch.equal(lse, lse2)


def _weighed(q, keys, values, scale):
    """Definition for one sequence and values that need not be finite: keys of a score of -infinity are absent, every
    other value belongs in the result.  (out, the largest finite |value| per head and dim, lse)."""
    heads, dim = q.shape
    g = heads // keys.shape[1]
    K, V = np.repeat(keys, g, axis=1), np.repeat(values, g, axis=1)
    out, lse = np.zeros((heads, dim)), np.full(heads, -np.inf)
    with np.errstate(all="ignore"):
        for h in range(heads):
            z = (K[:, h] * q[h]).sum(axis=1) * scale
            on = z > -np.inf
            if not on.any():
                continue
            w = np.exp(z[on] - z[on].max())
            lse[h] = z[on].max() + np.log(w.sum())
            w = w / w.sum()
            v = V[on, h]
            out[h] = np.where(np.isfinite(v), w[:, None] * np.where(np.isfinite(v), v, 0), v).sum(axis=0)
    return out, lse


def _check_infinite(got, want, rel):
    got = _np(got)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(np.isinf(got) & ok, np.isinf(want) & ok) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    f = np.isfinite(want)
    off = np.abs(got[f] - want[f]) - rel(np.where(f, want, 0))[f]
    assert (off <= 0).all(), float(off.max())


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,heads,kv,dim,page", [([40, 3, 700], 4, 1, 64, 16), ([2500, 60], 8, 8, 128, 16), ([300, 9, 9], 6, 2, 96, 24),
                                                    ([90, 5000], 12, 1, 64, 5), ([100] * 40, 4, 4, 64, 16)])
def test_attention_values_of_infinity_and_nan(cuda, kind, reach, lens, heads, kv, dim, page):
    """A value of infinity or NaN belongs in the result at any key that counts, however small its weight is, and in none where the
    key's score is -infinity; the other dims and heads are what they are without it."""
    rng = _rng(kind, dim, len(lens), heads)
    table, n_pages = _pages(rng, lens, page, width=-(-reach // page))
    kc, vc = _pool(n_pages, page, kv, dim, kind, "slot", math.nan)
    parts = _fill(rng, lens, table, kc, vc, page)
    q = _t(np.abs(rng.standard_normal((len(lens), heads, dim))) + 0.1, kind)

    def put(pool, which, s, j, h, e, x):
        pool[int(table[s, j // page]), j % page, h, e] = x
        parts[s][which][j, h, e] = x
    inf, nan = math.inf, math.nan
    for s, n in enumerate(lens):
        put(vc, 1, s, 0, 0, 3, inf)
        put(vc, 1, s, n - 1, kv - 1, 5, -inf)
        put(vc, 1, s, n // 2, 0, 7, nan)
        put(vc, 1, s, n - 1, 0, 9, inf), put(vc, 1, s, 0, 0, 9, -inf)
        if n > 30:
            put(kc, 0, s, 11, 0, 0, -inf), put(vc, 1, s, 11, 0, 11, nan), put(vc, 1, s, 11, 0, 12, inf)  # absent
            put(kc, 0, s, 20, 0, 1, -3000.0), put(vc, 1, s, 20, 0, 13, inf)  # a weight far below fp32
            parts[s][0][20, 0, 1] = _np(kc[int(table[s, 20 // page]), 20 % page, 0, 1])
    out, lse = B.decode_attention(q, kc, vc, _i(table), _i(lens))
    for s, (k, v) in enumerate(parts):
        want, wl = _weighed(_np(q)[s], k, v, dim ** -0.5)
        g = heads // kv
        spread = np.repeat(np.where(np.isfinite(v), np.abs(v), 0).max(axis=0), g, axis=0)
        # weights as in _attention, with scores of at most 300 in size where they count: their bound there, and of the mean of the values
        z = np.einsum("hd,nhd->hn", _np(q)[s], np.repeat(np.where(np.abs(k) < 100, np.abs(k), 0), g, axis=1)).max() * dim ** -0.5
        dw = ((dim + 4) * U + 4 * U) * z + 2.0 ** -15 + (len(k) + 8) * U
        _check_infinite(out[s], want, lambda w: 2 * dw * spread + (2.0 ** -8 * (np.abs(w) + 2 * dw * spread) if kind == "bf16" else 0))
        _check(lse[s], wl, dw + 4 * U * np.abs(wl))


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,heads,kv", [([700, 3], 4, 1), ([6000], 2, 2), ([64] * 50, 2, 2), ([2000], 8, 1)])
def test_attention_of_the_largest_values(cuda, kind, reach, lens, heads, kv):
    """Values at half of the type's range: their mean is finite, whatever their sum is."""
    rng = _rng(kind, len(lens), heads)
    page, dim = 16, 64
    table, n_pages = _pages(rng, lens, page, width=reach // page)
    kc, vc = _pool(n_pages, page, kv, dim, kind, "slot", math.nan)
    parts = _fill(rng, lens, table, kc, vc, page)
    q = _t(rng.standard_normal((len(lens), heads, dim)), kind)
    big = 2.0 ** 127
    for s, n in enumerate(lens):
        j = np.arange(n)
        at = torch.from_numpy(table[s, j // page].astype(np.int64)).cuda(), torch.from_numpy(j % page).cuda()
        sign = np.where(np.arange(dim) % 3 == 0, -1.0, 1.0) * np.ones((n, kv, dim))
        sign[:, :, 1::5] = rng.integers(0, 2, (n, kv, len(range(1, dim, 5)))) * 2.0 - 1
        vc[at] = (_t(sign) * big).to(vc.dtype)
        parts[s][1] = sign
    out, lse = B.decode_attention(q, kc, vc, _i(table), _i(lens))
    assert torch.isfinite(out).all()
    for s, (k, v) in enumerate(parts):
        want, wl, tol, tl = _attention(_np(q)[s], k, v, dim ** -0.5)
        _check(_np(out[s]) / big, want, tol + ((np.abs(want) + tol) * 2.0 ** -8 if kind == "bf16" else 0))
        _check(lse[s], wl, tl + 2.0 ** -20)


@pytest.mark.parametrize("change", [
    dict(page_stride=256, slot_stride=256), dict(page_stride=16 * 256 - 64), dict(slot_stride=64, head_stride=64),
    dict(slot_stride=192), dict(head_stride=16 * 64, slot_stride=64, page_stride=4096 - 64), dict(page_stride=64, slot_stride=64 * 31, head_stride=64 * 31 * 16)])
def test_append_into_dimensions_on_top_of_one_another_is_refused(lib, change):
    """Strides of a head and more each, but together two indices for one address."""
    assert lib.gpt_kv_append(ctypes.byref(_cache(**change)), ctypes.byref(_append()), None) == -1
    assert "smaller" in lib.gpt_last_error(None).decode()


@pytest.mark.parametrize("row,head", [(64, 64), (448, 64), (64, 128), (512, 512)])
def test_outputs_on_top_of_one_another_are_refused(lib, row, head):
    assert lib.gpt_kv_append(ctypes.byref(_cache()), ctypes.byref(_append(qo_row=row, qo_head=head)), None) == -1
    assert "smaller" in lib.gpt_last_error(None).decode()
    assert lib.gpt_decode_attention(ctypes.byref(_cache()), ctypes.byref(_attend(out_row=row, out_head=head)), None) == -1
    assert "smaller" in lib.gpt_last_error(None).decode()


@pytest.mark.parametrize("change", [dict(qo_row=1024), dict(qo_head=128, qo_row=1024)])
def test_queries_in_place_with_other_strides_are_refused(lib, change):
    args = {"q": FAKE, "q_out": FAKE, **change}
    assert lib.gpt_kv_append(ctypes.byref(_cache()), ctypes.byref(_append(**args)), None) == -1
    assert "strides" in lib.gpt_last_error(None).decode()


@pytest.mark.parametrize("cache,out", [
    (dict(page_stride=64, slot_stride=64 * 32, head_stride=64 * 32 * 16), (64, 192)),  # pages innermost; heads outermost
    (dict(head_stride=80, slot_stride=80 * 4 - 16, page_stride=(80 * 4 - 16) * 16), (72 * 8, 72)),  # gaps, but for the last
    (dict(page_stride=8, n_pages=1), (0, 64)), (dict(slot_stride=0, page_size=1), (512, 64))])
def test_layouts_that_do_not_overlap_are_taken(lib, cache, out):
    """Any order of the dimensions, gaps between them, any stride of a dimension of one entry: refused by nothing but the
    missing device (or, where there is one, not called)."""
    row, head = out
    n_seq = 1 if row == 0 else 3
    a, t = _append(q_out=FAKE + 65536, qo_row=row, qo_head=head, n_tokens=n_seq), _attend(out_row=row, out_head=head)
    c = _cache(n_seq=n_seq, **cache)
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real ones")
    assert lib.gpt_kv_append(ctypes.byref(c), ctypes.byref(a), None) == -2
    assert lib.gpt_decode_attention(ctypes.byref(c), ctypes.byref(t), None) == -2


def _small(dtype=torch.float32):
    z = lambda *s, t=dtype: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    i32 = torch.int32
    return dict(k=z(2, 4, 64), v=z(2, 4, 64), kc=z(8, 16, 4, 64), vc=z(8, 16, 4, 64), table=z(2, 4, t=i32) + torch.tensor([[0], [1]], dtype=i32, device="cuda"),
                at=z(2, t=i32), q=z(2, 8, 64), out=z(2, 8, 64), logits=z(3, 50), status=z(1, t=i32))


def _small_calls(x):
    return [("k", lambda: B.kv_append(x["k"], x["v"], x["kc"], x["vc"], x["table"], x["at"], q=x["q"], q_out=x["out"])),
            ("q", lambda: B.decode_attention(x["q"], x["kc"], x["vc"], x["table"], x["at"] + 1, out=x["out"])),
            ("logits", lambda: B.next_token(x["logits"], repetition=x["rep"], out=x["z"]))]


@gpu
@pytest.mark.parametrize("who", ["k", "v", "kc", "vc", "q", "out", "logits", "rep", "z"])
def test_tensors_that_require_gradients_are_refused_while_these_are_recorded(cuda, who):
    x = {**_small(), "rep": torch.ones(3, device="cuda"), "z": torch.zeros(3, 50, device="cuda")}
    x[who].requires_grad_()
    refused = 0
    for _, call in _small_calls(x):
        with torch.no_grad():
            call()
        try:
            call()
        except B.GptError as e:
            assert e.name == "INVALID_ARG" and "gradient" in str(e)
            refused += 1
    assert refused == {"kc": 2, "vc": 2, "q": 2, "out": 2}.get(who, 1)


@gpu
def test_written_tensors_are_new_versions(cuda):
    """Autograd finds a tensor that it has saved and a call has written since."""
    x = {**_small(), "rep": torch.ones(3, device="cuda"), "z": torch.zeros(3, 50, device="cuda")}
    for names, (_, call) in zip((("kc", "vc", "out"), ("out",), ("z",)), _small_calls(x)):
        before = {n: t._version for n, t in x.items()}
        call()
        assert {n for n, t in x.items() if t._version != before[n]} == set(names)
    w = torch.ones(64, device="cuda", requires_grad=True)
    loss = (x["kc"] * w).sum()
    B.kv_append(x["k"], x["v"], x["kc"][2:], x["vc"][2:], x["table"], x["at"])  # a view of the same memory
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        y = _small()
        B.kv_append(y["k"], y["v"], y["kc"], y["vc"], y["table"], y["at"], status=y["status"])
        B.decode_attention(y["q"], y["kc"], y["vc"], y["table"], y["at"] + 1, status=y["status"])
        B.next_token(y["logits"], status=y["status"])


@gpu
@pytest.mark.parametrize("rope", [-(1 << 32), -(1 << 33) + 2, 1 << 32, (1 << 32) + 64, -(1 << 63)])
def test_rope_dims_past_32_bits_are_refused(cuda, rope):
    x = _small()
    with pytest.raises(B.GptError) as e:
        B.kv_append(x["k"], x["v"], x["kc"], x["vc"], x["table"], x["at"], rope_dims=rope)
    assert e.value.name == "INVALID_ARG"


@gpu
def test_arguments_that_are_no_numbers(cuda):
    x = _small()
    for kw in (dict(rope_dims="8"), dict(rope_dims=1 << 70), dict(rope_dims=8, rope_base="x"), dict(stream=3)):
        with pytest.raises((TypeError, OverflowError, AttributeError)):
            B.kv_append(x["k"], x["v"], x["kc"], x["vc"], x["table"], x["at"], **kw)
    with pytest.raises(TypeError):
        B.decode_attention(x["q"], x["kc"], x["vc"], x["table"], x["at"], scale="x")


@gpu
@pytest.mark.parametrize("vocab", [60, 40000])
def test_next_token_prompt_lengths_out_of_range(cuda, vocab):
    """A negative prompt length is reported and counts as none; one past the history leaves nothing behind it, and is no error."""
    x = _token_inputs(_rng(vocab), 3, vocab, 20, "fp32")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x["pl"][:] = [20, 21, 1 << 30]
    _check_next(_run_next(x, "fp32", status=status), _next(**x))
    assert int(status) == 0
    x["pl"][:] = [3, -1, -(1 << 31)]
    got = _run_next(x, "fp32", status=status)
    x["pl"][:] = [3, 0, 0]
    _check_next(got, _next(**x))
    assert int(status) == B.STATUS_BAD_POS


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("page", [16, 24, 5])
@pytest.mark.parametrize("dim,heads", [(64, 4), (96, 10), (128, 6), (128, 34)])
def test_attention_bad_pages_and_lengths_in_every_form(cuda, kind, reach, page, dim, heads):
    """Bad pages at the start, inside and at the end of rows, rows of bad pages only, lengths below zero and past the
    table: both kernels, whole-group and other pages, exact and other heads."""
    rng = _rng(kind, reach, page, dim, heads)
    width = max(12, reach // page)
    lens = [5 * page + 3, 7 * page, 4 * page + 1, 3 * page, -3, 10 ** 9, 0, 6 * page - 1, 9 * page + 2, -(1 << 31)]
    there = [n if 0 <= n < 10 ** 9 else 0 for n in lens]
    table, n_pages = _pages(rng, [9 * page + 2] * len(lens), page, spare=2, width=width)
    bad = np.array([-1, n_pages, 1 << 30, -(1 << 31), (1 << 31) - 1])
    used = np.zeros((len(lens), width), dtype=bool)
    for s, n in enumerate(there):
        used[s, :-(-n // page)] = True
    used[5, [0, width - 1]] = True  # of the longest: the first page and the last that the table has
    table[5, width - 1] = table[5, 1]
    used[0, 0] = used[1, 3] = used[2, 4] = False
    used[3, :] = used[8, 4:7] = False
    table = np.where(used, table, bad[rng.integers(0, len(bad), table.shape)])
    kc, vc = _pool(n_pages, page, 2, dim, kind, "slot", math.nan)
    keep = []
    for s, n in enumerate(there):
        n = width * page if s == 5 else n
        rows = [j for i in np.nonzero(used[s])[0] for j in range(i * page, min((i + 1) * page, n))]
        j = np.array(rows, dtype=np.int64)
        at = torch.from_numpy(table[s, j // page].astype(np.int64)).cuda(), torch.from_numpy(j % page).cuda()
        kv = [_t(rng.standard_normal((len(j), 2, dim)), kind) for _ in range(2)]
        kc[at], vc[at] = kv
        keep.append([_np(x) for x in kv])
    q = _t(rng.standard_normal((len(lens), heads, dim)), kind)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = B.decode_attention(q, kc, vc, _i(table), _i(lens), status=status)
    assert int(status) == B.STATUS_BAD_PAGE | B.STATUS_BAD_POS
    for s, (k, v) in enumerate(keep):
        want, wl, tol, tl = _attention(_np(q)[s], k, v, dim ** -0.5)
        _check(out[s], want, tol + ((np.abs(want) + tol) * 2.0 ** -8 if kind == "bf16" else 0))
        if len(k):
            _check(lse[s], wl, tl)
        else:
            assert bool((lse[s] == -math.inf).all())
    # each kind of fault by itself, and no status word
    one = lambda rows, n: (B.decode_attention(q[rows], kc, vc, _i(table[rows]), _i(n), status=status.zero_())[0], int(status))  # noqa: E731
    assert one([7], [-1])[1] == B.STATUS_BAD_POS and one([0], [1])[1] == B.STATUS_BAD_PAGE
    got, bits = one([7], [6 * page - 1])
    assert bits == 0 and torch.equal(got[0], B.decode_attention(q[7:8], kc, vc, _i(table[7:8]), _i([6 * page - 1]))[0][0])
    again = B.decode_attention(q, kc, vc, _i(table), _i(lens))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@gpu
@pytest.mark.parametrize("reach", [0, 400000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,heads,kv", [([700, 3], 4, 2), ([5000], 4, 4), ([64] * 50, 2, 2)])
def test_attention_scores_that_are_no_numbers(cuda, kind, reach, lens, heads, kv):
    """A key of NaN, or a score of +infinity, makes its head NaN, lse too; the other heads and sequences do not see it."""
    rng = _rng(kind, reach, len(lens), heads)
    table, n_pages = _pages(rng, lens, 16, width=reach // 16)
    kc, vc = _pool(n_pages, 16, kv, 64, kind, "slot", math.nan)
    parts = _fill(rng, lens, table, kc, vc, 16)
    q = _t(np.abs(rng.standard_normal((len(lens), heads, 64))) + 0.1, kind)
    clean = B.decode_attention(q, kc, vc, _i(table), _i(lens))
    j = lens[0] // 2
    kc[int(table[0, j // 16]), j % 16, 0, 3] = math.nan
    last = lens[-1] - 1
    kc[int(table[-1, last // 16]), last % 16, kv - 1, 5] = math.inf
    out, lse = B.decode_attention(q, kc, vc, _i(table), _i(lens))
    gone = torch.zeros(len(lens), heads, dtype=torch.bool, device="cuda")
    gone[0, :heads // kv] = True
    gone[-1, heads - heads // kv:] = True
    assert torch.equal(torch.isnan(lse), gone) and torch.equal(torch.isnan(out).all(-1), gone) and torch.equal(torch.isnan(out).any(-1), gone)
    assert torch.equal(out[~gone], clean[0][~gone]) and torch.equal(lse[~gone], clean[1][~gone])
