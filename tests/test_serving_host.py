"""Serving operators without a GPU: the header's functions are exported and
bound, arguments are refused before anything is launched, sizes of the stored
forms, and calls run with their tensors' device current."""
import contextlib
import ctypes
import os
import re

import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tensor_scaled_fp8_amd import _lib, serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def test_header_functions_all_exported():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8lin_serve.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*[A-Za-z_][\w\s\*]*?\b(fp[48]_\w+)\s*\(", src, flags=re.M))
    assert len(names) == 14
    lib = tsf.load()
    for n in names:
        assert hasattr(lib, n) and n in _lib.SIGNATURES, n


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_tokens", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class Batch(ctypes.Structure):
    _fields_ = [("tables", ctypes.c_void_p), ("ld", ctypes.c_int64), ("table_pages", ctypes.c_int64),
                ("lengths", ctypes.c_void_p), ("starts", ctypes.c_void_p), ("sequences", ctypes.c_int64),
                ("tokens", ctypes.c_int64)]


class Rows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


OK = 4096                          # a 16-byte aligned address that is never read
CACHE = dict(k=OK, v=OK, scales=OK, pages=4, page_tokens=16, heads=2, head_dim=64)
BATCH = dict(tables=OK, ld=2, table_pages=2, lengths=OK, starts=None, sequences=3, tokens=3)
INV, UNS = _lib.FP8_ERR_INVALID, _lib.FP8_ERR_UNSUPPORTED


def calls(cache=CACHE, batch=BATCH, rows=(OK, 128, 64), **how):
    """(append, read, attention) with these arguments."""
    lib, r = tsf.load(), ctypes.byref
    c, b, x = Cache(**cache), Batch(**batch), Rows(*rows)
    freqs, rot, heads = how.get("freqs", OK), how.get("rot", 64), how.get("q_heads", 4)
    return (lib.fp8_cache_append(r(c), r(b), r(x), r(x), r(x), r(x), heads, freqs, rot, 0, None),
            lib.fp8_cache_read(r(c), r(b), r(x), r(x), None),
            lib.fp8_cache_attention(r(c), r(b), r(x), heads, how.get("scale", 1.0), how.get("cap", 0.0), how.get("window", 0), r(x),
                                    how.get("lse", OK), how.get("ws", OK), 1 << 40, None))


@pytest.mark.parametrize("change", [
    dict(k=None), dict(v=OK + 8), dict(scales=OK + 2), dict(pages=-1), dict(page_tokens=8), dict(page_tokens=48),
    dict(page_tokens=8192), dict(heads=0), dict(heads=2000), dict(head_dim=80), dict(head_dim=512)])
def test_caches_that_are_refused(change):
    assert calls(cache={**CACHE, **change}) == (INV,) * 3


@pytest.mark.parametrize("change", [
    dict(tables=None), dict(tables=OK + 2), dict(ld=-1), dict(table_pages=-1), dict(lengths=None), dict(lengths=OK + 1),
    dict(starts=OK + 2), dict(sequences=-1), dict(tokens=-1), dict(tokens=4), dict(sequences=2)])
def test_batches_that_are_refused(change):
    assert calls(batch={**BATCH, **change}) == (INV,) * 3


def test_rows_and_numbers_that_are_refused():
    assert calls(rows=(None, 128, 64)) == (INV,) * 3
    assert calls(rows=(OK + 1, 128, 64)) == (INV,) * 3
    assert calls(batch={**BATCH, "starts": OK, "tokens": 1 << 40}) == (UNS,) * 3
    assert calls(batch={**BATCH, "sequences": 1 << 30, "tokens": 1 << 30}) == (UNS,) * 3
    bad = dict(batch={**BATCH, "sequences": 1 << 30, "tokens": 1 << 30})       # nothing is launched whatever else is right
    for rot in (-16, 8, 80, 128):
        assert calls(rot=rot, **bad)[0] == INV
    assert calls(freqs=None, **bad)[0] == INV and calls(freqs=OK + 2, **bad)[0] == INV
    assert calls(q_heads=3, **bad)[::2] == (INV, INV)
    nan, inf = float("nan"), float("inf")
    for how in (dict(scale=nan), dict(scale=inf), dict(cap=-1.0), dict(cap=nan), dict(cap=inf), dict(cap=1e-20), dict(cap=1e20), dict(scale=-1e20), dict(window=-1), dict(lse=OK + 2),
                dict(ws=OK + 8)):
        assert calls(**how, **bad)[2] == INV, how
    lib, r = tsf.load(), ctypes.byref
    assert lib.fp8_cache_append(None, None, None, None, None, None, 0, None, 0, 0, None) == INV
    assert lib.fp8_cache_read(r(Cache(**CACHE)), None, None, None, None) == INV
    assert lib.fp8_cache_attention_workspace_bytes(None, None, 4) == 0


def test_sizes():
    lib = tsf.load()
    assert lib.fp8_cache_codes_bytes(3, 64, 8, 128) == 3 * 64 * 8 * 128
    assert lib.fp8_cache_scales_bytes(3, 64, 8, 128) == 3 * 4 * 8 * 2
    assert lib.fp8_cache_codes_bytes(3, 40, 8, 128) == lib.fp8_cache_scales_bytes(3, 64, 0, 128) == 0
    assert lib.fp4_codes_bytes(512, 16) == 4096 and lib.fp4_scales_bytes(512, 16) == 256
    assert lib.fp4_codes_bytes(513, 17) == 4 * 4096 and lib.fp4_codes_bytes(0, 5) == lib.fp4_codes_bytes(-1, 5) == 0


def plan(tokens, sequences, q_heads, heads, d, starts=True, table_pages=64):
    rows, form = ctypes.c_int(), ctypes.c_int()
    c, b = Cache(**{**CACHE, "heads": heads, "head_dim": d}), Batch(**{**BATCH, "tokens": tokens, "sequences": sequences,
                                                                      "starts": OK if starts else None, "table_pages": table_pages})
    assert tsf.load().fp8_cache_attention_plan(ctypes.byref(c), ctypes.byref(b), q_heads, ctypes.byref(rows),
                                               ctypes.byref(form)) == 0
    return rows.value, form.value


def test_attention_forms():
    """The sizes that the GPU tests take reach every form."""
    from tests.test_gpu_cache_attention_forms import CASES, SHARES, TILES, ROWS
    seen = {}
    for form, heads, hq, d, lens, new in CASES:
        got = plan(sum(new), len(new), hq, heads, d)
        assert got[1] == form, (heads, hq, d, got)
        seen.setdefault(form, set()).add((d, got[0]))
    wide = {(64, 64), (128, 64), (256, 32)}
    assert seen[TILES] == seen[ROWS] == wide and seen[SHARES] == wide | {(64, 32), (128, 32), (64, 16), (128, 16), (256, 16)}
    assert plan(0, 3, 4, 2, 64) == (0, 0) and plan(5, 5, 4, 2, 64, starts=False) == (16, SHARES)
    lib, r = tsf.load(), ctypes.c_int()
    assert lib.fp8_cache_attention_plan(None, None, 4, ctypes.byref(r), ctypes.byref(r)) == INV
    bad = Batch(**{**BATCH, "starts": OK, "tokens": 1 << 40})
    assert lib.fp8_cache_attention_plan(ctypes.byref(Cache(**CACHE)), ctypes.byref(bad), 4, ctypes.byref(r), ctypes.byref(r)) == UNS


def test_fp4_forms():
    """The sizes that the GPU tests take reach every form that any size up to 700 rows chooses."""
    from tests.test_gpu_fp4 import FORMS, blocks_of, is_exact

    def fp4_plan(M, K, N, exact):
        v = [ctypes.c_int() for _ in range(4)]
        assert tsf.load().fp4_linear_plan(M, K, N, exact, *map(ctypes.byref, v)) == 0
        return tuple(x.value for x in v)
    for form, (M, N) in FORMS.items():
        assert fp4_plan(M, blocks_of(form), N, is_exact(form)) == form
    seen = {fp4_plan(M, K, N, e) for M in (1, 2, 16, 17, 32, 33, 64, *range(65, 700, 13)) for K in (200, 4000) for e in (0, 1)
            for N in (1, 17, 300, 4096, 4097, 8193, *range(9000, 40000, 700))}
    assert seen <= set(FORMS), seen - set(FORMS)
    assert tsf.load().fp4_linear_plan(-1, 1, 1, 0, *[ctypes.byref(ctypes.c_int())] * 4) == INV
    assert tsf.load().fp4_linear_plan(1 << 40, 1, 1, 0, *[ctypes.byref(ctypes.c_int())] * 4) == UNS
    assert tsf.load().fp4_linear_plan(1, 1, 1, 0, None, None, None, None) == INV


def test_fp4_arguments_without_launch():
    lib = tsf.load()
    q, d, f = lib.fp4_quantize, lib.fp4_dequantize, lib.fp4_linear_fwd_cached
    for g, last in ((q, None), (d, None)):
        args = (lambda w=OK, ld=16, K=32, N=16, c=OK, s=OK: (w, ld, K, N, c, s) if g is q else (c, s, K, N, w, ld))
        for change in (dict(w=None), dict(w=OK + 1), dict(K=-1), dict(N=-1), dict(c=None), dict(c=OK + 8), dict(s=None),
                       dict(s=OK + 4), dict(ld=-1)):
            assert g(*args(**change), None) == INV, change
        assert g(*args(K=(1 << 20) + 1), None) == UNS
    assert d(OK, OK, 32, 16, OK, 8, None) == INV
    ok = dict(X=OK, ldx=32, M=20, K=32, N=16, c=OK, s=OK, exact=0, ws=OK, n=1 << 30, Y=OK)
    for change in (dict(X=None), dict(X=OK + 1), dict(M=-1), dict(ldx=-1), dict(c=None), dict(s=OK + 8), dict(ws=None),
                   dict(ws=OK + 8), dict(n=0), dict(Y=None)):
        assert f(*{**ok, **change}.values(), None) == INV, change
    assert f(*{**ok, "M": 1 << 40}.values(), None) == UNS
    assert f(*{**ok, "N": 1 << 40}.values(), None) == UNS


# ---- Python ------------------------------------------------------------------------------

def cache():
    return tsf.BlockKVCache(4, 16, 2, 64, device="cpu")


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_cache_sizes():
    c = tsf.BlockKVCache(5, 32, 3, 128, device="cpu")
    assert c.nbytes == 2 * 5 * 32 * 3 * 128 + 5 * 2 * 3 * 2 and not c.data.any()
    for bad in ((4, 8, 2, 64), (4, 24, 2, 64), (4, 8192, 2, 64), (4, 16, 0, 64), (4, 16, 2, 96), (-1, 16, 2, 64)):
        with pytest.raises(ValueError, match="no cache of"):
            tsf.BlockKVCache(*bad, device="cpu")


GOOD = dict(k=lambda: z(3, 2, 64), v=lambda: z(3, 2, 64), q=lambda: z(3, 4, 64), tables=lambda: z(3, 5, dtype=I32),
            lengths=lambda: z(3, dtype=I32), starts=lambda: None, freqs=lambda: torch.zeros(32), q_out=lambda: None)


def append(**change):
    a = {n: f() for n, f in GOOD.items()} | change
    return tsf.fp8_cache_append(cache(), a["k"], a["v"], a["tables"], a["lengths"], a["starts"], a["q"], a["freqs"], False, a["q_out"])


def attention(**change):
    a = {n: f() for n, f in GOOD.items()} | change
    return tsf.fp8_cache_attention(a["q"], cache(), a["tables"], a["lengths"], a["starts"],
                                   **{n: a[n] for n in ("scale", "softcap", "window", "out") if n in a})


BATCHES = [
    (dict(tables=z(3, 5, dtype=torch.int64)), "tables must be int32"), (dict(tables=z(2, 5, dtype=I32)), "tables must be"),
    (dict(tables=z(3, dtype=I32)), "tables must be"), (dict(tables=z(3, 10, dtype=I32)[:, ::2]), "contiguous rows"),
    (dict(lengths=z(3)), "lengths must be int32"), (dict(lengths=z(3, 1, dtype=I32)), "lengths must be 1-D"),
    (dict(lengths=z(6, dtype=I32)[::2]), "lengths must be 1-D"), (dict(starts=z(3, dtype=I32)), "starts must be"),
    (dict(starts=z(4)), "starts must be int32"), (dict(starts=z(8, dtype=I32)[::2]), "starts must be contiguous"),
    (dict(lengths=z(4, dtype=I32), tables=z(4, 5, dtype=I32)), "one row a sequence"),
    (dict(q=z(3, 3, 64)), "not a multiple"), (dict(q=z(3, 0, 64)), "not a multiple"), (dict(q=z(3, 4, 64, dtype=torch.float16)), "q must be"),
    (dict(q=z(3, 4, 128)), "q must be"), (dict(q=z(3, 64, 4).transpose(1, 2)), "contiguous last"), ({}, "device tensor")]


@pytest.mark.parametrize("change,said", BATCHES + [
    (dict(k=z(3, 1, 64)), "k must be"), (dict(v=z(4, 2, 64)), "v must be"), (dict(k=z(3, 128)), "k must be"),
    (dict(v=z(3, 2, 64, dtype=torch.float32)), "v must be bfloat16"), (dict(freqs=torch.zeros(20)), "multiple of 16"),
    (dict(freqs=torch.zeros(40)), "multiple of 16"), (dict(freqs=torch.zeros(32, dtype=torch.float64)), "float32"),
    (dict(freqs=torch.zeros(64)[::2]), "contiguous"), (dict(q=None, q_out=z(3, 4, 64)), "without q"),
    (dict(q_out=z(3, 2, 64)), "q_out must be"), (dict(q_out=z(1, 4, 64).expand(3, 4, 64)), "expanded")])
def test_appends_that_are_refused(change, said):
    with pytest.raises(ValueError, match=said):
        append(**change)


@pytest.mark.parametrize("change,said", BATCHES + [
    (dict(q=z(4, 4, 64)), "one row a sequence"), (dict(scale=float("nan")), "scale must be"), (dict(scale=1e39), "scale must be"),
    (dict(scale=-1e20), "scale must be"), (dict(softcap=1e-20), "softcap must be"), (dict(softcap=1e20), "softcap must be"),
    (dict(softcap=-1.0), "softcap must be"), (dict(softcap=float("inf")), "softcap must be"), (dict(window=-1), "window must be"),
    (dict(window=2 ** 31), "window must be"), (dict(out=z(3, 4, 64, dtype=torch.float32)), "out must be"),
    (dict(out=z(3, 1, 64).expand(3, 4, 64)), "expanded")])
def test_attentions_that_are_refused(change, said):
    with pytest.raises(ValueError, match=said):
        attention(**change)


def test_reads_that_are_refused():
    t, n = z(3, 5, dtype=I32), z(3, dtype=I32)
    for args, said in (((t, n, z(4, dtype=I32)), "tokens"), ((t, n, None, 4), "one row a sequence"),
                       ((t, n, None, -1), "negative"), ((t, n, None, 3, z(3, 2, 128)), "k must be"),
                       ((t, n, None, 3, None, z(3, 1, 64).expand(3, 2, 64)), "expanded"), ((t, n), "device tensor")):
        with pytest.raises(ValueError, match=said):
            tsf.fp8_cache_read(cache(), *args)


def test_gradients_are_refused():
    for name in ("k", "v", "q", "freqs"):
        with pytest.raises(NotImplementedError, match=f"{name} wants a gradient"):
            append(**{name: GOOD[name]().requires_grad_()})
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
            append(**{name: GOOD[name]().requires_grad_()})
    with pytest.raises(NotImplementedError, match="q wants a gradient"):
        attention(q=z(3, 4, 64).requires_grad_())
    w = tsf.FP4Tensor(torch.zeros(4096 + 256, dtype=U8), 512, 16)
    with pytest.raises(NotImplementedError, match="X wants a gradient"):
        tsf.fp4_linear_fwd_cached(z(2, 512).requires_grad_(), w)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(z(2, 512), z(2, 512))
        with pytest.raises(NotImplementedError, match="X wants a gradient"):
            tsf.fp4_linear_fwd_cached(dual, w)


def test_fp4_that_is_refused():
    with pytest.raises(ValueError, match="4352 contiguous bytes"):
        tsf.FP4Tensor(torch.zeros(4096, dtype=U8), 512, 16)
    with pytest.raises(ValueError, match="contiguous bytes"):
        tsf.FP4Tensor(torch.zeros(0, dtype=U8), -1, 16)
    w = tsf.FP4Tensor(torch.zeros(4352, dtype=U8), 512, 16)
    for args, said in (((z(2, 500), w), "does not go with"), ((z(2, 512, dtype=torch.float16), w), "X must be bfloat16"),
                       ((z(512), w), "X must be 2-D"), ((z(512, 2).t(), w), "contiguous rows"),
                       ((z(2, 512), w, z(2, 15)), "Y must be contiguous"), ((z(2, 512), w, z(16, 2).t()), "Y must be contiguous"),
                       ((z(2, 512), w), "device tensor")):
        with pytest.raises(ValueError, match=said):
            tsf.fp4_linear_fwd_cached(*args)
    square, x = tsf.FP4Tensor(torch.zeros(4 * 4352 * 8, dtype=U8), 512, 512), z(2 * 512 + 1)
    for y in (x[:-1], x[1:]):
        with pytest.raises(ValueError, match="overlap"):
            tsf.fp4_linear_fwd_cached(x[:-1].view(2, 512), square, y.view(2, 512))
    with pytest.raises(ValueError, match="device tensor"):
        w.dequantize()
    for bad, said in ((z(2, 3, 4), "2-D"), (z(4, 4, dtype=torch.float32), "bfloat16"), (z(4, 4), "device tensor")):
        with pytest.raises(ValueError, match=said):
            tsf.prepare_fp4_weight(bad)
    for args in ((z(8, 5 * 64), z(128, 8), 2, 1, 64), (z(8, 4 * 64), z(64, 8), 2, 1, 64)):
        with pytest.raises(ValueError, match="shape mismatch"):
            tsf.InferenceAttention(*args)
    with pytest.raises(ValueError, match="4 or 8 bits"):
        tsf.InferenceAttention(z(8, 4 * 64), z(128, 8), 2, 1, 64, bits=5)
    for freqs in (torch.zeros(32, dtype=torch.float64), torch.zeros(1, 32)):
        with pytest.raises(ValueError, match="freqs must be float32"):
            tsf.InferenceAttention(z(8, 4 * 64), z(128, 8), 2, 1, 64, freqs=freqs)


def test_calls_run_on_their_tensors_device(monkeypatch):
    """The library, the devices and the tensors' device are stand-ins: a launch goes to the current device."""
    from tensor_scaled_fp8_amd import binding
    current, seen = [0], []

    class Elsewhere(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1

    class Compiled:
        def __getattr__(self, name):
            def call(*args):
                seen.append((name, current[-1]))
                return z(4, 4), None
            return call

    @contextlib.contextmanager
    def device(index):
        current.append(index)
        yield
        current.pop()
    monkeypatch.setattr(serving, "_binding", Compiled)
    monkeypatch.setattr(binding, "_current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    c = cache()
    c.data = c.data.as_subclass(Elsewhere)
    x = z(3, 2, 64).as_subclass(Elsewhere)
    t, n = GOOD["tables"](), GOOD["lengths"]()
    w = tsf.FP4Tensor(torch.zeros(4352, dtype=U8).as_subclass(Elsewhere), 512, 16)
    tsf.fp8_cache_append(c, x, x, t, n)
    tsf.fp8_cache_read(c, t, n)
    tsf.fp8_cache_attention(x, c, t, n)
    tsf.fp4_linear_fwd_cached(z(2, 512).as_subclass(Elsewhere), w)
    w.dequantize()
    monkeypatch.setattr(serving, "FP4Tensor", lambda *a: None)
    tsf.prepare_fp4_weight(z(512, 16).as_subclass(Elsewhere))
    assert seen == [(e, 1) for e in ("cache_append", "cache_read", "cache_attention", "fp4_serve", "fp4_restore", "fp4_store")]
