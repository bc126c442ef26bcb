"""The serving operators where their sizes end: 4-bit matrices past 32 bits,
the longest sequences, the most heads, and reading into views."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.serve_util import Model, attend, tolerance
from tests.test_gpu_cache import draw, host, ints, same, tables_of, up
from tests.test_gpu_cache_attention import compare, filled
from tests.test_gpu_fp4 import check, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,exact", [(2, False), (40, False), (40, True), (70, True)])
def test_a_weight_past_32_bits(M, exact):
    """2^23 columns, the most: 6.9 GB of codes. Products of some columns, the last among them."""
    K, N = 1100, 1 << 23
    g = np.random.Generator(np.random.PCG64(M))
    W = torch.zeros((K, N), dtype=torch.bfloat16, device="cuda")
    at = [0, N // 2 - 16, N - 32]
    some = [weight(g, K, 32) for _ in at]
    for i, w in zip(at, some):
        W[:, i:i + 32] = up(w)
    q = tsf.prepare_fp4_weight(W)
    assert q.nbytes > 2 ** 32
    del W
    x = host(up(g.standard_normal((M, K))))
    y = tsf.fp4_linear_fwd_cached(up(x), q, exact=exact)
    for i, w in zip(at, some):
        check(x, w, y[:, i:i + 32])
    assert not y[:, 32:N // 2 - 16].any() and not y[:, N // 2 + 16:N - 32].any()


@pytest.mark.parametrize("exact", [False, True])
def test_rows_past_32_bits(exact):
    """2^22 rows, the most, of 1100: 2^32 elements of X and more."""
    M, K, N = 1 << 22, 1100, 40
    g = np.random.Generator(np.random.PCG64(3))
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    at = [0, M // 2 - 7, M - 20]
    some = [host(up(g.standard_normal((20, K)))) for _ in at]
    for i, x in zip(at, some):
        X[i:i + 20] = up(x)
    w = weight(g, K, N)
    y = tsf.fp4_linear_fwd_cached(X, tsf.prepare_fp4_weight(up(w)), exact=exact)
    for i, x in zip(at, some):
        check(x, w, y[i:i + 20])
    assert not y[20:M // 2 - 7].any() and not y[M // 2 + 13:M - 20].any()


@pytest.mark.parametrize("new,starts", [(1, False), (3, True), (40, True)])
def test_the_longest_lengths(new, starts):
    """A length of 2^31 - 1 over a table of a few pages: its queries see what the table holds, and through a window nothing."""
    g = np.random.Generator(np.random.PCG64(new))
    held = 96
    cache, model, tables = filled(g, [held], 2, 64, 32, tables=np.array([[2, 0, 1]], dtype=np.int32), pages=3)
    q = up(draw(g, (new, 4, 64), 1))
    s = ints([0, new]) if starts else None
    t, most = ints(tables), ints([2 ** 31 - 1])
    out, lse = tsf.fp8_cache_attention(q, cache, t, most, s, lse=True)
    for r in range(new):               # each as if it were at the last held token
        want, wl, mass, size = attend(host(q[r:r + 1]), model, tables, [held])
        assert (np.abs(host(out[r:r + 1]) - want) <= tolerance(want, mass, size, 64)).all(), r
        assert (np.abs(lse[r:r + 1].cpu().numpy() - wl) <= 1e-4).all()
    out, lse = tsf.fp8_cache_attention(q, cache, t, most, s, window=1000, lse=True)
    assert (out == 0).all() and (lse == -np.inf).all()
    before = cache.data.clone()
    k = up(draw(g, (new, 2, 64), 1))
    tsf.fp8_cache_append(cache, k, k, t, most, s, q=q, freqs=torch.full((32,), 0.5, device="cuda"))
    assert torch.equal(cache.data, before)
    assert not any(x.any() for x in tsf.fp8_cache_read(cache, t, most, s, new))


@pytest.mark.parametrize("heads,hq,d,starts", [(1024, 1024, 64, False), (1024, 16384, 64, True), (1, 16384, 64, False),
                                               (512, 4096, 256, False), (1, 3000, 128, True)])
def test_the_most_heads(heads, hq, d, starts):
    g = np.random.Generator(np.random.PCG64(hq))
    lens = [19, 2]
    tables, pages = tables_of(g, lens, 16)
    cache, model = tsf.BlockKVCache(pages, 16, heads, d, device="cuda"), Model(pages, 16, heads, d)
    for n in (18, 19):                 # whole, then a token a sequence
        new = [18, 1] if n == 18 else [1, 1]
        k, v, q = (draw(g, (sum(new), h, d), 1) for h in (heads, heads, hq))
        s = None if n == 19 and not starts else ints([0, new[0], sum(new)])
        at = [n, 1 if n == 18 else 2]
        tsf.fp8_cache_append(cache, up(k), up(v), ints(tables), ints(at), s)
        model.append(k, v, tables, at, [0, new[0], sum(new)])
    rk, rv = tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints([0, 19, 21]), 21)
    wk, wv = model.read(tables, lens, [0, 19, 21])
    same(host(rk), wk)
    same(host(rv), wv)
    compare(q, cache, model, tables, lens, [0, 1, 2] if starts else None)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_reading_into_views(d):
    """Keys and values beside each other at 2-byte alignment, and with the heads outermost; nothing else is written."""
    g = np.random.Generator(np.random.PCG64(d))
    lens, heads = [37, 16, 5], 3
    cache, model, tables = filled(g, lens, heads, d, 16)
    a, starts = (ints(tables), ints(lens)), [0, 20, 21, 26]
    wk, wv = model.read(tables, lens, starts)
    wide = torch.full((30, heads, 2, d + 1), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = wide[:, :, 0, 1:], wide[:, :, 1, 1:]
    got = tsf.fp8_cache_read(cache, *a, ints(starts), 30, k, v)
    assert got[0].data_ptr() == k.data_ptr() and got[1].data_ptr() == v.data_ptr()
    same(host(k[:26]), wk)
    same(host(v[:26]), wv)
    assert (wide[26:] == 7).all() and (wide[..., 0] == 7).all()
    both = torch.full((2 * heads, 30, d), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    tsf.fp8_cache_read(cache, *a, ints(starts), 30, both[:, :heads], both[:, heads:])
    same(host(both[:26, :heads]), wk)
    same(host(both[:26, heads:]), wv)
    assert (both[26:] == 7).all()
