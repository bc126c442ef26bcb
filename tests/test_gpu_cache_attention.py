"""Attention over the paged 8-bit cache against the definition in 64 bits, at
the values that the cache holds."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.serve_util import Model, attend, tolerance
from tests.test_gpu_cache import draw, host, ints, tables_of, up

pytestmark = pytest.mark.gpu


def filled(g, lens, heads, d, page, k=None, v=None, tables=None, pages=None):
    """A cache and its model with sequences of these lengths."""
    if tables is None:
        tables, pages = tables_of(g, lens, page)
    starts = np.concatenate([[0], np.cumsum(lens)])
    k = draw(g, (int(starts[-1]), heads, d), 1) if k is None else k
    v = draw(g, (int(starts[-1]), heads, d), 1) if v is None else v
    cache, model = tsf.BlockKVCache(pages, page, heads, d, device="cuda"), Model(pages, page, heads, d)
    tsf.fp8_cache_append(cache, up(k), up(v), ints(tables), ints(lens), ints(starts))
    model.append(k, v, tables, lens, starts)
    return cache, model, tables


def compare(q, cache, model, tables, lens, starts=None, **how):
    q = host(up(q))                      # what the kernel is given
    out, lse = tsf.fp8_cache_attention(up(q), cache, ints(tables), ints(lens), None if starts is None else ints(starts), lse=True,
                                       **how)
    want, wl, mass, size = attend(q, model, tables, lens, starts, **how)
    got = host(out)
    assert got.shape == want.shape
    nan = np.isnan(want)
    bad = ~((np.abs(got - want) <= tolerance(want, mass, size, q.shape[2])) | (nan & np.isnan(got)))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
    # lse: the scores' error, and the logarithm of a sum of weights that are 2^-18 off
    got = lse.cpu().numpy().astype(np.float64)
    err = size * ((q.shape[2] + 10) * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -17 + 2.0 ** -22 * np.abs(np.where(np.isfinite(wl), wl, 0))
    with np.errstate(invalid="ignore"):
        ok = (np.abs(got - wl) <= err) | (got == wl) | (np.isnan(wl) & np.isnan(got))
    assert ok.all(), (np.argwhere(~ok)[:4], got[~ok][:4], wl[~ok][:4])
    return out


@pytest.mark.parametrize("heads,hq,d,page,lens", [
    (1, 1, 128, 16, [1]), (1, 1, 64, 16, [2, 1]), (2, 8, 128, 32, [15, 16, 17, 33]), (8, 64, 128, 64, [100, 1, 257]),
    (2, 2, 256, 16, [31, 64, 129]), (1, 16, 128, 256, [500]), (1, 17, 64, 64, [77, 300]), (3, 15, 128, 128, [1000, 5]),
    (1, 48, 256, 64, [140]), (1, 70, 64, 16, [99, 40]), (2, 6, 64, 4096, [4097, 1]), (4, 4, 128, 64, [2049, 3, 700])])
def test_one_token(heads, hq, d, page, lens):
    g = np.random.Generator(np.random.PCG64(hq * d + lens[0]))
    cache, model, tables = filled(g, lens, heads, d, page)
    compare(draw(g, (len(lens), hq, d), 1), cache, model, tables, lens)


@pytest.mark.parametrize("heads,hq,d,page,lens,new", [
    (1, 1, 128, 16, [20], [20]), (2, 4, 64, 32, [70, 33, 1], [70, 5, 1]), (1, 8, 128, 64, [130, 64], [33, 64]),
    (2, 2, 256, 16, [47, 20], [47, 0]), (1, 5, 128, 128, [200, 100], [3, 50]), (3, 3, 64, 64, [150], [150]),
    (2, 14, 128, 16, [37, 90, 12], [2, 11, 12]), (1, 32, 64, 16, [40], [9]), (1, 33, 128, 64, [65], [65])])
def test_several_tokens(heads, hq, d, page, lens, new):
    g = np.random.Generator(np.random.PCG64(hq * d + lens[0] + 7))
    cache, model, tables = filled(g, lens, heads, d, page)
    starts = np.concatenate([[0], np.cumsum(new)])
    compare(draw(g, (int(starts[-1]), hq, d), 1), cache, model, tables, lens, starts)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 40, 100, 10 ** 9])
@pytest.mark.parametrize("new", [1, 30])
def test_window(window, new):
    g = np.random.Generator(np.random.PCG64(window % 1000 + new))
    lens = [130, 1 if new == 1 else 31, 64]
    cache, model, tables = filled(g, lens, 2, 64, 16)
    starts = None if new == 1 else np.arange(4) * new
    compare(draw(g, (3 * new, 6, 64), 1), cache, model, tables, lens, starts, window=window)


@pytest.mark.parametrize("softcap,scale", [(50.0, None), (0.5, 1.0), (1e6, 0.3), (3.0, -0.1), (0.0, 0.0), (20.0, 4.0)])
def test_softcap_and_scale(softcap, scale):
    g = np.random.Generator(np.random.PCG64(int(softcap) % 1000))
    lens = [77, 200]
    cache, model, tables = filled(g, lens, 2, 128, 32)
    compare(draw(g, (5, 4, 128), 1), cache, model, tables, lens, [0, 3, 5], softcap=softcap, scale=scale)


def test_what_is_not_there():
    """Missing pages, padded sequences, lengths past the table, rows that see nothing, rows behind the last sequence."""
    g = np.random.Generator(np.random.PCG64(3))
    heads, d, page = 2, 128, 16
    lens = [60, 0, 40, -7, 100, 2, 33]
    new = [3, 1, 40, 2, 9, 5, 2]
    tables = np.array([[4, -1, 2, 0], [0] * 4, [7, 2 ** 31 - 1, 1, -1], [0] * 4, [3, 6, 5, 8], [9] + [-1] * 3, [-1] * 4],
                      dtype=np.int32)
    held = [max(n, 0) for n in lens]
    cache, model, _ = filled(g, held, heads, d, page, tables=tables, pages=10)
    starts = np.concatenate([[0], np.cumsum(new)])
    q = draw(g, (int(starts[-1]), 6, d), 1)
    compare(q, cache, model, tables, lens, starts)
    compare(q, cache, model, tables, lens, starts, window=20)
    more = np.concatenate([q, q[:3]])
    out = torch.full((len(more), 6, d + 3), 9.0, dtype=torch.bfloat16, device="cuda")
    tsf.fp8_cache_attention(up(more), cache, ints(tables), ints(lens), ints(starts), out=out[..., 2:d + 2])
    assert (out[..., :2] == 9).all() and (out[..., d + 2:] == 9).all() and (out[len(q):] == 9).all()
    want = tsf.fp8_cache_attention(up(q), cache, ints(tables), ints(lens), ints(starts))
    assert torch.equal(out[:len(q), :, 2:d + 2], want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_reaches_only_who_sees_it(d):
    """NaN in the keys and values of a token in the middle of a prompt, and in stale tokens behind the last one."""
    g = np.random.Generator(np.random.PCG64(d))
    n, heads = 70, 2
    k, v = draw(g, (n, heads, d), 1), draw(g, (n, heads, d), 1)
    v[41, 0, 5] = np.nan                 # one element of one head's value
    k[50, 1, d - 1] = np.nan             # a key: the whole score
    v[60:] = np.nan
    k[60:] = np.nan
    cache, model, tables = filled(g, [n], heads, d, 16, k, v)
    q = draw(g, (60, 4, d), 1)
    out = compare(q, cache, model, tables, [60], [0, 60])
    got = host(out)
    assert not np.isnan(got[:41]).any() and np.isnan(got[41:, :2, 5]).all() and np.isnan(got[50:, 2:]).all()
    assert np.isnan(got).sum() == 19 * 2 + 10 * 2 * d
    for length in (41, 42, 50, 51, 59):
        compare(q[:1], cache, model, tables, [length])
        compare(q[:1], cache, model, tables, [length], window=8)
    compare(q[:2], cache, model, tables, [44], [0, 2], window=2)


def test_extreme_scores():
    """Scores of thousands, one token far above the others at the end, rows of infinities and NaN in q."""
    g = np.random.Generator(np.random.PCG64(9))
    n, d = 200, 64
    k, v = draw(g, (n, 1, d), 1), draw(g, (n, 1, d), 1)
    q = draw(g, (6, 2, d), 1)
    k[190] = 8.0
    q[1] *= 300
    q[2] = 30.0
    q[3] *= 2.0 ** -60
    cache, model, tables = filled(g, [n], 1, d, 64, k, v)
    compare(q, cache, model, tables, [n], [0, 6])
    q[4, 0, 3] = np.nan
    out = host(tsf.fp8_cache_attention(up(q), cache, ints(tables), ints([n]), ints([0, 6])))
    assert np.isnan(out[4, 0]).all() and np.isfinite(np.delete(out.reshape(12, d), 8, axis=0)).all()
    q[4, 0, 3] = np.inf
    out = host(tsf.fp8_cache_attention(up(q), cache, ints(tables), ints([n]), ints([0, 6])))
    assert np.isnan(out[4, 0]).all() and np.isfinite(np.delete(out.reshape(12, d), 8, axis=0)).all()


@pytest.mark.parametrize("new,hq", [(1, 6), (40, 6), (40, 2)])
def test_largest_values_in_hidden_places(new, hq):
    """bf16's largest values that a window or the order of tokens hides, and codes that an earlier sequence left behind the
    last token of a block whose scale is the largest, change no bit."""
    g = np.random.Generator(np.random.PCG64(60 + new + hq))
    heads, d, n, most = 2, 64, 100, 255 / 128 * 2.0 ** 127
    k, v, q = draw(g, (n, heads, d), 1), draw(g, (n, heads, d), 1), up(draw(g, (new, hq, d), 1))
    how, hidden = (dict(window=20), slice(64, 80)) if new == 1 else (dict(), slice(96, 100))
    outs = []
    for far in (False, True):
        if far:
            v[hidden] = most * np.sign(v[hidden])
        cache, model, tables = filled(np.random.Generator(np.random.PCG64(1)), [n], heads, d, 16, k, v)
        outs.append(tsf.fp8_cache_attention(q, cache, ints(tables), ints([n]), ints([0, new]), **how))
    rows = slice(0, new - (0 if new == 1 else 4))         # those that see none of them
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0][rows], outs[1][rows])
    # the same pages for a shorter sequence, with a value of the largest scale, and pages that are new
    v[33, :, 5] = most
    new = min(new, 35)
    fresh = tsf.BlockKVCache(cache.pages, 16, heads, d, device="cuda")
    for c in (cache, fresh):
        if c is cache:
            c.data[:c.pages * 16 * heads * d * 2] = 126                                 # the largest code everywhere
        tsf.fp8_cache_append(c, up(k[:35]), up(v[:35]), ints(tables), ints([35]), ints([0, 35]))
    outs = [tsf.fp8_cache_attention(q[:new], c, ints(tables), ints([35]), ints([0, new])) for c in (cache, fresh)]
    assert torch.equal(outs[0][..., :5], outs[1][..., :5]) and torch.isfinite(outs[0][..., :5]).all()


def test_strides_streams_and_equal_bits():
    g = np.random.Generator(np.random.PCG64(10))
    lens, hq, d = [300, 45], 8, 128
    cache, model, tables = filled(g, lens, 2, d, 16)
    q = up(draw(g, (7, hq, d), 1))
    a = (cache, ints(tables), ints(lens), ints([0, 4, 7]))
    want = tsf.fp8_cache_attention(q, *a)
    wide = torch.zeros((7, hq * d + 3), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:-2] = q.reshape(7, -1)
    assert torch.equal(tsf.fp8_cache_attention(wide[:, 1:-2].unflatten(1, (hq, d)), *a), want)
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((hq, 7, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert torch.equal(tsf.fp8_cache_attention(turned, *a, out=out), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = tsf.fp8_cache_attention(q, *a)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    wider = np.concatenate([tables, np.full((2, 500), -1, dtype=np.int32)], 1)
    y = tsf.fp8_cache_attention(q, cache, ints(wider)[:, :tables.shape[1] + 400], ints(lens), ints([0, 4, 7]))
    assert torch.equal(y, want)          # a table with room for more, and of another pitch


def test_attention_in_a_graph():
    """Lengths grow from replay to replay; two graphs of the same shapes replayed in turn."""
    g = np.random.Generator(np.random.PCG64(11))
    lens, hq, d = np.array([700, 30, 1]), 8, 64
    cache, model, tables = filled(g, [800, 100, 80], 2, d, 64)
    q, lengths, t = up(draw(g, (3, hq, d), 1)), ints(lens), ints(tables)
    tsf.fp8_cache_attention(q, cache, t, lengths)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(tsf.fp8_cache_attention(q, cache, t, lengths))
    for _ in range(4):
        lengths += 17
        q.copy_(up(draw(g, (3, hq, d), 1)))
        want = tsf.fp8_cache_attention(q, cache, t, lengths)
        for graph, out in zip(graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_empty_batches():
    cache = tsf.BlockKVCache(2, 16, 2, 64, device="cuda")
    t0 = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    none = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = tsf.fp8_cache_attention(none, cache, t0, ints([]), lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert tsf.fp8_cache_attention(none, cache, ints([[0], [1]]), ints([5, 6]), ints([0, 0, 0])).shape == (0, 4, 64)
    q = torch.ones((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full((2, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    tsf.fp8_cache_attention(q, cache, t0, ints([]), ints([0]), out=out)
    assert (out == 3).all()
    narrow = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    out, lse = tsf.fp8_cache_attention(q, cache, narrow, ints([5, 6]), lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
