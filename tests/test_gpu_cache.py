"""The paged 8-bit cache: appended and read back against the definition in 64
bits, exactly (codes are the nearest to the rotated keys; read-back values are
exact in bf16)."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import BF16_HALF, to_bf16
from tests.serve_util import Model, rotate

pytestmark = pytest.mark.gpu


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def same(got, want):
    """Equal, NaN with NaN."""
    assert got.shape == want.shape
    bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def tables_of(g, lens, page, extra=1):
    """Shuffled pages; a table of one column more than the longest needs, -1 where there is no page."""
    need = [-(-n // page) for n in lens]
    order = g.permutation(sum(need) + extra)
    t = np.full((len(lens), max(need, default=0) + 1), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, sum(need) + extra


def freqs_of(rot):
    return (10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)


def draw(g, shape, spread=3):
    return to_bf16(g.standard_normal(shape) * np.exp2(g.integers(-spread, spread + 1, size=(shape[0], 1, 1))))


# heads, query heads, d, page, rotated, interleaved, lengths after each call (a call's tokens are what is new)
CASES = [
    (1, 1, 128, 16, 128, False, [[1], [2], [3], [15], [16], [17], [50]]),
    (2, 8, 64, 32, 64, True, [[5, 0, 33], [6, 1, 34], [37, 1, 64], [38, 2, 65]]),
    (3, 3, 256, 64, 256, False, [[70, 16], [71, 31], [90, 32]]),
    (4, 20, 128, 128, 64, False, [[7, 200, 1, 129], [8, 201, 2, 130], [9, 217, 18, 131]]),
    (1, 5, 64, 16, 16, True, [[100], [117]]),
    (2, 2, 128, 256, 0, False, [[31, 300], [63, 301]]),
    (2, 4, 256, 16, 48, False, [[9, 17], [10, 40]]),
    (8, 64, 128, 64, 128, True, [[1000], [1001]]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_and_read(case):
    heads, hq, d, page, rot, inter, calls = CASES[case]
    g = np.random.Generator(np.random.PCG64(case))
    tables, pages = tables_of(g, calls[-1], page)
    cache, model = tsf.BlockKVCache(pages, page, heads, d, device="cuda"), Model(pages, page, heads, d)
    freqs = freqs_of(rot)
    before = np.zeros(len(calls[0]), dtype=int)
    for lens in calls:
        new = np.array(lens) - before
        starts = np.concatenate([[0], np.cumsum(new)])
        T = int(starts[-1])
        k, v, q = draw(g, (T, heads, d)), draw(g, (T, heads, d)), draw(g, (T, hq, d))
        one = (new == 1).all()
        args = (ints(tables), ints(lens), None if one else ints(starts))
        got = tsf.fp8_cache_append(cache, up(k), up(v), *args, q=up(q), freqs=torch.from_numpy(freqs).cuda() if rot else None,
                                   interleaved=inter)
        model.append(k, v, tables, lens, starts, freqs, inter)
        pos = np.concatenate([np.arange(b, n) for b, n in zip(before, lens)])
        want = rotate(q, pos, freqs, inter)
        # two products and a sum in 32 bits, cos and sin rounded to 32 bits: 4 roundings of 2^-24 of |a| + |b|
        size = np.abs(q) + np.abs(rotate_partner(q, rot, inter))
        assert (np.abs(host(got) - want) <= BF16_HALF * np.abs(want) + 2.0 ** -22 * size + 2.0 ** -133).all()
        before = np.array(lens)
        all_starts = np.concatenate([[0], np.cumsum(lens)])
        rk, rv = tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints(all_starts), int(all_starts[-1]))
        wk, wv = model.read(tables, lens, all_starts)
        same(host(rk), wk)
        same(host(rv), wv)
    last_k, last_v = tsf.fp8_cache_read(cache, ints(tables), ints(calls[-1]))
    wk, wv = model.read(tables, calls[-1])
    same(host(last_k), wk)
    same(host(last_v), wv)


def rotate_partner(x, rot, inter):
    """Each rotated element's partner."""
    y = np.array(x)
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = x[..., 1:rot:2], x[..., 0:rot:2]
    elif rot:
        y[..., :rot // 2], y[..., rot // 2:rot] = x[..., rot // 2:rot], x[..., :rot // 2]
    return y


def test_far_positions():
    """Angles in 64 bits: position 2^24 + 1 and beyond."""
    g = np.random.Generator(np.random.PCG64(50))
    d, page = 128, 4096
    lens = [2 ** 24 + 3, 2 ** 27 + 17]
    tables = np.full((2, 2 ** 27 // page + 1), -1, dtype=np.int32)
    tables[0, (2 ** 24) // page], tables[1, 2 ** 27 // page] = 1, 0
    starts = [0, 3, 20]
    k, v, q = (draw(g, (20, 2, d)) for _ in range(3))
    freqs = freqs_of(d)
    cache, model = tsf.BlockKVCache(2, page, 2, d, device="cuda"), Model(2, page, 2, d)
    tsf.fp8_cache_append(cache, up(k), up(v), ints(tables), ints(lens), ints(starts), freqs=torch.from_numpy(freqs).cuda())
    model.append(k, v, tables, lens, starts, freqs, False)
    rk, rv = tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints(starts), 20)
    wk, wv = model.read(tables, lens, starts)
    same(host(rk), wk)
    same(host(rv), wv)


def test_extremes():
    """Zeros first, subnormal and largest values, infinities and NaN, in blocks that grow token by token."""
    g = np.random.Generator(np.random.PCG64(51))
    d, page, n = 64, 16, 40
    x = draw(g, (n, 2, d), 20)
    x[0] = 0
    x[1] *= 2.0 ** -100
    x[17, 0, 3], x[18, 1, 5], x[19, 0, 0] = np.inf, -np.inf, np.nan
    x[33] = np.nan
    x[35, 1] = 3.3895e38 * np.sign(x[35, 1])
    x[36, 0] = 2.0 ** -133
    x = np.where(np.isfinite(x), to_bf16(np.where(np.isfinite(x), x, 0)), x)
    tables, pages = tables_of(g, [n], page)
    cache, model = tsf.BlockKVCache(pages, page, 2, d, device="cuda"), Model(pages, page, 2, d)
    for i in range(n):
        tsf.fp8_cache_append(cache, up(x[i:i + 1]), up(-x[i:i + 1]), ints(tables), ints([i + 1]))
        model.append(x[i:i + 1], -x[i:i + 1], tables, [i + 1])
    rk, rv = tsf.fp8_cache_read(cache, ints(tables), ints([n]), ints([0, n]), n)
    wk, wv = model.read(tables, [n], [0, n])
    for got, want in ((host(rk), wk), (host(rv), wv)):
        # a value next to bf16's largest is held as 1.875 2^127; below bf16's normal range read-back rounds
        assert np.nanmax(np.abs(want)) == 1.875 * 2.0 ** 127
        small = np.abs(want) < 2.0 ** -126
        same(np.where(small, 0, got), np.where(small, 0, want))
        assert (np.abs(got[small]) <= 2.0 ** -126).all()


def test_what_is_not_there():
    """No page, pages that are none, positions past the table, lengths of 0, negative ones, rows behind the last sequence:
    nothing else is written, reads give zeros."""
    g = np.random.Generator(np.random.PCG64(52))
    heads, d, page = 2, 128, 32
    lens = [70, 0, 40, -5, 100, 3]
    new = [70, 2, 40, 3, 30, 5]
    starts = np.concatenate([[0], np.cumsum(new)])
    T = int(starts[-1]) + 7
    tables = np.array([[4, -1, 2], [0, 0, 0], [7, 2 ** 31 - 1, 1], [0, 0, 0], [3, 6, 5], [1, -1, -1]], dtype=np.int32)
    cache, model = tsf.BlockKVCache(7, page, heads, d, device="cuda"), Model(7, page, heads, d)
    k, v, q = (draw(g, (T, heads, d)) for _ in range(3))
    freqs = freqs_of(128)
    wide = torch.full((T, heads, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[..., 3:d + 3]
    tsf.fp8_cache_append(cache, up(k), up(v), ints(tables), ints(lens), ints(starts), q=up(q),
                         freqs=torch.from_numpy(freqs).cuda(), q_out=out)
    model.append(k[:starts[-1]], v[:starts[-1]], tables, lens, starts, freqs, False)
    assert (wide[..., :3] == 7).all() and (wide[..., d + 3:] == 7).all() and (out[starts[-1]:] == 7).all()
    pos = np.concatenate([np.arange(max(n, 0) - m, max(n, 0)) for n, m in zip(lens, new)])
    want = rotate(q[:starts[-1]], pos, freqs, False)
    assert (np.abs(host(out)[:starts[-1]] - want) <= BF16_HALF * np.abs(want) + 2.0 ** -22 * 2 * np.abs(q).max()).all()
    ko, vo = (torch.full((T, heads, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints(starts), T, ko, vo)
    wk, wv = model.read(tables, lens, starts)
    same(host(ko)[:starts[-1]], wk)
    same(host(vo)[:starts[-1]], wv)
    assert (ko[starts[-1]:] == 5).all() and (vo[starts[-1]:] == 5).all()
    # every other byte of the cache is as it was: 0
    full = np.concatenate([[0], np.cumsum([7 * page])])
    rk, _ = tsf.fp8_cache_read(cache, ints(np.arange(7)[None]), ints([7 * page]), ints(full), 7 * page)
    wk, _ = model.read(np.arange(7)[None], [7 * page], full)
    same(host(rk), wk)


def test_views_and_in_place():
    """Views of one projection at 2-byte alignment, q rotated where it lies, heads outermost, the same bits."""
    g = np.random.Generator(np.random.PCG64(53))
    T, hq, hk, d = 37, 6, 2, 64
    x = up(draw(g, (T, hq + 2 * hk, d)))
    freqs = torch.from_numpy(freqs_of(64)).cuda()
    tables, pages = tables_of(g, [T], 16)
    a = (ints(tables), ints([T]), ints([0, T]))
    one, two, three = (tsf.BlockKVCache(pages, 16, hk, d, device="cuda") for _ in range(3))
    want = tsf.fp8_cache_append(one, x[:, hq:hq + hk].contiguous(), x[:, hq + hk:].contiguous(), *a, q=x[:, :hq].contiguous(),
                                freqs=freqs)
    wide = torch.zeros((T, (hq + 2 * hk) * d + 5), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:-4] = x.reshape(T, -1)
    y = wide[:, 1:-4].unflatten(1, (-1, d))
    q = y[:, :hq]
    got = tsf.fp8_cache_append(two, y[:, hq:hq + hk], y[:, hq + hk:], *a, q=q, freqs=freqs, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want) and torch.equal(one.data, two.data)
    assert torch.equal(y[:, hq:], x[:, hq:]) and (wide[:, 0] == 0).all() and (wide[:, -4:] == 0).all()
    z = x.transpose(0, 1).contiguous().transpose(0, 1)
    got = tsf.fp8_cache_append(three, z[:, hq:hq + hk], z[:, hq + hk:], *a, q=z[:, :hq], freqs=freqs,
                               q_out=torch.empty((hq, T, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1))
    assert torch.equal(got, want) and torch.equal(one.data, three.data)
    # without a rotation q is copied
    assert torch.equal(tsf.fp8_cache_append(three, z[:, hq:hq + hk], z[:, hq + hk:], *a, q=z[:, :hq]), x[:, :hq])


def test_past_32_bits():
    """A cache of more than 2^32 codes."""
    g = np.random.Generator(np.random.PCG64(54))
    page, heads, d = 4096, 8, 256
    pages = 2 ** 32 // (page * heads * d) + 2
    cache = tsf.BlockKVCache(pages, page, heads, d, device="cuda")
    tables, lens, starts = [[pages - 1], [0]], [20, 4096], [0, 20, 52]
    k, v = draw(g, (52, heads, d)), draw(g, (52, heads, d))
    tsf.fp8_cache_append(cache, up(k), up(v), ints(tables), ints(lens), ints(starts))
    small = Model(2, page, heads, d)
    small.append(k, v, [[1], [0]], lens, starts)
    rk, rv = tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints(starts), 52)
    wk, wv = small.read([[1], [0]], lens, starts)
    same(host(rk), wk)
    same(host(rv), wv)


def test_append_in_a_graph():
    """A captured decode step: lengths, tables and rows are what the device holds at the replay."""
    g = np.random.Generator(np.random.PCG64(55))
    B, heads, hq, d, page = 3, 2, 4, 128, 16
    tables = g.permutation(12).reshape(3, 4).astype(np.int32)
    freqs = torch.from_numpy(freqs_of(128)).cuda()
    caches = [tsf.BlockKVCache(12, page, heads, d, device="cuda") for _ in range(2)]
    t, lengths = ints(tables), ints([14, 0, 31])
    k, v, q = (torch.zeros((B, n, d), dtype=torch.bfloat16, device="cuda") for n in (heads, heads, hq))
    tsf.fp8_cache_append(caches[0], k, v, t, ints([0, 0, 0]), q=q, freqs=freqs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tsf.fp8_cache_append(caches[0], k, v, t, lengths, q=q, freqs=freqs)
        rk, rv = tsf.fp8_cache_read(caches[0], t, lengths)
    for _ in range(5):
        lengths += 1
        for x in (k, v, q):
            x.copy_(up(draw(g, tuple(x.shape))))
        want = tsf.fp8_cache_append(caches[1], k, v, t, lengths, q=q, freqs=freqs)
        wk, wv = tsf.fp8_cache_read(caches[1], t, lengths)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(caches[0].data, caches[1].data)
        assert torch.equal(rk, wk) and torch.equal(rv, wv)


def test_empty_batches():
    cache = tsf.BlockKVCache(2, 16, 2, 64, device="cuda")
    none = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    t0 = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    tsf.fp8_cache_append(cache, none, none, t0, ints([]), q=none)
    tsf.fp8_cache_append(cache, none, none, ints([[0], [1]]), ints([5, 6]), ints([0, 0, 0]))
    tsf.fp8_cache_append(cache, none.new_ones((3, 2, 64)), none.new_ones((3, 2, 64)), ints([[0], [1]]), ints([5, 6]), ints([0, 0, 0]))
    tsf.fp8_cache_append(cache, none.new_ones((3, 2, 64)), none.new_ones((3, 2, 64)), t0, ints([]), ints([0]))
    k, v = tsf.fp8_cache_read(cache, t0, ints([]))
    assert k.shape == v.shape == (0, 2, 64)
    assert (cache.data == 0).all()
    empty = tsf.BlockKVCache(0, 16, 2, 64, device="cuda")
    tsf.fp8_cache_append(empty, none.new_ones((1, 2, 64)), none.new_ones((1, 2, 64)), ints([[0]]), ints([1]))
    assert (tsf.fp8_cache_read(empty, ints([[0]]), ints([1]))[0] == 0).all()
