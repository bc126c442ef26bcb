"""Attention over the paged 8-bit cache in each of the forms that its sizes
choose (equal shares, a tile of rows a workgroup, a tile of rows a wave; each
number of rows), on prompts and drafted tokens: sampled rows against the
definition in 64 bits at the values that the cache holds (read back, which
other tests hold to the definition)."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.serve_util import tolerance
from tests.test_gpu_cache import draw, host, ints, tables_of, up

pytestmark = pytest.mark.gpu

SHARES, TILES, ROWS = 0, 1, 2
# form, key heads, query heads, head_dim, lengths, new tokens
CASES = [
    (SHARES, 2, 8, 64, [900, 70, 5], [4, 4, 4]), (SHARES, 1, 5, 128, [700, 33], [3, 2]), (SHARES, 2, 6, 256, [300, 45], [2, 3]),
    (SHARES, 2, 8, 64, [700, 70, 9], [8, 8, 8]), (SHARES, 1, 6, 128, [400, 333], [5, 4]), (SHARES, 3, 3, 256, [350, 90], [20, 30]),
    (SHARES, 2, 4, 64, [300, 1000], [300, 20]), (SHARES, 1, 8, 128, [260, 131], [40, 131]), (SHARES, 1, 3, 256, [150], [150]),
    (TILES, 128, 128, 64, [130, 64, 97, 300], [130, 64, 97, 200]), (TILES, 64, 192, 128, [140, 250, 60], [140, 250, 60]),
    (TILES, 64, 128, 256, [140, 77, 210], [140, 77, 200]),
    (ROWS, 128, 512, 64, [300, 171, 65], [300, 171, 65]), (ROWS, 64, 512, 128, [200, 120, 97, 31], [200, 120, 97, 31]),
    (ROWS, 64, 256, 256, [150, 99, 190], [150, 99, 100]),
    # 256 tiles and more: three workgroups a CU share them
    (SHARES, 64, 128, 64, [600, 70, 5, 33, 1000], [2, 2, 2, 2, 2]), (SHARES, 40, 80, 128, [700, 33, 5, 1, 90, 300, 64], [1] * 7)]


def reference(q, k, v, pos, there, softcap, window):
    """q [d] at pos over k, v [tokens, d]: (out, lse, mass, size)."""
    j = np.arange(len(k))
    seen = there & (j <= pos) & ((j > pos - window) if window else True)
    if not seen.any():
        return np.zeros(len(q)), -np.inf, np.zeros(len(q)), 0.0
    s = k[seen] @ q / np.sqrt(len(q))
    size = np.max(np.abs(k[seen]) @ np.abs(q)) / np.sqrt(len(q))
    if softcap:
        s = softcap * np.tanh(s / softcap)
    e = np.exp(s - s.max())
    return e @ v[seen] / e.sum(), s.max() + np.log(e.sum()), e @ np.abs(v[seen]) / e.sum(), size


@pytest.mark.parametrize("how", [dict(), dict(softcap=20.0, window=70)], ids=["plain", "cap-window"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_form(case, how):
    form, heads, hq, d, lens, new = CASES[case]
    g = np.random.Generator(np.random.PCG64(case))
    page = (16, 64, 128)[case % 3]
    tables, pages = tables_of(g, lens, page)
    if case % 2 and lens[0] > page:
        tables[0, 0] = -1                        # a page that is not there
    all_starts, starts = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(new)])
    cache = tsf.BlockKVCache(pages, page, heads, d, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(case)
    k, v = (torch.randn((int(all_starts[-1]), heads, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = (torch.randn((int(starts[-1]), hq, d), generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
    tsf.fp8_cache_append(cache, k, v, ints(tables), ints(lens), ints(all_starts))
    rk, rv = tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints(all_starts), int(all_starts[-1]))
    out, lse = tsf.fp8_cache_attention(q, cache, ints(tables), ints(lens), ints(starts), lse=True, **how)
    again = tsf.fp8_cache_attention(q, cache, ints(tables), ints(lens), ints(starts), **how)
    assert torch.equal(out, again)
    place = q.clone()                            # in place
    assert tsf.fp8_cache_attention(place, cache, ints(tables), ints(lens), ints(starts), out=place, **how) is place
    assert torch.equal(out, place)
    out, lse, rk, rv, q = host(out), lse.cpu().numpy().astype(np.float64), host(rk), host(rv), host(q)
    # every sequence's first and last row, and others, of the first and last head and others
    for i, (length, n) in enumerate(zip(lens, new)):
        there = np.array([tables[i, p // page] >= 0 for p in range(length)])
        for t in sorted({0, n - 1, n // 2, *g.integers(0, n, 6).tolist()}):
            for h in sorted({0, hq - 1, *g.integers(0, hq, 3).tolist()}):
                rows = slice(all_starts[i], all_starts[i + 1])
                kv = h // (hq // heads)
                want, wl, mass, size = reference(q[starts[i] + t, h], rk[rows, kv], rv[rows, kv], length - n + t, there,
                                                 how.get("softcap", 0.0), how.get("window", 0))
                got = out[starts[i] + t, h]
                # sums of rounded weights: 2^-8 more of what they weigh
                tol = tolerance(want[None], mass[None], np.array([size]), d)[0] + 2.0 ** -8 * np.abs(want)
                assert (np.abs(got - want) <= tol).all(), (i, t, h, np.abs(got - want).max(), got[:4], want[:4])
                err = size * ((d + 10) * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -8 + 2.0 ** -22 * abs(wl if np.isfinite(wl) else 0)
                assert got_near(lse[starts[i] + t, h], wl, err), (i, t, h, lse[starts[i] + t, h], wl)


def got_near(got, want, err):
    return got == want or abs(got - want) <= err


@pytest.mark.parametrize("case", [c for c in range(len(CASES)) if CASES[c][0] != SHARES])
def test_nan_and_padding(case):
    """A NaN value in the middle of a prompt reaches its own head's queries from its token on; rows behind the last
    sequence stay as they were."""
    form, heads, hq, d, lens, new = CASES[case]
    tables, pages = tables_of(np.random.Generator(np.random.PCG64(case)), lens, 32)
    all_starts, starts = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(new)])
    cache = tsf.BlockKVCache(pages, 32, heads, d, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(case)
    k, v = (torch.randn((int(all_starts[-1]), heads, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((int(starts[-1]) + 5, hq, d), generator=gen, device="cuda").to(torch.bfloat16)
    t, h, G = lens[0] - new[0] + 37, heads - 1, hq // heads
    v[t, h, 11] = float("nan")
    tsf.fp8_cache_append(cache, k, v, ints(tables), ints(lens), ints(all_starts))
    out = torch.full((int(starts[-1]) + 5, hq, d), 4.0, dtype=torch.bfloat16, device="cuda")
    tsf.fp8_cache_attention(q, cache, ints(tables), ints(lens), ints(starts), out=out)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[37:new[0], h * G:(h + 1) * G, 11] = True
    assert torch.equal(torch.isnan(out), nan) and (out[int(starts[-1]):] == 4).all()
