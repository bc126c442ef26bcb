"""Batches of several kinds in one call: decoded tokens over long caches beside
a prompt's chunk, and drafted tokens of many ragged sequences, in the forms
that the whole batch's sizes choose; sampled rows against the definition in 64
bits at the values that the cache holds. And starts that the contract bars."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.serve_util import tolerance
from tests.test_gpu_cache import host, ints, tables_of
from tests.test_gpu_cache_attention_forms import ROWS, SHARES, TILES, reference

pytestmark = pytest.mark.gpu


def ragged(n, lo, hi):
    """Lengths spread over [lo, hi] by their logarithm, in no order."""
    return [int(lo * (hi / lo) ** ((i * 37 % n) / max(1, n - 1))) for i in range(n)]


# form, rows a tile, key heads, query heads, d, lengths, new tokens
CASES = [
    (ROWS, 64, 8, 64, 128, ragged(63, 100, 9000) + [2500], [1] * 63 + [2048]),
    (TILES, 64, 8, 64, 128, [1200] + ragged(40, 50, 5000), [700] + [1] * 40),
    (SHARES, 64, 8, 64, 64, ragged(30, 60, 3000) + [256], [1] * 30 + [256]),
    (ROWS, 64, 8, 64, 64, ragged(200, 10, 3000), [5] * 200),
    (TILES, 32, 8, 32, 256, ragged(50, 20, 2000) + [600, 9], [1] * 50 + [600, 9])]


def made(case, page=64):
    _, _, heads, hq, d, lens, new = CASES[case]
    new = [min(a, b) for a, b in zip(new, lens)]
    g = np.random.Generator(np.random.PCG64(case))
    tables, pages = tables_of(g, lens, page)
    gen = torch.Generator(device="cuda").manual_seed(case)
    all_starts, starts = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(new)])
    k, v = (torch.randn((int(all_starts[-1]), heads, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = (torch.randn((int(starts[-1]), hq, d), generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
    cache = tsf.BlockKVCache(pages, page, heads, d, device="cuda")
    tsf.fp8_cache_append(cache, k, v, ints(tables), ints(lens), ints(all_starts))
    held = tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints(all_starts), len(k))
    return cache, q, held, tables, lens, new, all_starts, starts, g


@pytest.mark.parametrize("how", [dict(), dict(softcap=30.0, window=777)], ids=["plain", "cap-window"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_batch(case, how):
    _, _, heads, hq, d, _, _ = CASES[case]
    cache, q, (rk, rv), tables, lens, new, all_starts, starts, g = made(case)
    out, lse = tsf.fp8_cache_attention(q, cache, ints(tables), ints(lens), ints(starts), lse=True, **how)
    out, lse, q = host(out), lse.cpu().numpy().astype(np.float64), host(q)
    for i in sorted({0, 1, len(lens) // 2, len(lens) - 2, len(lens) - 1, int(np.argmax(lens)), int(np.argmin(lens))}):
        rows = slice(int(all_starts[i]), int(all_starts[i + 1]))
        k, v = host(rk[rows]), host(rv[rows])
        for t in sorted({0, new[i] - 1, int(g.integers(new[i]))}):
            for h in (0, hq - 1, int(g.integers(hq))):
                kv, r = h // (hq // heads), starts[i] + t
                want, wl, mass, size = reference(q[r, h], k[:, kv], v[:, kv], lens[i] - new[i] + t, np.ones(lens[i], dtype=bool),
                                                 how.get("softcap", 0.0), how.get("window", 0))
                # as for the forms: a weight in one bf16, and sums of rounded weights
                tol = tolerance(want[None], mass[None], np.array([size]), d)[0] + 2.0 ** -8 * np.abs(want)
                assert (np.abs(out[r, h] - want) <= tol).all(), (i, t, h, np.abs(out[r, h] - want).max())
                # a lane's sum of up to 9000 / 32 steps and 5 more, 2^-24 each; the rest as for the logarithms of prompts
                err = size * ((d + 10) * 2.0 ** -24 + 2.0 ** -20) + how.get("softcap", 0) * 2.0 ** -22 + \
                    (lens[i] / 32 + 5) * 2.0 ** -24 + 2.0 ** -22 * (1 + abs(wl)) + 17 * 2.0 ** -23
                assert abs(lse[r, h] - wl) <= err, (i, t, h, lse[r, h], wl)


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("bad", ["decreasing", "negative", "past the end", "from the middle"])
def test_starts_that_are_none(case, bad):
    """What is in bounds stays so: nothing outside of the batch's rows and pages is written, and the next call is right."""
    _, _, heads, hq, d, _, _ = CASES[case]
    cache, q, _, tables, lens, new, _, starts, g = made(case)
    t, n, T = ints(tables), ints(lens), len(q)
    want = tsf.fp8_cache_attention(q, cache, t, n, ints(starts))
    s = {"decreasing": np.concatenate([starts[::-1][:-1], [T]]), "negative": starts - 2 ** 31 // 2,
         "past the end": np.minimum(starts.astype(np.int64) * 1000, 2 ** 31 - 1), "from the middle": starts + T // 2}[bad]
    room = torch.full((T + 64, hq, d), 6.0, dtype=torch.bfloat16, device="cuda")
    out = room[32:T + 32]
    tsf.fp8_cache_attention(q, cache, t, n, ints(s), out=out)
    assert (room[:32] == 6).all() and (room[T + 32:] == 6).all()
    big = tsf.BlockKVCache(cache.pages + 2, cache.page_tokens, heads, d, device="cuda")
    k = torch.randn((T, heads, d), device="cuda").to(torch.bfloat16)
    tsf.fp8_cache_append(big, k, k, ints(tables), n, ints(s), q=q, q_out=out)
    assert (room[:32] == 6).all() and (room[T + 32:] == 6).all()
    none = np.setdiff1d(np.arange(cache.pages + 2), tables[tables >= 0])         # pages of no sequence
    page = heads * d * cache.page_tokens
    codes = big.data[:2 * big.pages * page].view(2, big.pages, page)
    assert (codes[:, torch.from_numpy(none).cuda()] == 0).all()
    wide = torch.full((2, T + 64, heads, d), 6.0, dtype=torch.bfloat16, device="cuda")
    tsf.fp8_cache_read(big, t, n, ints(s), T, wide[0, 32:T + 32], wide[1, 32:T + 32])
    assert (wide[:, :32] == 6).all() and (wide[:, T + 32:] == 6).all()
    assert torch.equal(tsf.fp8_cache_attention(q, cache, t, n, ints(starts)), want)
