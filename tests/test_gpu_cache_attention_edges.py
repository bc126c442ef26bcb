"""Attention over the paged 8-bit cache where its numbers end: against the
definition in 64 bits at the values that the cache holds."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.test_gpu_cache import draw, host, ints, tables_of, up
from tests.test_gpu_cache_attention import compare, filled
from tests.test_gpu_cache_attention_forms import CASES, SHARES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,hq", [(1, 2), (5, 8), (40, 2)])
@pytest.mark.parametrize("scale,softcap", [(0.0, 0.0), (-0.0, 0.0), (0.0, 30.0), (0.0, 1000.0)])
def test_scale_of_zero(new, hq, scale, softcap):
    """0 times a query that is not finite is NaN, of its own head and row alone; of the others it is 0: the mean of values."""
    g = np.random.Generator(np.random.PCG64(new))
    cache, model, tables = filled(g, [50], 2, 64, 16)
    q = draw(g, (new, hq, 64), 1)
    q[0, 1, 5], q[new // 2, 0, 63] = np.nan, -np.inf
    out = compare(q, cache, model, tables, [50], [0, new], scale=scale, softcap=softcap)
    bad = torch.zeros((new, hq), dtype=torch.bool)
    bad[0, 1] = bad[new // 2, 0] = True
    assert torch.equal(torch.isnan(out).all(2).cpu(), bad) and torch.equal(torch.isnan(out).any(2).cpu(), bad)
    # where nothing is seen it makes no difference
    none = tsf.fp8_cache_attention(up(q), cache, ints(np.full_like(tables, -1)), ints([50]), ints([0, new]), scale=scale, lse=True)
    assert (none[0] == 0).all() and (none[1] == -np.inf).all()


@pytest.mark.parametrize("how", [dict(), dict(softcap=20.0, window=70)], ids=["plain", "cap-window"])
@pytest.mark.parametrize("case", [c for c in range(len(CASES)) if CASES[c][0] != SHARES])
def test_lse_of_prompts(case, how):
    """The logarithms of the sums are the 32-bit softmax's, also where weights enter the product in one bf16."""
    _, heads, hq, d, lens, new = CASES[case]
    tables, pages = tables_of(np.random.Generator(np.random.PCG64(case)), lens, 16)
    all_starts, starts = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(new)])
    cache = tsf.BlockKVCache(pages, 16, heads, d, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(case)
    k, v = (torch.randn((int(all_starts[-1]), heads, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = (torch.randn((int(starts[-1]), hq, d), generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
    tsf.fp8_cache_append(cache, k, v, ints(tables), ints(lens), ints(all_starts))
    rk, _ = tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints(all_starts), int(all_starts[-1]))
    _, lse = tsf.fp8_cache_attention(q, cache, ints(tables), ints(lens), ints(starts), lse=True, **how)
    lse, rk, q = lse.cpu().numpy().astype(np.float64), host(rk), host(q)
    for i, (length, n) in enumerate(zip(lens, new)):
        for t in {0, 1, n // 3, n - 1}:
            p = length - n + t
            low = max(0, p - how["window"] + 1) if "window" in how else 0
            keys = np.repeat(rk[all_starts[i] + low:all_starts[i] + p + 1], hq // heads, axis=1)
            s = np.einsum("hd,jhd->hj", q[starts[i] + t], keys) / np.sqrt(d)
            size = np.einsum("hd,jhd->hj", np.abs(q[starts[i] + t]), np.abs(keys)).max(1) / np.sqrt(d)
            if "softcap" in how:
                s = how["softcap"] * np.tanh(s / how["softcap"])
            want = s.max(1) + np.log(np.exp(s - s.max(1, keepdims=True)).sum(1))
            # a score as in serve_util's tolerance; tanh by 1 - 2 / (exp(2 x) + 1), 3 2^-24 of the cap, or its rounding; a weight
            # within 2^-22; a lane's sum of n / 32 steps and 5 more, 2^-24 each; the base-2 logarithm of up to 2^17, 2^-23 of
            # it; the maximum added and the product with log(2), 2^-22 of it
            err = size * ((d + 10) * 2.0 ** -24 + 2.0 ** -20) + how.get("softcap", 0) * 2.0 ** -22 + \
                2.0 ** -22 + (length / 32 + 5) * 2.0 ** -24 + 2.0 ** -22 * np.abs(want) + 17 * 2.0 ** -23
            got = lse[starts[i] + t]
            assert (np.abs(got - want) <= err).all(), (i, t, np.abs(got - want).max(), err.min())
