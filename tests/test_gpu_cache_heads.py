"""Tokens appended one a sequence to caches of many heads, each a wave's lane:
codes and scales, in their stored order, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import to_bf16
from tests.serve_util import TOK, VALUES, Model
from tests.test_gpu_cache import freqs_of, ints, tables_of, up

pytestmark = pytest.mark.gpu


def stored(cache):
    """codes [2, pages, page tokens, heads, d] and scale bytes [2, pages, blocks, heads] of a cache, by the header's layout."""
    P, T, H, D = cache.pages, cache.page_tokens, cache.heads, cache.head_dim
    raw = cache.data.cpu().numpy()
    n, w = P * T * H * D, D // 16
    t, d = np.arange(TOK)[:, None], np.arange(D)[None]
    at = (1024 * (d // 64) + 256 * (d % 64 // 16) + 16 * t + d % 16,
          1024 * (d % w // 4) + 256 * (t // 4) + 16 * (d // w) + 4 * (d % 4) + t % 4)
    codes = np.stack([raw[i * n:(i + 1) * n].reshape(P, H, T // TOK, TOK * D)[..., at[i]] for i in range(2)])
    scales = raw[2 * n:].reshape(P, H, T // TOK, 2)
    return codes.transpose(0, 1, 3, 4, 2, 5).reshape(2, P, T, H, D), scales.transpose(3, 0, 2, 1)


@pytest.mark.parametrize("heads,hq,d,page,inter", [
    (10, 10, 128, 16, False), (20, 40, 64, 32, True), (17, 17, 256, 16, False), (32, 64, 128, 64, False), (40, 40, 64, 16, False),
    (33, 33, 256, 32, True), (1, 16, 128, 16, False), (16, 128, 64, 16, False)])
def test_scales_that_move_in_many_heads(heads, hq, d, page, inter):
    g = np.random.Generator(np.random.PCG64(heads * d))
    lens = np.array([0, 5, 14, 0])
    tables, pages = tables_of(g, lens + 20, page)
    tables[3] = -1                                                       # padding
    cache, model = tsf.BlockKVCache(pages, page, heads, d, device="cuda"), Model(pages, page, heads, d)
    freqs = freqs_of(d)
    f = torch.from_numpy(freqs).cuda()
    begin = np.concatenate([[0], np.cumsum(lens)])
    k, v = (to_bf16(g.standard_normal((int(begin[-1]), heads, d))) for _ in range(2))
    tsf.fp8_cache_append(cache, up(k), up(v), ints(tables), ints(lens), ints(begin), freqs=f, interleaved=inter)
    model.append(k, v, tables, lens, begin, freqs, inter)
    grows = 2.0 ** g.integers(-3, 4, size=(20, 4, heads, 1))             # some heads' scales at every token
    for step in range(20):
        lens = lens + [1, 1, 1, 0]
        k, v = (to_bf16(g.standard_normal((4, heads, d)) * grows[step] * 1.2 ** step) for _ in range(2))
        q = up(g.standard_normal((4, hq, d)))
        one = tsf.fp8_cache_append(cache, up(k), up(v), ints(tables), ints(lens), q=q, freqs=f, interleaved=inter)
        before = np.concatenate([[0], np.cumsum([1, 1, 1])])
        model.append(k[:3], v[:3], tables, lens[:3], before, freqs, inter)
        codes, scales = stored(cache)
        assert np.array_equal(scales, np.where(model.bias == 127, 0, 127 - model.bias)), step
        bad = VALUES[codes] != VALUES[model.codes]
        assert not bad.any(), (step, np.argwhere(bad)[:4])
        # queries: the same bits as by the kernel of several tokens
        other = tsf.BlockKVCache(pages, page, heads, d, device="cuda")
        many = tsf.fp8_cache_append(other, up(k), up(v), ints(tables), ints(lens), ints([0, 1, 2, 3, 4]), q=q, freqs=f,
                                    interleaved=inter)
        assert torch.equal(one, many)
