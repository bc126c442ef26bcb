"""The serving operators in their places: an attention layer's prompt, then
decode steps, against the same layer computed from its definition."""
import numpy as np
import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.block_util import held, to_bf16
from tests.serve_util import Model, attend, fp4_held, rotate
from tests.test_gpu_cache import freqs_of, host, ints, same, tables_of, up

pytestmark = pytest.mark.gpu


def near(got, want, far):
    """Relative to the size of want (rms)."""
    assert np.sqrt(((got - want) ** 2).mean() / (want ** 2).mean()) <= far


@pytest.mark.parametrize("bits,hq,hk,d,inter", [(4, 4, 2, 64, False), (8, 3, 1, 128, True)])
def test_prompt_then_decode(bits, hq, hk, d, inter):
    g = np.random.Generator(np.random.PCG64(bits))
    K, page = 320, 16
    wqkv, wo = to_bf16(g.standard_normal((K, (hq + 2 * hk) * d)) * K ** -0.5), to_bf16(g.standard_normal((hq * d, K)) * 0.1)
    freqs = freqs_of(d)
    layer = tsf.InferenceAttention(up(wqkv), up(wo), hq, hk, d, freqs=torch.from_numpy(freqs).cuda(), interleaved=inter,
                                   bits=bits)
    tables, pages = tables_of(g, [40, 23, 30], page)
    cache, model = tsf.BlockKVCache(pages, page, hk, d, device="cuda"), Model(pages, page, hk, d)
    lens = np.array([37, 20, 0])
    stored = [fp4_held(w) if bits == 4 else held(w.T).T for w in (wqkv, wo)]
    for step in range(4):
        new = lens.copy() if step == 0 else np.ones(3, dtype=int)
        if step:
            lens = lens + 1
        starts = np.concatenate([[0], np.cumsum(new)])
        x = to_bf16(g.standard_normal((int(starts[-1]), K)))
        s = None if step else ints(starts)
        y = layer(up(x), cache, ints(tables), ints(lens), s)
        # the projection as it is (its roundings to bf16 decide the codes), everything after it by the definition
        qkv = layer.qkv(up(x))
        near(host(qkv), held(x) @ stored[0], 0.0025)
        a = host(qkv).reshape(len(x), -1, d)
        pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
        model.append(a[:, hq:hq + hk], a[:, hq + hk:], tables, lens, starts, freqs, inter)
        all_starts = np.concatenate([[0], np.cumsum(lens)])
        rk, rv = tsf.fp8_cache_read(cache, ints(tables), ints(lens), ints(all_starts), int(all_starts[-1]))
        wk, wv = model.read(tables, lens, all_starts)
        same(host(rk), wk)
        same(host(rv), wv)
        q = to_bf16(rotate(a[:, :hq], pos, freqs, inter))
        o = to_bf16(attend(q, model, tables, lens, starts)[0]).reshape(len(x), -1)
        # o to bf16 twice as far off as its rounding, then to 8 bits (some next to a border), and Y's own rounding
        near(host(y), held(o) @ stored[1], 0.02)
        assert np.isfinite(host(y)).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_layer_refuses_gradients_and_keeps_its_angles(bits):
    g = np.random.Generator(np.random.PCG64(8))
    K, hq, hk, d = 128, 2, 1, 64
    bf = [up(to_bf16(g.standard_normal(s) * 0.06)) for s in ((K, (hq + 2 * hk) * d), (hq * d, K))]
    layer = tsf.InferenceAttention(*bf, hq, hk, d, freqs=torch.from_numpy(freqs_of(d)).cuda(), bits=bits)
    a = (tsf.BlockKVCache(1, 16, hk, d, device="cuda"), ints([[0]]), ints([5]), ints([0, 5]))
    x = up(g.standard_normal((5, K)))
    want = layer(x, *a)
    x.requires_grad_()
    with pytest.raises(NotImplementedError, match="x wants a gradient"):
        layer(x, *a)
    with torch.no_grad():
        assert torch.equal(layer(x, *a), want)
    layer.to(torch.bfloat16)
    assert layer.freqs.dtype == torch.float32
    with torch.inference_mode():
        assert torch.equal(layer(x.detach(), *a), want)
    other = tsf.InferenceAttention(*bf, hq, hk, d, freqs=torch.zeros(d // 2, device="cuda"), bits=bits)
    other.load_state_dict(layer.state_dict())
    with torch.no_grad():
        assert torch.equal(other(x, *a), want)


def test_layer_in_a_graph():
    """A captured decode step of a padded batch, replayed as sequences come and go."""
    g = np.random.Generator(np.random.PCG64(5))
    K, hq, hk, d, page, B = 256, 4, 2, 64, 16, 4
    bf = [up(to_bf16(g.standard_normal(s) * 0.06)) for s in ((K, (hq + 2 * hk) * d), (hq * d, K))]
    layer = tsf.InferenceAttention(*bf, hq, hk, d, freqs=torch.from_numpy(freqs_of(d)).cuda(), window=20, softcap=30.0, bits=4)
    caches = [tsf.BlockKVCache(20, page, hk, d, device="cuda") for _ in range(2)]
    t = ints(g.permutation(20)[:16].reshape(4, 4))
    x, lengths = torch.zeros((B, K), dtype=torch.bfloat16, device="cuda"), ints([0] * B)
    layer(x, caches[0], t, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, caches[0], t, lengths)
    for step in range(20):
        lengths.copy_(ints([step + 1, max(0, step - 4), 0 if step > 10 else step + 1, 0]))
        x.copy_(up(g.standard_normal((B, K))))
        want = layer(x, caches[1], t, lengths)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(caches[0].data, caches[1].data)
        assert (y[3] == 0).all()
