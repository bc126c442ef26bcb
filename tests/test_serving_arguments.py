"""Arguments of the serving operators, without a GPU: outputs that overlap an
input, each other or themselves are refused before anything is launched, by
the binding and by the library, and so is what would lose a gradient."""
import ctypes
import random

import pytest
import torch

import tensor_scaled_fp8_amd as tsf
from tests.test_serving_host import BATCH, CACHE, INV, Batch, Cache, Rows, append, attention, cache, z

D, T = 64, 3                               # of the arguments that test_serving_host gives


def rows(buf, at, heads, tok, head, tokens=T):
    return torch.as_strided(buf, (tokens, heads, D), (tok, head, 1), at)


def refused(call, **change):
    """What the refusal says; "device tensor" comes last of all."""
    with pytest.raises(ValueError) as e:
        call(**change)
    return str(e.value)


def read(k, v):
    t, n = z(T, 5, dtype=torch.int32), z(T, dtype=torch.int32)
    tsf.fp8_cache_read(cache(), t, n, None, T, k, v)


def projection(hq=4, hk=2):
    x = z(T, hq + 2 * hk, D)
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]


def test_views_of_one_projection_are_apart():
    q, k, v = projection()
    assert "device tensor" in refused(append, q=q, k=k, v=v, q_out=q)
    assert "device tensor" in refused(append, q=q, k=k, v=v)
    # query, key and value of each head beside each other, and heads outermost
    x = z(T, 2, 3, D)
    assert "device tensor" in refused(append, q=x[:, :, 0], k=x[:, :, 1], v=x[:, :, 2], q_out=x[:, :, 0])
    x = z(8, T, D).transpose(0, 1)
    assert "device tensor" in refused(append, q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], q_out=x[:, :4])
    # keys and values of a head beside each other, other strides than the queries
    x = z(T, 4 * D + 4 * D)
    kv = x[:, 4 * D:].unflatten(1, (2, 2, D))
    q = x[:, :4 * D].unflatten(1, (4, D))
    assert "device tensor" in refused(append, q=q, k=kv[:, :, 0], v=kv[:, :, 1], q_out=q)
    assert "device tensor" in refused(lambda: read(kv[:, :, 0], kv[:, :, 1]))
    assert "device tensor" in refused(attention, q=q, out=q)
    # another part of the same tensor
    x = z(2 * T, 4, D)
    assert "device tensor" in refused(attention, q=x[:T], out=x[T:])


def test_append_refuses_q_out_over_its_inputs():
    q, k, v = projection()
    wide = z(T + 1, 4, D)
    assert "q_out must be q itself or not overlap q" in refused(append, q=wide[:T], q_out=wide[1:])            # by a token
    x = z(T, 5, D)
    assert "q_out must be q itself or not overlap q" in refused(append, q=x[:, :4], q_out=x[:, 1:])            # by a head
    assert "q_out must be q itself or not overlap q" in refused(append, q=x.view(-1)[:-D].view(-1)[:T * 4 * D].view(T, 4, D),
                                                                q_out=x[:, :4])                                # other strides
    x = z(T, 8, D)
    assert "q_out must not overlap k" in refused(append, q=z(T, 4, D), k=x[:, 3:5], q_out=x[:, :4])
    assert "q_out must not overlap v" in refused(append, q=z(T, 4, D), v=x[:, 3:5], q_out=x[:, :4])
    assert "q_out must not overlap v" in refused(append, q=q, k=k, v=q[:, 2:], q_out=q)
    flat = torch.zeros(T * 4 * D + 1, dtype=torch.bfloat16)
    assert "q_out must be q itself" in refused(append, q=flat[:-1].view(T, 4, D), q_out=flat[1:].view(T, 4, D))


def test_attention_refuses_out_over_q():
    wide = z(T + 1, 4, D)
    assert "out must be q itself or not overlap q" in refused(attention, q=wide[:T], out=wide[1:])
    x = z(T, 5, D)
    assert "out must be q itself or not overlap q" in refused(attention, q=x[:, 1:], out=x[:, :4])


def test_read_refuses_k_over_v():
    x = z(T, 3, D)
    assert "k must not overlap v" in refused(lambda: read(x[:, :2], x[:, 1:]))
    assert "k must not overlap v" in refused(lambda: read(x[:, :2], x[:, :2]))


def test_outputs_over_themselves():
    buf = torch.zeros(4096, dtype=torch.bfloat16)
    for tok, head in ((D, D), (32, 4 * D), (4 * D, 32), (2 * D, D), (D, 2 * D), (3 * D - 1, D)):
        y = rows(buf, 0, 4, tok, head)
        assert "itself" in refused(attention, out=y) and "itself" in refused(append, q_out=y), (tok, head)
    for tok, head in ((4 * D, D), (D, 3 * D), (4 * D + 3, D), (2 * D, 7 * D), (3 * D, 4 * D)):
        assert "device tensor" in refused(attention, out=rows(buf, 0, 4, tok, head)), (tok, head)
    y = rows(buf, 0, 2, D, D)
    assert "k must not overlap itself" in refused(lambda: read(y, None)) and "v must not overlap itself" in refused(lambda: read(None, y))


def elements(t):
    return {t.storage_offset() + i * t.stride(0) + j * t.stride(1) + e for i in range(t.size(0)) for j in range(t.size(1))
            for e in range(D)}


def test_any_strides():
    """Every overlap is refused, and of rows of the same strides nothing but overlaps."""
    r, buf, seen = random.Random(1), torch.zeros(1 << 13, dtype=torch.bfloat16), [0, 0]
    for _ in range(3000):
        tok, head = (r.choice((D, 2 * D, 3 * D, 4 * D, 5 * D, 4 * D + 3, 9 * D, 12 * D)) for _ in range(2))
        same = r.random() < 0.7
        tok2, head2 = (tok, head) if same else (r.choice((D, 4 * D, 8 * D, 9 * D)), r.choice((D, 2 * D, 5 * D)))
        q = rows(buf, 1700 + r.choice((0, 1, D, 2 * D, 63)), 4, tok, head)
        out = rows(buf, 1700 + r.randrange(-12, 13) * r.choice((D, D, 2 * D, 61)), 4, tok2, head2)
        a, b = elements(q), elements(out)
        said = refused(attention, q=q, out=out)
        if len(b) < out.numel():
            assert "itself" in said
        elif q.storage_offset() == out.storage_offset() and q.stride() == out.stride():
            assert "device tensor" in said
        elif a & b:
            assert "not overlap q" in said, (q.storage_offset(), q.stride(), out.storage_offset(), out.stride())
            seen[0] += 1
        elif same:
            assert "device tensor" in said, (q.storage_offset(), q.stride(), out.storage_offset(), out.stride())
            seen[1] += 1
    assert min(seen) > 100


def test_library_refuses_them():
    """By the C interface: addresses that are never read."""
    lib, r = tsf.load(), ctypes.byref
    at = 1 << 20
    c, b = Cache(**CACHE), Batch(**BATCH)

    def row(p, tok=256, head=64):
        return Rows(at + 2 * p, tok, head)

    def run(q, out, k=row(1 << 16, 128), v=row(2 << 16, 128)):
        return (lib.fp8_cache_append(r(c), r(b), r(k), r(v), r(q), r(out), 4, at, 64, 0, None),
                lib.fp8_cache_attention(r(c), r(b), r(q), 4, 1.0, 0.0, 0, r(out), None, at, 1 << 40, None))
    assert run(row(0), row(256)) == (INV, INV) and run(row(0), row(64)) == (INV, INV) and run(row(0), row(1)) == (INV, INV)
    assert run(row(0), row(9999, 64)) == (INV, INV)                                        # its own rows
    assert run(row(0), row(0), k=row(128))[0] == INV and run(row(0), row(5000), v=row(5000))[0] == INV
    assert run(row(0), row(9999, -64)) == (INV, INV) and run(row(0, -256), row(-512)) == (INV, INV)
    for other in (0, 64, 128 * 2):
        assert lib.fp8_cache_read(r(c), r(b), r(row(0, 128)), r(row(other, 128)), None) == INV
    assert lib.fp4_linear_fwd_cached(at, 32, 20, 32, 16, at, at, 0, at, 1 << 30, at + 4, None) == INV


def test_outputs_that_want_a_gradient():
    def made(*shape):
        return z(*shape).requires_grad_()
    w = tsf.FP4Tensor(torch.zeros(4352, dtype=torch.uint8), 512, 16)
    calls = {"q_out": lambda: append(q_out=made(T, 4, D)), "out": lambda: attention(out=made(T, 4, D)),
             "k": lambda: read(made(T, 2, D), None), "v": lambda: read(None, made(T, 2, D)),
             "Y": lambda: tsf.fp4_linear_fwd_cached(z(2, 512), w, made(2, 16))}
    for name, call in calls.items():
        with pytest.raises(NotImplementedError, match=f"^{name} wants a gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
            call()
    with torch.autograd.forward_ad.dual_level(), pytest.raises(NotImplementedError, match="out wants a gradient"):
        attention(out=torch.autograd.forward_ad.make_dual(z(T, 4, D), z(T, 4, D)))


def test_weights_that_carry_a_tangent():
    """Stored ones are constants: a parameter may be, a tangent would be lost."""
    with torch.autograd.forward_ad.dual_level():
        def dual(*shape, dtype=torch.bfloat16):
            return torch.autograd.forward_ad.make_dual(z(*shape, dtype=dtype), z(*shape, dtype=dtype))
        for make in (tsf.prepare_fp4_weight, tsf.FP4InferenceLinear):
            with pytest.raises(NotImplementedError, match="W wants a gradient"):
                make(dual(8, 16))
            with pytest.raises(ValueError, match="device tensor"):
                make(torch.nn.Parameter(z(8, 16)))
        sizes = {"Wqkv": (8, 4 * D), "Wo": (2 * D, 8), "freqs": (D // 2,)}
        for name in sizes:
            for bits in (4, 8):
                w = {n: (dual if n == name else z)(*s, dtype=torch.float32 if n == "freqs" else torch.bfloat16)
                     for n, s in sizes.items()}
                with pytest.raises(NotImplementedError, match=f"{name} wants a gradient"):
                    tsf.InferenceAttention(w["Wqkv"], w["Wo"], 2, 1, D, freqs=w["freqs"], bits=bits)


NAN = float("nan")


@pytest.mark.parametrize("change,said", [
    (dict(scale=NAN), "scale must be"), (dict(scale=-1e20), "scale must be"), (dict(softcap=-1.0), "softcap must be"),
    (dict(softcap=NAN), "softcap must be"), (dict(softcap=1e20), "softcap must be"), (dict(window=-1), "window must be"),
    (dict(window=2 ** 31), "window must be"), (dict(heads=3, kv=2), "multiple of the key heads"),
    (dict(heads=2, kv=0), "multiple of the key heads"), (dict(d=80), "64, 128 or 256"), (dict(freqs=torch.zeros(20)), "multiple of 16"),
    (dict(freqs=torch.zeros(40)), "multiple of 16"), ({}, "device tensor"), (dict(softcap=30.0, window=5, scale=-0.1), "device tensor")])
@pytest.mark.parametrize("bits", [4, 8])
def test_layers_that_are_refused(bits, change, said):
    """When they are made, and not after their first call's tokens are in the cache."""
    how = dict(change)
    heads, kv, d = how.pop("heads", 2), how.pop("kv", 1), how.pop("d", D)
    with pytest.raises(ValueError, match=said):
        tsf.InferenceAttention(z(8, (heads + 2 * kv) * d), z(heads * d, 8), heads, kv, d, bits=bits, **how)
