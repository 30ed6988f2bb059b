"""Refusals of the entry points of the gated half of a decoder layer (no GPU needed): every call here is
invalid on purpose and is turned down on the host before anything is enqueued."""
import os

import pytest
import torch

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt
    if not os.path.exists(rt.LIB_PATH):
        from dynamic_scaling_scaled_amd import _build
        _build.build()
    rt.lib()
    return rt


def route(rt, **kw):
    a = dict(x=FAKE, lt=rt.F32, tokens=8, experts=64, ld=64, score=0, bias=FAKE, groups=4, top=2, best=2, k=8, renorm=1,
             scale=1.0, ids=FAKE, w=FAKE, slots=FAKE, order=FAKE, offsets=FAKE)
    a.update(kw)
    return rt.lib().fp8_expert_route(a["x"], a["lt"], a["tokens"], a["experts"], a["ld"], a["score"], a["bias"],
                                     a["groups"], a["top"], a["best"], a["k"], a["renorm"], a["scale"], a["ids"], a["w"],
                                     a["slots"], a["order"], a["offsets"], None)


ROUTE_BAD = [
    (dict(x=None), "EINVAL"), (dict(lt=3), "EINVAL"), (dict(tokens=0), "EINVAL"), (dict(experts=0), "EINVAL"),
    (dict(ld=63), "EINVAL"), (dict(score=2), "EINVAL"), (dict(score=-1), "EINVAL"), (dict(k=0), "EINVAL"),
    (dict(k=65), "EINVAL"), (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
    (dict(tokens=2 ** 31), "EINVAL"), (dict(tokens=2 ** 28, k=8), "EINVAL"), (dict(ld=2 ** 31), "EINVAL"),
    (dict(ids=None), "EINVAL"), (dict(experts=1025, ld=1025), "EUNSUPPORTED"), (dict(k=33), "EUNSUPPORTED"),
    (dict(x=FAKE + 2), "EALIGN"), (dict(lt=1, x=FAKE + 1), "EALIGN"), (dict(ids=FAKE + 2), "EALIGN"),
]


@pytest.mark.parametrize("kw,status", ROUTE_BAD + [
    (dict(w=None), "EINVAL"), (dict(slots=None), "EINVAL"), (dict(order=None), "EINVAL"), (dict(offsets=None), "EINVAL"),
    (dict(slots=None, order=None), "EINVAL"), (dict(groups=0), "EINVAL"), (dict(top=0), "EINVAL"),
    (dict(top=5), "EINVAL"), (dict(best=0), "EINVAL"), (dict(best=3), "EINVAL"), (dict(groups=5, top=5), "EINVAL"),
    (dict(k=17, top=1), "EINVAL"), (dict(experts=130, ld=130, groups=65), "EUNSUPPORTED"),
    (dict(tokens=2 ** 27 + 1, k=1), "EUNSUPPORTED"),
    (dict(w=FAKE + 1), "EALIGN"), (dict(bias=FAKE + 2), "EALIGN"), (dict(slots=FAKE + 2), "EALIGN"),
    (dict(order=FAKE + 3), "EALIGN"), (dict(offsets=FAKE + 1), "EALIGN"),
])
def test_route_refusals(rt, kw, status):
    assert route(rt, **kw) == getattr(rt, status)


def route_grad(rt, **kw):
    a = dict(x=FAKE, lt=rt.F32, tokens=8, experts=64, ld=64, score=0, k=8, renorm=1, scale=1.0, ids=FAKE, dw=FAKE,
             dl=FAKE * 2, ldd=64)
    a.update(kw)
    return rt.lib().fp8_expert_route_backward(a["x"], a["lt"], a["tokens"], a["experts"], a["ld"], a["score"], a["k"],
                                              a["renorm"], a["scale"], a["ids"], a["dw"], a["dl"], a["ldd"], None)


@pytest.mark.parametrize("kw,status", ROUTE_BAD + [
    (dict(dw=None), "EINVAL"), (dict(dl=None), "EINVAL"), (dict(ldd=63), "EINVAL"), (dict(ldd=2 ** 31), "EINVAL"),
    (dict(dl=FAKE, ldd=128), "EINVAL"), (dict(dw=FAKE + 2), "EALIGN"), (dict(dl=FAKE + 2), "EALIGN"),
])
def test_route_gradient_refusals(rt, kw, status):
    assert route_grad(rt, **kw) == getattr(rt, status)


def gemm(rt, **kw):
    a = dict(a=FAKE, fa=0, rows=8, lda=256, ga=(1, 0), sa=FAKE, order=FAKE, choices=2, b=FAKE, fb=0, gb=(1, 0), sb=FAKE,
             offsets=FAKE, experts=4, slots=16, N=64, K=256, y=FAKE, yt=rt.BF16, ldy=64, flags=2)
    a.update(kw)
    return rt.lib().fp8_expert_gemm(a["a"], a["fa"], a["rows"], a["lda"], rt.Gran(*a["ga"]), a["sa"], a["order"],
                                    a["choices"], a["b"], a["fb"], rt.Gran(*a["gb"]), a["sb"], a["offsets"], a["experts"],
                                    a["slots"], a["N"], a["K"], a["y"], a["yt"], a["ldy"], a["flags"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), "EINVAL"), (dict(sa=None), "EINVAL"), (dict(b=None), "EINVAL"), (dict(sb=None), "EINVAL"),
    (dict(offsets=None), "EINVAL"), (dict(y=None), "EINVAL"), (dict(fa=2), "EINVAL"), (dict(fb=-1), "EINVAL"),
    (dict(yt=2), "EINVAL"), (dict(rows=0), "EINVAL"), (dict(experts=0), "EINVAL"), (dict(slots=0), "EINVAL"),
    (dict(N=0), "EINVAL"), (dict(K=0), "EINVAL"), (dict(lda=128), "EINVAL"), (dict(ldy=48), "EINVAL"),
    (dict(choices=0), "EINVAL"), (dict(ga=(-1, 0)), "EINVAL"), (dict(gb=(1, -1)), "EINVAL"), (dict(flags=3), "EINVAL"),
    (dict(flags=6), "EINVAL"), (dict(slots=2 ** 31), "EINVAL"), (dict(rows=2 ** 31), "EINVAL"),
    (dict(choices=2 ** 31), "EINVAL"), (dict(N=2 ** 31), "EINVAL"), (dict(lda=2 ** 31), "EINVAL"),
    (dict(flags=0), "EUNSUPPORTED"), (dict(fb=1), "EUNSUPPORTED"), (dict(experts=1025), "EUNSUPPORTED"),
    (dict(rows=2 ** 24, lda=256), "EUNSUPPORTED"), (dict(K=2 ** 20 + 128, lda=2 ** 21), "EUNSUPPORTED"),
    (dict(slots=2 ** 30, N=64), "EUNSUPPORTED"), (dict(ga=(1, 128)), "EUNSUPPORTED"), (dict(gb=(128, 128)), "EUNSUPPORTED"),
    (dict(ga=(2, 0)), "EUNSUPPORTED"), (dict(gb=(2, 0)), "EUNSUPPORTED"), (dict(gb=(128, 0)), "EUNSUPPORTED"),
    (dict(N=72, ldy=72), "EALIGN"), (dict(K=192), "EALIGN"), (dict(lda=264), "EALIGN"), (dict(ldy=68), "EALIGN"),
    (dict(yt=0, ldy=66), "EALIGN"), (dict(a=FAKE + 8), "EALIGN"), (dict(b=FAKE + 8), "EALIGN"),
    (dict(y=FAKE + 8), "EALIGN"), (dict(sa=FAKE + 2), "EALIGN"), (dict(sb=FAKE + 2), "EALIGN"),
    (dict(offsets=FAKE + 2), "EALIGN"), (dict(order=FAKE + 2), "EALIGN"),
])
def test_gemm_refusals(rt, kw, status):
    assert gemm(rt, **kw) == getattr(rt, status)


def gated(rt, **kw):
    a = dict(x=FAKE, xt=rt.BF16, rows=8, cols=256, ldx=512, act=0, g=(1, 0), f=0, mode=0, eps=1e-12, pow2=0, s=FAKE,
             inv=None, q=FAKE, ldq=256, kept=FAKE, kf=0, ldk=512, ks=FAKE, amax=None, live=None)
    a.update(kw)
    return rt.lib().fp8_gated_quantize(a["x"], a["xt"], a["rows"], a["cols"], a["ldx"], a["act"], rt.Gran(*a["g"]), a["f"],
                                       a["mode"], a["eps"], a["pow2"], a["s"], a["inv"], a["q"], a["ldq"], a["kept"],
                                       a["kf"], a["ldk"], a["ks"], a["amax"], a["live"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), "EINVAL"), (dict(s=None), "EINVAL"), (dict(q=None), "EINVAL"), (dict(kept=None), "EINVAL"),
    (dict(ks=None), "EINVAL"), (dict(xt=2), "EINVAL"), (dict(f=2), "EINVAL"), (dict(kf=7), "EINVAL"),
    (dict(act=2), "EINVAL"), (dict(act=-1), "EINVAL"), (dict(mode=2), "EINVAL"), (dict(eps=0.0), "EINVAL"),
    (dict(mode=1, eps=0.0), "EINVAL"),                 # the checkpoint's own scales need it
    (dict(rows=0), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(ldx=256), "EINVAL"), (dict(ldq=240), "EINVAL"),
    (dict(ldk=256), "EINVAL"), (dict(g=(-1, 0)), "EINVAL"), (dict(g=(1, -2)), "EINVAL"),
    (dict(cols=264, ldx=528), "EALIGN"), (dict(ldx=520), "EALIGN"), (dict(ldq=264), "EALIGN"), (dict(ldk=520), "EALIGN"),
    (dict(g=(1, 24)), "EALIGN"), (dict(x=FAKE + 8), "EALIGN"), (dict(q=FAKE + 8), "EALIGN"), (dict(kept=FAKE + 8), "EALIGN"),
    (dict(s=FAKE + 2), "EALIGN"), (dict(ks=FAKE + 2), "EALIGN"), (dict(amax=FAKE + 1), "EALIGN"),
    (dict(inv=FAKE + 1), "EALIGN"), (dict(live=FAKE + 2), "EALIGN"),
    (dict(g=(0, 0)), "EUNSUPPORTED"), (dict(g=(2, 0)), "EUNSUPPORTED"), (dict(g=(1, 48)), "EUNSUPPORTED"),
    (dict(g=(0, 128), mode=1), "EUNSUPPORTED"), (dict(cols=2048, ldx=4096, ldq=2048, ldk=4096, g=(1, 1024)), "EUNSUPPORTED"),
    (dict(cols=65552, ldx=131104, ldq=65552, ldk=131104), "EUNSUPPORTED"),
])
def test_gated_refusals(rt, kw, status):
    assert gated(rt, **kw) == getattr(rt, status)


def gated_grad(rt, **kw):
    a = dict(dz=FAKE, t=rt.BF16, rows=8, cols=256, lddz=256, kept=FAKE, kf=0, ldk=512, ks=FAKE, act=0, dx=FAKE, lddx=512,
             z=FAKE, ldz=256, live=None)
    a.update(kw)
    return rt.lib().fp8_gated_backward(a["dz"], a["t"], a["rows"], a["cols"], a["lddz"], a["kept"], a["kf"], a["ldk"],
                                       a["ks"], a["act"], a["dx"], a["lddx"], a["z"], a["ldz"], a["live"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dz=None), "EINVAL"), (dict(kept=None), "EINVAL"), (dict(ks=None), "EINVAL"), (dict(dx=None), "EINVAL"),
    (dict(t=2), "EINVAL"), (dict(kf=2), "EINVAL"), (dict(act=5), "EINVAL"), (dict(rows=0), "EINVAL"),
    (dict(cols=0), "EINVAL"), (dict(lddz=240), "EINVAL"), (dict(ldk=256), "EINVAL"), (dict(lddx=256), "EINVAL"),
    (dict(ldz=240), "EINVAL"), (dict(cols=264, lddz=272, ldk=544, lddx=544, ldz=272), "EALIGN"),
    (dict(lddz=264), "EALIGN"), (dict(ldk=520), "EALIGN"), (dict(lddx=520), "EALIGN"), (dict(ldz=264), "EALIGN"),
    (dict(dz=FAKE + 8), "EALIGN"), (dict(kept=FAKE + 8), "EALIGN"), (dict(dx=FAKE + 8), "EALIGN"),
    (dict(z=FAKE + 8), "EALIGN"), (dict(ks=FAKE + 2), "EALIGN"), (dict(live=FAKE + 2), "EALIGN"),
    (dict(cols=65552, lddz=65552, ldk=131104, lddx=131104, ldz=65552), "EUNSUPPORTED"),
])
def test_gated_gradient_refusals(rt, kw, status):
    assert gated_grad(rt, **kw) == getattr(rt, status)


def combine(rt, **kw):
    a = dict(x=FAKE, xt=rt.BF16, x_rows=16, cols=256, ldx=256, slots=FAKE, w=FAKE, tokens=8, k=2, res=FAKE * 2, ldr=256,
             y=FAKE * 3, ldy=256)
    a.update(kw)
    return rt.lib().fp8_expert_combine(a["x"], a["xt"], a["x_rows"], a["cols"], a["ldx"], a["slots"], a["w"], a["tokens"],
                                       a["k"], a["res"], a["ldr"], a["y"], a["ldy"], None)


COMBINE_BAD = [
    (dict(x=None), "EINVAL"), (dict(slots=None), "EINVAL"), (dict(w=None), "EINVAL"), (dict(xt=2), "EINVAL"),
    (dict(x_rows=0), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(ldx=128), "EINVAL"), (dict(tokens=0), "EINVAL"),
    (dict(k=0), "EINVAL"), (dict(x_rows=2 ** 31), "EINVAL"), (dict(tokens=2 ** 31), "EINVAL"),
    (dict(k=33), "EUNSUPPORTED"), (dict(cols=252), "EALIGN"), (dict(ldx=260), "EALIGN"), (dict(x=FAKE + 8), "EALIGN"),
    (dict(slots=FAKE + 2), "EALIGN"), (dict(w=FAKE + 2), "EALIGN"),
]


@pytest.mark.parametrize("kw,status", COMBINE_BAD + [
    (dict(y=None), "EINVAL"), (dict(y=FAKE), "EINVAL"), (dict(ldy=128), "EINVAL"), (dict(ldr=128), "EINVAL"),
    (dict(y=FAKE * 2, ldy=512), "EINVAL"), (dict(ldy=260), "EALIGN"), (dict(ldr=260), "EALIGN"),
    (dict(y=FAKE * 3 + 8), "EALIGN"), (dict(res=FAKE * 2 + 8), "EALIGN"),
])
def test_combine_refusals(rt, kw, status):
    assert combine(rt, **kw) == getattr(rt, status)


def combine_grad(rt, **kw):
    a = dict(dy=FAKE * 2, xt=rt.BF16, tokens=8, cols=256, lddy=256, x=FAKE, x_rows=16, ldx=256, slots=FAKE, w=FAKE, k=2,
             dx=FAKE * 3, lddx=256, dw=FAKE)
    a.update(kw)
    return rt.lib().fp8_expert_combine_backward(a["dy"], a["xt"], a["tokens"], a["cols"], a["lddy"], a["x"], a["x_rows"],
                                                a["ldx"], a["slots"], a["w"], a["k"], a["dx"], a["lddx"], a["dw"], None)


@pytest.mark.parametrize("kw,status", COMBINE_BAD + [
    (dict(dy=None), "EINVAL"), (dict(dx=None), "EINVAL"), (dict(dw=None), "EINVAL"), (dict(dx=FAKE * 2), "EINVAL"),
    (dict(lddy=128), "EINVAL"), (dict(lddx=128), "EINVAL"), (dict(dx=FAKE, lddx=512), "EINVAL"),
    (dict(lddy=260), "EALIGN"), (dict(lddx=260), "EALIGN"), (dict(dy=FAKE * 2 + 8), "EALIGN"),
    (dict(dx=FAKE * 3 + 8), "EALIGN"), (dict(dw=FAKE + 2), "EALIGN"),
])
def test_combine_gradient_refusals(rt, kw, status):
    assert combine_grad(rt, **kw) == getattr(rt, status)


def test_packed_calls(rt):
    """Arguments as 64-bit words: each call with its own number of words, and its refusals."""
    import struct

    L = rt.lib()

    def packed(fmt, *words):
        record = struct.pack(fmt, *words)
        return L.fp8_call_packed(record, len(record) // 8)

    good = {4: (rt._ROUTE, 20), 5: (rt._ROUTE_GRAD, 15), 6: (rt._EXPERTS, 25), 7: (rt._GATED, 24), 8: (rt._GATED_GRAD, 17),
            9: (rt._COMBINE, 15), 10: (rt._COMBINE_GRAD, 16)}
    for call, (record, words) in good.items():
        assert record.size == 8 * words
        for n in range(1, 40):
            zeros = struct.pack("%dq" % n, call, *([0] * (n - 1)))
            assert L.fp8_call_packed(zeros, n) == rt.EINVAL  # null pointers, or another call's number of words
    route = [4, FAKE, 0, 8, 64, 64, 0, 0, 1, 1, 1, 8, 1]
    tail = [FAKE, FAKE, FAKE, FAKE, FAKE, 0]
    assert packed("13qd6q", *route, float("inf"), *tail) == rt.EINVAL
    assert packed("13qd6q", *route[:4], 1025, 1025, *route[6:], 1.0, *tail) == rt.EUNSUPPORTED
    assert packed("13qd6q", *route[:6], 2 ** 32, *route[7:], 1.0, *tail) == rt.EINVAL  # an enumerator does not wrap
    assert packed("13qd6q", *route, 1.0, FAKE + 2, *tail[1:]) == rt.EALIGN
    assert packed("15q", 11, *([0] * 14)) == rt.EINVAL


def test_binding_refusals(rt):
    """Shapes and types the binding turns down before it passes pointers (CPU tensors: never used)."""
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32

    def refused(f, good, *changes):
        for kw in changes:
            with pytest.raises((ValueError, TypeError)):
                f(**dict(good, **kw))

    l, ids, w = torch.zeros(4, 16), torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2)
    order, off = torch.zeros(8, dtype=i32), torch.zeros(17, dtype=i32)
    refused(rt.fp8_expert_route, dict(logits=l, ids=ids, weights=w, slots=ids, order=order, offsets=off),
            dict(logits=l.half()), dict(logits=l.t()), dict(ids=ids.long()), dict(ids=ids[:3]), dict(ids=ids[0]),
            dict(weights=w[:, :1]), dict(weights=w.double()), dict(slots=ids[:, :1]), dict(order=order[:7]),
            dict(offsets=off[:16]), dict(slots=None), dict(offsets=None), dict(bias=torch.zeros(15)),
            dict(bias=torch.zeros(16, dtype=bf)))
    refused(rt.fp8_expert_route_backward, dict(logits=l, ids=ids, dweights=w, dlogits=l.clone()),
            dict(dlogits=l.bfloat16()), dict(dlogits=l[:3]), dict(dweights=w[:3]), dict(ids=ids.long()), dict(ids=ids[:2]))
    a, s = torch.zeros(4, 128, dtype=u8), torch.zeros(4, 1)
    b = rt.PackedWeights(torch.zeros(2 * 16 * 128, dtype=u8), 32, 128)
    y, sb = torch.zeros(8, 16, dtype=bf), torch.zeros(2, 16)
    refused(rt.fp8_expert_gemm, dict(a=a, fa=0, ga=(1, 0), scale_a=s, b=b, fb=0, gb=(1, 0), scale_b=sb, offsets=off[:3],
                                     y=y, order=order, choices=2),
            dict(a=a.int()), dict(a=a[:, ::2]), dict(b=b.data), dict(b=rt.PackedWeights(b.data, 16, 128)),
            dict(scale_a=s[:3]), dict(scale_b=sb[:1]), dict(offsets=off[:4]), dict(offsets=off[:3].long()),
            dict(offsets=off[:1]), dict(order=order[:4]), dict(y=y.half()), dict(y=y[:, :8]))
    x, q, sc = torch.zeros(4, 64, dtype=bf), torch.zeros(4, 32, dtype=u8), torch.zeros(4, 1)
    kept, ks = torch.zeros(4, 64, dtype=u8), torch.zeros(4, 2, 1)
    one = torch.zeros(1, dtype=i32)
    refused(rt.fp8_gated_quantize, dict(x=x, gran=(1, 0), fmt=0, mode=0, eps=1e-12, pow2_round_up=False, scale=sc, q=q,
                                        kept=kept, kept_scale=ks, live=one),
            dict(x=x[:, :63]), dict(x=x.half()), dict(q=q.int()), dict(q=q[:, :16]), dict(scale=sc[:3]),
            dict(scale=sc.double()), dict(kept=None), dict(kept_scale=None), dict(kept=q), dict(kept_scale=ks[:3]),
            dict(kept_scale=ks.double()), dict(live=off), dict(live=one.long()), dict(amax_out=sc[:2]))
    refused(rt.fp8_gated_backward, dict(dz=x[:, :32], kept=kept, kept_scale=ks, dx=x, z=x[:, 32:], live=one),
            dict(dx=x.float()), dict(dx=x[:, :32]), dict(z=x), dict(z=x[:, :32].float()), dict(kept=q),
            dict(kept_scale=ks[:, :1]), dict(live=off), dict(dz=x[:, :32].half()))
    xs, yy = torch.zeros(8, 32, dtype=bf), torch.zeros(4, 32, dtype=bf)
    refused(rt.fp8_expert_combine, dict(x=xs, slots=ids, weights=w, y=yy, residual=yy.clone()),
            dict(x=xs.half()), dict(slots=ids.long()), dict(slots=ids.t()), dict(weights=w[:3]), dict(y=yy.float()),
            dict(y=yy[:3]), dict(residual=yy.float()), dict(residual=yy[:, :16]))
    refused(rt.fp8_expert_combine_backward, dict(dy=yy, x=xs, slots=ids, weights=w, dx=xs.clone(), dweights=w.clone()),
            dict(dy=yy[:3]), dict(x=xs.float()), dict(x=xs[:, :16]), dict(dx=xs[:7]), dict(dx=xs.float()),
            dict(dweights=w[:3]), dict(weights=w.double()), dict(slots=ids[:3]))
