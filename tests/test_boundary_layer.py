"""Refusals of the decoder-layer entry points (no GPU needed): every call here
is invalid on purpose and is turned down on the host before anything is
enqueued."""
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


def norm(rt, **kw):
    a = dict(x=FAKE, xt=rt.BF16, rows=8, cols=256, ldx=256, res=FAKE * 2, ldr=256, w=FAKE, wt=rt.BF16, ne=1e-6,
             g=(1, 0), f=rt.E4M3, mode=rt.DYNAMIC, eps=1e-12, pow2=0, s=FAKE, inv=None, q=FAKE, ldq=256, h=FAKE * 3,
             ldh=256, rstd=FAKE, amax=None)
    a.update(kw)
    return rt.lib().fp8_rmsnorm_quantize(a["x"], a["xt"], a["rows"], a["cols"], a["ldx"], a["res"], a["ldr"], a["w"],
                                         a["wt"], a["ne"], rt.Gran(*a["g"]), a["f"], a["mode"], a["eps"], a["pow2"],
                                         a["s"], a["inv"], a["q"], a["ldq"], a["h"], a["ldh"], a["rstd"], a["amax"],
                                         None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), "EINVAL"), (dict(w=None), "EINVAL"), (dict(s=None), "EINVAL"), (dict(q=None), "EINVAL"),
    (dict(rows=0), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(xt=7), "EINVAL"), (dict(wt=-1), "EINVAL"),
    (dict(f=2), "EINVAL"), (dict(mode=3), "EINVAL"), (dict(eps=0.0), "EINVAL"), (dict(ne=-1.0), "EINVAL"),
    (dict(ne=float("nan")), "EINVAL"), (dict(ldx=128), "EINVAL"), (dict(ldr=128), "EINVAL"),
    (dict(ldh=128), "EINVAL"), (dict(ldq=128), "EINVAL"), (dict(g=(-1, 0)), "EINVAL"),
    (dict(h=FAKE, ldh=512), "EINVAL"),                 # in place with another pitch
    (dict(h=FAKE * 2, ldh=512), "EINVAL"),
    (dict(cols=200, ldx=208, ldr=208, ldq=208, ldh=208), "EALIGN"), (dict(ldx=260), "EALIGN"),
    (dict(ldr=264), "EALIGN"), (dict(ldh=264), "EALIGN"), (dict(ldq=264), "EALIGN"), (dict(g=(1, 24)), "EALIGN"),
    (dict(x=FAKE + 8), "EALIGN"), (dict(res=FAKE + 8), "EALIGN"), (dict(w=FAKE + 8), "EALIGN"),
    (dict(q=FAKE + 8), "EALIGN"), (dict(h=FAKE + 8), "EALIGN"), (dict(s=FAKE + 2), "EALIGN"),
    (dict(rstd=FAKE + 2), "EALIGN"), (dict(amax=FAKE + 1), "EALIGN"), (dict(inv=FAKE + 1), "EALIGN"),
    (dict(g=(0, 0)), "EUNSUPPORTED"),                  # per tensor needs a given scale
    (dict(g=(2, 0)), "EUNSUPPORTED"), (dict(g=(2, 128)), "EUNSUPPORTED"), (dict(g=(1, 48)), "EUNSUPPORTED"),
    (dict(g=(0, 128), mode=1), "EUNSUPPORTED"),
    (dict(cols=32784, ldx=32784, ldr=32784, ldq=32784, ldh=32784), "EUNSUPPORTED"),
])
def test_norm_refusals(rt, kw, status):
    assert norm(rt, **kw) == getattr(rt, status)


def grad(rt, **kw):
    a = dict(dy=FAKE, dyt=rt.BF16, rows=8, cols=256, lddy=256, h=FAKE * 2, ht=rt.BF16, ldh=256, w=FAKE, wt=rt.BF16,
             rstd=FAKE, dres=None, lddr=0, dx=FAKE * 3, lddx=256, dw=FAKE)
    a.update(kw)
    return rt.lib().fp8_rmsnorm_backward(a["dy"], a["dyt"], a["rows"], a["cols"], a["lddy"], a["h"], a["ht"],
                                         a["ldh"], a["w"], a["wt"], a["rstd"], a["dres"], a["lddr"], a["dx"],
                                         a["lddx"], a["dw"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), "EINVAL"), (dict(h=None), "EINVAL"), (dict(w=None), "EINVAL"), (dict(rstd=None), "EINVAL"),
    (dict(dx=None), "EINVAL"), (dict(rows=0), "EINVAL"), (dict(dyt=3), "EINVAL"), (dict(ht=3), "EINVAL"),
    (dict(lddy=128), "EINVAL"), (dict(ldh=128), "EINVAL"), (dict(lddx=128), "EINVAL"),
    (dict(dres=FAKE * 4, lddr=128), "EINVAL"), (dict(dx=FAKE, lddx=512), "EINVAL"), (dict(dx=FAKE * 2), "EINVAL"),
    (dict(dres=FAKE * 4, lddr=256, dx=FAKE * 4, lddx=512), "EINVAL"),
    (dict(cols=264, lddy=272, ldh=272, lddx=272), "EALIGN"), (dict(lddy=264), "EALIGN"), (dict(ldh=264), "EALIGN"),
    (dict(lddx=264), "EALIGN"), (dict(dres=FAKE * 4, lddr=264), "EALIGN"), (dict(h=FAKE + 8), "EALIGN"),
    (dict(dw=FAKE + 4), "EALIGN"), (dict(rstd=FAKE + 2), "EALIGN"), (dict(dx=FAKE + 4), "EALIGN"),
    (dict(cols=32784, lddy=32784, ldh=32784, lddx=32784), "EUNSUPPORTED"),
])
def test_gradient_refusals(rt, kw, status):
    assert grad(rt, **kw) == getattr(rt, status)


PLAN = dict(tokens=4, start=FAKE, kv=FAKE, seqs=2, max_new=2, table=FAKE, width=4, ldt=4, f=0, kc=FAKE, vc=FAKE, ks=FAKE,
            vs=FAKE, pages=8, heads=2, page=16, dim=64)
PLAN_BAD = [
    (dict(tokens=0), "EINVAL"), (dict(start=None), "EINVAL"), (dict(kv=None), "EINVAL"), (dict(seqs=0), "EINVAL"),
    (dict(max_new=0), "EINVAL"), (dict(table=None), "EINVAL"), (dict(width=0), "EINVAL"), (dict(ldt=3), "EINVAL"), (dict(f=5), "EINVAL"),
    (dict(kc=None), "EINVAL"), (dict(vc=None), "EINVAL"), (dict(ks=None), "EINVAL"), (dict(vs=None), "EINVAL"),
    (dict(pages=0), "EINVAL"), (dict(heads=0), "EINVAL"), (dict(page=0), "EINVAL"), (dict(dim=-64), "EINVAL"),
    (dict(tokens=2 ** 31), "EINVAL"), (dict(pages=2 ** 31), "EINVAL"), (dict(seqs=2 ** 31), "EINVAL"),
    (dict(page=8), "EUNSUPPORTED"), (dict(page=48), "EUNSUPPORTED"), (dict(page=256), "EUNSUPPORTED"),
    (dict(dim=32), "EUNSUPPORTED"), (dict(dim=96), "EUNSUPPORTED"), (dict(dim=256), "EUNSUPPORTED"),
    (dict(start=FAKE + 2), "EALIGN"), (dict(kv=FAKE + 1), "EALIGN"), (dict(table=FAKE + 2), "EALIGN"),
    (dict(kc=FAKE + 8), "EALIGN"), (dict(vc=FAKE + 4), "EALIGN"), (dict(ks=FAKE + 2), "EALIGN"),
    (dict(vs=FAKE + 3), "EALIGN"),
    (dict(seqs=2 ** 30, max_new=2 ** 30, tokens=2 ** 30), "EUNSUPPORTED"),  # a grid past the device's limit
]


def append(rt, **kw):
    a = dict(PLAN, k=FAKE, v=FAKE, xt=rt.BF16, ldk=128, hdk=64, ldv=128, hdv=64, eps=1e-12)
    a.update(kw)
    return rt.lib().fp8_kv_append(a["k"], a["v"], a["xt"], a["tokens"], a["ldk"], a["hdk"], a["ldv"], a["hdv"],
                                  a["start"], a["kv"], a["seqs"], a["max_new"], a["table"], a["width"], a["ldt"], a["f"],
                                  a["eps"], 0, a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["heads"], a["page"],
                                  a["dim"], None)


@pytest.mark.parametrize("kw,status", PLAN_BAD + [
    (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(xt=4), "EINVAL"), (dict(eps=0.0), "EINVAL"),
    (dict(ldk=-128), "EINVAL"), (dict(hdv=-64), "EINVAL"), (dict(ldk=132), "EALIGN"), (dict(hdk=68), "EALIGN"),
    (dict(ldv=132), "EALIGN"), (dict(hdv=4), "EALIGN"), (dict(k=FAKE + 8), "EALIGN"), (dict(v=FAKE + 2), "EALIGN"),
])
def test_append_refusals(rt, kw, status):
    assert append(rt, **kw) == getattr(rt, status)


def attend(rt, **kw):
    a = dict(PLAN, q=FAKE, qt=rt.BF16, qh=4, ldq=256, hdq=64, max_kv=64, sm=0.1, causal=1, window=0, y=FAKE,
             yt=rt.BF16, ldy=256, hdy=64, lse=FAKE)
    a.update(kw)
    return rt.lib().fp8_paged_attention(a["q"], a["qt"], a["tokens"], a["qh"], a["ldq"], a["hdq"], a["kc"], a["vc"],
                                        a["ks"], a["vs"], a["f"], a["pages"], a["heads"], a["page"], a["dim"],
                                        a["table"], a["width"], a["ldt"], a["start"], a["kv"], a["seqs"], a["max_new"],
                                        a["max_kv"], a["sm"], a["causal"], a["window"], a["y"], a["yt"], a["ldy"],
                                        a["hdy"], a["lse"], None)


@pytest.mark.parametrize("kw,status", PLAN_BAD + [
    (dict(q=None), "EINVAL"), (dict(y=None), "EINVAL"), (dict(qt=9), "EINVAL"), (dict(yt=9), "EINVAL"),
    (dict(qh=0), "EINVAL"), (dict(qh=3), "EINVAL"), (dict(max_kv=0), "EINVAL"), (dict(window=-1), "EINVAL"),
    (dict(sm=float("inf")), "EINVAL"), (dict(sm=float("nan")), "EINVAL"), (dict(ldq=-256), "EINVAL"),
    (dict(qt=0), "EUNSUPPORTED"), (dict(yt=0), "EUNSUPPORTED"),
    (dict(ldq=260), "EALIGN"), (dict(hdq=60), "EALIGN"), (dict(ldy=258), "EALIGN"), (dict(hdy=62), "EALIGN"),
    (dict(q=FAKE + 8), "EALIGN"), (dict(y=FAKE + 4), "EALIGN"), (dict(lse=FAKE + 2), "EALIGN"),
])
def test_attention_refusals(rt, kw, status):
    assert attend(rt, **kw) == getattr(rt, status)


def test_packed_call(rt):
    """Arguments as 64-bit words: the same refusals as the call itself, and its own."""
    import struct

    L = rt.lib()

    def packed(fmt, *words):
        record = struct.pack(fmt, *words)
        return L.fp8_call_packed(record, len(record) // 8)

    def grad(dy=FAKE, rows=8, lddy=256, dyt=1, h=FAKE * 2, call=1, fmt="18q", extra=()):
        return packed(fmt, call, dy, dyt, rows, 256, lddy, h, 1, 256, FAKE, 1, FAKE, 0, 0, FAKE * 3, 256, FAKE, 0, *extra)

    assert grad(dy=0) == rt.EINVAL and grad(rows=0) == rt.EINVAL and grad(lddy=128) == rt.EINVAL
    assert grad(lddy=264) == rt.EALIGN and grad(h=FAKE + 8) == rt.EALIGN
    assert grad(dyt=1 + 2 ** 32) == rt.EINVAL        # an enumerator does not wrap
    assert grad(call=4) == rt.EINVAL and grad(call=-1) == rt.EINVAL
    assert grad(call=0) == rt.EINVAL and grad(call=2) == rt.EINVAL  # another call's number of words
    assert grad(fmt="19q", extra=(0,)) == rt.EINVAL
    assert L.fp8_call_packed(None, 18) == rt.EINVAL and L.fp8_call_packed(b"", 0) == rt.EINVAL

    def norm(eps=1e-12, norm_eps=1e-6, gr=1, gc=0, mode=0):
        return packed("10qd4qd10q", 0, FAKE, 1, 8, 256, 256, 0, 0, FAKE, 1,
                      norm_eps, gr, gc, 0, mode, eps, 0, FAKE, 0, FAKE, 256, 0, 0, 0, 0, 0)

    assert norm(eps=0.0) == rt.EINVAL and norm(norm_eps=-1.0) == rt.EINVAL and norm(mode=7) == rt.EINVAL
    assert norm(gr=2) == rt.EUNSUPPORTED and norm(gr=0) == rt.EUNSUPPORTED and norm(gc=48) == rt.EUNSUPPORTED
    assert norm(gr=2 ** 40) == rt.EINVAL


def test_binding_refusals(rt):
    """Shapes and types the binding turns down before it passes pointers (CPU tensors: never used)."""
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    x, w, q = torch.zeros(4, 64, dtype=bf), torch.zeros(64, dtype=bf), torch.zeros(4, 64, dtype=u8)
    s = torch.zeros(4, 1)

    def n(**kw):
        a = dict(x=x, weight=w, norm_eps=1e-6, gran=(1, 0), fmt=0, mode=0, eps=1e-12, pow2_round_up=False, scale=s, q=q)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            rt.fp8_rmsnorm_quantize(**a)
    n(x=x.half())
    n(x=x.t())
    n(q=q[:, :48])
    n(q=q.int())
    n(weight=w[:32])
    n(residual=x.float())
    n(residual=x[:3])
    n(h=x.float())
    n(rstd=torch.zeros(3))
    n(scale=torch.zeros(3, 1))
    n(scale=s.double())
    n(amax_out=torch.zeros(2))
    for kw in (dict(h=x[:3]), dict(dx=x.float()), dict(rstd=torch.zeros(4, dtype=bf)), dict(dweight=torch.zeros(63)),
               dict(dresidual=x.float()), dict(weight=w[::2])):
        a = dict(dy=x, h=x, weight=w, rstd=torch.zeros(4), dx=x.clone(), dweight=torch.zeros(64))
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            rt.fp8_rmsnorm_backward(**a)
    c, sc = torch.zeros(8, 2, 16, 64, dtype=u8), torch.zeros(8, 2)
    tb, st, kv = torch.zeros(2, 4, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    k = torch.zeros(4, 2, 64, dtype=bf)
    plan = dict(k_cache=c, v_cache=c, k_scale=sc, v_scale=sc, fmt=0, block_table=tb, seq_start=st, kv_len=kv)
    for kw in (dict(k_cache=c.int()), dict(v_cache=c[:4]), dict(k_scale=sc[:4]), dict(v_scale=sc.double()),
               dict(block_table=tb.long()), dict(block_table=tb[:1]), dict(seq_start=st[:2]), dict(kv_len=kv.long()),
               dict(k=k[:, :1]), dict(v=k[:3]), dict(v=k.float()), dict(k=k.transpose(1, 2)),
               dict(k_cache=c.transpose(1, 2))):
        a = dict(plan, k=k, v=k, max_new=2)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            rt.fp8_kv_append(**a)
    qq = torch.zeros(4, 4, 64, dtype=bf)
    for kw in (dict(q=qq[:, :, :32]), dict(y=qq[:3]), dict(lse=torch.zeros(4, 3)), dict(lse=torch.zeros(4, 4, dtype=bf)),
               dict(q=qq.half()), dict(y=qq.half())):
        a = dict(plan, q=qq, max_new=2, max_kv=64, sm_scale=0.1, y=qq.clone())
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            rt.fp8_paged_attention(**a)
