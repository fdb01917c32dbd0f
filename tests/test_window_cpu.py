"""Refusals of the rotary, logits and acceptance calls: every bad argument is
turned down on the host, with its code, before anything is launched, by the C ABI
(fake addresses) and by the binding; and the frequencies, which are the host's."""
import ctypes
import math
import os

import pytest
import torch

from speculative_verify_gdn_amd import gdn
from tests.test_kv_binding_cpu import BF, Stream, fake
from tests.test_kv_cpu import p

E, U = gdn.GDN_EINVAL, gdn.GDN_EUNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.skip("libgdn.so not built")
    return gdn.load()


def st(*s):
    return (ctypes.c_longlong * 3)(*s)


TURN = dict(pos=None, lens=p(10), parent=p(11), count=p(12), freqs=p(13), rot=32, layout=0, mscale=1.0, B=2, K=3, D=64,
            dtype=gdn.GDN_BF16)
CALLS = {
    "gdn_rope": ("x x_strides y y_strides pos lens parent count freqs rot layout mscale B K H D dtype",
                 dict(TURN, x=p(1), x_strides=None, y=p(2), y_strides=None, H=4)),
    "gdn_qk_norm_rope": ("q q_strides k k_strides wq wk eps q_out k_out pos lens parent count freqs rot layout mscale B K Hq "
                         "Hk D dtype",
                         dict(TURN, q=p(1), q_strides=st(4608, 1536, 64), k=p(2), k_strides=None, wq=p(3), wk=p(4), eps=1e-6,
                              q_out=p(5), k_out=p(6), Hq=4, Hk=2)),
    "gdn_kv_append_rope": ("q q_strides k k_strides v v_strides wq wk eps q_out k_pages v_pages pos lens parent count table "
                           "freqs rot layout mscale B K Hq Hkv D page n_pages P dtype",
                           dict(TURN, q=p(1), q_strides=None, k=p(2), k_strides=None, v=p(3), v_strides=None, wq=p(4),
                                wk=p(5), eps=1e-6, q_out=p(6), k_pages=p(7), v_pages=p(8), table=p(9), Hq=4, Hkv=2, page=16,
                                n_pages=8, P=4)),
    "gdn_logits_adjust": ("logits logits_stride out out_stride best history history_lens history_start capacity tokens "
                          "parent count params bias_ids bias_values n_bias mask noise workspace workspace_bytes B K V dtype "
                          "out_dtype",
                          dict(logits=p(1), logits_stride=1000, out=p(2), out_stride=1000, best=p(3), history=p(4),
                               history_lens=p(5), history_start=p(6), capacity=100, tokens=p(7), parent=p(8), count=p(9),
                               params=p(10), bias_ids=p(11), bias_values=p(12), n_bias=5, mask=p(13), noise=p(14),
                               workspace=p(15), workspace_bytes=1 << 20, B=2, K=3, V=1000, dtype=0, out_dtype=1)),
    "gdn_accept_tree": ("target tokens parent count root node next history lens lens_out capacity B K",
                        dict(target=p(1), tokens=p(2), parent=p(3), count=p(4), root=p(5), node=p(6), next=p(7),
                             history=p(8), lens=p(9), lens_out=p(10), capacity=50, B=2, K=3)),
}


def call(lib, name, **kw):
    order, args = CALLS[name]
    args = dict(args, **kw)
    return getattr(lib, name)(*[args[a] for a in order.split()], None)


inf, nan = float("inf"), float("nan")
BAD_TURN = [(dict(rot=31), E), (dict(rot=-2), E), (dict(rot=66), E), (dict(layout=2), E), (dict(layout=-1), E),
            (dict(mscale=inf), E), (dict(mscale=nan), E), (dict(freqs=None), E), (dict(freqs=p(13, 4)), E), (dict(dtype=2), E),
            (dict(B=-1), E), (dict(K=0), E), (dict(B=65536), U), (dict(K=65537, parent=None), U),
            (dict(B=65535, K=65536, parent=None), U), (dict(K=65), U), (dict(lens=p(10, 2)), E),
            (dict(pos=p(14, 1)), E), (dict(count=p(12, 2)), E), (dict(parent=p(11, 3)), E)]
BAD = {
    "gdn_rope": BAD_TURN + [(dict(D=0), E), (dict(rot=0), E), (dict(D=40, rot=32), U), (dict(D=528), U), (dict(H=0), E), (dict(H=1025), U),
                            (dict(x=None), E), (dict(y=None), E), (dict(x=p(1, 8)), E), (dict(y=p(2, 4)), E),
                            (dict(x_strides=st(768, 256, 60)), E), (dict(x_strides=st(-768, 256, 64)), E),
                            (dict(x_strides=st(1 << 41, 256, 64)), E), (dict(y_strides=st(768, 256, 0)), E),
                            (dict(y_strides=st(768, 128, 64)), E), (dict(y_strides=st(256, 256, 64)), E),
                            (dict(y_strides=st(64, 128, 200)), E), (dict(y=p(1, 512)), E),
                            (dict(y=p(1), y_strides=st(1024, 256, 64)), E), (dict(y=p(10)), E), (dict(y=p(13)), E),
                            (dict(x_strides=st(1 << 38, 1 << 38, 64), K=60000, parent=None), U)],
    "gdn_qk_norm_rope": BAD_TURN + [(dict(Hq=0), E), (dict(Hk=0), E), (dict(Hq=1025), U), (dict(q=None), E), (dict(wk=None), E),
                                    (dict(k_out=None), E), (dict(eps=-1.0), E), (dict(eps=nan), E), (dict(eps=inf), E),
                                    (dict(wq=p(3, 2)), E), (dict(q_out=p(1)), E), (dict(q_out=p(2)), E), (dict(k_out=p(5)), E),
                                    (dict(k_out=p(3)), E), (dict(q_out=p(5, 8)), E), (dict(k_out=p(1)), E),
                                    (dict(q_strides=st(4608, 1536, 63)), E)],
    "gdn_kv_append_rope": BAD_TURN + [(dict(D=96), U), (dict(page=24), U), (dict(page=8), U), (dict(Hkv=0), E), (dict(n_pages=0), E),
                                      (dict(P=0), E), (dict(Hq=-1), E), (dict(Hq=2000), U), (dict(q=None), E),
                                      (dict(q_out=None), E), (dict(Hq=0), E), (dict(q=None, q_out=None, Hq=0), E),
                                      (dict(k=None), E), (dict(v=None), E), (dict(lens=None), E), (dict(table=None), E),
                                      (dict(k_pages=p(8)), E), (dict(v_pages=p(3)), E), (dict(q_out=p(7)), E),
                                      (dict(k_pages=p(1)), E), (dict(v_pages=p(9)), E), (dict(v=p(3, 8)), E),
                                      (dict(table=p(9, 2)), E), (dict(eps=-1e-6), E), (dict(q_out=p(2)), E),
                                      (dict(v_strides=st(64, 32, 60)), E)],
    "gdn_logits_adjust": [(dict(B=-1), E), (dict(K=0), E), (dict(V=0), E), (dict(K=65), U), (dict(B=65536), U),
                          (dict(V=(1 << 24) + 1), U), (dict(dtype=5), E), (dict(out_dtype=-1), E), (dict(logits=None), E),
                          (dict(out=None, best=None, noise=None), E), (dict(out=None, best=None), E), (dict(best=None), E),
                          (dict(logits_stride=999), E), (dict(out_stride=10), E), (dict(logits=p(1, 8)), E),
                          (dict(noise=p(14, 4)), E), (dict(workspace=p(15, 8)), E), (dict(best=p(3, 2)), E),
                          (dict(history_lens=None), E), (dict(capacity=0), E), (dict(capacity=(1 << 29) + 1), E),
                          (dict(n_bias=-1), E), (dict(n_bias=(1 << 20) + 1), E), (dict(bias_ids=None), E),
                          (dict(bias_values=None), E), (dict(workspace=None), E), (dict(workspace_bytes=8), E),
                          (dict(out=p(1)), E), (dict(out=p(1, 16)), E), (dict(best=p(1, 64)), E), (dict(workspace=p(2)), E),
                          (dict(out=p(14)), E), (dict(best=p(9)), E), (dict(mask=p(13, 2)), E), (dict(params=p(10, 2)), E)],
    "gdn_accept_tree": [(dict(B=-1), E), (dict(K=0), E), (dict(K=65), U), (dict(B=(1 << 20) + 1), U), (dict(target=None), E),
                        (dict(tokens=None), E), (dict(node=None), E), (dict(next=None), E), (dict(history=None), E),
                        (dict(lens=None), E), (dict(lens_out=None), E), (dict(capacity=0), E), (dict(target=p(1, 2)), E),
                        (dict(node=p(1)), E), (dict(next=p(6)), E), (dict(lens_out=p(9, 4)), E), (dict(history=p(5)), E),
                        (dict(next=p(3)), E)],
}


@pytest.mark.parametrize("name,kw,code", [(n, kw, c) for n in BAD for kw, c in BAD[n]])
def test_refused_on_the_host(lib, name, kw, code):
    assert call(lib, name, **kw) == code
    assert lib.gdn_last_error().decode().startswith(name)


@pytest.mark.parametrize("name", CALLS)
def test_empty_calls_are_ok(lib, name):
    assert call(lib, name, B=0) == gdn.GDN_OK


def test_logits_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.gdn_logits_workspace(2, 3, 1000, ctypes.byref(n)) == gdn.GDN_OK and n.value >= 48
    assert lib.gdn_logits_workspace(2, 3, 0, ctypes.byref(n)) == E
    assert lib.gdn_logits_workspace(2, 65, 10, ctypes.byref(n)) == U
    assert lib.gdn_logits_workspace(2, 3, 1000, None) == E
    assert lib.gdn_logits_workspace(0, 3, 1000, ctypes.byref(n)) == gdn.GDN_OK


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 1e6), (30, 500000.0), (512, 1.5)])
def test_frequencies(rot, base):
    i = torch.arange(rot // 2, dtype=torch.float64)
    plain = torch.tensor([base ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float64)
    close = dict(rtol=1e-13, atol=0)
    f, m = gdn.rope_freqs(rot, base, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0
    torch.testing.assert_close(f, plain, **close)
    f, m = gdn.rope_freqs(rot, base, "linear", 4.0, device="cpu")
    torch.testing.assert_close(f, plain / 4, **close)
    assert m == 1.0
    if rot > 2:
        f, m = gdn.rope_freqs(rot, base, "ntk", 4.0, device="cpu")
        # the slowest pair turns as with linear scaling, the fastest as without
        torch.testing.assert_close(f[0], plain[0], **close)
        torch.testing.assert_close(f[-1], plain[-1] / 4, rtol=1e-12, atol=0)
    turns = 4096 * plain / (2 * math.pi)
    for scaling, at in (("bands", lambda n: (n - 1) / (4 - 1)), ("yarn", lambda n: torch.log(n) / math.log(4.0))):
        f, m = gdn.rope_freqs(rot, base, scaling, 8.0, low=1.0, high=4.0, original=4096, device="cpu")
        k = at(turns).clamp(0, 1)
        torch.testing.assert_close(f, k * plain + (1 - k) * plain / 8, rtol=1e-12, atol=0)
        assert m == (1.0 if scaling == "bands" else pytest.approx(0.1 * math.log(8) + 1, rel=2 ** -24))
        torch.testing.assert_close(f[turns >= 4.001], plain[turns >= 4.001], **close)
        torch.testing.assert_close(f[turns <= 0.999], plain[turns <= 0.999] / 8, **close)


@pytest.mark.parametrize("kw,code", [(dict(rot=0), E), (dict(rot=7), E), (dict(rot=514), U), (dict(base=1.0), E),
                                     (dict(base=nan), E), (dict(factor=0.5, scaling="linear"), E),
                                     (dict(factor=inf, scaling="ntk"), E), (dict(rot=2, scaling="ntk", factor=2.0), E),
                                     (dict(scaling="yarn", factor=2.0), E), (dict(scaling="bands", factor=2.0, original=-1.0), E),
                                     (dict(scaling="yarn", factor=2.0, original=100.0, low=4.0, high=4.0), E)])
def test_frequencies_refused(kw, code):
    with pytest.raises(gdn.GdnError) as e:
        gdn.rope_freqs(**dict(dict(rot=64, device="cpu"), **kw))
    assert e.value.code == code


def test_frequencies_of_no_such_scaling():
    with pytest.raises(ValueError, match="scaling"):
        gdn.rope_freqs(64, scaling="none", device="cpu")


# ---------------------------------------------------------------- the binding
F32, F64, I32 = torch.float32, torch.float64, torch.int32
SHAPES = dict(x=(2, 3, 4, 64), y=(2, 3, 4, 64), q=(2, 3, 4, 64), q_out=(2, 3, 4, 64), k=(2, 3, 2, 64), v=(2, 3, 2, 64),
              k_out=(2, 3, 2, 64), k_pages=(8, 2, 16, 64), v_pages=(8, 2, 16, 64), table=(2, 4), wq=(64,), wk=(64,), freqs=(16,),
              pos=(2, 3), lens=(2,), parent=(2, 3), count=(2,), logits=(2, 3, 100), out=(2, 3, 100), best=(2, 3),
              history=(2, 20), history_lens=(2,), history_start=(2,), tokens=(2, 3), params=(2, 4), bias_ids=(2, 5),
              bias_values=(2, 5), mask=(2, 3, 4), noise=(2, 3, 100), workspace=(1024,), target=(2, 3), node=(2,), next=(2,),
              root=(2,), lens_out=(2,))
TYPES = dict(dict.fromkeys("x y q q_out k v k_out k_pages v_pages logits out".split(), BF),
             **dict.fromkeys("wq wk params bias_values noise".split(), F32), freqs=F64, workspace=torch.uint8)
BOUND = {
    "rope": "x y freqs pos lens parent count",
    "qk_norm_rope": "q k wq wk freqs q_out k_out pos lens parent count",
    "kv_append_rope": "k v k_pages v_pages lens table freqs q q_out wq wk pos parent count",
    "logits_adjust": "logits out best history history_lens history_start tokens parent count params bias_ids bias_values mask "
                     "noise workspace",
    "accept_tree": "target tokens node next parent count root history lens lens_out",
}


def bound(name, **other):
    args = {a: fake(*SHAPES[a], dtype=TYPES.get(a, I32)) for a in BOUND[name].split()}
    args.update(other)
    return getattr(gdn, name)(**args, stream=Stream)


@pytest.mark.parametrize("name,arg", [(n, a) for n in BOUND for a in BOUND[n].split()])
def test_binding_checks_each_tensor(lib, name, arg):
    shape, dtype = SHAPES[arg], TYPES.get(arg, I32)
    with pytest.raises(ValueError, match="one device"):
        bound(name, **{arg: fake(*shape, dtype=dtype, device="cuda:1")})
    with pytest.raises(ValueError, match="device tensors"):
        bound(name, **{arg: fake(*shape, dtype=dtype, device="cpu")})
    with pytest.raises((TypeError, ValueError)):
        bound(name, **{arg: 7})
    if arg != "workspace":
        with pytest.raises((TypeError, ValueError)):
            bound(name, **{arg: fake(*shape, dtype=torch.float16)})
        with pytest.raises((TypeError, ValueError)):
            bound(name, **{arg: fake(*shape, 1, dtype=dtype)})
        if name != "accept_tree" or arg != "history":
            with pytest.raises((TypeError, ValueError, gdn.GdnError)):
                bound(name, **{arg: fake(*shape[:-1], shape[-1] + 1, dtype=dtype)})


@pytest.mark.parametrize("name,kw", [("rope", dict(freqs=None)), ("kv_append_rope", dict(q=None)), ("kv_append_rope", dict(q_out=None)),
                                     ("logits_adjust", dict(workspace=None)), ("logits_adjust", dict(history_lens=None)),
                                     ("logits_adjust", dict(bias_values=None)), ("rope", dict(mscale="1")),
                                     ("qk_norm_rope", dict(eps=None)), ("accept_tree", dict(node=None))])
def test_binding_needs_them_together(lib, name, kw):
    with pytest.raises((TypeError, ValueError)):
        bound(name, **kw)


def test_binding_strides(lib):
    with pytest.raises(ValueError, match="dense heads"):
        bound("rope", x=fake(2, 3, 4, 128, dtype=BF)[..., ::2])
    with pytest.raises(ValueError, match="evenly spaced"):
        bound("logits_adjust", logits=fake(3, 2, 100, dtype=BF).transpose(0, 1))
    with pytest.raises(gdn.GdnError):   # no multiple of 16 bytes
        bound("rope", x=fake(2, 3, 4, 68, dtype=BF)[..., :64])
