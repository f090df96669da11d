"""Refusals of the speculative decoding operators on the host, before any CUDA call (CPU only)."""
import ctypes

import pytest
import torch

from invariant_paged_kv_gb300 import build, pa

P = 1 << 12


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pa.load()


@pytest.fixture(autouse=True)
def nothing_launched(lib):
    before = lib.pa_kernel_launches()
    yield
    assert lib.pa_kernel_launches() == before


def tree(lib, **kw):
    a = dict(q=P, kc=P, vc=P, bt=P, mb=4, cu=P, ctx=P, par=P, slot=None, kn=None, vn=None, out=P, B=1,
             T=1, H=4, Hkv=2, D=64, bs=16, NB=8, mq=1, mc=16, scale=0.125, dt=1, ks=1.0, vs=1.0, ws=P,
             wsb=1 << 20, st=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pa_attention_tree(*a.values())


def test_attention_tree(lib):
    assert tree(lib, B=0, T=0) == 0
    assert tree(lib, T=0) == 0
    for bad in (dict(B=-1), dict(T=-1), dict(NB=0), dict(mq=-1), dict(mc=-1), dict(H=0), dict(B=0, T=1),
                dict(q=None), dict(kc=None), dict(vc=None), dict(bt=None), dict(cu=None), dict(ctx=None),
                dict(par=None), dict(out=None), dict(mb=0), dict(q=P + 8), dict(out=P + 8), dict(kc=P + 8),
                dict(slot=P), dict(slot=P, kn=P), dict(slot=P, kn=P + 8, vn=P), dict(scale=0.0),
                dict(scale=float("nan")), dict(dt=2, ks=0.0), dict(dt=2, vs=float("inf"))):
        assert tree(lib, **bad) == 1, bad
    for bad in (dict(D=96), dict(bs=8), dict(H=6, Hkv=4), dict(H=34), dict(dt=5), dict(mq=257),
                dict(mc=(1 << 30) + 1), dict(NB=1 << 27, bs=32)):
        assert tree(lib, **bad) == 2, bad
    for dt, mc in ((1, 257), (2, 5000), (0, 257)):
        for bad in (dict(ws=None), dict(ws=P + 16), dict(wsb=64)):
            assert tree(lib, dt=dt, mc=mc, **bad) == 3, bad


def test_tree_workspace_bytes(lib):
    f = lib.pa_tree_workspace_bytes
    row = 40 * (128 + 2) * 4
    # ceil(max_ctx / 256) splits a row, at most 32; none up to one split
    assert f(8, 100, 16, 256, 40, 8, 128, 16, 1) == 256
    assert 17 * 100 * row <= f(8, 100, 16, 4100, 40, 8, 128, 16, 1) < 17 * 100 * row + 1024
    # e4m3: and q in two 8-bit pieces, with a byte per row
    extra = 100 * 40 * (2 * 128 + 1)
    assert 32 * 100 * row + extra <= f(8, 100, 16, 1 << 20, 40, 8, 128, 16, 2) < 32 * 100 * row + extra + 2048
    assert extra <= f(8, 100, 16, 100, 40, 8, 128, 16, 2) < extra + 1024
    # fp32: / 128
    assert 8 * 100 * row <= f(8, 100, 16, 1000, 40, 8, 128, 16, 0) < 8 * 100 * row + 1024
    assert f(8, 0, 16, 4100, 40, 8, 128, 16, 1) == 256
    for bad in ((-1, 1, 1, 1, 4, 2, 64, 16, 1), (1, 1, 257, 300, 4, 2, 64, 16, 1), (1, 1, 1, 1, 4, 2, 96, 16, 1),
                (1, -1, 1, 1, 4, 2, 64, 16, 1), (1, 1, 1, -1, 4, 2, 64, 16, 1)):
        assert f(*bad) == 0
    with pytest.raises(pa.PaError, match="PA_ERR_UNSUPPORTED"):
        pa.tree_workspace_bytes(1, 1, 257, 300, 4, 2, 64, 16, torch.bfloat16)


def test_verify_tree(lib):
    def f(**kw):
        a = dict(p=P, q=P, tok=P, par=P, cu=P, ua=P, us=P, n=P, path=P, out=P, B=1, T=4, V=100, mq=4,
                 st=None, stream=None)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.pa_verify_tree(*a.values())
    assert f(B=0, T=0) == 0
    for bad in (dict(B=-1), dict(T=-1), dict(V=0), dict(V=-5), dict(mq=0), dict(B=0), dict(p=None),
                dict(tok=None), dict(par=None), dict(cu=None), dict(ua=None), dict(us=None), dict(n=None),
                dict(path=None), dict(out=None), dict(p=P + 4), dict(q=P + 8), dict(tok=P + 2)):
        assert f(**bad) == 1, bad
    for bad in (dict(mq=257), dict(V=(1 << 24) + 1)):
        assert f(**bad) == 2, bad


def test_page_operators(lib):
    arr = (ctypes.c_void_p * 2)(P, P)
    odd = (ctypes.c_void_p * 2)(P, P + 8)
    hole = (ctypes.c_void_p * 2)(P, None)

    def compact(**kw):
        a = dict(k=arr, v=arr, L=2, bt=P, mb=4, cu=P, ctx=P, path=P, n=P, new=2 * P, B=1, T=1, NB=8, bs=16,
                 Hkv=2, D=64, dt=1, st=None, stream=None)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.pa_compact_kv(*a.values())
    assert compact(B=0, T=0) == 0
    for bad in (dict(L=-1), dict(L=0), dict(B=-1), dict(T=-1), dict(NB=0), dict(B=0), dict(k=None), dict(v=None),
                dict(bt=None), dict(mb=0), dict(cu=None), dict(ctx=None), dict(path=None), dict(n=None),
                dict(new=None), dict(new=P), dict(k=odd), dict(v=hole), dict(Hkv=0)):
        assert compact(**bad) == 1, bad
    for bad in (dict(D=96), dict(bs=8), dict(dt=5), dict(NB=1 << 27, bs=32)):
        assert compact(**bad) == 2, bad

    def copy(**kw):
        a = dict(k=arr, v=arr, L=2, pairs=P, n=1, NB=8, bs=16, Hkv=2, D=64, dt=1, st=None, stream=None)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.pa_copy_blocks(*a.values())
    assert copy(n=0) == 0 and copy(L=0) == 0
    for bad in (dict(L=-1), dict(n=-1), dict(NB=0), dict(k=None), dict(v=None), dict(pairs=None),
                dict(pairs=P + 4), dict(k=odd), dict(v=hole), dict(Hkv=0)):
        assert copy(**bad) == 1, bad
    for bad in (dict(D=96), dict(bs=8), dict(dt=5), dict(NB=1 << 27, bs=32), dict(n=(1 << 16) + 1)):
        assert copy(**bad) == 2, bad


def test_binding_refuses_before_the_library(lib):
    """Host tensors, wrong types and shapes raise in the binding: no pointer of theirs reaches a kernel."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, kc = torch.zeros(3, 4, 64), torch.zeros(8, 16, 2, 64)
    good = dict(q=q, k_cache=kc, v_cache=kc.clone(), block_tables=i(1, 4), cu_seqlens_q=i(2), ctx_lens=i(1),
                tree_parents=i(3), out=q.clone())
    kw = dict(max_q_len=3, max_ctx_len=9, scale=0.1, workspace=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        pa.attention_tree(*good.values(), **kw)
    for name, value in [("v_cache", torch.zeros(8, 16, 2, 128)), ("out", torch.zeros(2, 4, 64)),
                        ("block_tables", i(2, 4)), ("cu_seqlens_q", i(3)), ("tree_parents", i(2)),
                        ("block_tables", i(4))]:
        with pytest.raises(ValueError):
            pa.attention_tree(*dict(good, **{name: value}).values(), **kw)
    with pytest.raises(TypeError):
        pa.attention_tree(*dict(good, q=q.half(), out=q.half()).values(), **kw)
    with pytest.raises(ValueError, match="slot_mapping|k_new"):
        pa.attention_tree(*good.values(), **kw, k_new=torch.zeros(3, 1, 64), v_new=torch.zeros(3, 2, 64),
                          slot_mapping=torch.zeros(3, dtype=torch.int64))
    p = torch.zeros(4, 10)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        pa.verify_tree(p, None, i(4), i(4), i(2), f, torch.zeros(1), i(1), i(4), i(4), max_q_len=4)
    with pytest.raises(ValueError, match="draft_probs"):
        pa.verify_tree(p, torch.zeros(4, 9), i(4), i(4), i(2), f, torch.zeros(1), i(1), i(4), i(4), max_q_len=4)
    with pytest.raises(ValueError, match="path"):
        pa.verify_tree(p, None, i(4), i(4), i(2), f, torch.zeros(1), i(1), i(3), i(4), max_q_len=4)
    for k, v in [([], []), ([kc], []), ([kc], [torch.zeros(8, 16, 2, 128)]), ([kc], [kc]), ([kc[0]], [kc[0]])]:
        with pytest.raises(ValueError):
            pa.LayerCaches(k, v)
    with pytest.raises(TypeError):
        pa.LayerCaches([kc.half()], [kc.half()])


@pytest.mark.parametrize("given", [("k_new",), ("v_new",), ("slot_mapping",), ("k_new", "v_new"), ("k_new", "slot_mapping")])
def test_binding_wants_the_write_whole(lib, given):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, kc = torch.zeros(3, 4, 64), torch.zeros(8, 16, 2, 64)
    new = dict(k_new=torch.zeros(3, 2, 64), v_new=torch.zeros(3, 2, 64), slot_mapping=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="go together"):
        pa.attention_tree(q, kc, kc.clone(), i(1, 4), i(2), i(1), i(3), q.clone(), max_q_len=3, max_ctx_len=9,
                          scale=0.1, workspace=torch.zeros(256, dtype=torch.uint8), **{k: new[k] for k in given})


def test_compact_wants_its_output_apart(lib):
    """new_ctx_lens over any part of an input is refused: the kernel's CTAs would read what another wrote."""
    arr = (ctypes.c_void_p * 1)(P)
    place = dict(bt=2 * P, cu=3 * P, ctx=4 * P, path=5 * P, n=6 * P)  # 40 lanes, 4 blocks each, 100 rows
    size = dict(bt=640, cu=164, ctx=160, path=400, n=160)
    for name, at in place.items():
        for new in (at, at - 156, at + size[name] - 4):
            a = dict(k=arr, v=arr, L=1, bt=2 * P, mb=4, cu=3 * P, ctx=4 * P, path=5 * P, n=6 * P, new=new, B=40,
                     T=100, NB=8, bs=16, Hkv=2, D=64, dt=1, st=None, stream=None)
            assert lib.pa_compact_kv(*a.values()) == 1, (name, new - at)


def test_arrays_off_their_elements_boundary(lib):
    """A 32-bit (64-bit) array that does not start on a 4 (8) byte boundary would fault in a kernel: refused."""
    for name in ("bt", "cu", "ctx", "par", "st"):
        for off in (1, 2):
            assert tree(lib, **{name: P + off}) == 1, name
    assert tree(lib, slot=P + 4, kn=P, vn=P) == 1
    verify = dict(p=P, q=P, tok=P, par=P, cu=P, ua=P, us=P, n=P, path=P, out=P, B=1, T=4, V=100, mq=4, st=P,
                  stream=None)
    for name in ("tok", "par", "cu", "ua", "us", "n", "path", "out", "st"):
        assert lib.pa_verify_tree(*dict(verify, **{name: P + 2}).values()) == 1, name
    arr = (ctypes.c_void_p * 1)(P)
    compact = dict(k=arr, v=arr, L=1, bt=P, mb=4, cu=P, ctx=P, path=P, n=P, new=2 * P, B=1, T=1, NB=8, bs=16, Hkv=2,
                   D=64, dt=1, st=P, stream=None)
    for name in ("bt", "cu", "ctx", "path", "n", "new", "st"):
        assert lib.pa_compact_kv(*dict(compact, **{name: compact[name] + 2}).values()) == 1, name
    copy = dict(k=arr, v=arr, L=1, pairs=P, n=1, NB=8, bs=16, Hkv=2, D=64, dt=1, st=P + 2, stream=None)
    assert lib.pa_copy_blocks(*copy.values()) == 1
