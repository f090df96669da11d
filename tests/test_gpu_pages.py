"""pa_compact_kv and pa_copy_blocks: bit-exact against the definition, every type, layers beyond one
launch, overlapping moves, refusals, streams and graphs."""
import numpy as np
import pytest
import torch

import oracle.speculative as osp
from invariant_paged_kv_gb300 import build, pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    pa.load()


KIND = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.uint8}


def layers(L, NB, bs, Hkv, D, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(2 * L):
        raw = torch.randint(0, 256, (NB, bs, Hkv, D * KIND[dtype].itemsize), generator=g, device="cuda",
                            dtype=torch.uint8)  # any bytes: NaN patterns too
        out.append(raw.view(KIND[dtype]))
    return out[:L], out[L:]


def raw(ts):
    return [t.view(torch.uint8).cpu().numpy() for t in ts]


def lanes(seed, B, n_max, past_max, bs, fixed=None):
    rng = np.random.default_rng(seed)
    n = rng.integers(0, n_max + 1, B) if fixed is None else np.array(fixed)
    past = rng.integers(0, past_max + 1, B)
    keep, path = [], []
    for k in n:
        if k == 0:
            keep.append(-1)
            continue
        a = int(rng.integers(0, k))
        p = [0] + sorted(rng.choice(np.arange(1, k), a, replace=False).tolist()) if k > 1 else [0]
        keep.append(len(p) - 1)
        path += p + [-1] * (int(k) - len(p))
    ctx = (past + n).astype(np.int32)
    need = [-(-int(c) // bs) for c in ctx]
    NB = sum(need) + 2
    ids = rng.permutation(NB)
    table = np.full((B, max(need + [1])), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return dict(tables=table, cu=cu, ctx=ctx, path=np.array(path, np.int32), keep=np.array(keep, np.int32), NB=NB)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def compact(k, v, s, status=None, stream=None, **over):
    s = dict(s, **over)
    new = torch.full((len(s["ctx"]),), -9, dtype=torch.int32, device="cuda")
    st = pa.new_status() if status is None else status
    pa.compact_kv(pa.LayerCaches(k, v), dev(s["tables"]), dev(s["cu"]), dev(s["ctx"]), dev(s["path"]),
                  dev(s["keep"]), new, status=st, stream=stream)
    return new.cpu().numpy(), pa.read_status(st)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("B,n_max,L,Hkv,D,bs", [(1, 4, 1, 2, 64, 16), (7, 9, 3, 8, 128, 16),
                                                (40, 33, 2, 1, 64, 32), (3, 256, 5, 3, 128, 32)])
def test_compact(dtype, B, n_max, L, Hkv, D, bs):
    s = lanes(B + L, B, n_max, 70, bs, fixed=[4] if B == 1 else None)
    k, v = layers(L, s["NB"], bs, Hkv, D, dtype, seed=B)
    want, new = osp.compact_kv(raw(k + v), s["tables"], s["cu"], s["ctx"], s["path"], s["keep"])
    got_new, flags = compact(k, v, s)
    assert flags == 0
    np.testing.assert_array_equal(got_new, new)
    for a, b in zip(raw(k + v), want):  # every other byte as it was
        np.testing.assert_array_equal(a, b)


def test_compact_moves_that_overlap():
    """Rows that are both read and written over: the read comes first, in any length of path."""
    for a in (2, 3, 4, 5, 9, 64, 255):
        n = a + 1
        path = [0] + list(range(2, n)) + [-1]  # each row moves one place down
        s = dict(tables=np.arange(20, dtype=np.int32)[None], cu=np.array([0, n], np.int32),
                 ctx=np.array([13 + n], np.int32), path=np.array(path, np.int32),
                 keep=np.array([n - 2], np.int32), NB=20)
        k, v = layers(2, 20, 16, 2, 64, "bf16", seed=a)
        want, new = osp.compact_kv(raw(k + v), s["tables"], s["cu"], s["ctx"], s["path"], s["keep"])
        got_new, flags = compact(k, v, s)
        assert flags == 0 and got_new.tolist() == new.tolist()
        for x, y in zip(raw(k + v), want):
            np.testing.assert_array_equal(x, y)


def test_compact_many_layers():
    s = lanes(3, 5, 8, 40, 16, fixed=[8, 3, 0, 1, 6])
    k, v = layers(230, s["NB"], 16, 1, 64, "bf16")  # three launches
    want, new = osp.compact_kv(raw(k + v), s["tables"], s["cu"], s["ctx"], s["path"], s["keep"])
    got_new, flags = compact(k, v, s)
    assert flags == 0
    np.testing.assert_array_equal(got_new, new)
    for a, b in zip(raw(k + v), want):
        np.testing.assert_array_equal(a, b)


def test_compact_refused_lanes():
    s = lanes(1, 3, 8, 40, 16, fixed=[6, 6, 6])
    s["path"] = np.array([0, 2, 4, -1, -1, -1] * 3, np.int32)
    s["keep"] = np.array([2, 2, 2], np.int32)
    F = pa.FLAGS

    def case(flag, skip=(1,), dropped=False, **over):
        k, v = layers(2, s["NB"], 16, 2, 64, "bf16")
        keep = s["keep"].copy()
        for b in skip:
            keep[b] = -1
        want, new = osp.compact_kv(raw(k + v), s["tables"], s["cu"], s["ctx"], s["path"], keep)
        got_new, flags = compact(k, v, s, **over)
        assert flags == (F[flag] if flag else 0)
        for a, b in zip(raw(k + v), want):
            np.testing.assert_array_equal(a, b)
        for b in range(3):
            if b not in skip:
                assert got_new[b] == new[b]
        return got_new

    def path(*p):
        a = s["path"].copy()
        a[6:12] = p
        return a
    for p in ((1, 2, 4, -1, -1, -1), (0, 4, 2, -1, -1, -1), (0, 2, 2, -1, -1, -1), (0, 2, 6, -1, -1, -1),
              (0, -1, 4, -1, -1, -1), (0, 2, 1 << 30, -1, -1, -1)):
        assert case("TREE", path=path(*p))[1] == s["ctx"][1]
    assert case("TREE", keep=np.array([2, 6, 2], np.int32))[1] == s["ctx"][1]
    # a lane that was not verified keeps none of the step's rows
    assert case(None, keep=np.array([2, -1, 2], np.int32))[1] == s["ctx"][1] - 6
    assert case("QLEN_RANGE", ctx=np.array([s["ctx"][0], 5, s["ctx"][2]], np.int32))[1] == 5
    case("CTX_RANGE", ctx=np.array([s["ctx"][0], 1 << 20, s["ctx"][2]], np.int32))
    # an unknown block leaves the rows there where they are
    t = s["tables"].copy()
    t[1] = s["NB"]
    case("BLOCK_RANGE", tables=t)
    t[1] = -1
    case("BLOCK_RANGE", tables=t)
    case("CU_SEQLENS", skip=(0, 1, 2), cu=s["cu"] + np.array([0, 50, 50, 50], np.int32))


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("n,L,NB,Hkv,D,bs", [(1, 1, 5, 1, 64, 16), (3, 2, 40, 2, 64, 16),
                                             (300, 3, 700, 8, 128, 32), (700, 1, 1500, 3, 64, 16)])
def test_copy(dtype, n, L, NB, Hkv, D, bs):
    rng = np.random.default_rng(n)
    ids = rng.permutation(NB)
    dst = ids[:n]
    src = rng.choice(ids[n:], n)  # sources repeat
    pairs = np.stack([src, dst], 1).astype(np.int32)
    k, v = layers(L, NB, bs, Hkv, D, dtype, seed=n)
    want = osp.copy_blocks(raw(k + v), pairs)
    st = pa.new_status()
    pa.copy_blocks(pa.LayerCaches(k, v), dev(pairs), status=st)
    assert pa.read_status(st) == 0
    for a, b in zip(raw(k + v), want):
        np.testing.assert_array_equal(a, b)


def test_copy_refused_pairs():
    F = pa.FLAGS
    for pairs, done, flag in [([(0, 5), (1, 5), (2, 6)], [(2, 6)], "ALIAS"),     # one destination twice
                              ([(0, 5), (0, 5), (2, 6)], [(2, 6)], "ALIAS"),     # the same pair twice
                              ([(0, 5), (5, 6), (2, 7)], [(5, 6), (2, 7)], "ALIAS"),  # a source written over
                              ([(0, 5), (10, 6), (2, 7)], [(0, 5), (2, 7)], "BLOCK_RANGE"),
                              ([(0, 5), (1, -1), (2, 7)], [(0, 5), (2, 7)], "BLOCK_RANGE"),
                              ([(4, 4), (2, 7)], [(2, 7)], None),                # itself: nothing to do
                              ([], [], None)]:
        k, v = layers(2, 10, 16, 2, 64, "bf16", seed=1)
        want = osp.copy_blocks(raw(k + v), done)
        st = pa.new_status()
        pa.copy_blocks(pa.LayerCaches(k, v), dev(np.array(pairs, np.int32).reshape(-1, 2)), status=st)
        assert pa.read_status(st) == (F[flag] if flag else 0), pairs
        for a, b in zip(raw(k + v), want):
            np.testing.assert_array_equal(a, b)


def test_offsets_past_32_bits():
    NB = (1 << 31) // (32 * 8 * 128) + 8
    k = [torch.zeros(NB, 32, 8, 128, dtype=torch.bfloat16, device="cuda")]
    v = [torch.zeros(NB, 32, 8, 128, dtype=torch.bfloat16, device="cuda")]
    g = torch.Generator(device="cuda").manual_seed(1)
    k[0][NB - 2] = torch.randn(32, 8, 128, generator=g, device="cuda").bfloat16()
    c = pa.LayerCaches(k, v)
    pa.copy_blocks(c, dev(np.array([[NB - 2, NB - 1], [NB - 2, 0]], np.int32)))
    assert torch.equal(k[0][NB - 1], k[0][NB - 2]) and torch.equal(k[0][0], k[0][NB - 2])
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    row = k[0][NB - 1, 20].clone()
    pa.compact_kv(c, dev(np.array([[NB - 1]], np.int32)), dev(np.array([0, 4], np.int32)),
                  dev(np.array([22], np.int32)), dev(np.array([0, 2, -1, -1], np.int32)),
                  dev(np.array([1], np.int32)), new)
    assert new.tolist() == [20] and torch.equal(k[0][NB - 1, 19], row)


def test_streams_and_graphs():
    s = lanes(5, 6, 12, 50, 16, fixed=[12, 5, 1, 8, 3, 9])
    k, v = layers(3, s["NB"], 16, 2, 64, "bf16", seed=3)
    k0, v0 = [t.clone() for t in k], [t.clone() for t in v]
    want, new = osp.compact_kv(raw(k + v), s["tables"], s["cu"], s["ctx"], s["path"], s["keep"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c = pa.LayerCaches(k, v)
    args = [dev(s[x]) for x in ("tables", "cu", "ctx", "path", "keep")]
    out = torch.empty(6, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    pa.compact_kv(c, *args, out, stream=side)
    side.synchronize()
    for a, b in zip(raw(k + v), want):
        np.testing.assert_array_equal(a, b)
    g = torch.cuda.CUDAGraph()
    pairs = dev(np.array([[0, s["NB"] - 1]], np.int32))
    with torch.cuda.graph(g):
        pa.compact_kv(c, *args, out)
        pa.copy_blocks(c, pairs)
    for t, o in zip(k + v, k0 + v0):
        t.copy_(o)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    want = osp.copy_blocks(want, [(0, s["NB"] - 1)])
    np.testing.assert_array_equal(out.cpu().numpy(), new)
    for a, b in zip(raw(k + v), want):
        np.testing.assert_array_equal(a, b)


def test_compact_a_step_without_rows():
    """Lanes and no row at all (an empty path has no address): the lengths are passed on."""
    k, v = layers(2, 6, 16, 2, 64, "bf16")
    before = raw(k + v)
    s = dict(tables=np.arange(6, dtype=np.int32).reshape(3, 2), cu=np.zeros(4, np.int32),
             ctx=np.array([0, 17, 32], np.int32), path=np.zeros(0, np.int32), keep=np.full(3, -1, np.int32))
    new, flags = compact(k, v, s)
    assert flags == 0 and new.tolist() == [0, 17, 32]
    for a, b in zip(raw(k + v), before):
        np.testing.assert_array_equal(a, b)
