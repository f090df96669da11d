"""pa_attention_tree against the 64-bit definition: geometries, types, tree shapes, lengths around
every border, masked values, invariance, streams, graphs and refusals on the device."""
import numpy as np
import pytest
import torch

import spec_harness as sh
from invariant_paged_kv_gb300 import build, pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    pa.load()


def lanes_of(seed, spec):
    rng = np.random.default_rng(seed)
    make = {"chain": lambda n: sh.chain(n), "tree": lambda n: sh.tree(rng, n),
            "forest": lambda n: sh.forest(rng, n)}
    return [(past, make[kind](n) if n else []) for past, n, kind in spec]


SMALL = [(5, 1, "chain"), (0, 3, "chain"), (40, 7, "tree"), (17, 0, "chain"), (100, 12, "forest")]


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("H,Hkv,D,bs", [(4, 2, 64, 16), (8, 8, 128, 16), (8, 2, 128, 32),
                                        (10, 2, 128, 16), (16, 1, 64, 32), (7, 1, 128, 16)])
def test_small(dtype, H, Hkv, D, bs):
    s = sh.Step(lanes_of(1, SMALL), H, Hkv, D, bs, dtype, seed=11)
    out, flags = s.run()
    assert flags == 0
    s.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("n", [1, 3, 33])
def test_lengths_around_borders(dtype, n):
    pasts = [0, 1, 15, 16, 127 - n % 7, 127, 128, 129, 255, 256, 257, 1023, 1024, 1025, 1153, 2049]
    s = sh.Step(lanes_of(n, [(p, n, "tree") for p in pasts]), 8, 2, 128, 16, dtype, seed=n)
    out, flags = s.run()
    assert flags == 0
    s.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("kind", ["chain", "tree", "forest"])
def test_many_nodes(dtype, kind):
    # one and several row tiles, trees over one, two and three key tiles
    s = sh.Step(lanes_of(5, [(0, 256, kind), (130, 255, kind), (127, 130, kind), (2100, 65, kind),
                             (1024, 64, kind), (300, 16, kind)]), 8, 2, 64, 16, dtype, seed=3)
    out, flags = s.run()
    assert flags == 0
    s.check(out)


@pytest.mark.parametrize("dtype,H,Hkv,D", [("bf16", 16, 2, 128), ("fp8", 10, 2, 128), ("f32", 4, 2, 64)])
def test_long_context(dtype, H, Hkv, D):
    # more splits than the fold loads at once, and splits longer than the shortest
    s = sh.Step(lanes_of(7, [(9000, 5, "tree"), (34000, 20, "tree"), (3, 2, "chain")]), H, Hkv, D, 32,
                dtype, seed=5)
    out, flags = s.run()
    assert flags == 0
    s.check(out)


def test_many_lanes():
    # more lanes than one window of the walk, lanes without rows among them
    rng = np.random.default_rng(0)
    spec = [(int(rng.integers(0, 1500)), int(rng.integers(0, 9)), "tree") for _ in range(100)]
    s = sh.Step(lanes_of(2, spec), 8, 2, 64, 16, "bf16", seed=9)
    out, flags = s.run()
    assert flags == 0
    s.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_hidden_values_do_not_reach_a_row(dtype):
    """Infinities and NaN in the K and V of nodes a row does not attend leave it bitwise as it is."""
    lanes = lanes_of(3, [(1100, 20, "tree"), (50, 140, "tree"), (120, 30, "forest")])
    s = sh.Step(lanes, 8, 2, 128, 16, dtype, seed=21)
    clean, _ = s.run()
    rng = np.random.default_rng(4)
    bad = {}
    for b, (past, par) in enumerate(lanes):
        for j in rng.choice(len(par), 6, replace=False):
            bad.setdefault(b, set()).add(int(j))
            i, r = s.row(b, past + int(j))
            if dtype == "fp8":
                s.k[i, r, :, 3], s.v[i, r, :, 5] = 0x7F, 0xFF
            else:
                s.k[i, r, :, 3] = float(rng.choice([np.nan, np.inf, -np.inf]))
                s.v[i, r, :, 5] = float(rng.choice([np.nan, np.inf, -np.inf]))
    got, flags = s.run()
    assert flags == 0
    import oracle.speculative as osp
    hit = 0
    for b, (past, par) in enumerate(lanes):
        for j in range(len(par)):
            row = int(s.cu[b]) + j
            if bad[b] & set(osp.ancestors(par, j)):
                hit += 1
                continue
            assert torch.equal(got[row], clean[row]), (b, j)
    assert 0 < hit < s.T


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("past", [40, 1500])
def test_values_not_finite_reach_the_rows_that_attend_them(dtype, past):
    """An infinity in V arrives as an infinity of its sign, a NaN as NaN, in its own element only."""
    s = sh.Step([(past, [-1, 0, 0, 1, 2])], 8, 2, 64, 16, dtype, seed=2)
    clean, _ = s.run()
    i, r = s.row(0, past + 1)
    s.v[i, r, 0, 7] = float("inf")
    i2, r2 = s.row(0, past + 2)
    s.v[i2, r2, 1, 9] = float("nan")
    got, flags = s.run()
    assert flags == 0
    want = clean.clone()
    want[[1, 3], :4, 7] = float("inf")
    want[[2, 4], 4:, 9] = float("nan")
    assert torch.equal(torch.nan_to_num(got, nan=12345.0), torch.nan_to_num(want, nan=12345.0))


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_spoils_its_own_head_only(dtype, value):
    s = sh.Step([(70, [-1, 0, 0, 1]), (1300, sh.chain(30))], 8, 2, 128, 16, dtype, seed=5)
    clean, _ = s.run()
    s.q[2, 3, 17] = value
    s.q[20, 7, 0] = value
    got, flags = s.run()
    assert flags == 0
    assert torch.isnan(got[2, 3]).all() and torch.isnan(got[20, 7]).all()
    got[2, 3], got[20, 7] = clean[2, 3], clean[20, 7]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_queries_of_any_size(dtype):
    """Rows of zeros, of tiny and of huge elements, and single large ones among small: scores from
    uniform to one-hot, each row within its own bound."""
    s = sh.Step([(300, sh.chain(12)), (2500, sh.chain(6))], 8, 2, 128, 16, dtype, seed=15)
    size = torch.tensor([0.0, 1e-30, 1e-6, 1e-3, 0.1, 1, 3, 10, 30, 1, 1, 1])
    s.q[:12] = (s.q[:12].float() * size[:, None, None]).to(s.q.dtype)
    s.q[9, :, 5] = 40.0
    s.q[10, :, :64] *= 1e-4
    out, flags = s.run()
    assert flags == 0
    s.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_batch_invariance(dtype):
    """A lane's rows are bitwise the same alone, among other lanes, and in another order."""
    lanes = lanes_of(9, [(1500, 6, "tree"), (3000, 40, "tree"), (64, 2, "chain"), (900, 130, "forest"),
                         (5000, 1, "chain")])
    s = sh.Step(lanes, 8, 2, 128, 16, dtype, seed=31)
    dev = s.to_device()
    all_rows, _ = s.run(dev)
    again, _ = s.run(dev)
    assert torch.equal(all_rows, again)
    for order in ([0], [4], [3, 0], [4, 2, 1, 0], [1, 1]):
        rows = np.concatenate([np.arange(s.cu[b], s.cu[b + 1]) for b in order])
        t = torch.from_numpy(rows).cuda()
        sub = dict(dev, q=dev["q"][t].contiguous(), tree_parents=dev["tree_parents"][t].contiguous(),
                   block_tables=dev["block_tables"][order].contiguous(),
                   ctx_lens=dev["ctx_lens"][order].contiguous(),
                   cu_seqlens_q=torch.tensor(np.concatenate([[0], np.cumsum([s.n[b] for b in order])]),
                                             dtype=torch.int32, device="cuda"))
        out = torch.full_like(sub["q"], float("nan"))
        mq, mc = max(s.n[b] for b in order), max(int(s.ctx[b]) for b in order)
        n = pa.tree_workspace_bytes(len(order), len(rows), mq, mc, 8, 2, 128, 16, s.kind)
        pa.attention_tree(sub["q"], sub["k_cache"], sub["v_cache"], sub["block_tables"],
                          sub["cu_seqlens_q"], sub["ctx_lens"], sub["tree_parents"], out,
                          workspace=torch.empty(n, dtype=torch.uint8, device="cuda"),
                          **s.kwargs(max_q_len=mq, max_ctx_len=mc))
        assert torch.equal(out, all_rows[t]), order


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_new_rows_are_written_first(dtype):
    lanes = lanes_of(4, [(200, 9, "tree"), (1030, 3, "chain")])
    s = sh.Step(lanes, 8, 2, 64, 16, dtype, seed=8)
    dev = s.to_device()
    slots = np.array([int(s.tables[b, key // 16]) * 16 + key % 16 for b, (past, par) in enumerate(lanes)
                      for key in range(past, past + len(par))], np.int64)
    st = torch.from_numpy(slots).cuda()
    g = torch.Generator().manual_seed(77)
    kn, vn = (torch.randn(s.T, 2, 64, generator=g).to(s.qt).cuda() for _ in range(2))
    want_k, want_v = dev["k_cache"].clone(), dev["v_cache"].clone()
    pa.write_kv(kn, vn, want_k, want_v, st, k_scale=s.k_scale, v_scale=s.v_scale)
    want, _ = s.run(dict(dev, k_cache=want_k, v_cache=want_v))
    out = torch.full_like(dev["q"], float("nan"))
    pa.attention_tree(*[dev[k] for k in ("q", "k_cache", "v_cache", "block_tables", "cu_seqlens_q",
                                         "ctx_lens", "tree_parents")], out, workspace=s.workspace(),
                      slot_mapping=st, k_new=kn, v_new=vn, **s.kwargs())
    assert torch.equal(out, want)
    assert torch.equal(dev["k_cache"].view(torch.uint8), want_k.view(torch.uint8))
    assert torch.equal(dev["v_cache"].view(torch.uint8), want_v.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chain_is_a_causal_chunk(dtype):
    """A chain gives what pa_attention gives for the chunk, within both kernels' bound."""
    lanes = [(700, sh.chain(30)), (10, sh.chain(1)), (2000, sh.chain(100))]
    s = sh.Step(lanes, 8, 2, 128, 16, dtype, seed=6)
    dev = s.to_device()
    out, _ = s.run(dev)
    ref = torch.full_like(out, float("nan"))
    n = pa.workspace_bytes(s.B, s.T, max(s.n), int(s.ctx.max()), -1, 8, 2, 128, 16, s.kind)
    pa.attention(dev["q"], dev["k_cache"], dev["v_cache"], dev["block_tables"], dev["cu_seqlens_q"],
                 dev["ctx_lens"], ref, max_q_len=max(s.n), max_ctx_len=int(s.ctx.max()), scale=s.scale,
                 workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    s.check(out)
    s.check(ref)


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements, blocks from all over it."""
    s = sh.Step(lanes_of(1, [(300, 5, "tree"), (1200, 3, "tree")]), 16, 8, 128, 16, "bf16", seed=4,
                num_blocks=(1 << 31) // (16 * 8 * 128) + 64)
    assert s.tables.max() == s.NB - 1
    out, flags = s.run()
    assert flags == 0
    s.check(out)


def test_another_stream_and_a_graph():
    lanes = lanes_of(6, [(1500, 6, "tree"), (64, 20, "tree")])
    s = sh.Step(lanes, 8, 2, 128, 16, "bf16", seed=13)
    dev = s.to_device()
    want, _ = s.run(dev)
    args = [dev[k] for k in ("q", "k_cache", "v_cache", "block_tables", "cu_seqlens_q", "ctx_lens",
                             "tree_parents")]
    side = torch.cuda.Stream()
    out, ws = torch.full_like(want, float("nan")), s.workspace()
    side.wait_stream(torch.cuda.current_stream())
    pa.attention_tree(*args, out, workspace=ws, stream=side, **s.kwargs())
    side.synchronize()
    assert torch.equal(out, want)
    # a graph, replayed on changed inputs (lengths and trees too)
    g = torch.cuda.CUDAGraph()
    out2, ws2 = torch.full_like(want, float("nan")), s.workspace()
    with torch.cuda.graph(g):
        pa.attention_tree(*args, out2, workspace=ws2, **s.kwargs())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, want)
    dev["q"].copy_(torch.flip(dev["q"], [0]))
    dev["ctx_lens"].copy_(torch.tensor([700, 64], dtype=torch.int32))
    dev["tree_parents"].copy_(torch.tensor(sh.chain(6) + sh.chain(20), dtype=torch.int32))
    g.replay()
    now, _ = s.run(dev)
    assert torch.equal(out2, now) and not torch.equal(now, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_more_items_than_the_gpu_holds(dtype):
    """Items taken from the counter, by class of length, over several windows of lanes: every row as in
    a step of its lane alone, whichever workspace and however often."""
    rng = np.random.default_rng(8)
    spec = [(int(x), int(n), "tree") for x, n in zip(rng.integers(0, 5000, 70), rng.integers(0, 40, 70))]
    s = sh.Step(lanes_of(3, spec), 16, 4, 64, 16, dtype, seed=2)
    dev = s.to_device()
    out, flags = s.run(dev)
    assert flags == 0
    again, _ = s.run(dev)
    assert torch.equal(out, again)
    for b in (0, 33, 69, int(np.argmax(s.n))):
        r = slice(int(s.cu[b]), int(s.cu[b + 1]))
        if s.n[b] == 0:
            continue
        sub = dict(dev, q=dev["q"][r].contiguous(), tree_parents=dev["tree_parents"][r].contiguous(),
                   block_tables=dev["block_tables"][b:b + 1].contiguous(), ctx_lens=dev["ctx_lens"][b:b + 1].clone(),
                   cu_seqlens_q=torch.tensor([0, s.n[b]], dtype=torch.int32, device="cuda"))
        one = torch.full_like(sub["q"], float("nan"))
        n = pa.tree_workspace_bytes(1, s.n[b], s.n[b], int(s.ctx[b]), 16, 4, 64, 16, s.kind)
        pa.attention_tree(*[sub[k] for k in ("q", "k_cache", "v_cache", "block_tables", "cu_seqlens_q", "ctx_lens",
                                             "tree_parents")], one,
                          workspace=torch.empty(n, dtype=torch.uint8, device="cuda"),
                          **s.kwargs(max_q_len=s.n[b], max_ctx_len=int(s.ctx[b])))
        assert torch.equal(one, out[r]), b


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    s = sh.Step(lanes_of(6, [(4000, 12, "tree")] * 20), 8, 2, 128, 16, "bf16", seed=13)
    dev = s.to_device()
    want, _ = s.run(dev)
    args = [dev[k] for k in ("q", "k_cache", "v_cache", "block_tables", "cu_seqlens_q", "ctx_lens",
                             "tree_parents")]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [torch.empty_like(want) for _ in streams], [s.workspace() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, o, w in zip(streams, outs, wss):
            pa.attention_tree(*args, o, workspace=w, stream=st, **s.kwargs())
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_bad_lanes_raise_flags_and_leave_the_others(dtype):
    lanes = lanes_of(8, [(300, 6, "tree"), (40, 4, "tree"), (1100, 5, "tree")])
    s = sh.Step(lanes, 8, 2, 64, 16, dtype, seed=1)
    dev = s.to_device()
    good, _ = s.run(dev)
    r = lambda b: slice(int(s.cu[b]), int(s.cu[b + 1]))  # noqa: E731
    F = pa.FLAGS

    def but(name, at, value):
        t = dev[name].clone()
        t[at] = value
        return dict(dev, **{name: t})

    for changed, flag, lane in [
            (but("ctx_lens", 1, 3), "QLEN_RANGE", 1),
            (but("ctx_lens", 1, -1), "CTX_RANGE", 1),
            (but("ctx_lens", 1, 1 << 30), "CTX_RANGE", 1),
            (but("block_tables", (1, 0), s.NB), "BLOCK_RANGE", 1),
            (but("block_tables", (1, 0), -1), "BLOCK_RANGE", 1),
            (but("tree_parents", int(s.cu[1]) + 2, 2), "TREE", 1),
            (but("tree_parents", int(s.cu[1]) + 2, -2), "TREE", 1),
            (but("tree_parents", int(s.cu[1]) + 2, 1 << 30), "TREE", 1)]:
        out, flags = s.run(changed)
        assert flags == F[flag], (flag, flags)
        for b in range(3):
            if b != lane:
                assert torch.equal(out[r(b)], good[r(b)]), (flag, b)
    # a bad parent is taken as a root
    out, _ = s.run(but("tree_parents", int(s.cu[1]) + 2, 3))
    want, _ = s.run(but("tree_parents", int(s.cu[1]) + 2, -1))
    assert torch.equal(out[r(1)], want[r(1)])
    out, flags = s.run(dev, max_ctx_len=1000)
    assert flags == F["HOST_BOUND"] and torch.equal(out[r(0)], good[r(0)])
    out, flags = s.run(dev, max_q_len=5)
    assert flags == F["HOST_BOUND"] and torch.equal(out[r(2)], good[r(2)])
    cu = dev["cu_seqlens_q"].clone()
    cu[1:] += 100
    _, flags = s.run(dict(dev, cu_seqlens_q=cu))
    assert flags & F["CU_SEQLENS"]


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_wait_that_runs_out(dtype):
    """One K tile never comes: its CTA gives up, the others end as ever, and the fold touches nothing
    out of bounds for the lanes whose entries the CTA had yet to leave (those past the first 32; the
    workspace holds small whole numbers there). The next call is right."""
    s = sh.Step([(700, sh.chain(3))] * 40, 8, 2, 128, 16, dtype, seed=31)
    dev, kw = s.to_device(), s.kwargs()
    want, flags = s.run(dev)
    assert flags == 0
    ws = s.workspace()
    ws = torch.full((ws.numel() // 4,), 3, dtype=torch.int32, device="cuda").view(torch.uint8)
    out, st, L = torch.zeros_like(dev["q"]), pa.new_status(), pa.load()
    call = lambda: pa.attention_tree(  # noqa: E731
        *[dev[k] for k in ("q", "k_cache", "v_cache", "block_tables", "cu_seqlens_q", "ctx_lens", "tree_parents")],
        out, workspace=ws, status=st, **kw)
    try:
        L.pa_test_set_wait_cycles(2_000_000)  # about a millisecond of SM clock
        L.pa_test_skip_split_item(0)
        call()
        flags = pa.read_status(st)
    finally:
        L.pa_test_skip_split_item(-1)
        L.pa_test_set_wait_cycles(0)
    assert flags == pa.FLAGS["TIMEOUT"], f"flags {flags:#x}"
    call()
    assert pa.read_status(st) == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys_shut_out_by_an_infinity(dtype):
    """Scores of -inf in whole splits, one after another: as if those keys were not there, that is as
    with keys so far below the others that nothing is left of them, bit for bit."""
    outs = []
    for value in (-float("inf"), -1e4):
        s = sh.Step([(700, sh.chain(3)), (1500, sh.chain(20))], 8, 2, 128, 16, dtype, seed=8)
        s.q[..., 0] = 1.0
        for b, upto in ((0, 600), (1, 1400)):
            for key in range(upto):
                i, r = s.row(b, key)
                s.k[i, r] = 0.0
                s.k[i, r, :, 0] = value
        out, flags = s.run()
        assert flags == 0
        outs.append(out)
    s.check(outs[1])
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_loose_bounds_change_nothing(dtype):
    s = sh.Step(lanes_of(3, [(600, 5, "tree"), (40, 1, "chain"), (0, 9, "forest")]), 8, 2, 128, 16, dtype, seed=6)
    dev = s.to_device()
    want, flags = s.run(dev)
    assert flags == 0
    for q_len, ctx in ((9, 5000), (256, 605), (256, 1 << 17)):
        got, flags = s.run(dev, max_q_len=q_len, max_ctx_len=ctx)
        assert flags == 0 and torch.equal(got, want), (q_len, ctx)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_wait_that_runs_out_leaves_the_other_lanes(dtype):
    """The CTA that leaves the fold its entries gives up in the first of two windows of lanes, over a
    workspace in which an earlier step had other lanes (more nodes, more splits): every lane that it
    does not work on has its ordinary bits all the same, the split ones too."""
    old = sh.Step([(900, sh.chain(5))] * 40, 8, 2, 128, 16, dtype, seed=30)
    s = sh.Step([(1500, sh.chain(32))] + [(700, sh.chain(2)), (40, sh.chain(3))] * 22, 8, 2, 128, 16, dtype, seed=31)
    dev, kw = s.to_device(), s.kwargs()
    want, flags = s.run(dev)
    assert flags == 0
    need = [pa.tree_workspace_bytes(x.B, x.T, max(x.n), int(x.ctx.max()), 8, 2, 128, 16, x.kind) for x in (old, s)]
    # what the earlier step leaves where this one keeps its entries: theirs, of other lanes
    ws = torch.zeros(max(need), dtype=torch.uint8, device="cuda")
    entries = torch.zeros(len(ws) // 16, 4, dtype=torch.int32, device="cuda")
    entries[:, 2], entries[:, 3] = 5, 2
    ws[:entries.numel() * 4] = entries.view(torch.uint8).view(-1)
    out, st, L = torch.zeros_like(dev["q"]), pa.new_status(), pa.load()
    args = [dev[k] for k in ("q", "k_cache", "v_cache", "block_tables", "cu_seqlens_q", "ctx_lens", "tree_parents")]
    try:
        L.pa_test_set_wait_cycles(2_000_000)  # about a millisecond of SM clock
        L.pa_test_skip_split_item(0)
        pa.attention_tree(*args, out, workspace=ws, status=st, **kw)
        flags = pa.read_status(st)
    finally:
        L.pa_test_skip_split_item(-1)
        L.pa_test_set_wait_cycles(0)
    assert flags == pa.FLAGS["TIMEOUT"], f"flags {flags:#x}"
    assert not torch.equal(out[:32], want[:32])  # the lane of the item that was given up
    bad = [b for b in range(1, s.B) if not torch.equal(out[s.cu[b]:s.cu[b + 1]], want[s.cu[b]:s.cu[b + 1]])]
    assert not bad, bad
    pa.attention_tree(*args, out, workspace=ws, status=st, **kw)
    assert pa.read_status(st) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("dtype,scale,k_scale", [
    ("fp8", None, 1e-12), ("fp8", None, 1e-30), ("fp8", 1e-30, 1e-20), ("fp8", 1e-12, 1e-30), ("fp8", 3e38, 1e-38),
    ("bf16", 1e-45, 1.0), ("bf16", 3e38, 1.0), ("f32", 1e-45, 1.0), ("f32", 3e38, 1.0)])
def test_scales_of_any_size(dtype, scale, k_scale):
    """Every finite positive scale, rows of zeros among them: a score is never 0 times infinity."""
    s = sh.Step([(300, [-1, 0, 0, 1]), (1300, sh.chain(5)), (20, sh.chain(70))], 8, 2, 128, 16, dtype, seed=17)
    s.k_scale = float(np.float32(k_scale))
    if scale is not None:
        s.scale = float(np.float32(scale))
    if scale == 3e38 and dtype != "fp8":
        s.k.mul_(0.0)  # (NaN past the lanes' ends stays)
    s.q[::2] = 0
    out, flags = s.run()
    assert flags == 0
    s.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_queries_near_the_largest(dtype):
    """Elements around 2^116 to 2^120 under a scale that brings the scores back to ordinary size."""
    s = sh.Step([(300, sh.chain(8)), (1300, sh.chain(5))], 8, 2, 128, 16, dtype, seed=16)
    s.q = (s.q.float() * 2.0 ** 116).to(s.q.dtype)
    s.q[3, :, 5], s.q[3, :, 6] = 2.0 ** 118, 2.0 ** 120
    s.q[10, :, 7] = -2.0 ** 119
    s.scale = float(np.float32(2.0 ** -116 / np.sqrt(128)))
    out, flags = s.run()
    assert flags == 0
    s.check(out)


def test_keys_of_zeros_under_any_scale():
    """The largest q and a large scale over codes of zero: every score is 0."""
    s = sh.Step([(300, [-1, 0, 0, 1]), (1300, sh.chain(5))], 8, 2, 128, 16, "fp8", seed=18)
    s.k[s.k != 0x7F] = 0
    s.q[1, :, 3] = 3e38
    s.k_scale, s.scale = 4096.0, 1.0
    out, flags = s.run()
    assert flags == 0
    s.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_queries_near_the_smallest(dtype):
    """Elements around 2^-122 under a scale that brings the scores up to ordinary size."""
    s = sh.Step([(300, sh.chain(8)), (1300, sh.chain(5))], 8, 2, 128, 16, dtype, seed=16)
    s.q = (s.q.float() * 2.0 ** -122).to(s.q.dtype)
    s.q[3, :, 5] = 2.0 ** -118
    s.scale = float(np.float32(2.0 ** 122 / np.sqrt(128)))
    out, flags = s.run()
    assert flags == 0
    s.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("past", [40, 1500])
@pytest.mark.parametrize("low", [-float("inf"), -1e4])
def test_an_infinity_of_weight_zero_is_nan(dtype, past, low):
    """0 times infinity, as for a key of the cache, not infinity: a node's V whose weight is nothing."""
    s = sh.Step([(past, [-1, 0, 0, 1, 2]), (past, sh.chain(40))], 8, 2, 64, 16, dtype, seed=2)
    s.q[..., 0] = 1.0
    for b, j in ((0, 1), (1, 2)):
        i, r = s.row(b, past + j)
        s.k[i, r] = 0.0
        s.k[i, r, :, 0] = low * 8
    clean, flags = s.run()
    assert flags == 0
    s.check(clean)
    for b, j, value in ((0, 1, float("inf")), (0, 2, -float("inf")), (1, 2, -float("inf"))):
        i, r = s.row(b, past + j)
        s.v[i, r, 0, 7] = value
    got, flags = s.run()
    assert flags == 0
    want = clean.clone()
    want[[1, 3], :4, 7] = float("nan")   # node 1 and its child: weight 0
    want[[2, 4], :4, 7] = -float("inf")  # node 2 and its child: an ordinary weight
    want[5 + 2:, :4, 7] = float("nan")
    assert torch.equal(torch.nan_to_num(got, nan=12345.0), torch.nan_to_num(want, nan=12345.0))


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("ctx", [0, 100, 2000])
def test_a_bound_of_no_rows_is_raised(dtype, ctx):
    """max_q_len = 0 with lanes that have rows: every one exceeds it, which is said; nothing is written
    but the new K/V rows."""
    s = sh.Step([(30, sh.chain(3)), (1400, sh.chain(5))], 8, 2, 64, 16, dtype, seed=1)
    out, flags = s.run(max_q_len=0, max_ctx_len=ctx)
    assert flags == pa.FLAGS["HOST_BOUND"]
    assert torch.isnan(out).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("past", [40, 1500])
def test_values_not_finite_in_any_tile(dtype, past):
    """As above in trees of several row tiles and key tiles, and for the codes of NaN: element 5 of the
    rows that attend such a node is what the formula gives, the rest of them and every other row as with
    finite values."""
    rng = np.random.default_rng(past)
    lanes = [(past, sh.tree(rng, 140)), (past + 3, sh.chain(30)), (past + 9, sh.forest(rng, 200))]
    s = sh.Step(lanes, 8, 2, 128, 16, dtype, seed=22)
    clean, _ = s.run()
    odd = {}
    for b, (p, par) in enumerate(lanes):
        for j in rng.choice(len(par), 5, replace=False).tolist() + [len(par) - 1]:
            i, r = s.row(b, p + j)
            value = float(rng.choice([np.nan, np.inf, -np.inf])) if dtype != "fp8" else int(rng.choice([0x7F, 0xFF]))
            s.v[i, r, 1, 5] = value
            odd[int(s.cu[b]) + j] = value if dtype != "fp8" else float("nan")
    got, flags = s.run()
    assert flags == 0
    import oracle.speculative as osp
    want, hit = clean.clone(), 0
    for b, (p, par) in enumerate(lanes):
        for j in range(len(par)):
            met = [odd[int(s.cu[b]) + a] for a in osp.ancestors(par, j) if int(s.cu[b]) + a in odd]
            if met:
                hit += 1
                want[int(s.cu[b]) + j, 4:, 5] = sum(met)
    assert 0 < hit < s.T
    assert torch.equal(torch.nan_to_num(got, nan=12345.0), torch.nan_to_num(want, nan=12345.0))


@pytest.mark.parametrize("dtype", ["fp8", "f32"])
def test_a_graph_of_each_type(dtype):
    """Captured and replayed on changed inputs, as the eager call gives them."""
    s = sh.Step(lanes_of(6, [(1500, 6, "tree"), (64, 20, "tree")]), 8, 2, 128, 16, dtype, seed=13)
    dev = s.to_device()
    want, _ = s.run(dev)
    args = [dev[k] for k in ("q", "k_cache", "v_cache", "block_tables", "cu_seqlens_q", "ctx_lens", "tree_parents")]
    g, out, ws = torch.cuda.CUDAGraph(), torch.full_like(want, float("nan")), s.workspace()
    with torch.cuda.graph(g):
        pa.attention_tree(*args, out, workspace=ws, **s.kwargs())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    dev["q"].copy_(torch.flip(dev["q"], [0]))
    dev["ctx_lens"].copy_(torch.tensor([700, 64], dtype=torch.int32))
    g.replay()
    now, _ = s.run(dev)
    assert torch.equal(out, now) and not torch.equal(now, want)


def test_an_e4m3_chain_is_a_causal_chunk():
    """Over e4m3 caches a chain gives what pa_attention gives for the chunk, within both kernels' bound."""
    s = sh.Step([(700, sh.chain(30)), (10, sh.chain(1)), (2000, sh.chain(100))], 8, 2, 128, 16, "fp8", seed=6)
    dev = s.to_device()
    out, _ = s.run(dev)
    ref = torch.full_like(out, float("nan"))
    mq, mc = max(s.n), int(s.ctx.max())
    n = pa.workspace_bytes(s.B, s.T, mq, mc, -1, 8, 2, 128, 16, s.kind)
    pa.attention(dev["q"], dev["k_cache"], dev["v_cache"], dev["block_tables"], dev["cu_seqlens_q"],
                 dev["ctx_lens"], ref, max_q_len=mq, max_ctx_len=mc, scale=s.scale, k_scale=s.k_scale,
                 v_scale=s.v_scale, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    s.check(out)
    s.check(ref)
