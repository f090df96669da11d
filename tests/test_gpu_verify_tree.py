"""pa_verify_tree against the definition: exact rationals on small vocabularies, float64 on large
ones; the distribution it leaves; ties, zeros, refusals and invariance."""
import numpy as np
import pytest
import torch

import oracle.speculative as osp
import spec_harness as sh
from invariant_paged_kv_gb300 import build, pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    pa.load()


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def make(seed, trees, V, near=1.0, sharp=2.0):
    """Target and draft rows, tokens drawn from the parent's draft row, random numbers."""
    rng = np.random.default_rng(seed)
    T = sum(len(t) for t in trees)
    logits = rng.normal(size=(T, V)) * sharp
    p, q = softmax(logits), softmax(logits + near * rng.normal(size=(T, V)))
    tokens, at = np.zeros(T, np.int32), 0
    for t in trees:
        for j, par in enumerate(t):
            if j:
                cum = np.cumsum(q[at + par].astype(np.float64))
                tokens[at + j] = min(int(np.searchsorted(cum, rng.random() * cum[-1], side="right")), V - 1)
        at += len(t)
    u, us = rng.random(T).astype(np.float32), rng.random(len(trees)).astype(np.float32)
    us = np.minimum(us, np.float32(1 - 2.0 ** -24))
    return p, q, tokens, u, us


def cu_of(trees):
    return np.concatenate([[0], np.cumsum([len(t) for t in trees])]).astype(np.int32)


def run(p, q, tokens, trees, u, us, stream=None, max_q_len=None, status=None, extra=0):
    c = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    T, B = len(tokens), len(us)
    parents = np.array([x for t in trees for x in t], np.int32)
    out = [torch.full((n,), -77, dtype=torch.int32, device="cuda") for n in (B, T, T)]
    st = pa.new_status() if status is None else status
    pa.verify_tree(c(p), None if q is None else c(q), c(tokens), c(parents), c(cu_of(trees)), c(u),
                   c(us), *out, max_q_len=max_q_len or max(len(t) for t in trees), status=st,
                   stream=stream)
    flags = pa.read_status(st)
    return [o.cpu().numpy() for o in out], flags


def same(got, want):
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)


TREES = {
    "chains": lambda r: [sh.chain(int(n)) for n in r.integers(1, 9, 12)],
    "trees": lambda r: [sh.tree(r, int(n)) for n in r.integers(1, 25, 12)],
    "wide": lambda r: [[-1] + [0] * 40, [-1] + [0] * 255],
    "deep": lambda r: [sh.chain(256), sh.chain(255)],
    "empty": lambda r: [sh.chain(3), [], sh.chain(1), []],
}


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("kind", sorted(TREES))
@pytest.mark.parametrize("V", [1, 2, 5, 129])
def test_small_vocabularies_exactly(kind, V, drafts):
    rng = np.random.default_rng(V)
    trees = TREES[kind](rng)
    for near in (0.2, 1.5):
        p, q, tokens, u, us = make(V + 7, trees, V, near)
        q = q if drafts else None
        got, flags = run(p, q, tokens, trees, u, us)
        want = osp.verify_tree(p, q, tokens, np.array([x for t in trees for x in t]), cu_of(trees), u,
                               us, exact=V <= 5 or kind in ("chains", "empty"))
        assert flags == 0
        same(got, want)


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("V", [2047, 2048, 4099, 16385, 32000, 100003, 248320])
def test_large_vocabularies(V, drafts):
    # odd sizes put rows at every 4-byte offset of a 16-byte boundary
    rng = np.random.default_rng(V)
    trees = [sh.tree(rng, 9), sh.chain(4), sh.tree(rng, 5), [-1]]
    p, q, tokens, u, us = make(V, trees, V, 0.7, 3.0)
    q = q if drafts else None
    got, flags = run(p, q, tokens, trees, u, us)
    assert flags == 0
    same(got, osp.verify_tree(p, q, tokens, np.array([x for t in trees for x in t]), cu_of(trees), u, us))


def test_decisions_on_the_border():
    """u q = p exactly is a rejection; a draw exactly at a running sum goes to the next entry; zero
    entries are never drawn; u = 0 takes whatever has any probability."""
    V = 8
    p = np.zeros((2, V), np.float32)
    p[0, [1, 3]] = 0.25, 0.75
    p[1, [0, 2, 5]] = 0.25, 0.25, 0.5
    q = np.zeros((2, V), np.float32)
    q[0, [1, 3]] = 0.5, 0.5
    q[1] = 1 / 8
    trees = [[-1, 0]]
    for u, us, want in [(0.5, 0.5, (0, [0, -1], [3, -1])),        # 0.5 * 0.5 = 0.25: rejected
                        (0.499, 0.25, (1, [0, 1], [1, 2])),       # accepted; 0.25 -> the second entry
                        (0.0, 0.0, (1, [0, 1], [1, 0])),
                        (0.0, 0.5, (1, [0, 1], [1, 5])),
                        (0.0, 1 - 2.0 ** -24, (1, [0, 1], [1, 5]))]:
        got, flags = run(p, q, np.array([0, 1], np.int32), trees, np.array([0, u], np.float32),
                         np.array([us], np.float32))
        assert flags == 0
        assert (got[0][0], got[1].tolist(), got[2].tolist()) == want, (u, us)


def test_nothing_left_of_the_residual_draws_from_the_target():
    """p <= q everywhere (p is q, its last bits cut): the rejected walk draws from p itself."""
    rng = np.random.default_rng(0)
    V = 300
    q = softmax(rng.normal(size=(1, V)))
    p = (q * np.float32(1 - 2.0 ** -12)).astype(np.float32)
    x = int(p.argmax())
    p2, q2 = np.repeat(p, 3, 0), np.repeat(q, 3, 0)
    trees, tok = [[-1, 0, 0]], np.array([0, x, x], np.int32)
    u, us = np.array([0, 1 - 2.0 ** -24, 1 - 2.0 ** -24], np.float32), np.array([0.3], np.float32)
    got, flags = run(p2, q2, tok, trees, u, us)
    assert flags == 0
    cum = np.cumsum(p[0].astype(np.float64))
    want = int(np.searchsorted(cum, float(us[0]) * cum[-1], side="right"))
    assert got[0][0] == 0 and got[2].tolist() == [want, -1, -1]


def test_output_token_has_the_targets_distribution():
    """Over many draws the first output token (kept draft or drawn) follows the target's row: a
    chi-square over 8 tokens stays under its 1 - 1e-6 quantile."""
    rng = np.random.default_rng(3)
    V, N = 8, 4000
    p, q = softmax(rng.normal(size=(1, V)) * 1.5), softmax(rng.normal(size=(1, V)) * 1.5)
    trees = [[-1, 0, 0]] * N
    P, Q = np.repeat(p, 3 * N, 0), np.repeat(q, 3 * N, 0)
    cum = np.cumsum(q[0].astype(np.float64))
    tok = np.minimum(np.searchsorted(cum, rng.random(3 * N) * cum[-1], side="right"), V - 1).astype(np.int32)
    u, us = rng.random(3 * N).astype(np.float32), rng.random(N).astype(np.float32)
    us = np.minimum(us, np.float32(1 - 2.0 ** -24))
    got, flags = run(P, Q, tok, trees, u, us)
    assert flags == 0
    first = got[2].reshape(N, 3)[:, 0]
    seen = np.bincount(first, minlength=V)
    want = p[0].astype(np.float64) * N
    chi2 = float(((seen - want) ** 2 / want).sum())
    assert chi2 < 40.5, chi2  # 7 degrees of freedom: P(chi2 > 40.5) < 1e-6


def test_lanes_do_not_depend_on_one_another():
    rng = np.random.default_rng(11)
    trees = [sh.tree(rng, int(n)) for n in rng.integers(1, 20, 40)]
    V = 5003
    p, q, tokens, u, us = make(5, trees, V, 0.6)
    got, _ = run(p, q, tokens, trees, u, us)
    again, _ = run(p, q, tokens, trees, u, us)
    same(got, again)
    cu = cu_of(trees)
    for b in (0, 7, 39):
        r = slice(cu[b], cu[b + 1])
        one, _ = run(p[r], q[r], tokens[r], [trees[b]], u[r], us[b:b + 1], max_q_len=256)
        same(one, (got[0][b:b + 1], got[1][r], got[2][r]))


def test_refused_lanes():
    """Trees that are none, tokens outside the vocabulary, rows that are no probabilities: a flag,
    -1 in every output of the lane, the other lanes as they are."""
    trees = [sh.chain(4), [-1, 0, 0, 1], sh.chain(4)]
    V = 100
    p, q, tokens, u, us = make(2, trees, V)
    u[:] = np.float32(1 - 2.0 ** -24)
    good, flags = run(p, q, tokens, trees, u, us)
    assert flags == 0
    F = pa.FLAGS

    def case(flag, p=p, q=q, tokens=tokens, trees=trees, us=us):
        got, flags = run(p, q, tokens, trees, u, us)
        assert flags == F[flag]
        assert got[0][1] == -1 and (got[1][4:8] == -1).all() and (got[2][4:8] == -1).all()
        for b in (0, 2):
            assert got[0][b] == good[0][b]
            for a, w in zip(got[1:], good[1:]):
                np.testing.assert_array_equal(a[4 * b:4 * b + 4], w[4 * b:4 * b + 4])

    for bad in ([0, 0, 0, 1], [-1, -1, 0, 1], [-1, 0, 2, 1], [-1, 0, -2, 1], [-1, 5, 0, 1]):
        case("TREE", trees=[trees[0], bad, trees[2]])
    for x in (-1, V, 1 << 30):
        t = tokens.copy()
        t[5] = x
        case("TREE", tokens=t)
    for x in (np.nan, -0.1, 2.5, np.inf, 1.9):
        a = p.copy()
        a[4, 3] = a[4, 7] = x
        case("PROB", p=a)
    for x in (np.nan, -0.1, np.inf):
        a = q.copy()
        a[4, 3] = x
        case("PROB", q=a)
    a = p.copy()
    a[4] = 0
    case("PROB", p=a)
    for x in (1.0, -0.25, np.nan, np.inf):
        a = us.copy()
        a[1] = x
        case("PROB", us=a)
    got, flags = run(p, q, tokens, trees, u, us, max_q_len=3)
    assert flags == F["HOST_BOUND"] and (got[0] == -1).all() and (got[1] == -77).all()


def test_another_stream_and_a_graph():
    rng = np.random.default_rng(1)
    trees = [sh.tree(rng, 12) for _ in range(6)]
    V = 20001
    p, q, tokens, u, us = make(4, trees, V, 0.5)
    want, _ = run(p, q, tokens, trees, u, us)
    side = torch.cuda.Stream()
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    par = c(np.array([x for t in trees for x in t], np.int32))
    args = [c(p), c(q), c(tokens), par, c(cu_of(trees)), c(u), c(us)]
    outs = [[torch.empty(n, dtype=torch.int32, device="cuda") for n in (6, 72, 72)] for _ in range(2)]
    torch.cuda.synchronize()
    pa.verify_tree(*args, *outs[0], max_q_len=12, stream=side)
    side.synchronize()
    same([o.cpu().numpy() for o in outs[0]], want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.verify_tree(*args, *outs[1], max_q_len=12)
    args[5].copy_(c(np.zeros_like(u)))
    g.replay()
    torch.cuda.synchronize()
    zero, _ = run(p, q, tokens, trees, np.zeros_like(u), us)
    same([o.cpu().numpy() for o in outs[1]], zero)
    assert not np.array_equal(zero[0], want[0])


def test_offsets_past_32_bits():
    """More than 2^31 probabilities."""
    V = 248320
    T = (1 << 31) // V + 40
    p = torch.zeros(T, V, device="cuda")
    n = T - 6
    lanes = [sh.chain(1)] * n + [sh.chain(6)]
    p[:, 0] = 1.0
    p[-6:, 0], p[-6:, 9] = 0.0, 1.0
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    tok = i([0] * n + [9] * 6)
    out = [torch.empty(k, dtype=torch.int32, device="cuda") for k in (n + 1, T, T)]
    st = pa.new_status()
    pa.verify_tree(p, None, tok, i([x for t in lanes for x in t]), torch.from_numpy(cu_of(lanes)).cuda(),
                   torch.full((T,), 0.5, device="cuda"), torch.full((n + 1,), 0.5, device="cuda"), *out,
                   max_q_len=6, status=st)
    assert pa.read_status(st) == 0
    assert out[0].tolist() == [0] * n + [5]
    assert out[2].tolist() == [0] * n + [9] * 6


def test_one_token_rejected_many_times():
    """Ten children of one token that the draft is nearly sure of: A q of it passes 4, far beyond any p."""
    V = 1000
    p, q = np.full(V, 0.7 / (V - 1)), np.full(V, 0.1 / (V - 1))
    p[500], q[500] = 0.3, 0.9
    lanes = 64
    trees = [[-1] + [0] * 10] * lanes
    T = 11 * lanes
    rows = lambda x: np.repeat(x.astype(np.float32)[None], T, 0)  # noqa: E731
    tokens, u = np.full(T, 500, np.int32), np.full(T, 0.99, np.float32)
    us = ((np.arange(lanes) + 0.5) / lanes).astype(np.float32)
    got, flags = run(rows(p), rows(q), tokens, trees, u, us)
    assert flags == 0
    want = osp.verify_tree(rows(p), rows(q), tokens, np.array([x for t in trees for x in t]), cu_of(trees), u, us)
    assert 500 not in want[2][::11]
    same(got, want)


@pytest.mark.parametrize("drafts", [True, False])
def test_minus_zero_is_zero(drafts):
    """-0 lies in [0, 2): rows that hold it give what they give with 0."""
    rng = np.random.default_rng(4)
    trees = [sh.tree(rng, 9), [-1] + [0] * 5, sh.chain(4)]
    p, q, tokens, u, us = make(11, trees, 2049, 1.5, 3.0)
    hole = rng.random(p.shape) < 0.5
    hole[np.arange(len(p)), p.argmax(-1)] = False  # (something stays; tokens may fall into holes)
    res = []
    for zero in (0.0, -0.0):
        a, b = np.where(hole, np.float32(zero), p), np.where(hole[::-1], np.float32(zero), q)
        got, flags = run(a, b if drafts else None, tokens, trees, u, us)
        assert flags == 0
        res.append(got)
    same(*res)


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("x", [-0.1, 1.0, 2.5, np.nan, np.inf, -np.inf])
def test_a_random_number_outside_its_range(x, drafts):
    """u_accept outside [0, 1): the lane is refused where the walk comes to that node, and takes no
    notice of it where it does not."""
    trees = [sh.chain(4), [-1, 0, 0, 1], sh.chain(4)]
    p, q, tokens, u, us = make(2, trees, 100)
    q = q if drafts else None
    u[:], u[5] = 0.5, 1 - 2.0 ** -24
    p[4, tokens[5]] = 0  # node 1 of the second lane is tried and never kept: node 3 is not reached
    good, flags = run(p, q, tokens, trees, u, us)
    assert flags == 0 and 3 not in good[1][4:8]
    away = u.copy()
    away[[0, 4, 7]] = x  # roots' numbers are not read, node 3's is not used
    got, flags = run(p, q, tokens, trees, away, us)
    assert flags == 0
    same(got, good)
    bad = u.copy()
    bad[5] = x
    got, flags = run(p, q, tokens, trees, bad, us)
    assert flags == pa.FLAGS["PROB"]
    assert got[0][1] == -1 and (got[1][4:8] == -1).all() and (got[2][4:8] == -1).all()
    for b in (0, 2):
        same([got[0][b], got[1][4 * b:4 * b + 4], got[2][4 * b:4 * b + 4]],
             [good[0][b], good[1][4 * b:4 * b + 4], good[2][4 * b:4 * b + 4]])


@pytest.mark.parametrize("children", [1, 3])
def test_rows_that_are_no_distribution(children):
    """A row that is read and sums to nothing, or to 2 and more, refuses the lane, a draft row as a
    target row; one that is not read does not."""
    V = 257
    trees = [[-1] + [0] * children] * 3
    n = children + 1
    p, q, tokens, u, us = make(3, trees, V)
    u[:] = 0.5
    p[n, tokens[n + 1:2 * n]] = 0  # the second lane rejects every child: both its rows are read
    good, flags = run(p, q, tokens, trees, u, us)
    assert flags == 0 and good[0][1] == 0
    one = lambda value: np.eye(1, V, 200, dtype=np.float32)[0] * np.float32(value)  # noqa: E731

    def case(which, row, flag):
        a, b = p.copy(), q.copy()
        (a if which == "p" else b)[row[0]] = row[1]
        got, flags = run(a, b, tokens, trees, u, us)
        assert flags == flag, (which, flags)
        if flag:
            assert got[0][1] == -1 and (got[1][n:2 * n] == -1).all() and (got[2][n:2 * n] == -1).all()
            for i in (0, 2):
                same([got[0][i], got[1][i * n:i * n + n], got[2][i * n:i * n + n]],
                     [good[0][i], good[1][i * n:i * n + n], good[2][i * n:i * n + n]])
        else:
            same(got, good)

    full = np.full(V, 2.0 / (V - children), np.float32) * np.float32(1 + 2.0 ** -10)
    full[tokens[n + 1:2 * n]] = 0
    for which in "pq":
        for row in (np.zeros(V, np.float32), one(2.0 ** -42), full, 4 * full, 40 * full):
            case(which, (n, row), pa.FLAGS["PROB"])
        case(which, (n + 1, np.zeros(V, np.float32)), 0)  # a row that no walk comes to


def border_row(rng, V, drafts):
    """A row (with a draft row whose only drawn token is always rejected), u_sample = k / 2^24 and the
    token that follows, by whole numbers: the residual's entries are multiples of 2^-58, and u_sample
    times their sum lies within a few of these units of a running sum."""
    unit = 2.0 ** 58
    while True:
        x = rng.normal(size=V) * 2.0
        p = np.exp(x - x.max())
        p = (p / p.sum()).astype(np.float32)
        p = (np.rint(p.astype(np.float64) * unit) / unit).astype(np.float32)  # (fewer bits, so exact)
        q = np.zeros(V, np.float32)
        if drafts:
            q = p[rng.permutation(V)] * np.float32(0.9)
            q = (np.rint(q.astype(np.float64) * unit) / unit).astype(np.float32)
        z = V - 1
        p[z], q[z] = 0.0, 2.0 ** -12
        fine = 5
        p[fine], q[fine] = 2.0 ** 23 / unit, 0.0
        whole = lambda a: np.rint(a.astype(np.float64) * unit).astype(np.int64)  # noqa: E731
        k = int(rng.integers(1 << 21, 1 << 22))
        r = np.maximum(whole(p) - whole(q), 0)
        cum = np.cumsum(r)
        at = int(np.searchsorted(cum, (k * int(cum[-1])) >> 24, side="right"))
        if not 100 < at < V - 100:
            continue
        # off the entry what the running sum there has beyond u_sample times the whole, first coarsely
        # (a float's last place), then by an entry small enough to hold any whole number of units
        q[at] = 0.0
        for place, want in ((at, 0), (fine, int(rng.integers(-3, 4)))):
            r = np.maximum(whole(p) - whole(q), 0)
            cum = np.cumsum(r)
            gap = (int(cum[at]) << 24) - k * int(cum[-1])  # in 2^-24 units; (1 - u) of a change reaches it
            p[place] = (int(r[place]) + round((want * 2 ** 24 - gap) / (2 ** 24 - k))) / unit
            if not p[place] > 0:
                break
        r = np.maximum(whole(p) - whole(q), 0)
        cum = np.cumsum(r)
        gap = (int(cum[at]) << 24) - k * int(cum[-1])
        if p[at] <= 0 or not 0 < p[fine] < 2.0 ** -34 or abs(gap) > 8 << 24:
            continue
        y = int(np.searchsorted(cum, (k * int(cum[-1])) >> 24, side="right"))
        return p, q, z, np.float32(k / 2 ** 24), y


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("V,lanes", [(2049, 16), (100003, 16), (248320, 12), (1 << 24, 4)])
def test_draws_within_a_hair_of_a_running_sum(V, lanes, drafts):
    """Sums of rows keep what their entries hold: a draw that misses a running sum by 2^-57 of a row
    falls on the right side of it, up to the largest vocabulary."""
    rng = np.random.default_rng(V + drafts)
    rows = [border_row(rng, V, drafts) for _ in range(lanes)]
    trees = [[-1, 0] if drafts else [-1]] * lanes
    n = len(trees[0])
    p = np.repeat(np.stack([r[0] for r in rows]), n, 0)
    q = np.repeat(np.stack([r[1] for r in rows]), n, 0) if drafts else None
    tokens = np.repeat(np.array([r[2] for r in rows], np.int32), n)
    got, flags = run(p, q, tokens, trees, np.full(n * lanes, 0.5, np.float32),
                     np.array([r[3] for r in rows], np.float32))
    assert flags == 0 and (got[0] == 0).all()
    np.testing.assert_array_equal(got[2][::n], [r[4] for r in rows])


@pytest.mark.parametrize("V", [300, 2500, 40000])
def test_a_draw_of_zero_takes_the_first_entry_that_is_left(V):
    """u_sample = 0 over rows that are nearly all zeros: tokens taken out, of any size and with any last
    bits, leave nothing behind that could be drawn in their place."""
    rng = np.random.default_rng(V)
    lanes, n = 64, 6
    p = np.zeros((lanes * n, V), np.float32)
    tokens = np.zeros(lanes * n, np.int32)
    want = []
    for b in range(lanes):
        places = np.sort(rng.choice(V - 40, n - 1, replace=False))
        p[b * n, places] = 2.0 ** -rng.uniform(20, 45, n - 1) * rng.uniform(1, 2, n - 1)
        p[b * n, V - 40 + b % 40] = 0.9
        tokens[b * n + 1:b * n + n] = places
        want.append(V - 40 + b % 40)
    u, us = np.full(lanes * n, 0.999, np.float32), np.zeros(lanes, np.float32)
    got, flags = run(p, None, tokens, [[-1] + [0] * (n - 1)] * lanes, u, us)
    assert flags == 0 and (got[0] == 0).all()
    np.testing.assert_array_equal(got[2][::n], want)


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("V", [130, 700])
def test_draws_at_the_ends_of_cut_rows(V, drafts):
    """Rows of a few entries of all sizes, several rejections, u_sample 0 and next to 1: exactly as by
    rationals."""
    rng = np.random.default_rng(V)
    trees = [[-1] + [0] * int(rng.integers(1, 6)) for _ in range(60)]
    p, q, tokens, u, us = make(V, trees, V, 1.0, 6.0)
    cut = rng.random(p.shape) < 0.97
    cut[np.arange(len(p)), p.argmax(-1)] = False
    p = np.where(cut, np.float32(0), p)
    u[:] = np.float32(1 - 2.0 ** -24)
    us[::2], us[1::2] = 0, 1 - 2.0 ** -24
    q = q if drafts else None
    got, flags = run(p, q, tokens, trees, u, us)
    assert flags == 0
    same(got, osp.verify_tree(p, q, tokens, np.array([x for t in trees for x in t]), cu_of(trees), u, us, exact=True))
