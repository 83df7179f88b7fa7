"""Dense attention at its edges on the GPU: NaN and infinities in rows that count, key axes that are cut,
calls that meet on several streams and graphs (needs a B200)."""
import pytest
import torch

import dense_ref
from block_sparse_spherical_b200 import abi, api
from test_gpu_cross import inputs, lens_of, normal

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    abi.load()


# n_q, n_k, key_len: whole units; few rows cut into two parts, into more than four, into more than 32; many rows cut
# into two or three parts and into more than four; a cut unit beside an empty entry
CUT = [(1, 700, None), (1, 1300, None), (3, 9000, None), (32, 30000, None), (200, 3000, None), (200, 30000, None),
       (1, 20000, [20000, 0])]


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", CUT, ids=str)
def test_a_query_row_that_is_not_finite_gives_nan(shape, d, bad):
    """Scores of a NaN query are NaN, those of an infinite one infinite of both signs: out, lse and dq are NaN in that
    row, dk and dv in every state it meets, however many parts its keys are cut into. Other rows stay."""
    nq, nk, lens = shape
    b = len(lens) if lens else 1
    q, k, v, g = inputs(b, 2, 2, nq, nk, d, seed=31)
    row = nq // 2
    q[0, 1, row, 5] = bad
    layer = api.CrossAttentionTrain(b, 2, nq, nk, d)
    out = layer(q, k, v, lens_of(lens))
    lse = layer._saved[5]
    dq, dk, dv = layer.backward(g)
    assert layer.check_status() == 0
    for x in (out, lse, dq):
        assert torch.isnan(x[0, 1, row]).all()
    assert torch.isnan(dk[0, 1]).all() and torch.isnan(dv[0, 1]).all()
    keep = [i for i in range(nq) if i != row]
    for x in (out, lse, dq):
        assert torch.isfinite(x[0, 0]).all() and torch.isfinite(x[0, 1, keep]).all()
    assert torch.isfinite(dk[0, 0]).all() and torch.isfinite(dv[0, 0]).all()
    if lens:
        assert not out[1].any() and not dq[1].any() and not dk[1].any() and (lse[1] == -INF).all()


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", [(2, 1, 300, 20), (4, 3, 20000, 77), (4, 150, 30000, 300), (2, 1, 30000, 20000)],
                         ids=str)
def test_a_query_row_that_is_not_finite_gives_nan_over_a_prefix(shape, d, bad):
    b, nq, npre, nown = shape
    gen = torch.Generator(device="cuda").manual_seed(32)
    q = normal(gen, b, 2, nq, d, size=2.0)
    kp, vp, ko, vo = (normal(gen, *s) for s in ((1, 2, npre, d), (1, 2, npre, d), (b, 2, nown, d), (b, 2, nown, d)))
    q[1, 1, nq // 2, 3] = bad
    layer = api.PrefixAttention(b, 2, nq, npre, nown, d)
    for plen, olen in ((None, None), ([npre], [0] * b), ([0], [nown] * b)):
        out = layer(q, kp, vp, ko, vo, lens_of(plen), lens_of(olen))
        assert torch.isnan(out[1, 1, nq // 2]).all()
        out[1, 1, nq // 2] = 0
        assert torch.isfinite(out).all() and layer.check_status() == 0


def test_backward_on_another_stream_outlives_inputs_that_only_the_layer_holds():
    """A forward() that replaces the saved q, k, v and key_len while a backward on a side stream still waits for them:
    their memory is not handed out to what the first stream allocates next."""
    shape = (1, 4, 2, 400, 3000, 64)
    first, second = inputs(*shape, seed=41), inputs(*shape, seed=42)
    lens, full = lens_of([2999]), lens_of([3000])
    layer = api.CrossAttentionTrain(1, 4, 400, 3000, 64, kv_heads=2)
    layer(*first[:3], lens)
    want = layer.backward(first[3])
    side, busy = torch.cuda.Stream(), torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        layer(*(x.clone() for x in first[:3]), lens.clone())         # nobody else keeps these
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                busy.fill_(1)
            got = layer.backward(first[3])
        layer(*second[:3], full)
        junk = [torch.full_like(x, NAN) for x in first[:3] for _ in range(3)] + [torch.zeros_like(lens) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        del junk


# n_q, n_k: few rows whole and cut, many rows whole and cut
FORMS = [(2, 300), (2, 20000), (150, 300), (150, 20000)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", FORMS, ids=str)
def test_rows_whose_scores_are_all_minus_infinity_give_zeros(shape, d):
    nq, nk = shape
    q, k, v, _ = inputs(1, 2, 2, nq, nk, d, seed=51)
    q[0, 1, :, 0] = q[0, 1, :, 0].abs() + 1
    k[0, 1, :, 0] = -INF
    layer = api.CrossAttentionTrain(1, 2, nq, nk, d)
    out = layer(q, k, v)
    lse = layer._saved[5]
    assert not out[0, 1].any() and (lse[0, 1] == -INF).all()
    ref = dense_ref.cross(q[:, :1], k[:, :1], v[:, :1])
    dense_ref.check(out[:, :1], ref, "out")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", FORMS, ids=str)
def test_a_weight_that_is_nothing_meets_large_values(shape, d):
    """Every other pair of keys lies 200 below the rest (a weight of e^-200) and holds values of 3e38."""
    nq, nk = shape
    q, k, v, _ = inputs(1, 2, 2, nq, nk, d, seed=52)
    low = torch.arange(nk, device="cuda") // 2 % 2 == 0
    q[..., 0] = 16
    k[..., 0] = torch.where(low, -200 * d ** 0.5 / 16, 0.0).to(BF)
    v[:, :, low] = 3e38
    dense_ref.check(api.CrossAttention(1, 2, nq, nk, d)(q, k, v), dense_ref.cross(q, k, v), "out")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", FORMS + [(32, 77), (1, 5), (9, 40000)], ids=str)
def test_infinite_values_give_infinities_in_their_columns(shape, d):
    """One sign in a column: that infinity in all rows that meet it; both signs, or NaN: NaN. Other columns stay."""
    nq, nk = shape
    q, k, v, _ = inputs(2, 2, 1, nq, nk, d, seed=53, size=1.0)
    lens = [nk, max(1, nk - 150)]
    v[0, 0, nk // 2, 3], v[0, 0, nk - 1, d - 2] = INF, -INF
    v[0, 0, 0, 17], v[0, 0, nk - 1, 17] = INF, -INF
    v[0, 0, nk // 3, 40] = NAN
    v[1, 0, lens[1]:] = INF                       # not used
    out = api.CrossAttention(2, 2, nq, nk, d, kv_heads=1)(q, k, v, lens_of(lens))
    assert (out[0, :, :, 3] == INF).all() and (out[0, :, :, d - 2] == -INF).all()
    assert torch.isnan(out[0, :, :, [17, 40]]).all()
    at = [c for c in range(d) if c not in (3, 17, 40, d - 2)]
    ref = dense_ref.cross(q, k, torch.where(torch.isfinite(v), v, 0), lens)
    ref = {x: t[..., at] if t.dim() == 4 else t for x, t in ref.items()}
    dense_ref.check(out[..., at], ref, "out")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [1, 5, 40])
def test_infinite_values_of_a_prefix_and_of_own_states(nq, d):
    gen = torch.Generator(device="cuda").manual_seed(54)
    b, npre, nown = 3, 5000, 40
    q = normal(gen, b, 1, nq, d)
    kp, vp, ko, vo = (normal(gen, *s) for s in ((1, 1, npre, d), (1, 1, npre, d), (b, 1, nown, d), (b, 1, nown, d)))
    vp[0, 0, 4000, 6] = INF
    vo[1, 0, 7, 9] = -INF
    vo[2, 0, 39, 6] = -INF
    out = api.PrefixAttention(b, 1, nq, npre, nown, d)(q, kp, vp, ko, vo)
    assert (out[:2, ..., 6] == INF).all() and torch.isnan(out[2, ..., 6]).all() and (out[1, ..., 9] == -INF).all()
    out[..., 6], out[1, ..., 9] = 0, 0
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [128, 1, 150, 333])
def test_an_infinite_key_without_weight_has_no_gradient(nq, d):
    """Scores of -inf with every row (and so a weight of 0): dk and dv are 0 there whether or not the rows fill their
    last tile, and those of the other keys are what they are without it."""
    q, k, v, g = inputs(1, 2, 2, nq, 300, d, seed=55)
    q[..., 0] = q[..., 0].abs() + 1
    k[:, :, 77, 0] = -INF
    layer = api.CrossAttentionTrain(1, 2, nq, 300, d)
    out = layer(q, k, v)
    _, dk, dv = layer.backward(g)                     # dq is 0 times infinity in that column
    assert not dk[:, :, 77].any() and not dv[:, :, 77].any()
    rest = [j for j in range(300) if j != 77]
    ref = dense_ref.cross(q, k[:, :, rest], v[:, :, rest], dout=g)
    for name, x in (("out", out), ("dk", dk[:, :, rest]), ("dv", dv[:, :, rest])):
        dense_ref.check(x, ref, name)


def test_a_backward_captured_alone_replays_after_later_forwards():
    """An eager forward, its backward in a graph: replays read the rows' statistics of that forward, which only the
    layer holds, with other calls and allocations in between."""
    q, k, v, g = inputs(2, 4, 2, 130, 1000, 128, seed=43)
    lens = lens_of([1000, 301])
    layer = api.CrossAttentionTrain(2, 4, 130, 1000, 128, kv_heads=2)
    layer(q, k, v, lens)
    layer.backward(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = layer.backward(g)
    for seed in range(3):
        other = inputs(2, 4, 2, 130, 1000, 128, seed=60 + seed)
        junk = []
        for _ in range(3):
            layer(*other[:3])
            junk.append([torch.full(s, NAN, dtype=t, device="cuda") for s, t in
                         ((layer.shape, BF), (layer.shape[:3], torch.float32), (layer.shape, BF))])
        g.copy_(other[3])
        graph.replay()
        ref = dense_ref.cross(q, k, v, [1000, 301], dout=g)
        for name, x in zip(("dq", "dk", "dv"), grads):
            dense_ref.check(x, ref, name)
        del junk


def test_outputs_that_share_memory_are_refused_and_neighbours_are_not():
    """One buffer for all tensors of a call, end to end; then with an output moved by 16 bytes onto its neighbour."""
    b, h, nq, nk, d = 2, 2, 40, 300, 64
    q, k, v, g = inputs(b, h, h, nq, nk, d, seed=44)
    layer = api.CrossAttentionTrain(b, h, nq, nk, d)
    want = [layer(q, k, v), *layer.backward(g)]
    buf = torch.zeros(4 * q.numel() + 4 * k.numel(), dtype=BF, device="cuda")
    at, views = 0, []
    for x in (q, k, v, g, q, q, k, v):                     # q k v dout, out dq dk dv
        views.append(buf[at:at + x.numel()].view(x.shape))
        at += x.numel()
    for x, y in zip(views, (q, k, v, g)):
        x.copy_(y)
    got = [layer(*views[:3], out=views[4]), *layer.backward(views[3], grads=views[5:])]
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and layer.check_status() == 0
    shifted = buf[3 * q.numel() + 2 * k.numel() - 8:][:q.numel()].view(q.shape)    # dq, 16 bytes into out
    with pytest.raises(abi.BsaError) as e:
        layer.backward(views[3], grads=[shifted, *views[6:]])
    assert e.value.code == 1
    shifted = buf[3 * q.numel():][:q.numel()].view(q.shape)                        # inside k
    with pytest.raises(abi.BsaError) as e:
        layer(*views[:3], out=shifted)
    assert e.value.code == 1


def test_a_bad_length_on_a_busy_stream_is_reported():
    q, k, v, _ = inputs(2, 2, 2, 40, 200, 64, seed=45)
    layer = api.CrossAttention(2, 2, 40, 200, 64)
    busy, side = torch.empty(1 << 30, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    bad = lens_of([201, 5])
    layer(q, k, v, lens_of([200, 5]))             # (the first call of a kernel waits for the device by itself)
    assert layer.check_status() == 0
    with torch.cuda.stream(side):
        for _ in range(50):
            busy.fill_(1)
        layer(q, k, v, bad)
    assert layer.check_status() == 7 and layer.check_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [0.0, 30.0])
@pytest.mark.parametrize("nq", [1, 7, 150])
@pytest.mark.parametrize("nk", [700, 9000])
def test_flat_and_peaked_rows_in_cut_units(nq, nk, size, d):
    """Logits in the hundreds that grow along the keys, in either order: the running maximum moves from tile to tile by
    more than it may lag, and parts of a unit lie far apart; or all logits equal."""
    q, k, v, g = inputs(1, 2, 1, nq, nk, d, seed=46, size=size)
    ramp = torch.linspace(0.1, 2.0, nk, device="cuda")[:, None]
    for r in (ramp, ramp.flip(0)):
        kr = (k.float() * r).to(BF)
        ref = dense_ref.cross(q, kr, v, dout=g)
        layer = api.CrossAttentionTrain(1, 2, nq, nk, d, kv_heads=1)
        dense_ref.check(layer(q, kr, v), ref, "out")
        dense_ref.check(layer._saved[5], ref, "lse")
        for name, x in zip(("dq", "dk", "dv"), layer.backward(g)):
            dense_ref.check(x, ref, name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [1, 5, 100])
@pytest.mark.parametrize("large", ["own", "prefix"])
def test_prefix_and_own_states_far_apart(large, nq, d):
    gen = torch.Generator(device="cuda").manual_seed(47)
    b, npre, nown = 4, 9000, 300
    q = normal(gen, b, 2, nq, d, size=2.0)
    kp, vp, ko, vo = (normal(gen, *s) for s in ((1, 1, npre, d), (1, 1, npre, d), (b, 1, nown, d), (b, 1, nown, d)))
    (ko if large == "own" else kp).mul_(40)
    layer = api.PrefixAttention(b, 2, nq, npre, nown, d, kv_heads=1)
    for own in (None, [300, 0, 1, 129]):
        out = layer(q, kp, vp, ko, vo, own_len=lens_of(own))
        dense_ref.check(out, dense_ref.prefix(q, kp, vp, ko, vo, None, own), "out")
    assert layer.check_status() == 0
