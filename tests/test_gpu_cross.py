"""Cross attention, its gradients and shared-prefix attention on the GPU, against 64 bits within the
bounds of dense_ref (needs a B200)."""
import pytest
import torch

import dense_ref
from block_sparse_spherical_b200 import abi, api

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    abi.load()


def normal(gen, *shape, size=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * size).to(BF)


def lens_of(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def spoil(x, lens):
    """What lies behind a length must not matter: NaN and infinities there."""
    x = x.clone()
    for i, n in enumerate([] if lens is None else lens):
        x[i, :, n:] = float("nan")
        x[i, :, n + 1::2] = float("inf")
    return x


def inputs(b, h, hk, nq, nk, d, seed=0, size=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (normal(gen, b, h, nq, d, size=size), normal(gen, b, hk, nk, d), normal(gen, b, hk, nk, d),
            normal(gen, b, h, nq, d))


# batch, heads, kv_heads, n_q, n_k, d, key_len: one row and one key, tiles met exactly, one more and
# one less, several key tiles, shared heads whose rows fill a quarter, a half, one and several tiles,
# empty entries, lengths that end inside a tile, key axes long enough to be split
SHAPES = [
    (1, 1, 1, 1, 1, 64, None),
    (1, 1, 1, 1, 1, 128, [0]),
    (2, 2, 1, 1, 128, 64, None),
    (2, 4, 2, 5, 129, 64, [0, 129]),
    (3, 3, 3, 128, 127, 128, [127, 1, 64]),
    (1, 2, 2, 129, 300, 64, None),
    (2, 8, 2, 64, 257, 128, [1, 256]),
    (3, 2, 1, 300, 64, 64, [63, 0, 64]),
    (1, 8, 2, 1, 5000, 128, None),
    (2, 4, 1, 7, 4099, 64, [4099, 130]),
    (1, 3, 1, 11, 2000, 128, [1999]),
    (2, 16, 4, 12, 1500, 64, [700, 1500]),
    (1, 6, 2, 41, 999, 128, None),
    (2, 2, 2, 257, 640, 64, [639, 385]),
    (1, 2, 1, 500, 1100, 128, [1027]),
    (5, 5, 5, 33, 65, 64, [0, 65, 0, 1, 2]),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:6])))
def test_forward_and_gradients(shape):
    b, h, hk, nq, nk, d, lens = shape
    q, k, v, g = inputs(b, h, hk, nq, nk, d)
    k, v = spoil(k, lens), spoil(v, lens)
    ref = dense_ref.cross(q, k, v, lens, dout=g)
    layer = api.CrossAttentionTrain(b, h, nq, nk, d, kv_heads=hk)
    out = layer(q, k, v, lens_of(lens))
    lse, low = layer._saved[5:]
    grads = layer.backward(g)
    plain = api.CrossAttention(b, h, nq, nk, d, kv_heads=hk)(q, k, v, lens_of(lens))
    assert layer.check_status() == 0
    dense_ref.check(out, ref, "out")
    dense_ref.check(lse, ref, "lse")
    # out + out_low: off by the weights' rounding and 2^-17 of the value, without the result's own rounding
    ref["both"], ref["both_tol"] = ref["out"], ref["out_tol"] - 1.01 * (dense_ref.U - dense_ref.TWO) * ref["out"].abs()
    dense_ref.check(out.double() + low.double(), ref, "both")
    for name, x in zip(("dq", "dk", "dv"), grads):
        dense_ref.check(x, ref, name)
    assert torch.equal(plain, out)
    again = layer.backward(g)
    assert all(torch.equal(x, y) for x, y in zip(grads, again)), "gradients change from call to call"


# more units than SMs, so that a CTA takes several, whole and cut; few rows and many; more entries with lengths
# than are added up to cut units
LONG = [
    (40, 8, 8, 2, 700, 64, [0, 1, 128, 129, 700] * 8),
    (40, 8, 8, 3, 260, 128, None),
    (30, 8, 4, 9, 2600, 128, None),
    (30, 8, 4, 9, 2600, 64, list(range(0, 2600, 87))),
    (4, 8, 8, 1100, 200, 128, [200, 0, 1, 130]),
    (5, 8, 8, 1030, 130, 64, None),
    (2, 8, 8, 2500, 520, 64, [520, 77]),
    (2, 8, 4, 1250, 520, 128, [520, 385]),
    (1, 16, 4, 8, 30000, 64, None),
    (1100, 1, 1, 2, 140, 64, [i % 141 for i in range(1100)]),
    (1100, 2, 1, 70, 129, 128, [(7 * i) % 130 for i in range(1100)]),
]


@pytest.mark.parametrize("shape", LONG, ids=lambda s: "-".join(map(str, s[:6])))
def test_many_units(shape):
    test_forward_and_gradients(shape)


def test_offsets_past_32_bits():
    """Keys and values of 2.3e9 elements (the last slab holds what is compared), then rows of as many."""
    b, hk, n, d = 17, 8, 132000, 128
    gen = torch.Generator(device="cuda").manual_seed(20)
    k, v = (torch.empty((b, hk, n, d), dtype=BF, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    for t in (k, v):
        t[:] = normal(gen, n, d)
        t[-1, -1] = normal(gen, n, d)
    q = normal(gen, b, hk, 1, d, size=2.0)
    out = api.CrossAttention(b, hk, 1, n, d)(q, k, v)
    for i, e in ((0, 0), (b - 1, hk - 1)):
        ref = dense_ref.attend(q[i, e], k[i, e], v[i, e], d ** -0.5)
        dense_ref.check(out[i, e], ref, "out", f"slab {i}, {e}")
    del k, v, out
    rows, n, d = 2 ** 25 + 300, 130, 64
    q, g = (torch.empty((1, 1, rows, d), dtype=BF, device="cuda") for _ in range(2))
    assert q.numel() > 2 ** 31
    q[:], g[:] = normal(gen, d), 0.0
    last = slice(rows - 1000, rows)
    q[0, 0, last], g[0, 0, last] = normal(gen, 1000, d, size=2.0), normal(gen, 1000, d)
    k, v = normal(gen, 1, 1, n, d), normal(gen, 1, 1, n, d)
    layer = api.CrossAttentionTrain(1, 1, rows, n, d)
    out = layer(q, k, v)
    dq, dk, dv = layer.backward(g)
    ref = dense_ref.attend(q[0, 0, last], k[0, 0], v[0, 0], d ** -0.5, g[0, 0, last])     # the others have no gradient
    dense_ref.check(out[0, 0, last], ref, "out")
    for name, x in (("dq", dq[0, 0, last]), ("dk", dk[0, 0]), ("dv", dv[0, 0])):
        dense_ref.check(x, ref, name)
    assert not dq[0, 0, :rows - 1000].any() and layer.check_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [0.0, 30.0])
def test_flat_and_peaked_rows(d, size):
    """All logits equal, and rows that one key takes whole (logits in the hundreds, growing along the keys
    so that the running maximum moves from tile to tile)."""
    q, k, v, g = inputs(1, 2, 1, 150, 700, d, seed=5, size=size)
    k = (k.float() * torch.linspace(0.1, 2.0, 700, device="cuda")[:, None]).to(BF)
    ref = dense_ref.cross(q, k, v, dout=g)
    layer = api.CrossAttentionTrain(1, 2, 150, 700, d, kv_heads=1)
    dense_ref.check(layer(q, k, v), ref, "out")
    for name, x in zip(("dq", "dk", "dv"), layer.backward(g)):
        dense_ref.check(x, ref, name)


def test_scale_and_given_outputs():
    q, k, v, g = inputs(2, 2, 2, 70, 90, 64, seed=6)
    ref = dense_ref.cross(q, k, v, scale=0.3, dout=g)
    layer = api.CrossAttentionTrain(2, 2, 70, 90, 64, scale=0.3)
    # outputs inside larger buffers: what lies around them stays as it was
    bufs = [torch.full((x.numel() + 256,), 7.0, dtype=BF, device="cuda") for x in (q, q, k, v)]
    views = [t[128:-128].view(x.shape) for t, x in zip(bufs, (q, q, k, v))]
    assert layer(q, k, v, out=views[0]) is views[0]
    assert layer.backward(g, grads=tuple(views[1:]))[0] is views[1]
    for name, x in zip(("out", "dq", "dk", "dv"), views):
        dense_ref.check(x, ref, name)
    assert all(bool((t[:128] == 7).all() and (t[-128:] == 7).all()) for t in bufs)


def test_nan_in_a_state_that_counts_stays_in_its_rows():
    q, k, v, _ = inputs(2, 2, 2, 40, 200, 64, seed=7)
    v[1, 0, 150] = float("nan")
    out = api.CrossAttention(2, 2, 40, 200, 64)(q, k, v)
    assert torch.isnan(out[1, 0]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[1, 1]).all()


@pytest.mark.parametrize("row", range(0, 64, 7))
def test_nan_in_a_key_or_query_reaches_all_that_it_meets(row):
    q, k, v, g = inputs(1, 2, 2, 70, 150, 64, seed=17)
    k[0, 0, row] = float("nan")
    q[0, 1, row] = float("nan")
    layer = api.CrossAttentionTrain(1, 2, 70, 150, 64)
    out = layer(q, k, v)
    dq, dk, dv = layer.backward(g)
    assert torch.isnan(out[0, 0]).all() and torch.isnan(out[0, 1, row]).all()
    rest = [i for i in range(70) if i != row]
    assert torch.isfinite(out[0, 1, rest]).all() and torch.isfinite(dq[0, 1, rest]).all()
    assert torch.isnan(dq[0, 0]).all() and torch.isnan(dk[0]).all() and torch.isnan(dv[0]).all()


def test_lengths_outside_the_buffer_are_clamped_and_flagged():
    q, k, v, g = inputs(2, 2, 2, 40, 200, 64, seed=8)
    layer = api.CrossAttentionTrain(2, 2, 40, 200, 64)
    out = layer(q, k, v, lens_of([-5, 1 << 30]))
    assert layer.check_status() == 7 and layer.check_status() == 0
    grads = layer.backward(g)
    assert layer.check_status() == 7
    ref = dense_ref.cross(q, k, v, [0, 200], dout=g)
    for name, x in zip(("out", "dq", "dk", "dv"), (out, *grads)):
        dense_ref.check(x, ref, name)


# groups, batch, heads, kv_heads, n_q, n_prefix, n_own, d, prefix_len, own_len
PREFIX = [
    (1, 1, 1, 1, 1, 1, 1, 64, None, None),
    (1, 4, 8, 8, 3, 777, 77, 64, None, [0, 25, 51, 77]),
    (2, 6, 4, 2, 5, 300, 40, 128, [0, 300], [0, 40, 3, 0, 1, 39]),
    (1, 24, 16, 4, 1, 4096, 40, 128, None, None),
    (3, 6, 2, 1, 100, 129, 260, 64, [129, 128, 1], [260, 0, 129, 128, 127, 1]),
    (1, 3, 2, 2, 200, 500, 130, 128, [499], [0, 130, 64]),
    (2, 70, 2, 1, 1, 1000, 9, 64, None, None),
    (1, 5, 3, 1, 11, 128, 128, 64, [0], [0, 1, 0, 128, 100]),
    (2, 2, 1, 1, 300, 640, 200, 64, None, [200, 0]),
    (1, 8, 8, 8, 300, 2000, 300, 64, None, None),
    (2, 8, 8, 8, 300, 1500, 400, 128, [1500, 1], [400, 0, 399, 128, 129, 1, 5, 77]),
    (1, 60, 8, 4, 3, 6000, 50, 64, None, None),
    (5, 200, 4, 2, 3, 700, 30, 128, [700, 0, 128, 1, 300], None),
    (1, 2, 8, 8, 1, 30000, 3, 128, None, [3, 0]),
]


@pytest.mark.parametrize("shape", PREFIX, ids=lambda s: "-".join(map(str, s[:8])))
def test_prefix(shape):
    g, b, h, hk, nq, npre, nown, d, pl, ol = shape
    gen = torch.Generator(device="cuda").manual_seed(9)
    q = normal(gen, b, h, nq, d, size=2.0)
    kp, vp = (spoil(normal(gen, g, hk, npre, d), pl) for _ in range(2))
    ko, vo = (spoil(normal(gen, b, hk, nown, d), ol) for _ in range(2))
    ref = dense_ref.prefix(q, kp, vp, ko, vo, pl, ol)
    layer = api.PrefixAttention(b, h, nq, npre, nown, d, kv_heads=hk, groups=g)
    out = layer(q, kp, vp, ko, vo, lens_of(pl), lens_of(ol))
    assert layer.check_status() == 0
    dense_ref.check(out, ref, "out")
    assert torch.equal(out, layer(q, kp, vp, ko, vo, lens_of(pl), lens_of(ol)))


def test_prefix_lengths_outside_the_buffers_are_flagged():
    gen = torch.Generator(device="cuda").manual_seed(10)
    q, kp, vp = (normal(gen, *s) for s in ((2, 1, 3, 64), (1, 1, 50, 64), (1, 1, 50, 64)))
    ko, vo = normal(gen, 2, 1, 20, 64), normal(gen, 2, 1, 20, 64)
    layer = api.PrefixAttention(2, 1, 3, 50, 20, 64)
    out = layer(q, kp, vp, ko, vo, lens_of([51]), lens_of([-1, 21]))
    assert layer.check_status() == 7
    dense_ref.check(out, dense_ref.prefix(q, kp, vp, ko, vo, [50], [0, 20]), "out")


@pytest.mark.parametrize("shape", [(38, 35, 5, 2, 4733, 64), (38, 20, 5, 2, 4733, 128), (12, 8, 8, 120, 3000, 64),
                                   (12, 8, 8, 120, 3000, 128), (6, 8, 8, 700, 1500, 64), (6, 8, 8, 700, 1500, 128)],
                         ids=lambda s: "-".join(map(str, s)))
def test_results_do_not_depend_on_when_tiles_arrive(shape):
    """Keys that come from memory behind a long queue of writes arrive late and out of order: the results are those
    of keys at hand, bit for bit (few rows, whose pipelines take alternate tiles; units of one tile of rows)."""
    b, h, hk, nq, nk, d = shape
    q, k, v, g = inputs(b, h, hk, nq, nk, d, seed=21)
    layer = api.CrossAttentionTrain(b, h, nq, nk, d, kv_heads=hk)
    want = [layer(q, k, v)]
    want += layer.backward(g)
    ref = dense_ref.cross(q, k, v, dout=g)
    for name, x in zip(("out", "dq", "dk", "dv"), want):
        dense_ref.check(x, ref, name)
    queue = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(40):
        queue.fill_(i)
        out = layer(q, k, v)
        queue.fill_(i + 1)
        got = [out, *layer.backward(g)]
        assert all(torch.equal(x, y) for x, y in zip(got, want)), f"call {i}"
    assert layer.check_status() == 0


def test_another_stream_and_two_at_once():
    """Calls of one layer that overlap on two streams do not touch one another's workspace."""
    args = [inputs(1, 4, 1, 2, 9000, 64, seed=s)[:3] for s in (11, 12)]
    layer = api.CrossAttention(1, 4, 2, 9000, 64, kv_heads=1)
    want = [layer(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[], []]
    for _ in range(20):
        for a, s, o in zip(args, streams, got):
            with torch.cuda.stream(s):
                o.append(layer(*a))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for o, w in zip(got, want) for x in o)


def test_prefix_on_two_streams_and_in_graphs():
    """One layer's calls that overlap, eager ones and two graphs' of the same capture-time buffers."""
    gen = torch.Generator(device="cuda").manual_seed(18)
    g, b, h, hk, nq, npre, nown, d = 2, 12, 4, 2, 9, 3000, 200, 64
    layer = api.PrefixAttention(b, h, nq, npre, nown, d, kv_heads=hk, groups=g)
    shapes = ((b, h, nq, d), (g, hk, npre, d), (g, hk, npre, d), (b, hk, nown, d), (b, hk, nown, d))
    args = [normal(gen, *s) for s in shapes]
    own = lens_of([(37 * i) % 201 for i in range(b)])
    call = lambda: layer(*args, own_len=own)
    call()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call())
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        for x in args:
            x.copy_(normal(gen, *x.shape))
        own.copy_(own.roll(1))
        want = call()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        with torch.cuda.stream(streams[2]):
            got = call()
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in (*outs, got))
    dense_ref.check(got, dense_ref.prefix(*args, None, own.tolist()), "out")
    assert layer.check_status() == 0


def test_backward_on_another_stream_than_the_forward():
    """What the layer keeps for the backward outlives a forward that replaces it while that backward waits."""
    q, k, v, g = inputs(1, 4, 2, 400, 3000, 64, seed=19)
    layer = api.CrossAttentionTrain(1, 4, 400, 3000, 64, kv_heads=2)
    layer(q, k, v)
    want = layer.backward(g)
    side = torch.cuda.Stream()
    for _ in range(5):
        layer(q, k, v)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                layer.backward(g)
            got = layer.backward(g)
        junk = api.CrossAttentionTrain(1, 4, 400, 3000, 64, kv_heads=2)
        layer(v[:, :, :400].repeat(1, 2, 1, 1), k, v)                # replaces what was kept
        junk(v[:, :, :400].repeat(1, 2, 1, 1), k, v)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_captured_graphs_replay_with_new_inputs():
    """A training step and a prefix call captured from one layer each, two graphs, replayed in turn
    and at once on two streams with eager calls between."""
    q, k, v, g = inputs(1, 4, 2, 130, 400, 64, seed=13)
    layer = api.CrossAttentionTrain(1, 4, 130, 400, 64, kv_heads=2)
    serve = api.CrossAttention(1, 4, 130, 400, 64, kv_heads=2)
    step = lambda: (layer(q, k, v), *layer.backward(g), serve(q[:, :, :130], k, v))
    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step())
        graphs.append(gr)
    for seed in (14, 15):
        for x, y in zip((q, k, v, g), inputs(1, 4, 2, 130, 400, 64, seed=seed)):
            x.copy_(y)
        want = step()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(x, y) for x, y in zip(o, want))
    assert layer.check_status() == 0


def test_refusals_of_tensors():
    q, k, v, g = inputs(1, 2, 1, 8, 16, 64)
    layer = api.CrossAttentionTrain(1, 2, 8, 16, 64, kv_heads=1)
    with pytest.raises(RuntimeError, match="forward"):
        layer.backward(g)
    with pytest.raises(ValueError, match="CUDA"):
        layer(q.cpu(), k, v)
    with pytest.raises(TypeError):
        layer(q.float(), k, v)
    with pytest.raises(ValueError, match="shape"):
        layer(q[:, :1], k, v)
    with pytest.raises(ValueError, match="contiguous"):
        layer(q.transpose(2, 3).contiguous().transpose(2, 3), k, v)
    with pytest.raises(TypeError):
        layer(q, k, v, torch.tensor([16], device="cuda"))           # int64 lengths
    with pytest.raises(ValueError, match="shape"):
        layer(q, k, v, lens_of([16, 16]))
    with pytest.raises(abi.BsaError):
        layer(q, k, v, out=q)
    layer(q, k, v)
    with pytest.raises(ValueError, match="shape"):
        layer.backward(g, grads=(q, q, q))
    with pytest.raises(abi.BsaError):
        api.CrossAttention(1, 2, 8, 16, 96)
    with pytest.raises(abi.BsaError):
        api.CrossAttention(1, 2, 8, 16, 64, dtype=torch.float32)


def test_a_run_of_them_together():
    """A lat-lon field brought to the Nside 8 pixels, block-sparse attention among them, cross attention
    to the field itself, and an ensemble of three continuing from those states, one row each."""
    nside, nlat, nlon, h, d = 8, 25, 48, 2, 64
    npix, n = 12 * nside * nside, nlat * nlon
    gen = torch.Generator(device="cuda").manual_seed(16)
    field_k, field_v = normal(gen, h, n, d), normal(gen, h, n, d)
    wq = torch.randn((d, 3), generator=gen, device="cuda")
    x = api.LatLonToHealpix(nside, nlat, nlon)(field_k, field_v, wq)[None]            # [1, H, npix, d]
    gates = torch.rand((1, h, npix, 3), generator=gen, device="cuda")
    y = api.BSA(1, h, npix, d, 64, 4)(x, x, x, gates)
    cross = api.CrossAttentionTrain(1, h, npix, n, d)
    z = cross(y, field_k[None], field_v[None])
    g = normal(gen, 1, h, npix, d)
    grads = cross.backward(g)
    ref = dense_ref.cross(y, field_k[None], field_v[None], dout=g)
    for name, t in zip(("out", "dq", "dk", "dv"), (z, *grads)):
        dense_ref.check(t, ref, name)
    rows, own = normal(gen, 3, h, 1, d, size=2.0), normal(gen, 3, h, 5, d)
    members = api.PrefixAttention(3, h, 1, npix, 5, d)
    out = members(rows, z, z, own, own, own_len=lens_of([0, 2, 5]))
    dense_ref.check(out, dense_ref.prefix(rows, z, z, own, own, None, [0, 2, 5]), "out")
    # without own states it is cross attention to the prefix, of each member
    alone = members(rows, z, z, own, own, own_len=lens_of([0, 0, 0]))
    ref = dense_ref.cross(rows, z.expand(3, -1, -1, -1), z.expand(3, -1, -1, -1))
    dense_ref.check(alone, ref, "out")
    assert cross.check_status() == 0 and members.check_status() == 0
