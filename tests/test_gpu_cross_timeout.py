"""The dense attention kernels' bounded waits, exercised without faulting the GPU.

A test hook withholds one copy of the first CTA of each pass. The waits for it expire after their bound (about
2 s); the kernels record a timeout and return, the joins behind them run on what there is, nothing outside of the
results and the workspace is touched, and the next call gives the usual result.
"""
import ctypes

import pytest
import torch

from block_sparse_spherical_b200 import abi, api
from test_gpu_cross import inputs, lens_of, normal

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    abi.load()


class Guarded:
    """Memory for one result or workspace between two stretches that have to stay as they are. It is filled with the
    numbers 0, 140, 0, 140, ...: read as the first and last CTA of a unit, they name CTAs that there are."""

    def __init__(self, nbytes):
        self.words = torch.tensor([0, 140], dtype=torch.int32, device="cuda").repeat(GUARD + (nbytes + 511) // 512 * 64)
        self.used = (GUARD, GUARD + nbytes // 4)
        self.address = self.words.data_ptr() + 4 * GUARD
        assert self.address % 256 == 0

    def tensor(self, like):
        return self.words.view(torch.uint8)[4 * GUARD:][:like.numel() * like.element_size()].view(like.dtype).view(like.shape)

    def untouched(self):
        a, b = self.used
        return all(bool((x[::2] == 0).all() and (x[1::2] == 140).all()) for x in
                   (self.words[:a], self.words[b + b % 2:]))


def expired(call, written, status):
    assert call() == 0
    assert abi.bsa_check_status(status) == 5 and abi.bsa_check_status(status) == 0
    assert all(w.untouched() for w in written)


# heads, kv_heads, n_q, n_k, d: few rows whole and cut; many rows whole and cut, units with one tile of rows among them
SHAPES = [(8, 8, 1, 512, 64), (8, 2, 3, 20000, 128), (8, 8, 300, 700, 64), (2, 2, 100, 30000, 64), (4, 1, 700, 5000, 128)]


@pytest.mark.parametrize("number", [0, 3])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, number):
    h, hk, nq, nk, d = shape
    q, k, v, g = inputs(1, h, hk, nq, nk, d, seed=71)
    key_len = lens_of([nk - 5])
    layer = api.CrossAttentionTrain(1, h, nq, nk, d, kv_heads=hk)
    want = layer(q, k, v, key_len)
    grads = layer.backward(g)
    lse, low = layer._saved[5:]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    new = [Guarded(t.numel() * t.element_size()) for t in (want, lse, low)]
    ws = Guarded(layer.workspace_bytes)
    call = lambda n: abi.load().bsa_testing_cross_attention_withhold(
        ctypes.byref(layer.cfg), q.data_ptr(), k.data_ptr(), v.data_ptr(), key_len.data_ptr(), new[0].address,
        new[1].address, new[2].address, ws.address, layer.workspace_bytes, status.data_ptr(), stream, n)
    expired(lambda: call(number), [*new, ws], status)
    assert call(1 << 40) == 0 and abi.bsa_check_status(status) == 0
    assert all(torch.equal(x.tensor(y), y) for x, y in zip(new, (want, lse, low)))
    new = [Guarded(t.numel() * t.element_size()) for t in grads]
    ws = Guarded(layer.bwd_workspace_bytes)
    back = lambda n: abi.load().bsa_testing_cross_attention_backward_withhold(
        ctypes.byref(layer.cfg), q.data_ptr(), k.data_ptr(), v.data_ptr(), key_len.data_ptr(), want.data_ptr(),
        lse.data_ptr(), low.data_ptr(), g.data_ptr(), new[0].address, new[1].address, new[2].address, ws.address,
        layer.bwd_workspace_bytes, status.data_ptr(), stream, n)
    expired(lambda: back(0), [*new, ws], status)
    assert back(1 << 40) == 0 and abi.bsa_check_status(status) == 0
    assert all(torch.equal(x.tensor(y), y) for x, y in zip(new, grads))


# groups, batch, heads, kv_heads, n_q, n_prefix, n_own, d: own states in more whole units than the first CTA has noted
# when its waits expire (a unit that was never noted holds what was in the workspace), and in cut ones
@pytest.mark.parametrize("number", [0, 1])
@pytest.mark.parametrize("shape", [(1, 1200, 2, 2, 1, 3000, 5, 128), (1, 1200, 2, 2, 1, 3000, 5, 64),
                                   (2, 8, 4, 4, 300, 3000, 2000, 64)], ids=str)
def test_prefix(shape, number):
    grp, b, h, hk, nq, npre, nown, d = shape
    gen = torch.Generator(device="cuda").manual_seed(72)
    args = [normal(gen, *s) for s in ((b, h, nq, d), (grp, hk, npre, d), (grp, hk, npre, d), (b, hk, nown, d), (b, hk, nown, d))]
    layer = api.PrefixAttention(b, h, nq, npre, nown, d, kv_heads=hk, groups=grp)
    want = layer(*args)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, ws = Guarded(want.numel() * 2), Guarded(layer.workspace_bytes)
    q, kp, vp, ko, vo = (t.data_ptr() for t in args)
    call = lambda n: abi.load().bsa_testing_prefix_attention_withhold(
        ctypes.byref(layer.cfg), q, kp, vp, None, ko, vo, None, out.address, ws.address, layer.workspace_bytes,
        status.data_ptr(), torch.cuda.current_stream().cuda_stream, n)
    expired(lambda: call(number), [out, ws], status)
    assert call(1 << 40) == 0 and abi.bsa_check_status(status) == 0
    assert torch.equal(out.tensor(want), want)
