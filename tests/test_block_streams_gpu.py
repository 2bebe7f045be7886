"""Weights packed on another stream than the one that holds their memory."""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref

pytestmark = pytest.mark.gpu
N, K = 4096, 4096
LATE = 40_000_000  # cycles, about 20 ms


def _inputs():
    rng = np.random.default_rng(0)
    codes, scales = rng.integers(0, 16, (N, K), dtype=np.uint8), rng.integers(115, 130, (N, K // 32), dtype=np.uint8)
    return torch.from_numpy(ref.row_major_bytes(codes)).cuda(), torch.from_numpy(scales).cuda(), ref.values(codes, scales)


def _make(how, stream):
    codes, scales, w64 = _inputs()
    if how == "quantize":
        w = torch.from_numpy(w64).float().cuda()  # MXFP4's own values: packed as they are
        torch.cuda.synchronize()
        return lambda: block_ops.Fp4Weights.quantize(w, stream=stream())
    torch.cuda.synchronize()
    return lambda: block_ops.Fp4Weights.from_codes(codes, scales, stream=stream())


def _right(w):
    x = torch.eye(K, device="cuda", dtype=torch.bfloat16)[:8]
    y = block_ops.wd_fp4_matvec(w, x, torch.empty(8, N, device="cuda"))
    return np.array_equal(y.cpu().numpy(), _inputs()[2].T[:8].astype(np.float32))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("how", ["from_codes", "quantize"])
def test_memory_that_the_current_stream_still_writes(how, raw):
    """The weights take a block that a queued kernel of the current stream has yet to fill."""
    side = torch.cuda.Stream()
    make = _make(how, lambda: side.cuda_stream if raw else side)
    for _ in range(2):
        del_me = make()  # the sizes' blocks are in the allocator's hands afterwards
        torch.cuda.synchronize()
        sizes = [t.numel() for t in (del_me.codes, del_me.scales)]
        del del_me
        torch.cuda.synchronize()
        late = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda._sleep(LATE)
        for t in late:
            t.fill_(0x55)
        del late, t
        w = make()
        torch.cuda.synchronize()
        assert _right(w)
        del w


@pytest.mark.parametrize("how", ["from_codes", "quantize"])
def test_weights_freed_before_they_are_packed(how):
    """Their memory is not given out again while the other stream has yet to write it."""
    side = torch.cuda.Stream()
    make = _make(how, lambda: side)
    w = make()
    torch.cuda.synchronize()
    n = w.codes.numel()
    del w
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
    w = make()
    del w
    mine = torch.full((n,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert (mine == 7).all()


def test_the_current_stream_named():
    make = _make("from_codes", lambda: torch.cuda.current_stream())
    assert _right(make())
    make = _make("from_codes", lambda: 0)
    assert _right(make())
