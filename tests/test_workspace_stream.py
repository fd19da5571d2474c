"""The gradients' own workspace when they run on a stream other than the current
one: its memory has to come from that stream's pool. A block of the current
stream's pool may still be in use by work queued there."""
import pytest
import torch

import precision_quantization_row_amd as p


class _Block:
    is_cuda, device = True, torch.device("cuda", 0)

    def is_contiguous(self):
        return True

    def record_stream(self, stream):
        pass

    numel = element_size = lambda self: 64
    data_ptr = lambda self: 4096


def test_comes_from_the_pool_of_the_launch_stream(monkeypatch):
    """The allocator's view, on the host: which stream is current at the allocation."""
    current, taken = [None], []

    class Use:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.before, current[0] = current[0], self.s

        def __exit__(self, *_):
            current[0] = self.before

    def empty(*a, **k):
        taken.append(current[0])
        return _Block()

    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch, "empty", empty)
    side = object()
    p._workspace(None, 64, _Block.device, side)
    p._workspace(None, 64, _Block.device, None)
    assert taken == [side, None] and current == [None]


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["act", "norm"])
def test_leaves_queued_work_alone(which):
    """A tensor of the workspace's size, freed while queued work of the current
    stream has yet to read it: the gradient on a side stream neither disturbs
    that work nor is disturbed by it."""
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    dev = torch.device("cuda:0")
    M, N = 2048, 4096
    dy, z = torch.randn(M, N, device=dev), torch.randn(M, N, device=dev)
    w, r = torch.randn(N, device=dev), torch.rand(M, device=dev) + 0.5
    d, s = torch.empty_like(dy), torch.empty(N, device=dev)
    if which == "act":
        need = p.nvfp4_act_backward_workspace(M, N, p.NVFP4_ACT_SILU)
        call = lambda **k: p.nvfp4_act_backward(dy, z, p.NVFP4_ACT_SILU, d, dbias=s, **k)
    else:
        need = p.nvfp4_rmsnorm_backward_workspace(M, N)
        call = lambda **k: p.nvfp4_rmsnorm_backward(dy, z, w, r, d, dweight=s, **k)
    call(workspace=torch.empty(need, dtype=torch.uint8, device=dev))
    want = s.clone()
    big = torch.randn(4096, 4096, device=dev)
    out = torch.empty_like(big)
    copy = torch.empty(need, dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    for _ in range(3):
        s.fill_(float("nan"))
        block = torch.empty(need, dtype=torch.uint8, device=dev)
        block.fill_(77)
        torch.cuda.synchronize()
        for _ in range(40):              # tens of ms of work before the read below
            torch.mm(big, big, out=out)
        copy.copy_(block)
        block.fill_(0)
        del block                        # back to the current stream's pool, still in use
        call(stream=side)
        side.synchronize()
        got = s.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert bool((copy == 77).all())
