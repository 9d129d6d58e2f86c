"""Outputs that a call makes itself, on a stream that is not the current one: their memory belongs to
the stream that writes them (a block of the current stream's pool may still be in use there), and is
not given out again before the work that the current stream has queued on them is over.  Every class
of the binding, with the stream as an object and as a number."""
import pytest
import torch

from invariant_bi_gemm_gb300 import BiAttention, BiGemm, BiPreNorm, BiPromptAttention, BiQkRope, BiRmsNorm
from test_gpu_l_qkrope import make as make_rope
from test_gpu_m_prompt import Pack
from test_gpu_n_shared import Groups

pytestmark = pytest.mark.gpu


def owner(t):
    """The stream whose pool a tensor's memory comes from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


def rand(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()


def gemm():
    h, x, w = BiGemm(256, 64), rand(40, 256), rand(256, 64)
    return lambda s: [h.run(x, w, stream=s)]


def gathered():
    h, x, w = BiGemm(256, 64), rand(40, 256), rand(256, 64)
    return lambda s: list(h.run_gathered([x[:24].contiguous(), x[24:].contiguous()], w, stream=s)[:2])


def rmsnorm():
    h, x, g = BiRmsNorm(256), rand(40, 256), rand(256)
    return lambda s: [h.run(x, g, stream=s)]


def prenorm():
    h, x, w = BiPreNorm(4096, 32), rand(40, 4096), rand(4096, 32)
    return lambda s: [h.run(x, w, stream=s)]


def rope():
    h, a = BiQkRope(8, 2, 64, 16), make_rope(30, 8, 2, 64, 16, 64)
    return lambda s: [h.run(**a, stream=s)]


def prompt():
    h, a = BiPromptAttention(8, 2, 64, 16), Pack([(0, 70, 0), (1, 30, 5)], 8, 2, 64, 16).args()
    return lambda s: [h.run(*a, stream=s)]


def decode():
    gr = Groups([(600, [3, 4])], 8, 2, 64, 16)
    h, a = BiAttention(8, 2, 64, 16), gr.args()
    return lambda s: [h.run(*a, stream=s)]


def shared():
    gr = Groups([(600, [3, 4])], 8, 2, 64, 16)
    h, a = BiAttention(8, 2, 64, 16), gr.args() + [gr.start.cuda(), gr.len.cuda()]
    return lambda s: [h.run_shared(*a, stream=s)]


@pytest.mark.parametrize("as_number", [False, True])
@pytest.mark.parametrize("make", [gemm, gathered, rmsnorm, prenorm, rope, prompt, decode, shared])
def test_outputs_belong_to_the_stream_that_writes_them(make, as_number):
    call = make()
    want = [o.clone() for o in call(None)]
    torch.cuda.synchronize()
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    stream = side.cuda_stream if as_number else side
    for o in call(None) + call(current) + call(current.cuda_stream):
        assert owner(o) == current.cuda_stream
    got = call(stream)
    assert torch.cuda.current_stream() == current
    side.synchronize()
    for o, w in zip(got, want):
        assert owner(o) == side.cuda_stream
        assert torch.equal(o, w)
    # the current stream still has work on them when they are dropped: the side stream gets other memory
    torch.cuda._sleep(200_000_000)
    copies, at = [o.clone() for o in got], {o.data_ptr() for o in got}
    del got, o
    with torch.cuda.stream(side):
        again = [torch.empty_like(w) for w in want]
    assert not at & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert all(torch.equal(c, w) for c, w in zip(copies, want))


def test_the_default_stream_from_another():
    """Work for the default stream, asked for while another one is current."""
    call = rmsnorm()
    want = call(None)[0].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for s in (0, torch.cuda.default_stream()):
            o = call(s)[0]
            assert owner(o) == 0
            torch.cuda.synchronize()
            assert torch.equal(o, want)
