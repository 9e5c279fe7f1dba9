"""The binding's stream argument: what a call allocates belongs to the stream that it launches on (torch hands a
freed block out again at once, in the order of the stream it was allocated on)."""
import ast
import inspect

import pytest
import torch

import block_sparse_attention_kunlun_b200 as ba


def calls_of(tree):
    return [n for n in ast.walk(tree) if isinstance(n, ast.Call)]


def test_functions_with_a_stream_allocate_through_it():
    """Read from the source: no torch.empty and the like of their own, the stream passed on wherever memory is
    taken."""
    seen = 0
    for f in ast.parse(inspect.getsource(ba)).body:
        if not isinstance(f, ast.FunctionDef) or f.name in ("_empty", "_launch_stream"):
            continue
        if "stream" not in [a.arg for a in f.args.args]:
            continue
        for c in calls_of(f):
            name = ast.unparse(c.func)
            if name in ("_empty", "workspace_for"):
                assert "stream" in [ast.unparse(a) for a in c.args], f"{f.name}: {ast.unparse(c)}"
                seen += 1
            made = name.split(".")
            assert not (made[0] == "torch" and made[-1] in ("empty", "empty_like", "zeros", "zeros_like", "full")), \
                f"{f.name}: {ast.unparse(c)}"
    assert seen > 40


def busy_block(like):
    """Leaves a freed block of `like`'s size whose last write, on the current stream, is still to come."""
    x = torch.empty_like(like)
    torch.cuda._sleep(20_000_000)
    x.view(torch.uint8).fill_(0x7F)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["block", "sliding", "rope", "gdpa", "cross", "mx"])
def test_results_on_an_explicit_stream(kind):
    """Forward and backward on another stream, every buffer from the binding, while the current stream is busy."""
    g = torch.Generator().manual_seed(3)
    offs = torch.tensor([0, 300, 301, 700], dtype=torch.int32).cuda()
    q, k, v, dout = (torch.randn((700, 4, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    ang = torch.rand((400, 64), generator=g).cuda()
    cos, sin = ang.cos(), ang.sin()

    def run(**kw):
        if kind == "block":
            out, lse = ba.block_attention_fwd(q, k, v, offs, 64, 2, **kw)
            return out, lse, *ba.block_attention_bwd(q, k, v, out, lse, dout, offs, 64, 2, **kw)
        if kind == "sliding":
            out, lse = ba.sliding_window_attention_fwd(q, k, v, offs, 100, **kw)
            return out, lse, *ba.sliding_window_attention_bwd(q, k, v, out, lse, dout, offs, 100, **kw)
        if kind == "rope":
            out, lse = ba.rope_block_attention_fwd(q, k, v, offs, 64, 2, cos, sin, **kw)
            return out, lse, *ba.rope_block_attention_bwd(q, k, v, out, lse, dout, offs, 64, 2, cos, sin, **kw)
        if kind == "gdpa":
            return ba.gdpa_fwd(q, k, v, offs, 64, 2, **kw), *ba.gdpa_bwd(q, k, v, dout, offs, 64, 2, **kw)
        if kind == "cross":
            return ba.gdpa_cross_fwd(q, k, v, offs, offs, **kw), *ba.gdpa_cross_bwd(q, k, v, dout, offs, offs, **kw)
        out, lse = ba.mx_block_attention_fwd(q, k, v, offs, 64, 2, **kw)
        return out, lse, *ba.mx_block_attention_bwd(q, k, v, out, lse, dout, offs, 64, 2, **kw), *ba.mx_quantize(q, **kw)

    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(2):
        for t in want:
            busy_block(t)
        got = run(stream=side)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_streams_by_number():
    """CUDA's default streams by their numbers, a stream by its handle, and calls without rows."""
    offs = torch.tensor([0, 5, 90], dtype=torch.int32).cuda()
    q = torch.randn((90, 2, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want = ba.block_attention_fwd(q, q, q, offs, 16, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (0, 1, 2, side.cuda_stream, side, torch.cuda.default_stream()):
        out, lse = ba.block_attention_fwd(q, q, q, offs, 16, 2, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        out, _ = ba.block_attention_fwd(q[:0], q[:0], q[:0], offs * 0, 16, 2, stream=stream)
        assert out.shape == (0, 2, 64)
    with torch.cuda.stream(side):   # the caller's stream is the call's
        out, lse = ba.block_attention_fwd(q, q, q, offs, 16, 2, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0])
