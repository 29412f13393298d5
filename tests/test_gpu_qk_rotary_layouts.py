"""The norms and rotation on rows of heads in other orders than that of a
projection's output."""
import pytest

from gpu_support import say, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,heads,kv_heads,dim,rot", [(1, 4, 2, 64, 64), (9, 3, 1, 80, 32), (70, 8, 8, 128, 128)])
def test_heads_first(n, heads, kv_heads, dim, rot):
    """[heads][rows][dim] in and out, and in place: the bits of [rows][heads][dim]."""
    torch = torch_cuda()
    import lora_serving_mlora_amd as M
    say(f"heads first {n}x{heads}x{dim}")
    g = torch.Generator(device="cuda").manual_seed(n)
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    b = M.KVBatch(ints([[0]]), ints([1000 + n]), ints([0, n]), n)
    r = M.Rotary(rot)
    x = torch.randn(heads + kv_heads, n, dim, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.randn(dim, device="cuda", generator=g).to(torch.bfloat16)
    rows = x.transpose(0, 1)
    q, k = rows[:, :heads], rows[:, heads:]
    want = M.qk_norm_rotary(q.contiguous(), k.contiguous(), b, r, w, w)
    out = torch.full_like(x, 7.0).transpose(0, 1)
    got = M.qk_norm_rotary(q, k, b, r, w, w, q_out=out[:, :heads], k_out=out[:, heads:])
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    got = M.qk_norm_rotary(q, k, b, r, w, w, q_out=q, k_out=k)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
