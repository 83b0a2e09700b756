"""The autograd functions' backward passes have no derivative of their own: a second
one is refused, not dropped (CPU: the library's calls replaced by formulas in torch)."""
import pytest
import torch
import torch.utils.checkpoint


@pytest.fixture()
def A(monkeypatch):
    from exact_tiled_attention_22_gb300 import build
    build.build()
    from exact_tiled_attention_22_gb300 import attn

    def forward(q, k, v):
        with torch.no_grad():
            return torch.softmax(q.transpose(0, 1) @ k.permute(1, 2, 0), -1).matmul(v.transpose(0, 1)).transpose(0, 1)

    monkeypatch.setattr(attn, "varlen_fwd", lambda q, k, v, *a, o=None, **kw: (o.copy_(forward(q, k, v)), q[..., 0].t()))
    monkeypatch.setattr(attn, "varlen_bwd", lambda q, k, v, o, lse, do, *a, **kw: tuple(x.detach() * 2 for x in (q, k, v)))
    monkeypatch.setattr(attn, "fwd", lambda q, k, v, *a, **kw: (forward(q[0], k[0], v[0])[None], q[..., 0]))
    monkeypatch.setattr(attn, "bwd", lambda q, k, v, o, lse, do, *a, **kw: tuple(x.detach() * 2 for x in (q, k, v)))
    return attn


@pytest.mark.parametrize("packed", [False, True])
def test_second_derivatives_are_refused(A, packed):
    shape = (5, 2, 4) if packed else (1, 5, 2, 4)
    x = [torch.randn(shape, requires_grad=True) for _ in range(3)]
    call = (lambda: A.attention_varlen(*x, None, None)) if packed else (lambda: A.attention(*x))
    first = torch.autograd.grad(call().sum(), x)  # the first derivative is what it was
    assert all(torch.equal(g, 2 * t) for g, t in zip(first, x))
    # a gradient penalty beside a term that does have a second derivative
    with pytest.raises(RuntimeError, match="twice"):
        grads = torch.autograd.grad(call().sum(), x, create_graph=True)
        (sum((g ** 2).sum() for g in grads) + (x[0] ** 3).sum()).backward()
    # create_graph for the sake of something else goes through
    y = torch.randn(shape, requires_grad=True)
    gy, gx = torch.autograd.grad((call() * y ** 2).sum(), (y, x[0]), create_graph=True)
    assert gx.shape == x[0].shape
    with torch.no_grad():
        out = call()
    assert torch.equal(gy, 2 * out * y)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("create_graph", [False, True])
def test_in_a_checkpointed_block(A, packed, create_graph):
    """A recomputed forward hands each saved tensor out once."""
    shape = (5, 2, 4) if packed else (1, 5, 2, 4)
    x = [torch.randn(shape, requires_grad=True) for _ in range(3)]
    call = (lambda *t: A.attention_varlen(*t, None, None)) if packed else A.attention
    out = torch.utils.checkpoint.checkpoint(call, *x, use_reentrant=False)
    grads = torch.autograd.grad(out.sum(), x, create_graph=create_graph)
    assert all(torch.equal(g, 2 * t) for g, t in zip(grads, x))
