"""RMS norm, position bias and updates where offsets pass 32 bits, and updates beside other work."""
import pytest
import torch

import adaptive_gradient_summation_gb300 as ags
import more_reference as more
from training_reference import F8, HALF, TINY, close, u
from updates_reference import bound, orthogonal, updates

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32


def randn(*shape, seed=0, dtype=FP32):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


def test_rms_norm(native):
    """First, middle and last of rows of more than 2^31 elements."""
    cols = 8192
    rows = 2 ** 31 // cols + 3
    at = [0, 1, rows // 2, rows - 2, rows - 1]
    x = torch.ones(rows, cols, dtype=BF16, device=DEV)
    x[at] = randn(len(at), cols, seed=1, dtype=BF16)
    w, few = randn(cols, seed=2), x[at].clone()
    y, total, kept, rstd = ags.rms_norm_checkpointed(x, w, residual=x)
    y2, total2, kept2, rstd2 = ags.rms_norm_checkpointed(few, w, residual=few)
    for a, b in ((y, y2), (total, total2), (kept.codes, kept2.codes), (kept.scales, kept2.scales), (rstd, rstd2)):
        assert torch.equal(a[at], b)
    del y, total
    dx = ags.rms_norm_checkpointed_backward(x, kept, rstd, w, grad_residual=x, parameter_grads=False)[0]
    assert torch.equal(dx[at], ags.rms_norm_checkpointed_backward(few, kept2, rstd2, w, grad_residual=few, parameter_grads=False)[0])
    del kept, dx
    dx = ags.rms_norm_backward(x, x, rstd, w, grad_residual=x, parameter_grads=False)[0]
    assert torch.equal(dx[at], ags.rms_norm_backward(few, few, rstd2, w, grad_residual=few, parameter_grads=False)[0])


@pytest.mark.parametrize("queries,keys", [(4000, 4000), (4001, 4001)])
def test_position_bias(native, queries, keys):
    """The last of sequences of more than 2^31 scores: the bias added, and ones counted by bucket."""
    heads, batch = 8, 18
    table = randn(32, heads, seed=1)
    scores = torch.zeros(batch, heads, queries, keys, dtype=BF16, device=DEV)
    scores[-1] = randn(heads, queries, keys, seed=2, dtype=BF16)
    index = more.bucket_matrix(queries, keys, 0, 32, True, 128, DEV)
    out = ags.relative_position_bias(table, queries, keys, scores=scores)
    for h in (0, heads - 1):
        want = scores[-1, h].to(F8) + table.to(F8)[index, h]
        close(out[-1, h], want, (u + HALF[BF16]) * want.abs() + TINY)
    del out
    scores[-1] = 1.0
    grads = ags.relative_position_bias_backward(scores, 32, worker_offsets=[0, batch - 1, batch],
                                                grads=[torch.empty(32, heads, device=DEV) for _ in range(2)])
    assert not grads[0].any()
    # (counts below 2^24 are exact)
    count = torch.bincount(index.flatten(), minlength=32)
    assert count.max() < 2 ** 24
    assert torch.equal(grads[1].long(), count[:, None].expand(32, heads))


def test_updates(native):
    """Matrices whose elements lie beyond 2^31 others."""
    far = 2 ** 31 + 8
    room = torch.zeros(far + 64 * 104, dtype=BF16, device=DEV)
    x = room.as_strided((2, 64, 100), (far, 104, 1))
    x.copy_(updates(2, 64, 100, gen=torch.Generator(device=DEV).manual_seed(1)))
    got = ags.orthogonalize(x)
    want = orthogonal(x.contiguous())
    for a, b in zip(got, want):
        assert float((a.to(F8) - b).norm() / b.norm()) <= bound(b, BF16)
    del room
    n = far + 64 * 100
    grad = torch.zeros(n, dtype=BF16, device=DEV)
    g = updates(64, 100, gen=torch.Generator(device=DEV).manual_seed(2)).to(BF16)
    grad[far:] = g.flatten()
    w, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    ags.muon_step(grad, [0, far, n], [None, (64, 100)], w, v, lr=0.5, mu=0.5)
    assert torch.equal(v[far:], g.flatten().float()) and not v[:far].any() and not w[:far].any()
    want = -0.5 * orthogonal(g[None])[0]
    assert float((w[far:].view(64, 100).to(F8) - want).norm() / want.norm()) <= bound(g, FP32) + 2.0 ** -23
    assert ags.get_last_error() == 0


def test_updates_beside_the_combine(native):
    """The iteration's CTAs wait for each other while other streams' kernels come and go."""
    x = updates(4, 1024, 1024, gen=torch.Generator(device=DEV).manual_seed(1))
    grads = [randn(2 ** 22, seed=k, dtype=BF16) for k in range(8)]
    offsets = list(range(0, 2 ** 22 + 1, 2 ** 16))
    want, combined = ags.orthogonalize(x), ags.reduce(grads, offsets)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            got.append((ags.orthogonalize(x), want))
        with torch.cuda.stream(streams[1]):
            got.append((ags.reduce(grads, offsets), combined))
        with torch.cuda.stream(streams[2]):
            got.append((ags.orthogonalize(x), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    assert ags.get_last_error() == 0
