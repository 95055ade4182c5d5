"""Where the operators' sizes end: a grid has fewer than 2^32 threads in all, so what
would take more is refused with the shapes (host alone), and rows of logits, which
can be that many, go out in several launches."""
import pytest

from test_abi import FAKE, lib  # noqa: F401
from test_abi_ops import BIG, backward, book, linear
import ctypes

M = 1 << 24


def test_packed_codes_below_64_gib(lib):  # noqa: F811
    for K, d, chunk in ((16, 1, 128), (64, 1, 64), (65536, 8, 256)):
        n = 64 * chunk
        assert lib.mpq_pack_bytes(M - 16, n, K, d) == ((M - 16) // 16) * 64 * 1024
        assert lib.mpq_pack_bytes(M, n, K, d) == 0 and lib.mpq_pack_bytes(M // 2, 2 * n, K, d) == 0
        assert lib.mpq_pack(FAKE, M, n, ctypes.byref(book(K=K, d=d)), FAKE, BIG, None) == -2
        assert lib.mpq_linear_workspace_bytes(0, 1, M, n, K, d, 0) == 0
    assert linear(lib, m=M, n=8192, ldx=8192, ldy=M, cb=book(K=16)) == -2


def test_gradients_grids(lib):  # noqa: F811
    size = lib.mpq_linear_backward_workspace_bytes
    # tiles of du and x
    assert size(0, 64 * 63, M, 64, 16, 1, 0) > 0 and size(0, 64 * 64, M, 64, 16, 1, 0) == 0
    assert backward(lib, t=64 * 64, m=M, n=64, ldx=64, lddy=M, lddx=64) == -2
    # the affine's entries: 16 groups of 64 columns are too many for 2^24 rows, of 2^23 they are not
    assert size(0, 1, M, 15 * 64, 16, 1, 64) > 0 and size(0, 1, M, 16 * 64, 16, 1, 64) == 0
    assert size(0, 1, M // 2, 16 * 64, 16, 1, 64) > 0
    assert backward(lib, t=1, m=M, n=1024, ldx=1024, lddy=M, lddx=1024, cb=book(K=16), group=64) == -2
    # groups whose dW is formed a block of rows at a time
    assert size(0, 1, M, 1024, 16, 1, 32) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("V", [3, 8])
def test_more_rows_than_a_grid(V):
    """2^24 rows and some: log probabilities, lists and distillation against float64 in the same order, tolerances as in
    test_gpu_logits.py (sums of V terms)."""
    import torch
    import post_quantization_solver_amd as mpq
    t = (1 << 24) + 5
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(t, V, generator=g, device="cuda").mul_(2).bfloat16()
    tok = torch.randint(0, V, (t,), generator=g, device="cuda").int()
    r = mpq.token_logprobs(z, tok, top=2)
    teacher = torch.log_softmax(torch.randn(t, 2, generator=g, device="cuda"), 1) - 0.25
    weights = torch.rand(t, generator=g, device="cuda")
    d = mpq.distill(z, r["top_ids"], teacher, tail=True, weights=weights)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(0, 2000), torch.arange((1 << 21) - 1000, (1 << 21) + 1000),
                    torch.arange((1 << 23) - 1000, (1 << 23) + 1000), torch.arange(t - 2000, t)]).cuda()
    lq = torch.log_softmax(z[at].double(), 1)
    assert (r["logprob"][at] - lq.gather(1, tok[at].long()[:, None])[:, 0]).abs().max() < 2.0 ** -17
    order = torch.sort(z[at].float(), dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(r["top_ids"][at].long(), order)
    assert (r["top_logprobs"][at] - lq.gather(1, order)).abs().max() < 2.0 ** -17
    # distillation in closed form over the two listed tokens and the rest
    p, w = teacher[at].double().exp(), weights[at].double()
    hidden = torch.ones_like(lq, dtype=torch.bool).scatter_(1, order, False)
    pt, lr = 1 - p.sum(1), torch.logsumexp(lq.masked_fill(~hidden, float("-inf")), 1)
    loss = (p * (teacher[at].double() - lq.gather(1, order))).sum(1) + pt * (pt.log() - lr)
    assert (d["loss"][at] - w * loss).abs().max() < 2.0 ** -17
    grad = torch.where(hidden, lq.exp() - pt[:, None] * (lq - lr[:, None]).exp(), lq.exp().scatter_add(1, order, -p))
    grad = grad * w[:, None]
    assert ((d["grad"][at].double() - grad).abs() <= 2.0 ** -8 * grad.abs() + 2.0 ** -15).all()
    # no row is left out: the rows' losses and gradients add up
    assert torch.isfinite(d["loss"]).all() and torch.isfinite(r["lse"]).all()
    assert (r["logprob"] <= 0).all() and (r["entropy"] > 0).all()
