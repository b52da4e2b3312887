"""Router gradients for slots that name one expert more than once: the sum in slot order, in fp32."""
import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(24, 3), (64, 15), (256, 32), (1000, 8)])
def test_repeated_ids_add_in_slot_order(E, k):
    """With dlogits = sigmoid(l) (1 - sigmoid(l)) dw at logits of 0 (factor 1/4, exact) an element is the slots' sum,
    which depends on its order: large and small terms of both signs."""
    g = torch.Generator().manual_seed(E + k)
    T = 61
    l = torch.zeros(T, E, device="cuda")
    idx = torch.randint(0, 3, (T, k), generator=g, dtype=torch.int32)
    idx[0] = torch.arange(k)          # no repeats
    idx[1] = 2                        # one expert throughout
    idx[2, ::2] = -1                  # empty slots between
    idx[3] = E - 1
    dw = torch.randn(T, k, generator=g) * 10.0 ** torch.randint(-4, 8, (T, k), generator=g)
    want = torch.zeros(T, E)
    for j in range(k):                # fp32 additions, slot after slot
        on = (idx[:, j] >= 0).nonzero()[:, 0]
        want[on, idx[on, j].long()] += dw[on, j] * 0.25
    got = moe.route_topk_backward(l, idx.cuda(), dw.cuda(), score="sigmoid", renormalize=False)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_repeated_ids_against_the_formula(score, renormalize):
    """Each slot counts as one of the chosen, also in the renormalising sum."""
    g = torch.Generator().manual_seed(3)
    l = torch.randn(9, 40, generator=g)
    idx = torch.randint(0, 6, (9, 7), generator=g, dtype=torch.int32)
    dw = torch.randn(9, 7, generator=g)
    z = l.double().requires_grad_()
    a = z.gather(1, idx.long())
    if score == "softmax":
        p = torch.exp(a - torch.logsumexp(a if renormalize else z, 1, keepdim=True))
    else:
        p = torch.sigmoid(a) / torch.sigmoid(a).sum(1, keepdim=True)
    (p * dw.double()).sum().backward()
    got = moe.route_topk_backward(l.cuda(), idx.cuda(), dw.cuda(), score=score, renormalize=renormalize).double().cpu()
    # every term within 150 u at |l| < 5 (exponentials, sums of at most 40 terms), an element of at most 7 + 1 terms below max |dw|
    assert ((got - z.grad).abs() <= 150 * 2.0 ** -24 * 2 * dw.double().abs().sum(1, keepdim=True)).all()
