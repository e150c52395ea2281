"""layer_bounds' float64 gradients against those of layer_refs, which autograd checks."""
import torch

import layer_bounds
import layer_refs as ref


def test_recurrence_agrees():
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    Bt, Dn, L = 2, 5, 40
    p = dict(x=n(Bt, Dn, L), r=n(Bt, Dn, L), i=n(Bt, Dn, L), lam=2 * n(Dn) - 2, r_bias=n(Dn), i_bias=n(Dn), h0=n(Bt, Dn))
    kw = dict(reset=torch.rand(Bt, L, generator=g) < 0.1, lengths=torch.tensor([40, 17], dtype=torch.int32), dout=n(Bt, Dn, L),
              dh_last=n(Bt, Dn))
    a, b = ref.lru(**p, **kw), layer_bounds.lru(**p, **kw)
    assert set(a) == set(b)
    for k in a:
        assert torch.allclose(a[k][0], b[k][0], rtol=1e-12, atol=1e-13), k
        assert bool((b[k][1] >= 0).all()) and float(b[k][1].sum()) <= 1e-3 * float(b[k][0].abs().sum()), k
