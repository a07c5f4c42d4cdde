"""Rows of one slot far apart in a step (include/recur.h): they are that state's next
positions, in the rows' order, wherever they stand."""
import numpy as np
import pytest
import torch

from oracle import recur as orc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _states(rows, n):
    """The slot of each of n rows: rows[k] have slot k, the others one of their own."""
    slots = np.arange(n) + len(rows)
    for k, of in enumerate(rows):
        slots[of] = k
    return slots


CASES = [(3, [[0, 2]]), (64, [[0, 63]]), (65, [[0, 64], [1, 2, 63]]), (130, [[0, 63, 64, 65, 128, 129]]),
         (513, [[0, 512], [1, 511], [2, 510, 511]]), (1100, [[5, 517, 518, 1030], [6, 1099], [4, 1028, 1029], list(range(64, 576))]),
         (5000, [[0, 4999], [7, 519, 1031, 4615], list(range(100, 5000, 97))])]


@pytest.mark.parametrize("D", [40, 258])
@pytest.mark.parametrize("n,rows", CASES)
def test_rows_of_one_slot(n, rows, D):
    """Bound of a state: u 12 (|r| + 3) of a state's and an input's magnitude and 2 u, a position; their
    sum here, since what is off decays no slower than the state (a at most 1)."""
    from sparse_hashed_gram_amd import recur
    g = torch.Generator().manual_seed(n + D)
    x, r, i = (torch.randn(n, D, generator=g) for _ in range(3))
    lam = torch.linspace(-6, 0, D)
    slots = _states([[k for k in of] for of in rows], n)
    states = torch.randn(n + len(rows), D, generator=g)
    st = states.cuda()
    y = recur.step(recur.config(D, 1, "f32"), x.cuda(), r.cuda(), i.cuda(), lam.cuda(), st,
                   torch.from_numpy(slots.astype(np.int32)).cuda())
    oy, ost = orc.step(x.double().numpy(), r.double().numpy(), i.double().numpy(), lam.double().numpy(), 8.0,
                       states.double().numpy(), slots)
    most = max(len(of) for of in rows)
    size = np.abs(ost).max() + np.abs(states.numpy()).max() + x.abs().max().item()
    lim = most * U * (12 * (max(r.abs().max().item(), i.abs().max().item()) + 3) + 2) * size
    assert np.abs(y.double().cpu().numpy() - oy).max() <= lim and np.abs(st.double().cpu().numpy() - ost).max() <= lim
    # a row's order is what counts, not its place: the same rows side by side
    order = np.argsort(slots, kind="stable")
    st2 = states.cuda()
    o = torch.from_numpy(order)
    y2 = recur.step(recur.config(D, 1, "f32"), x[o].cuda(), r[o].cuda(), i[o].cuda(), lam.cuda(), st2,
                    torch.from_numpy(slots[order].astype(np.int32)).cuda())
    assert torch.equal(st, st2) and torch.equal(y.cpu()[o], y2.cpu())
