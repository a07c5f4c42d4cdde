"""Values with a bound on their fp32 error, for tolerances that follow from the
arithmetic: each operation carries its operands' bounds on to first order and
adds its own rounding, u = 2^-24 of the result (first order is enough: every
bound here is below 2^-10 of its value's scale, and 1 % is added at the end)."""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


class V:
    __array_priority__ = 1000   # a numpy array on the left hands over

    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, np.float64)
        self.e = np.broadcast_to(np.asarray(e, np.float64), self.v.shape) if np.ndim(e) == 0 else e

    def _rounded(self, v, e, steps=1):
        return V(v, e + steps * U * np.abs(v))

    def __add__(self, o):
        o = o if isinstance(o, V) else V(o)
        return self._rounded(self.v + o.v, self.e + o.e)

    __radd__ = __add__

    def __neg__(self):
        return V(-self.v, self.e)

    def __sub__(self, o):
        return self + (-o if isinstance(o, V) else V(-np.asarray(o)))

    def __mul__(self, o):
        o = o if isinstance(o, V) else V(o)
        return self._rounded(self.v * o.v, np.abs(self.v) * o.e + np.abs(o.v) * self.e)

    __rmul__ = __mul__

    def mean(self, steps):
        """Row means: sums in which a term passes through at most `steps` additions."""
        m = np.abs(self.v).mean(1, keepdims=True)
        return V(self.v.mean(1, keepdims=True), self.e.mean(1, keepdims=True) + steps * U * m)

    def total(self, steps):
        return V(self.v.sum(0), self.e.sum(0) + steps * U * np.abs(self.v).sum(0))

    def all(self, steps):
        return V(self.v.sum(keepdims=True).reshape(1), (self.e.sum() + steps * U * np.abs(self.v).sum()).reshape(1))

    def grow(self, rel):
        """A further relative error."""
        return V(self.v, self.e + rel * np.abs(self.v))


def within(got, want, v: V, out: str, name: str, at_least=0.0):
    """got (a tensor) against `want`, the oracle's values: no further off than the
    bound and the rounding to its type."""
    g = got.detach().double().cpu().numpy()
    assert g.shape == want.shape, name
    np.testing.assert_allclose(v.v, want, rtol=1e-9, atol=1e-9 * (np.abs(want).max(initial=0.0) + 1e-30), err_msg=name)
    lim = 1.01 * (v.e + HALF_STEP[out] * (np.abs(want) + v.e)) + at_least
    off = np.abs(g - want)
    bad = ~(off <= lim)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {bad.sum()} of {g.size} too far off, first at {i}: {g[i]} for {want[i]}, "
                             f"off {off[i]:.3g}, bound {lim[i]:.3g}")
