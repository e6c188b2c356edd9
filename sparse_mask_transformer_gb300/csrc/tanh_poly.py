"""Coefficients of the small-argument tanh of the capped scores
(score_tile.cuh, kTanh1 .. kTanh7).

For |y| <= 1/2, tanh y is computed as y (c1 + t (c3 + t (c5 + t c7))),
t = y^2, the odd polynomial of degree 7 whose largest absolute error on
[-1/2, 1/2] is as small as possible.  The coefficients come from the Remez
exchange algorithm (E. Remez, 1934) on (0, 1/2]: solve for the coefficients
and the levelled error E on a reference of five points, move the reference to
the extrema of the new error curve, repeat; rounded to fp32.

Run as a script to print them as C++ hex-float literals.  Double precision
suffices: the levelled error is 1.28e-7, with fp32
coefficients 1.30e-7.
"""
import numpy as np

LIMIT = 0.5


def remez_tanh(terms=4, iterations=40, grid=20001):
    """fp32 coefficients [c1, c3, c5, c7] and the levelled error."""
    n = terms + 1
    ref = LIMIT * np.cos(np.pi * (np.arange(n) + 0.5) / (2 * n))[::-1]
    y = np.linspace(0.0, LIMIT, grid)[1:]
    coef, level = None, None
    for _ in range(iterations):
        a = np.stack([ref ** (2 * j + 1) for j in range(terms)] + [(-1.0) ** np.arange(n)], axis=1)
        sol = np.linalg.solve(a, np.tanh(ref))
        coef, level = sol[:terms], abs(sol[terms])
        err = sum(c * y ** (2 * j + 1) for j, c in enumerate(coef)) - np.tanh(y)
        runs = []
        for k in range(len(y)):
            s = err[k] > 0
            if runs and runs[-1][0] == s:
                if abs(err[k]) > abs(err[runs[-1][1]]):
                    runs[-1][1] = k
            else:
                runs.append([s, k])
        if len(runs) < n:
            break
        best = max(range(len(runs) - n + 1), key=lambda i: min(abs(err[r[1]]) for r in runs[i:i + n]))
        new = np.array([y[r[1]] for r in runs[best:best + n]])
        if np.all(np.abs(new - ref) < LIMIT / grid):
            break
        ref = new
    return [float(np.float32(c)) for c in coef], float(level)


def largest_error(coef, n=200001):
    y = np.linspace(-LIMIT, LIMIT, n)
    t = y * y
    return float(np.max(np.abs(y * (coef[0] + t * (coef[1] + t * (coef[2] + t * coef[3]))) - np.tanh(y))))


if __name__ == "__main__":
    c, level = remez_tanh()
    for i, v in enumerate(c):
        print(f"c{2 * i + 1} = {v.hex()}f  ({v!r})")
    print(f"levelled error {level:.3e}; fp32 coefficients {largest_error(c):.3e}")
