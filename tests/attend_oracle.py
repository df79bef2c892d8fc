"""64-bit attention over selected rows and its gradients, in plain numpy, with
first-order bounds on the error of an fp32 computation (test infrastructure).

Bounds, per element. Products of bf16 values are exact in fp32; a dot product
of length d accumulated in fp32 is off by at most (d / 16 + 16) 2^-23 sum |q k|
(d / 16 accumulation steps that may truncate, 16 products inside each). `delta`
is that bound on a score plus 2^-20 for the exponential, its argument and the
normalisation, so a softmax weight is off by at most 2 delta relative. Gradients
propagate the bounds of p, dp and the row sum through their formulas."""
import numpy as np

U32 = 2.0 ** -23


def attend(q, k, v, idx, scale, out_bits=24, grad=None):
    """q [n,Hq,d], k and v [L,Hkv,d], idx [n,kt] (float64 values). Returns a dict of
    results and bounds: out, lse (+ dq, dk, dv), each with tol_<name>.
    out_bits: significand bits of the result and of the weights (8: bf16)."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    r = {"out": np.zeros((n, Hq, d)), "lse": np.full((n, Hq), -np.inf)}
    for name in ("out", "lse"):
        r["tol_" + name] = np.zeros(r[name].shape)
    if grad is not None:
        r["dq"], r["dk"], r["dv"] = np.zeros((n, Hq, d)), np.zeros((L, Hkv, d)), np.zeros((L, Hkv, d))
        for name in ("dq", "dk", "dv"):
            r["tol_" + name] = np.zeros(r[name].shape)
    steps = (d / 16 + 16) * U32
    round_out = 2.0 ** -out_bits
    for t in range(n):
        rows = idx[t]
        rows = rows[(rows >= 0) & (rows < L)].astype(np.int64)
        if rows.size == 0:
            continue
        for h in range(Hq):
            K, V, x = k[rows, h // G], v[rows, h // G], q[t, h]
            s = K @ x * scale
            top = s.max()
            e = np.exp(s - top)
            z = e.sum()
            p = e / z
            o = p @ V
            delta = steps * scale * (np.abs(K) @ np.abs(x)).max() + 2.0 ** -20 + \
                2.0 ** -22 * np.abs(s).max()
            weight = p @ np.abs(V)
            r["out"][t, h], r["lse"][t, h] = o, top + np.log(z)
            o_err = (2 * delta + steps) * weight
            r["tol_out"][t, h] = o_err + round_out * (np.abs(o) + weight)
            r["tol_lse"][t, h] = 2 * delta + 2.0 ** -22 * abs(r["lse"][t, h])
            if grad is None:
                continue
            g = grad[t, h]
            dp, D = V @ g, o @ g
            ds = p * (dp - D)
            e_dp = steps * (np.abs(V) @ np.abs(g))
            e_D = np.abs(g) @ o_err + steps * (np.abs(g) @ np.abs(o))
            e_p = p * 2 * delta
            e_ds = e_p * np.abs(dp - D) + p * (e_dp + e_D) + 2.0 ** -22 * np.abs(ds)
            r["dq"][t, h] = scale * (ds @ K)
            r["tol_dq"][t, h] = scale * ((e_ds + 4 * U32 * np.abs(ds) + steps * np.abs(ds)) @ np.abs(K))
            np.add.at(r["dk"], (rows, h // G), scale * ds[:, None] * x)
            np.add.at(r["dv"], (rows, h // G), p[:, None] * g)
            # + the order of the atomic additions: a few ulp of the sum of magnitudes
            np.add.at(r["tol_dk"], (rows, h // G),
                      scale * (e_ds + 32 * U32 * np.abs(ds))[:, None] * np.abs(x))
            np.add.at(r["tol_dv"], (rows, h // G), (e_p + 32 * U32 * p)[:, None] * np.abs(g))
    return r


def check(name, got, ref, tol, floor=1e-30):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, name
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), f"{name}: non-finite values differ"
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine]), name
    err = np.abs(got[fine] - ref[fine])
    over = err - (tol[fine] + floor)
    assert over.size == 0 or over.max() <= 0, \
        f"{name}: {int((over > 0).sum())} of {over.size} past the bound, worst error " \
        f"{err[over.argmax()]:.3g} against {tol[fine][over.argmax()]:.3g}"
