"""Float64 definitions of the block operators (numpy; test infrastructure, shares no code with the
library): the gated norm, the join and the gated recurrence with their gradients.

Each function also returns, for every output, a bound on what float32 arithmetic may leave of it:
per element, the sum of the absolute values of the terms that make it up times the number of
roundings on the way, in units of 2^-24. A test adds the rounding of the output's own type."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
# roundings of one element's path besides the sums: products, the reciprocal square root, and the
# gate's exponential, whose argument is rounded (an error of |g| units) and which the sigmoid and
# its slope use a few times
PATH = 32
# Additions that one term of a sum goes through, where fewer than all of them: a sum over a row is up to 16
# elements of a lane, 6 levels of lanes and 4 of waves (26); a weight gradient is a lane's own rows (10
# in the longest tests), up to 256 teams of a workgroup, and a column's partial rows: 64 threads of up to
# 2048 / 64 rows each and 6 levels (304).
ROW_SUM = 32
COLUMN_SUM = 304


def _row(n):
    return min(n, ROW_SUM) * U


def _column(n):
    return min(n, COLUMN_SUM) * U


def _sigmoid(g):
    with np.errstate(over="ignore"):
        return np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))),
                        np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def act_ref(g, act):
    """The gate's activation, its slope, and the size of the slope's terms."""
    s, t = _sigmoid(g), _sigmoid(g) * _sigmoid(-g)
    if act == "sigmoid":
        return s, t, t
    return g * s, s + g * t, s + np.abs(g) * t


def _units(g):
    return PATH + 4 * (np.abs(g) if g is not None else 0.0)


def gated_norm_ref(x, gate, weight, eps, act, dy=None):
    """x [rows, H, D]. Returns {name: (value, bound)} of y and, given dy, dx, dgate, dweight."""
    rows, H, D = x.shape
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    w = np.ones(D) if weight is None else weight
    a, slope, slope_abs = act_ref(gate, act) if gate is not None else (1.0, 0.0, 0.0)
    k = _units(gate)
    y = xh * w * a
    sums = _row(D)  # the mean of x^2, all terms of one sign
    out = {"y": (y, np.abs(y) * (k * U + sums))}
    if dy is None:
        return out
    e = dy * w * a
    c = (e * xh).mean(-1, keepdims=True)
    c_abs = np.abs(e * xh).mean(-1, keepdims=True)
    out["dx"] = (r * (e - xh * c),
                 r * (np.abs(e) + np.abs(xh) * c_abs) * (k.max() * U + 2 * sums
                                                         if gate is not None else k * U + 2 * sums))
    if gate is not None:
        out["dgate"] = (dy * xh * w * slope, np.abs(dy * xh * w) * slope_abs * (k * U + sums))
    if weight is not None:
        axes = (0,) if weight.ndim == 2 else (0, 1)
        t = dy * xh * a
        out["dweight"] = (t.sum(axes), (np.abs(t) * (k * U + sums)).sum(axes)
                          + np.abs(t).sum(axes) * _column(rows * (1 if weight.ndim == 2 else H)))
    return out


def join_ref(res, y, gate, w_post, scale, w_pre, alpha, eps, act, dres_out=None, dn=None):
    """[rows, C]. Returns {name: (value, bound)} of res_out, n and, given the gradients, the rest."""
    rows, C = y.shape
    k = _units(gate)
    k = float(np.max(k)) if np.size(k) else PATH
    sums = _row(C)
    one = np.ones(C)
    a, slope, slope_abs = act_ref(gate, act) if gate is not None else (1.0, None, None)
    ry = 1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + eps) if w_post is not None else 1.0
    yh = y * ry
    wp = w_post if w_post is not None else one
    s = alpha * (scale if scale is not None else one)
    u = yh * wp * a
    ro = res + s * u
    ro_abs = np.abs(res) + np.abs(s * u)
    e_ro = ro_abs * (k * U + sums)
    out = {"res_out": (ro, e_ro)}
    rr = rh = rh_err = 0.0
    if w_pre is not None:
        rr = 1.0 / np.sqrt((ro * ro).mean(-1, keepdims=True) + eps)
        rh = ro * rr
        # rstd' moves by at most the relative error of the root of the mean square
        rel = np.sqrt((e_ro ** 2).mean(-1, keepdims=True)) * rr + k * U + sums
        rh_err = e_ro * rr + np.abs(rh) * rel
        out["n"] = (rh * w_pre, np.abs(w_pre) * rh_err + np.abs(rh * w_pre) * k * U)
    if dres_out is None:
        return out
    G, G_abs = dres_out, np.abs(dres_out)
    e_G = G_abs * k * U
    if w_pre is not None:
        t = dn * w_pre
        c2, c2_abs = (t * rh).mean(-1, keepdims=True), np.abs(t * rh).mean(-1, keepdims=True)
        e_c2 = (np.abs(t) * rh_err).mean(-1, keepdims=True) + c2_abs * (k * U + sums)
        G = G + rr * (t - rh * c2)
        g_norm = rr * (np.abs(t) + np.abs(rh) * c2_abs)
        e_G = (e_G + g_norm * (rel + k * U)
               + rr * (rh_err * np.abs(c2) + np.abs(rh) * e_c2))
        G_abs = G_abs + g_norm
    out["dres"] = (G, e_G)
    du, e_du = s * G, np.abs(s) * e_G + np.abs(s * G) * k * U
    kk = k * U + 2 * sums
    if gate is not None:
        out["dgate"] = (du * yh * wp * slope,
                        np.abs(yh * wp) * slope_abs * (e_du + np.abs(du) * kk))
    e = du * wp * a
    e_e = e_du * np.abs(wp * a) + np.abs(e) * kk
    if w_post is not None:
        c1, c1_abs = (e * yh).mean(-1, keepdims=True), np.abs(e * yh).mean(-1, keepdims=True)
        e_c1 = (e_e * np.abs(yh)).mean(-1, keepdims=True) + c1_abs * kk
        out["dy"] = (ry * (e - yh * c1),
                     ry * (e_e + np.abs(yh) * e_c1 + (np.abs(e) + np.abs(yh) * c1_abs) * kk))
        t = du * a * yh
        out["dw_post"] = (t.sum(0), (np.abs(a * yh) * e_du + np.abs(t) * (kk + _column(rows))).sum(0))
    else:
        out["dy"] = (e, e_e)
    if scale is not None:
        t = alpha * G * u
        out["dscale"] = (t.sum(0), (np.abs(alpha * u) * e_G + np.abs(t) * (kk + _column(rows))).sum(0))
    if w_pre is not None:
        t = dn * rh
        out["dw_pre"] = (t.sum(0), (np.abs(dn) * rh_err + np.abs(t) * (kk + _column(rows))).sum(0))
    return out


def recur_ref(x, f, state=None, complement=True, dh=None, dstate=None):
    """x, f [B, T, C], token by token. Returns {name: (value, bound)} of h, state and, given dh, of
    dx, df and dstate. The bound follows the recurrence: every step adds its own roundings, and the
    earlier ones decay with the gate."""
    B, T, C = x.shape
    gamma, omg = _sigmoid(f), _sigmoid(-f)
    beta = omg if complement else np.ones_like(f)
    unit = (PATH + 4 * np.where(np.isfinite(f), np.abs(f), 0.0)) * U
    h = np.zeros((B, C)) if state is None else state.astype(np.float64)
    S, E = np.abs(h), np.zeros((B, C))
    hs, Ss, Es = np.empty((B, T + 1, C)), np.empty((B, T + 1, C)), np.empty((B, T + 1, C))
    hs[:, 0], Ss[:, 0], Es[:, 0] = h, S, E
    for t in range(T):
        h = gamma[:, t] * h + beta[:, t] * x[:, t]
        S = gamma[:, t] * S + np.abs(beta[:, t] * x[:, t])
        E = gamma[:, t] * E + unit[:, t] * S
        hs[:, t + 1], Ss[:, t + 1], Es[:, t + 1] = h, S, E
    out = {"h": (hs[:, 1:], Es[:, 1:]), "state": (h, E)}
    if dh is None:
        return out
    q = np.zeros((B, C)) if dstate is None else dstate.astype(np.float64)
    Sq, Eq = np.abs(q), np.zeros((B, C))
    dx, df = np.empty_like(x), np.empty_like(x)
    e_dx, e_df = np.empty_like(x), np.empty_like(x)
    for t in reversed(range(T)):
        g, o, un = gamma[:, t], omg[:, t], unit[:, t]
        q, Sq = q + dh[:, t], Sq + np.abs(dh[:, t])
        Eq = Eq + un * Sq
        dx[:, t] = beta[:, t] * q
        e_dx[:, t] = beta[:, t] * (Eq + un * Sq)
        d = hs[:, t] - x[:, t] if complement else hs[:, t]
        Sd = Ss[:, t] + (np.abs(x[:, t]) if complement else 0.0)
        df[:, t] = g * o * q * d
        e_df[:, t] = g * o * (Eq * np.abs(d) + Sq * (Es[:, t] + 2 * un * Sd))
        Eq = g * Eq + un * g * Sq
        q, Sq = g * q, g * Sq
    out.update(dx=(dx, e_dx), df=(df, e_df), dstate=(q, Eq))
    return out
