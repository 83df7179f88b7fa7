"""Plain 64-bit attention over states of another length, and how far a bf16 kernel may be from it.

Bounds, element by element. u = 2^-8 is half a bf16 step relative to the value. EPS bounds what
32-bit arithmetic and the exponential add to a softmax weight relative to it: the exponential's own
error (at most 1e-4 for its polynomial route), and logits summed in 32 bits, an absolute error of at
most (d + 2) 2^-24 s sum|q||k| (`logit`). Sums over n terms add n 2^-24.
  out:  a weight rounded to bf16 is off by u, the row sum by EPS, the result is rounded once:
        |err| <= (u + 2 eps) A + u |o|,  A = sum_j p_j |v_j|
  D = dout.(out + out_low), where out_low is what rounding out leaves off, itself rounded (2^-17 of out):
        |err D| <= sum_c |dout_c| ((u + 2 eps) A_c + 2^-17 |o_c|)
  dv:   |err| <= (u + 2 eps) sum_i p_i |dout_i| + u |dv|
  ds = p (dp - D), rounded to bf16: |err ds| <= p ((u + 2 eps) |dp - D| + err D + d 2^-24 sum|dout||v|)
  dk:   |err| <= s sum_i err ds_i |q_i| + (rows 2^-24) s sum |ds||q| + u |dk|
  dq:   the same over keys, with ds in two bf16 terms: 2^-17 in place of its u.
"""
import math

import torch

U = 2.0 ** -8
TWO = 2.0 ** -17        # of two bf16 terms: half a step of 8 bits below the first one's half step
F = 2.0 ** -24
EXP = 1e-4


def attend(q, k, v, scale, dout=None):
    """One key head: q [R, d], k, v [n, d] (n may be 0), dout [R, d] or None, any dtype.
    Returns a dict of 64-bit results and of the bounds on a bf16 kernel's error."""
    q, k, v = q.double(), k.double(), v.double()
    d, n = q.shape[-1], k.shape[0]
    if n == 0:
        zero, empty = torch.zeros_like(q), torch.zeros_like(k)
        lse = torch.full(q.shape[:1], -math.inf, dtype=q.dtype, device=q.device)
        return dict(out=zero, lse=lse, out_tol=zero, lse_tol=torch.zeros_like(lse), dq=zero, dk=empty, dv=empty,
                    dq_tol=zero, dk_tol=empty, dv_tol=empty)
    s = scale * (q @ k.T)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    o = p @ v
    logit = (d + 2) * F * scale * (q.abs() @ k.abs().T).amax(-1, keepdim=True)
    eps = EXP + logit + n * F
    out_tol = 1.01 * ((U + 2 * eps) * (p @ v.abs()) + U * o.abs())
    r = dict(out=o, lse=lse, out_tol=out_tol, lse_tol=(2 * eps[:, 0] + 4 * F * lse.abs()))
    if dout is None:
        return r
    g = dout.double()
    rows = q.shape[0]
    dp = g @ v.T
    dterm = (g * o).sum(-1, keepdim=True)
    ds = p * (dp - dterm)
    e = eps + (rows * F)
    both_tol = 1.01 * ((U + 2 * eps) * (p @ v.abs()) + TWO * o.abs())
    w, w2 = (p * ((u + 2 * e) * (dp - dterm).abs() + (g.abs() * both_tol).sum(-1, keepdim=True)
                  + d * F * (g.abs() @ v.abs().T)) for u in (U, TWO))
    r["dv"] = p.T @ g
    r["dv_tol"] = 1.01 * (((U + 2 * e) * p).T @ g.abs() + U * r["dv"].abs())
    r["dq"], r["dk"] = scale * (ds @ k), scale * (ds.T @ q)
    r["dq_tol"] = 1.01 * (scale * (w2 @ k.abs() + n * F * (ds.abs() @ k.abs())) + U * r["dq"].abs())
    r["dk_tol"] = 1.01 * (scale * (w.T @ q.abs() + rows * F * (ds.abs().T @ q.abs())) + U * r["dk"].abs())
    return r


def cross(q, k, v, key_len=None, scale=None, dout=None):
    """[B, H, n_q, d] queries against [B, H_kv, n_k, d] states: dicts as attend(), whole tensors."""
    b, h, nq, d = q.shape
    hk, nk = k.shape[1], k.shape[2]
    scale = scale or d ** -0.5
    names = ("out", "lse") + (("dq", "dk", "dv") if dout is not None else ())
    shapes = dict(out=q.shape, lse=q.shape[:3], dq=q.shape, dk=k.shape, dv=k.shape)
    res = {x + t: torch.zeros(shapes[x], dtype=torch.float64, device=q.device) for x in names for t in ("", "_tol")}
    qg = q.reshape(b, hk, -1, d)
    gg = dout.reshape(b, hk, -1, d) if dout is not None else None
    for i in range(b):
        n = nk if key_len is None else min(max(int(key_len[i]), 0), nk)
        for e in range(hk):
            r = attend(qg[i, e], k[i, e, :n], v[i, e, :n], scale, None if gg is None else gg[i, e])
            for x in res:
                base = x.replace("_tol", "")
                if base in ("dk", "dv"):
                    res[x][i, e, :n] = r[x]
                else:
                    t = res[x].view(b, hk, *(( -1, d) if base != "lse" else (-1,)))
                    t[i, e] = r[x]
    return res


def prefix(q, kp, vp, ko, vo, prefix_len=None, own_len=None, scale=None):
    b, h, nq, d = q.shape
    g, hk = kp.shape[:2]
    ks, vs, lens = [], [], []
    for i in range(b):
        gi = i // (b // g)
        np_ = kp.shape[2] if prefix_len is None else min(max(int(prefix_len[gi]), 0), kp.shape[2])
        no = ko.shape[2] if own_len is None else min(max(int(own_len[i]), 0), ko.shape[2])
        pad = kp.shape[2] + ko.shape[2] - np_ - no
        z = torch.zeros((hk, pad, d), dtype=q.dtype, device=q.device)
        ks.append(torch.cat([kp[gi, :, :np_], ko[i, :, :no], z], 1))
        vs.append(torch.cat([vp[gi, :, :np_], vo[i, :, :no], z], 1))
        lens.append(np_ + no)
    return cross(q, torch.stack(ks), torch.stack(vs), lens, scale)


def check(got, ref, name, what=""):
    """got against ref[name] within ref[name_tol], element by element; infinities have to match."""
    g, w, t = got.double(), ref[name], ref[name + "_tol"]
    fin = torch.isfinite(w)
    assert torch.equal(g[~fin], w[~fin]), f"{what} {name}: infinities differ"
    bad = ~((g - w).abs() <= t + 1e-30) & fin
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what} {name}: {int(bad.sum())} of {bad.numel()} off, first {i}: "
                             f"{float(g[i]):.6g} against {float(w[i]):.6g}, allowed {float(t[i]):.3g}")
