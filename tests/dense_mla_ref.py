"""Plain float64 definitions of the dense latent-attention calls, for their tests (CPU or GPU torch).

Bounds of the attention tests, per output element, with P the softmax weights and A = sum_j P_j |v_j|:
  * P is rounded to bf16 before it multiplies the values (relative 2^-8 each): 2^-8 A;
  * the output is rounded to bf16 once: 2^-8 |o|;
  * a score is an fp32 sum of K products (576 or 192), each product exact in fp32's 48-bit
    intermediate, added with a relative error of at most 2^-23 of the magnitude sum per addition
    (the tensor cores may truncate): |dS| <= K 2^-23 M, M = scale sum_d |q_d k_d|; the scaling and the
    base-2 exponential (2^-22 relative, argument rounding 2^-24 |S| log2 e) add at most
    2^-21 + 2^-22 |S|.  With d = their sum the weights move by a factor within e^{+-2d}: 2 d (1 + d) A;
  * the accumulation over n keys in fp32: n 2^-23 A at worst (the pieces of a split are joined in
    fp32: within the same bound).
lse: d + n 2^-23 + 2^-22 |lse|."""
import math

import torch


def attend(q, k, v, vis, scale):
    """q [n, d], k [m, d], v [m, e] (float64), vis [n]: (out, lse, bound_out, bound_lse)."""
    m = k.shape[0]
    s = scale * (q @ k.t())
    seen = torch.arange(m, device=q.device)[None] < vis[:, None]
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    mag = scale * (q.abs() @ k.abs().t())
    mag = torch.where(seen, mag, torch.zeros_like(mag)).amax(1) if m else torch.zeros(q.shape[0], device=q.device).double()
    top = torch.where(seen, s.abs(), torch.zeros_like(s)).amax(1) if m else torch.zeros_like(mag)
    some = vis > 0
    lse = torch.logsumexp(s, 1) if m else torch.full((q.shape[0],), -math.inf, device=q.device).double()
    p = torch.where(seen, torch.exp(s - torch.where(some, lse, torch.zeros_like(lse))[:, None]), torch.zeros_like(s))
    out = p @ v
    a = p @ v.abs()
    d = q.shape[1] * 2.0 ** -23 * mag + 2.0 ** -21 + 2.0 ** -22 * top
    n = vis.clamp_min(0).double()
    b_out = (2.0 ** -8 + 2 * d * (1 + d) + n * 2.0 ** -23)[:, None] * a + 2.0 ** -8 * out.abs() + 1e-30
    b_lse = d + n * 2.0 ** -23 + 2.0 ** -22 * torch.where(some, lse, torch.zeros_like(lse)).abs() + 1e-30
    return out, lse, b_out, b_lse


def decode(q, pool, table, seq_lens, q_lens, scale):
    """Dense absorbed attention.  Pages whose id is outside the pool are skipped."""
    T, H, _ = q.shape
    dev = q.device
    out = torch.zeros(T, H, 512, dtype=torch.float64, device=dev)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    b_out = torch.full_like(out, 1e-30)
    b_lse = torch.full_like(lse, 1e-30)
    r = 0
    for b, (n, ql) in enumerate(zip(seq_lens, q_lens)):
        for j in range(ql):
            v = max(0, n - ql + j + 1)
            pos = torch.arange(min(v, table.shape[1] * 64), device=dev)
            page = table[b].long()[pos // 64]
            ok = (page >= 0) & (page < pool.shape[0])
            c = pool[page[ok], pos[ok] % 64].double()
            if c.shape[0]:
                vis = torch.full((H,), c.shape[0], device=dev)
                out[r], lse[r], b_out[r], b_lse[r] = attend(q[r].double(), c, c[:, :512], vis, scale)
            r += 1
    return out, lse, b_out, b_lse


def prefill(q, k_nope, k_pe, v, q_lens, k_lens, scale, causal):
    T, H, _ = q.shape
    dev = q.device
    out = torch.zeros(T, H, 128, dtype=torch.float64, device=dev)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    b_out = torch.full_like(out, 1e-30)
    b_lse = torch.full_like(lse, 1e-30)
    r = k0 = 0
    for nq, nk in zip(q_lens, k_lens):
        vis = torch.full((nq,), nk, device=dev)
        if causal:
            vis = (nk - nq + 1 + torch.arange(nq, device=dev)).clamp_min(0)
        for h in range(H if nq else 0):
            k = torch.cat([k_nope[k0:k0 + nk, h], k_pe[k0:k0 + nk]], 1).double()
            o = attend(q[r:r + nq, h].double(), k, v[k0:k0 + nk, h].double(), vis, scale)
            out[r:r + nq, h], lse[r:r + nq, h], b_out[r:r + nq, h], b_lse[r:r + nq, h] = o
        r, k0 = r + nq, k0 + nk
    return out, lse, b_out, b_lse


def check(got, got_lse, ref):
    out, lse, b_out, b_lse = ref
    err = (got.double() - out).abs()
    assert bool((err <= b_out).all()), f"out: worst {float((err / b_out).max())} of the bound"
    if got_lse is not None:
        none = torch.isinf(lse)
        assert torch.equal(torch.isinf(got_lse), none) and bool((got_lse[none] < 0).all())
        e = (got_lse.double() - lse).abs()[~none]
        assert bool((e <= b_lse[~none]).all()), f"lse: worst {float((e / b_lse[~none]).max())} of the bound"


def store(raw, weight, eps, cs, pos, interleaved):
    """The rows [n, 576] in float64, unrounded, and the bound on the kernel's distance from them: one
    rounding to bf16 (2^-8 relative) plus fp32 arithmetic.  Norm: the sum of 512 squares, the square
    root, the division and two products, 520 2^-24 relative at worst (half of it through the root,
    counted in full).  Rope: two products and one sum, 3 2^-24 (|a c| + |b s|)."""
    x = raw.double()
    y = torch.empty_like(x)
    rstd = 1.0 / torch.sqrt((x[:, :512] ** 2).sum(1, keepdim=True) / 512 + eps)
    y[:, :512] = x[:, :512] * rstd * weight.double()
    c, s = cs[pos, :32].double(), cs[pos, 32:].double()
    ia = 512 + (torch.arange(32) * 2 if interleaved else torch.arange(32))
    ib = ia + (1 if interleaved else 32)
    a, b = x[:, ia], x[:, ib]
    y[:, ia], y[:, ib] = a * c - b * s, b * c + a * s
    bound = y.abs() * (2.0 ** -8 + 520 * 2.0 ** -24) + 1e-30
    bound[:, ia] += 3 * 2.0 ** -24 * ((a * c).abs() + (b * s).abs())
    bound[:, ib] += 3 * 2.0 ** -24 * ((b * c).abs() + (a * s).abs())
    return y, bound


def verify(target, draft, tokens, cu_q, u, u_s):
    """One row after the other, float64; returns (out_tokens, accepted)."""
    V = target.shape[1]
    out = [None] * len(tokens)
    acc = []
    for b in range(len(cu_q) - 1):
        r0, r1 = cu_q[b], cu_q[b + 1]
        if r1 <= r0:
            acc.append(0)
            continue
        r, x = r0, -1
        while True:
            x = tokens[r] if r < r1 - 1 and 0 <= tokens[r] < V else -1
            if x < 0:
                break
            q = float(draft[r, x]) if draft is not None else 1.0
            if not float(u[r]) * q < float(target[r, x]):
                break
            out[r] = x
            r += 1
        p = target[r].double()
        w = p.clone()
        if x >= 0:
            w = p - draft[r].double() if draft is not None else torch.where(torch.arange(V) == x, 0.0, p)
        clean = lambda t: torch.where((t > 0) & torch.isfinite(t), t, torch.zeros_like(t))  # noqa: E731
        w = clean(w)
        if float(w.sum()) == 0.0:
            w = clean(p)
        if float(w.sum()) == 0.0:
            out[r] = -1
        else:
            c = torch.cumsum(w, 0)
            past = torch.nonzero((c > float(u_s[b]) * float(c[-1])) & (w > 0))
            out[r] = int(past[0]) if past.numel() else int(torch.nonzero(w > 0)[-1])
        for i in range(r + 1, r1):
            out[i] = -1
        acc.append(r - r0)
    return out, acc
