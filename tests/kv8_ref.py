"""The paged 8-bit cache's operators in plain form: Python integers and float64.

Written from the definitions in include/ds.h, sharing no code with the library.
Tensors may live on any device; results are on the CPU.
"""
from __future__ import annotations

import math

import torch

MIN_SCALE = 2.0 ** -64


def qmax(dtype) -> float:
    return 127.0 if dtype == torch.int8 else 448.0


def _f32(x):
    """Rounded to fp32 where the definition holds a value in 32 bits."""
    return x.to(torch.float32).double()


def codes(x, dtype):
    """Nearest codes (ties to even) of float64 values that fp32 holds exactly."""
    q = qmax(dtype)
    x = torch.nan_to_num(x, nan=0.0, posinf=math.inf, neginf=-math.inf).clamp(-q, q)
    return torch.round(x).to(torch.int8) if dtype == torch.int8 else x.float().to(dtype)


def assign(lens, n_new, free, n_free, table, N, page):
    """(table, lens_out, n_free_out, cu, slots, refused) as lists; refused: 16 or 32 bits."""
    P, W = len(free), len(table[0])
    table = [list(r) for r in table]
    cu, slots, out, bits = [0], [-1] * N, [], 0
    e = used = 0
    for b, (l, n) in enumerate(zip(lens, n_new)):
        fits = l >= 0 and n >= 0 and l + n <= W * page
        have = -(-l // page) if fits else 0
        need = -(-(l + n) // page) - have if fits else 0
        roomy = fits and cu[-1] + max(n, 0) <= N
        ok = roomy and (need == 0 or e + need <= n_free)
        if not ok:
            bits |= 16 if not roomy else 32
        else:
            for j in range(need):
                page_id = free[n_free - 1 - e - j]
                if not 0 <= page_id < P:
                    bits |= 8
                    page_id = -1
                table[b][have + j] = page_id
            for i in range(n):
                pos = l + i
                page_id = table[b][pos // page]
                if not 0 <= page_id < P:
                    bits |= 8
                else:
                    slots[cu[-1] + i] = page_id * page + pos % page
            used = max(used, e + need if need else 0)
        out.append(l + n if ok else l)
        e += need
        cu.append(cu[-1] + max(n, 0))
    return table, out, n_free - used, cu, slots, bits


def release(lens, done, table, free, n_free, page):
    P, W = len(free), len(table[0])
    free, out, bits = list(free), [], 0
    for b, (l, d) in enumerate(zip(lens, done)):
        if not d:
            out.append(l)
            continue
        out.append(0)
        if not 0 <= l <= W * page:
            bits |= 16
        for j in range(min(max(-(-l // page), 0), W)):
            page_id = table[b][j]
            if n_free >= P:
                bits |= 16
                continue
            if not 0 <= page_id < P:
                bits |= 8
                page_id = -1
            free[n_free] = page_id
            n_free += 1
    return free, out, n_free, bits


def append(K, V, KV, scales, slots, cu, page):
    """KV, scales after the append (copies); K, V [N, Hkv, d]."""
    KV, scales = KV.cpu().clone(), scales.cpu().clone()
    u8 = KV.view(torch.uint8)
    K, V, slots, cu = K.cpu().double(), V.cpu().double(), slots.tolist(), cu.tolist()
    dt, q = KV.dtype, qmax(KV.dtype)
    for b in range(len(cu) - 1):
        i = cu[b]
        while i < cu[b + 1] and slots[i] >= 0:
            pg, off = divmod(slots[i], page)
            n = min(page - off, cu[b + 1] - i)
            for kv, X in enumerate((K, V)):
                x = X[i:i + n].transpose(0, 1)                      # [Hkv, n, d]
                a = torch.where(torch.isfinite(x), x, 0.0).abs().amax(dim=(1, 2))
                s = _f32(a / q).clamp(min=MIN_SCALE)
                if off:
                    s0 = scales[pg, :, kv].double()
                    s = torch.maximum(s, s0)
                    old = KV[pg, :, :off, kv].double() * _f32(s0 / s)[:, None, None]
                    grew = codes(_f32(old), dt).view(torch.uint8)
                    u8[pg, :, :off, kv] = torch.where((s > s0)[:, None, None], grew,
                                                      u8[pg, :, :off, kv])
                inv = _f32(1.0 / s)
                u8[pg, :, off:off + n, kv] = codes(_f32(x * inv[:, None, None]),
                                                   dt).view(torch.uint8)
                scales[pg, :, kv] = s.float()
            i += n
    return KV, scales


def rows(KV, scales, table, b, g, tokens, page):
    """K and V values [n, d] (float64) of the given tokens of sequence b, KV head g."""
    t = torch.as_tensor(tokens, dtype=torch.long)
    pg = table[b].cpu().long()[t // page]
    x = KV.cpu().view(torch.uint8)[pg, g, t % page].view(KV.dtype).double()
    x = x * scales.cpu()[pg, g].double()[..., None]
    return x[:, 0], x[:, 1]


def v_scales(scales, table, b, g, tokens, page):
    """The V scales [n] of the given tokens' pages."""
    pg = table[b].cpu().long()[torch.as_tensor(tokens, dtype=torch.long) // page]
    return scales.cpu()[pg, g, 1].double()


def attend(q, K, V, scale, sv=None):
    """(O, lse, bound on |O - exact| of the kernel, bound on its lse) of one query head.

    The bounds count fp32 roundings (u = 2^-24): a logit is a sum of 128 products
    (exact, added in any order, each addition off by u or, truncated, 2u of the
    partial sums), scaled by three factors and turned into a power of two
    (|l| * 4u); a weight is off by the logits' error relatively (twice: its own
    and the denominator's) plus 8u for the exponential (2 ulp) and the parts the
    weight is split into (2^-22); sums over n rows add at most one rounding for
    each 4 rows, and a merge some 64.

    sv: the rows' V scales.  The kernel holds a weight p_t sv_t relative to a
    power of two that is at most twice the largest of them, m, as two f16 of
    which the second ends at 2^-24 of a range of 2^14: beside the 2^-22 above
    it is off by up to half a step, 2^-25 / 2^14 = 2^-39, of 2m.  Over the rows
    that adds 2^-38 m sum |code_t|, which counts in the dims in which the rows
    of large weight hold a 0.
    """
    n, u = K.shape[0], 2.0 ** -24
    if n == 0:
        return torch.zeros(V.shape[1], dtype=torch.float64), -math.inf, 0.0, 0.0
    q = q.cpu().double()
    x = (K @ q) * scale
    lse = torch.logsumexp(x, 0).item()
    w = torch.softmax(x, 0)
    dl = ((K.abs() @ q.abs()) * scale * (2 * 128 + 8) * u).amax().item() \
        + 4 * u * x.abs().amax().item()
    rel = 2 * dl + (n / 4 + 64 + 32) * u
    tol = rel * (w @ V.abs()) + 1e-30
    if sv is not None:
        codes = torch.where(sv[:, None] > 0, V / sv[:, None], 0.0).abs()
        tol = tol + 2.0 ** -38 * (w * sv).amax() * codes.sum(0)
    return w @ V, lse, tol, dl + rel + u * abs(lse)
