"""Oracle of the serving calls: step plan, rotary positions with several axes,
token append and attention over records, in plain Python and float64."""
from __future__ import annotations

import numpy as np

from .hkv_oracle import (HEAD_DIM, dequant_records, f16_bits, pair_indices, quant_fp8_vectors,
                         quant_int4_vectors, rope_theta)


def plan_step(kv_len, new_tokens, block_table, free_blocks, free_count, block_tokens, n_tokens):
    """One step, request by request.  Returns a dict of copies: table, free,
    free_count, kv_len, q_start, positions, slots, refused."""
    table, free = block_table.copy(), free_blocks.copy()
    mb, cap = table.shape[1], free.size
    lens = [min(max(int(x), 0), mb * block_tokens) for x in kv_len]
    held = [-(-x // block_tokens) for x in lens]
    stack = [int(x) for x in free[:min(max(int(free_count), 0), cap)]]
    had = len(stack)
    for r, n in enumerate(new_tokens):
        if n < 0:
            stack += [int(x) for x in table[r, :held[r]]]
    stack = stack[:cap]
    free[had:len(stack)] = stack[had:]
    out_len, refused, short = [], [], False
    for r, n in enumerate(int(x) for x in new_tokens):
        if n < 0:
            out_len.append(0)
            refused.append(0)
            continue
        want = lens[r] + n
        if want > mb * block_tokens:
            out_len.append(lens[r])
            refused.append(1)
            continue
        need = -(-want // block_tokens) - held[r]
        if need > len(stack):
            short = True         # later requests that need blocks find none either
        if need > 0 and short:
            out_len.append(lens[r])
            refused.append(1)
            continue
        for i in range(need):
            table[r, held[r] + i] = stack.pop()
        out_len.append(want)
        refused.append(0)
    q_start = np.minimum(np.concatenate([[0], np.cumsum(np.maximum(np.asarray(new_tokens, np.int64), 0))]),
                         2 ** 31 - 1)
    positions = np.zeros(n_tokens, np.int64)
    slots = np.full(n_tokens, -1, np.int64)
    for r in range(len(lens)):
        for j in range(max(0, min(int(q_start[r + 1]), n_tokens) - int(q_start[r]))):
            i, pos = int(q_start[r]) + j, lens[r] + j
            positions[i] = pos
            if not refused[r] and table[r, pos // block_tokens] >= 0:
                slots[i] = int(table[r, pos // block_tokens]) * block_tokens + pos % block_tokens
    return dict(table=table, free=free, free_count=len(stack), kv_len=np.array(out_len, np.int64),
                q_start=q_start, positions=positions, slots=slots, refused=np.array(refused))


def rope_heads(x, positions, axis, freq, base, pairs, inverse=False):
    """x [n, H, 128] in float64 with pair i turned by positions[axis[i], t] /
    base^(2 freq[i] / 128); positions [n_axes, n]."""
    out = np.asarray(x, np.float64).copy()
    first, second = pair_indices(pairs)
    for i in range(HEAD_DIM // 2):
        if axis[i] < 0:
            continue
        phi = positions[axis[i]].astype(np.float64) / float(base) ** (2 * freq[i] / HEAD_DIM)
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None] * (-1 if inverse else 1)
        a, b = x[:, :, first[i]].astype(np.float64), x[:, :, second[i]].astype(np.float64)
        turned = phi[:, None] != 0
        out[:, :, first[i]] = np.where(turned, a * c - b * s, a)
        out[:, :, second[i]] = np.where(turned, a * s + b * c, b)
    return out


def append_tokens(k, v, slots, records, fmt, block_tokens):
    """Copy of one layer's records [n_blocks, bytes] with the tokens' vectors
    in their slots; slots outside the pool are skipped."""
    out = records.copy()
    nb, h = out.shape[0], k.shape[1]
    quant = quant_fp8_vectors if fmt == "fp8" else quant_int4_vectors
    n, c = block_tokens * h, HEAD_DIM if fmt == "fp8" else HEAD_DIM // 2
    for i, x in enumerate((k, v)):
        codes, scales = quant(np.asarray(x, np.float32))
        codes = np.ascontiguousarray(codes).view(np.uint8).reshape(x.shape[0], h, c)
        bits = np.ascontiguousarray(f16_bits(scales).astype("<u2")).view(np.uint8).reshape(x.shape[0], h, 2)
        for t, slot in enumerate(int(s) for s in slots):
            if not 0 <= slot < nb * block_tokens:
                continue
            b, at = slot // block_tokens, slot % block_tokens * h
            for j in range(h):
                p = i * n * c + (at + j) * c
                out[b, p:p + c] = codes[t, j]
                p = 2 * n * c + 2 * i * n + 2 * (at + j)
                out[b, p:p + 2] = bits[t, j]
    return out


def attend(q, records, fmt, block_tokens, n_kv_heads, block_table, kv_len, q_start=None,
           sm_scale=HEAD_DIM ** -0.5, causal=True, delta_m=None, rope_base=10000.0,
           pairs="half_split"):
    """(out, lse, spread, reach) in float64; rows of no request are NaN.
    spread [n, Hq, 128] = sum_m p_m |v_m| and reach [n, Hq] = the largest
    |sm_scale| * sum_d |q_d k_m,d| of the tokens seen: what rounding errors
    of weights and of scores are relative to."""
    q = np.asarray(q, np.float64)
    n, hq, _ = q.shape
    nb, mb = records.shape[0], block_table.shape[1]
    kd, vd = (x[0].astype(np.float64) for x in
              dequant_records(records[None], fmt, block_tokens, n_kv_heads)) if nb else (None, None)
    out = np.full(q.shape, np.nan)
    lse = np.full((n, hq), np.nan)
    spread, reach = np.zeros(q.shape), np.zeros((n, hq))
    first, second = pair_indices(pairs)
    for r in range(len(kv_len)):
        a, b = (r, r + 1) if q_start is None else (min(max(int(x), 0), n) for x in q_start[r:r + 2])
        ln = min(max(int(kv_len[r]), 0), mb * block_tokens)
        entries = block_table[r, :-(-ln // block_tokens)].astype(np.int64)
        tok = np.arange(ln)
        live = ((entries >= 0) & (entries < nb))[tok // block_tokens]
        tok = tok[live]
        if tok.size:
            blk, at = entries[tok // block_tokens], tok % block_tokens
            k, v = kd[blk, at].copy(), vd[blk, at]              # [T, H, 128]
            if delta_m is not None:
                phi = delta_m[r, tok // block_tokens].astype(np.float64)[:, None, None] * rope_theta(rope_base)
                x, y = k[..., first], k[..., second]
                k[..., first] = x * np.cos(phi) - y * np.sin(phi)
                k[..., second] = x * np.sin(phi) + y * np.cos(phi)
        for j in range(b - a):
            last = ln - (b - a) + j if causal else ln - 1
            sees = tok <= last
            if not sees.any():
                out[a + j], lse[a + j] = 0.0, -np.inf
                continue
            for h in range(hq):
                kh = h // (hq // n_kv_heads)
                s = k[sees, kh] @ q[a + j, h] * sm_scale
                top = s.max()
                p = np.exp(s - top)
                lse[a + j, h] = top + np.log(p.sum())
                out[a + j, h] = p @ v[sees, kh] / p.sum()
                spread[a + j, h] = p @ np.abs(v[sees, kh]) / p.sum()
                reach[a + j, h] = (np.abs(k[sees, kh]) @ np.abs(q[a + j, h])).max() * abs(sm_scale)
    return out, lse, spread, reach
