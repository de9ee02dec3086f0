"""64-bit references of the rotary positions and of the paged 8-bit cache, written from their
definitions on the host, one request, block and row at a time."""
import numpy as np
import torch

# the finite numbers of e4m3 from 0 to 448, in the order of their bytes
E4M3 = np.array([(m / 8.0 if e == 0 else 1.0 + m / 8.0) * 2.0 ** (max(e, 1) - 7)
                 for e in range(16) for m in range(8)][:127])


def rotary(x, positions, inv_freq, interleaved, first, magnitude, inverse=False):
    """x [T, H, d] in fp64: each pair as a complex number times magnitude e^{i angle}."""
    x = x.double().cpu().numpy().copy()
    f = inv_freq.double().cpu().numpy()
    angle = positions.cpu().numpy().astype(np.float64)[:, None] * f[None]
    turn = magnitude * np.exp((-1j if inverse else 1j) * angle)[:, None, :]
    n = len(f)
    j = np.arange(n)
    re = first + (2 * j if interleaved else j)
    im = re + (1 if interleaved else n)
    z = (x[..., re] + 1j * x[..., im]) * turn
    x[..., re], x[..., im] = z.real, z.imag
    return torch.from_numpy(x)


def rotary_size(x, inv_freq, interleaved, first):
    """|u| + |w| of each channel's pair (0 for the channels that are copied)."""
    x = x.double().cpu().abs()
    n = len(inv_freq)
    j = torch.arange(n)
    re = first + (2 * j if interleaved else j)
    im = re + (1 if interleaved else n)
    out = torch.zeros_like(x)
    out[..., re] = out[..., im] = x[..., re] + x[..., im]
    return out


def plan(past, new, table, free, n_free, block, rows):
    """The allocator as a loop over requests; lists in, a dict of lists out."""
    N, W, F = len(past), len(table[0]), len(free)
    table, free = [list(r) for r in table], list(free)
    top = min(max(n_free, 0), F)
    for i in range(N):      # ended requests first
        have = -(-past[i] // block)
        if new[i] == -1 and past[i] >= 0 and have <= W:
            for b in table[i][:have]:
                if top < F:
                    free[top] = b
                    top += 1
    cu, status, context = [0], [], []
    starved = False
    end = 0
    for i in range(N):
        n = max(new[i], 0)
        end += n
        cu.append(min(end, rows))
        have, want = -(-past[i] // block), -(-(past[i] + n) // block)
        st = 0
        if past[i] < 0 or new[i] < -1:
            st = 1
        elif want > W or past[i] + n > 0x7fffffff:
            st = 2
        elif n > 0 and end > rows:
            st = 4
        elif new[i] != -1 and want > have:
            if starved or want - have > top:
                st, starved = 3, True
            else:
                for b in range(have, want):
                    top -= 1
                    table[i][b] = free[top]
        status.append(st)
        context.append(past[i] + n if st == 0 and new[i] != -1 else 0)
    positions, slots = [0] * rows, [-1] * rows
    for i in range(N):
        for j in range(cu[i + 1] - cu[i]):
            p = past[i] + j
            positions[cu[i] + j] = min(p, 0x7fffffff)
            b = table[i][p // block] if status[i] == 0 else -1
            if 0 <= b and b * block + p % block < 1 << 31:
                slots[cu[i] + j] = b * block + p % block
    return dict(cu_seqlens=cu, context_lens=context, status=status, positions=positions,
                slots=slots, n_free=[top], block_table=table, free_blocks=free)


def scale_of(largest):
    """The smallest power of two, 2^-60 at least, under which `largest` is at most 448."""
    s = 2.0 ** -60
    while largest > 448.0 * s:
        s *= 2.0
    return s


def e4m3_bytes(x):
    """The bytes of the nearest e4m3 numbers, ties to even; at most 448; NaN 0x7f."""
    a = np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0))
    a = np.minimum(a, 448.0)
    hi = np.searchsorted(E4M3, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(E4M3[hi] == a, hi, code)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x) & ~np.isnan(x), 128, 0)).astype(np.uint8)


def e4m3_values(b):
    v = np.append(E4M3, np.nan)[b & 127]
    return np.where(b & 128, -v, v)


def write(x, slots, cache, scale, block):
    """x [T, H, d] into cache [nb, H, block, d] bytes and scale [nb, H], run by run."""
    x = x.double().cpu().numpy()
    cache, scale = cache.copy(), scale.astype(np.float64).copy()
    nb, H = scale.shape
    T, t = len(slots), 0
    while t < T:
        s = slots[t]
        if s < 0 or s >= nb * block:
            t += 1
            continue
        n = 1
        while t + n < T and slots[t + n] == s + n and (s + n) % block:
            n += 1
        b, off = s // block, s % block
        for h in range(H):
            rows = x[t:t + n, h]
            fine = np.abs(rows[np.isfinite(rows)])
            need = scale_of(fine.max() if fine.size else 0.0)
            old = scale[b, h]
            now = max(old, need) if off else need
            if off:
                cache[b, h, :off] = e4m3_bytes(e4m3_values(cache[b, h, :off]) * (old / now))
            cache[b, h, off:off + n] = e4m3_bytes(rows / now)
            scale[b, h] = now
        t += n
    return cache, scale


def attention(q, k, v, k_scale, v_scale, table, context, cu, scale, block):
    """(o, mass, size, least): o [T, Hq, d] in fp64, rows behind the last request's NaN, and what
    bounds on the error are multiples of: per element sum p |v| / sum p and sum |v| / v_scale times
    the scale of the heaviest key's block (heaviest by p v_scale), per row the largest scale
    sum |q| |k| and |log2 v_scale| over its keys.  k, v: the bytes [nb, H, block, d] as numpy."""
    q = q.double().cpu().numpy()
    T, Hq, d = q.shape
    nb, H = k_scale.shape
    G = Hq // H
    o, mass = np.full((T, Hq, d), np.nan), np.zeros((T, Hq, d))
    size, least = np.zeros((T, Hq, 2)), np.zeros((T, Hq, d))
    for i, c in enumerate(context):
        n = cu[i + 1] - cu[i]
        there = [x for x in range(max(c, 0)) if 0 <= table[i][x // block] < nb]
        b = np.array([table[i][x // block] for x in there], dtype=np.int64)
        at = np.array([x % block for x in there], dtype=np.int64)
        seen = np.array(there)[None] <= (c - n + np.arange(n))[:, None]       # [n, keys]
        any_key = seen.any(axis=1)
        for h in range(H):
            K = e4m3_values(k[b, h, at]) * k_scale[b, h].astype(np.float64)[:, None]
            V = e4m3_values(v[b, h, at]) * v_scale[b, h].astype(np.float64)[:, None]
            for hq in range(h * G, (h + 1) * G):
                x = q[cu[i]:cu[i + 1], hq]
                o[cu[i]:cu[i + 1], hq] = 0.0
                if not len(there):
                    continue
                s = np.where(seen, scale * (x @ K.T), -np.inf)
                top = np.where(any_key, np.max(s, axis=1, initial=-np.inf), 0.0)
                w = np.where(seen, np.exp(s - top[:, None]), 0.0)
                total = np.where(any_key, w.sum(axis=1), 1.0)[:, None]
                clean = np.nan_to_num(V) if np.isnan(V).any() else V
                vs = v_scale[b, h].astype(np.float64)
                heavy = vs[np.argmax(s + np.log(vs)[None], axis=1)]
                least[cu[i]:cu[i + 1], hq] = (seen @ np.abs(clean / vs[:, None])) * heavy[:, None]
                y, y_abs = w @ clean / total, w @ np.abs(clean) / total
                if np.isnan(V).any():
                    y = np.where((w @ np.isnan(V)) > 0, np.nan, y)
                rows = slice(cu[i], cu[i + 1])
                o[rows, hq] = np.where(any_key[:, None], y, 0.0)
                mass[rows, hq] = np.where(any_key[:, None], y_abs, 0.0)
                size[rows, hq, 0] = np.where(
                    any_key, abs(scale) * np.max(np.where(seen, np.abs(x) @ np.abs(K).T, 0.0),
                                                 axis=1, initial=0.0), 0.0)
                size[rows, hq, 1] = np.max(np.where(seen, np.abs(np.log2(vs))[None], 0.0), axis=1,
                                           initial=0.0)
    return o, mass, size, least


def attention_bound(o, mass, size, least, d, longest, bf16):
    """How far o may be off: a score's products carry 2^-22 of each (q in two halves of 11 bits)
    and d / 16 sums of two products rounded to 2^-22 of the whole; the weights' 2^-20 (exponent,
    its argument up to 16); the logarithm of a value scale in the argument, rounded itself, in the
    sum and in the reference, 3 ln 2 2^-24 < 2^-22 of its size; the running sums 2^-24 for each
    16 keys; for bf16 the weights' 11 bits and the result's rounding, 2^-8.  And an fp16 weight is off by up to 2^-25 however small it is, where
    the largest weight times its scale is 2^7 at least for bf16, 2^15 for fp32 (whose second half
    is an fp16 number too): 2^-32 or 2^-40 of `least`."""
    ds, log_scale = size[..., :1] * (1 + d / 8) * 2.0 ** -22, size[..., 1:]
    rel = 2 * ds + 2.0 ** -20 + 2 * log_scale * 2.0 ** -22 + (longest / 16 + 8) * 2.0 ** -23
    if bf16:
        return mass * (rel + 2.0 ** -11) + np.abs(o) * 2.0 ** -8 + least * 2.0 ** -32
    return mass * rel + least * 2.0 ** -40
