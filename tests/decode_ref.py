"""Plain forms of the decode operators, written from their definitions: whole
numbers in Python, computed numbers in 64 bits (the cache codes in numpy fp32,
whose single operations are the definition)."""
import math

import numpy as np
import torch


def plan(table, have, add, num_blocks, S, T):
    """(table, slots, sources, row_start, lens, report, refused any entry) as lists."""
    table = [list(r) for r in table]
    R, width = len(table), len(table[0])
    refs = [0] * num_blocks
    state = []
    for r in range(R):
        h, a = have[r], add[r]
        s = "refused" if h < 0 or a < 0 or h > width * S else "full" if h + a > width * S else "ok"
        if 0 <= h <= width * S:
            for p in table[r][:-(-h // S)]:
                if 0 <= p < num_blocks:
                    refs[p] += 1
                else:
                    s = "refused"
        state.append(s)
    free = [p for p in range(num_blocks) if refs[p] == 0]
    tails, needs = [], []
    for r in range(R):
        h, a = have[r], add[r]
        tail, need = None, 0
        if state[r] == "ok":
            need = -(-(h + a) // S) - -(-h // S)
            if h % S and a > 0 and refs[table[r][-(-h // S) - 1]] > 1:
                tail = table[r][-(-h // S) - 1]
                need += 1
        tails.append(tail)
        needs.append(need)
    slots, sources, start, lens = [-1] * T, [-1] * T, [0], []
    end = tok = failed = refused = 0
    for r in range(R):
        h, a = have[r], max(0, add[r])
        first, end = end, end + needs[r]
        t0, tok = tok, tok + a
        ok = state[r] == "ok" and (needs[r] == 0 or end <= len(free)) and (a == 0 or tok <= T)
        start.append(min(tok, T))
        lens.append(h + a if ok else -1)
        refused += state[r] == "refused"
        failed += not ok and state[r] != "refused"
        if not ok:
            continue
        used = -(-h // S) - (tails[r] is not None)
        table[r][used:used + needs[r]] = free[first:end]
        for i in range(a):
            p = h + i
            block = table[r][p // S]
            slots[t0 + i] = block * S + p % S
            sources[t0 + i] = tails[r] if tails[r] is not None and p // S == h // S else block
    return table, slots, sources, start, lens, [sum(needs), len(free), failed, refused]


def append(codes, scales, x, slots, sources):
    """codes int8 [blocks, heads, S, D], scales fp32 [blocks, heads] (numpy, changed in
    place), x fp32 [T, heads, D]."""
    blocks, heads, S, D = codes.shape
    T = len(slots)
    before, was = codes.copy(), scales.copy()
    t = 0
    while t < T:
        if slots[t] < 0 or slots[t] >= blocks * S:
            t += 1
            continue
        page, off = divmod(slots[t], S)
        n = 1
        while t + n < T and slots[t + n] == slots[t] + n and (off + n) < S:
            n += 1
        src = page if sources is None else sources[t]
        if off and not 0 <= src < blocks:
            t += n
            continue
        for h in range(heads):
            new = x[t:t + n, h].astype(np.float32)
            finite = np.abs(new[np.isfinite(new)])
            s0 = was[src, h] if off else np.float32(0)
            s = max(s0, np.float32(finite.max(initial=0)) / np.float32(127))
            s = s if s > np.float32(2.0 ** -100) else np.float32(0)
            turn = np.float32(1) / s if s else np.float32(0)
            ratio = s0 / s if s else np.float32(0)
            with np.errstate(invalid="ignore", over="ignore"):
                q = np.rint(new * turn)
            codes[page, h, off:off + n] = np.nan_to_num(np.clip(q, -127, 127), nan=0).astype(np.int8)
            codes[page, h, :off] = np.rint(before[src, h, :off].astype(np.float32) * ratio).astype(np.int8)
            scales[page, h] = s
        t += n


def attend(q, codes_k, codes_v, scale_k, scale_v, table, start, lens, scale, causal=True):
    """(out, tolerance parts) in 64 bits; q [T, Hq, D]. The parts: sum of
    weight * |value|, largest |value|, largest sum |q k| * scale of a head, keys."""
    q = q.double()
    T, Hq, D = q.shape
    blocks, H, S, _ = codes_k.shape
    G = Hq // H
    out = torch.zeros_like(q)
    mass, peak, big = torch.zeros_like(q), torch.zeros(T, Hq, 1, dtype=torch.float64), torch.zeros(T, Hq, 1, dtype=torch.float64)
    keys = torch.zeros(T, Hq, 1, dtype=torch.float64)
    for r, n in enumerate(lens):
        m = start[r + 1] - start[r]
        if n <= 0 or m == 0:
            continue
        at = [j for j in range(n) if 0 <= table[r][j // S] < blocks]
        if not at:
            continue
        page = torch.tensor([table[r][j // S] for j in at])
        off = torch.tensor([j % S for j in at])
        pos = torch.tensor(at)
        for h in range(Hq):
            k = codes_k[page, h // G, off].double() * scale_k[page, h // G].double()[:, None]
            v = codes_v[page, h // G, off].double() * scale_v[page, h // G].double()[:, None]
            x = q[start[r]:start[r + 1], h]
            w = (x @ k.T) * scale
            if causal:
                last = n - m + torch.arange(m)
                w = w.masked_fill(pos[None, :] > last[:, None], -math.inf)
            some = (w > -math.inf).any(1)
            some = some | w.isnan().any(1)
            p = torch.softmax(torch.where(some[:, None], w, 0.0), 1) * some[:, None]
            rows = slice(start[r], start[r + 1])
            out[rows, h] = p @ v
            mass[rows, h] = p @ v.abs()
            peak[rows, h] = v.abs().max()
            big[rows, h] = ((x.abs() @ k.abs().T) * abs(scale)).amax(1, keepdim=True) + 2.0 ** -1 * x.abs().amax(1, keepdim=True) * k.abs().amax() * D * abs(scale)
            keys[rows, h] = len(at)
    return out, (mass, peak, big, keys)


def attend_tolerance(out, parts, dtype, D):
    """Output rounding (half a step: eps / 2 of the value, tiny * eps / 2 below the normal numbers); each weight's rounding to 11 bits, half a
    step 2^-11 of it or 2^-25 of the largest (which is 1 before the division by
    a sum of at least 1); scores off by D + 8 fp32 roundings of their terms'
    sizes (the part of a query lost below fp16's range is within them), which
    move numerator and denominator by that factor each; 2^-20 for the fp32
    exponentials and sums."""
    mass, peak, big, keys = parts
    half = torch.finfo(dtype).eps / 2
    least = torch.finfo(dtype).tiny * half  # steps of subnormals are tiny * eps
    score = (D + 8) * 2.0 ** -24 * big
    return half * out.abs() + least + mass * (2.0 ** -11 + 2.0 ** -20 + 2 * score) * (1 + half) + keys * 2.0 ** -25 * peak * 2 + 1e-7 * (dtype == torch.float16)


def select(logits, scores, keep, allow=None, finished=None, end=0):
    """Per request the ordered [(score, parent, token)] in Python floats."""
    B, K, V = logits.shape
    x = logits.double().numpy()
    result = []
    for b in range(B):
        found = []
        for i in range(K):
            s0 = float(scores[b, i])
            if not math.isfinite(s0):
                continue
            if finished is not None and bool(finished[b, i]):
                found.append((np.array([s0]), np.array([i * V + end])))
                continue
            ok = np.isfinite(x[b, i])
            if allow is not None:
                words = allow[b, i].numpy().astype(np.int64) & 0xFFFFFFFF
                ok = ok & (((words[:, None] >> np.arange(32)) & 1).reshape(-1)[:V] > 0)
            at = np.nonzero(ok)[0]
            if not at.size:
                continue
            y = x[b, i, at]
            top = y.max()
            lse = top + math.log(math.fsum(np.exp(y - top)))
            found.append(((s0 - lse) + y, i * V + at))
        if not found:
            result.append([])
            continue
        val, idx = np.concatenate([f[0] for f in found]), np.concatenate([f[1] for f in found])
        order = np.lexsort((idx, -val))[:keep]
        result.append([(float(val[o]), int(idx[o]) // V, int(idx[o]) % V) for o in order])
    return result
