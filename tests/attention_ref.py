"""Plain 64-bit references of the page map, the rotary store and the attention
over a paged cache, and builders of their inputs. Row by row, for small sizes."""
import math

import torch

DEV = "cuda"
E4M3_MAX = 448.0


def i32(v, device=DEV):
    return torch.as_tensor(v, dtype=torch.int32).to(device)


def signed(word):
    """A 64-bit word as the int64 that holds it."""
    word &= (1 << 64) - 1
    return word - (1 << 64) if word >> 63 else word


# ----------------------------------------------------------------- page map
def page_map(B, page, width, M, cap, words, context, added, parent, table, ring, owned, ring_pos):
    """All outputs of moe_page_map as lists, from lists; arguments are not changed."""
    table, ring = [list(r) for r in table], list(ring)
    head, free = ring_pos[0] % cap, min(max(ring_pos[1], 0), cap)
    length, offsets, owned_out = [0] * B, [0] * (B + 1), list(owned)
    slot, position, mask = [-1] * M, [0] * M, [[0] * words for _ in range(M)]
    rows = need_all = taken = came_all = came = refused = bad = 0
    pushes = []
    for b in range(B):
        n = max(added[b], 0)
        offsets[b] = min(rows, M)
        total = context[b] + n
        want = -(-total // page)
        owns = 0 <= owned[b] <= width
        if added[b] < 0:
            if owns and came_all + owned[b] <= cap - free:
                pushes += [(came_all + i, table[b][i]) for i in range(owned[b])]
                owned_out[b] = 0
                came = came_all + owned[b]
            else:
                refused += 1
            came_all += owned[b] if owns else 0
            continue
        sound = (context[b] >= 0 and owns and want <= width and context[b] <= owned[b] * page and
                 rows + n <= M and (not words or n <= 64 * words))
        first = rows
        rows += n
        need = max(0, want - owned[b]) if sound else 0
        start, need_all = need_all, need_all + need
        if not sound or (need and need_all > free):
            refused += 1
            continue
        taken = max(taken, need_all if need else 0)
        for i in range(need):
            table[b][owned[b] + i] = ring[(head + start + i) % cap]
        owned_out[b] = max(owned[b], want)
        length[b] = total
        bits, depth = [0] * n, [0] * n
        for i in range(n):
            t, j = first + i, context[b] + i
            up = i - 1
            if parent is not None:
                up = parent[t]
                if not -1 <= up < i:
                    bad += 1
                    up = -1
            bits[i] = 1 << i | (bits[up] if up >= 0 else 0)
            depth[i] = depth[up] + 1 if up >= 0 else 0
            p = table[b][j // page]
            slot[t] = p * page + j % page if 0 <= p <= 0x7fffffff // page - 1 else -1
            position[t] = context[b] + depth[i]
            mask[t] = [signed(bits[i] >> 64 * w) for w in range(words)]
    offsets[B] = min(rows, M)
    for i, p in pushes:
        ring[(head + free + i) % cap] = p
    return dict(table=table, ring=ring, owned=owned_out,
                ring_pos=[(head + taken) % cap, free - taken + came], length=length,
                offsets=offsets, slot=slot, position=position, mask=mask,
                status=[offsets[B], taken, refused, max(0, need_all - free), bad])


# ------------------------------------------------------------ rotary, store
def frequencies(rotary, theta=10000.0, scaling="none", factor=1.0, low=1.0, high=32.0,
                original=4096):
    out = []
    for i in range(rotary // 2):
        f = theta ** (-2.0 * i / rotary)
        if scaling == "linear":
            f /= factor
        elif scaling == "by_parts":
            g = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f *= g + (1.0 - g) / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def turn(x, position, freqs, layout, gain=1.0):
    """x [T, H, D] in 64 bits, its leading 2 len(freqs) elements turned."""
    half = len(freqs)
    angle = position.double().cpu()[:, None] * freqs
    cos, sin = (gain * torch.cos(angle)).to(x.device)[:, None], (gain * torch.sin(angle)).to(x.device)[:, None]
    a = torch.arange(half)
    one, two = (a, a + half) if layout == "half" else (2 * a, 2 * a + 1)
    y = x.clone()
    y[..., one] = x[..., one] * cos - x[..., two] * sin
    y[..., two] = x[..., two] * cos + x[..., one] * sin
    return y


# ---------------------------------------------------------------- attention
def cache_of(g, pages, Hkv, page, D, kind):
    k = torch.randn(pages, Hkv, page, D, generator=g, device=DEV)
    v = torch.randn(pages, Hkv, page, D, generator=g, device=DEV)
    if kind == "bf16":
        return k.bfloat16(), v.bfloat16(), None, None
    ks = 0.01 + 0.01 * torch.rand(Hkv, generator=g, device=DEV)
    vs = 0.01 + 0.01 * torch.rand(Hkv, generator=g, device=DEV)
    code = lambda x, s: (x / s[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return code(k, ks), code(v, vs), ks, vs


def table_of(h, lengths, page, extra=3, width_extra=1):
    """A block table of shuffled pages; the entries past a request's pages are wrong ids."""
    held = [-(-n // page) for n in lengths]
    width = max(held + [1]) + width_extra
    pages = sum(held) + extra
    ids = torch.randperm(pages, generator=h).tolist()
    table = [[-7] * width for _ in lengths]
    for b, n in enumerate(held):
        for i in range(n):
            table[b][i] = ids.pop()
    return i32(table), pages


def random_tree(h, n, words):
    """Ancestor masks of a random tree: parents anywhere before, roots among them."""
    bits, rows = [], []
    for i in range(n):
        up = int(torch.randint(-1, i, (1,), generator=h)) if i else -1
        bits.append(1 << i | (bits[up] if up >= 0 else 0))
        rows.append([signed(bits[i] >> 64 * w) for w in range(words)])
    return rows


def visible(n, length, mask_rows):
    """[n, length] truth: which key each new token sees."""
    ctx = length - n
    see = torch.zeros(n, max(length, 0), dtype=torch.bool)
    if ctx < 0:
        return see
    for i in range(n):
        see[i, :ctx] = True
        for k in range(i + 1):
            if mask_rows is None:
                see[i, ctx + k] = True
            elif k < 64 * len(mask_rows[i]):
                see[i, ctx + k] = bool(mask_rows[i][k // 64] >> (k % 64) & 1)
    return see


def attention(q, kc, vc, ks, vs, table, lengths, news, masks, scale, start=0):
    """(out, bound): the definition in 64 bits [T, Hq, D] and how far the kernel may be off.
    masks: per request None or its rows' words. Keys not seen take no part at all.

    Bound, from the header's precision. A score is a sum of D products in FP32 (a unit in the last
    place, 2^-23, per addition, as tensor cores may truncate): es = (D + 8) 2^-23 scale sum|q k|.
    A weight exp(s - m) is then off by 2 es (s and m) and 2^-20 for the exponential, relative; V's
    weights are rounded to bf16 (2^-8); the sums over L keys add L 2^-23, numerator and
    denominator alike, and rescalings by powers add as many again. With A = sum p|v|:
    |err| <= A (2^-8 + 4 es + 2 (2^-20 + 2 L 2^-23)) and the output's rounding, 2^-8 |o|."""
    T, Hq, D = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(out)
    t = start
    for b, (L, n) in enumerate(zip(lengths, news)):
        see = visible(n, L, masks[b] if masks else None).to(DEV)
        if L < n or L == 0 or n == 0:
            t += n
            continue
        j = torch.arange(L, device=DEV)
        ids = table[b].long()[j // page]
        for h in range(Hkv):
            k, v = kc[ids, h, j % page].float().double(), vc[ids, h, j % page].float().double()
            if ks is not None:
                k, v = k * ks[h].double(), v * vs[h].double()
            qh = q[t:t + n, h * G:(h + 1) * G].double()
            s = torch.einsum("igd,kd->igk", qh, k) * scale
            s = s.masked_fill(~see[:, None], -math.inf)
            es = (D + 8) * 2.0 ** -23 * scale * torch.einsum("igd,kd->igk", qh.abs(), k.abs())
            es = es.masked_fill(~see[:, None], 0.0).amax(2)
            m = s.amax(2, keepdim=True)
            p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
            l = p.sum(2, keepdim=True)
            p = torch.where(l == 0, torch.zeros_like(p), p / l)     # (a NaN stays)
            # a key that no row of the request sees takes no part
            any_see = see.any(0)
            v = torch.where(any_see[:, None], v, torch.zeros_like(v))
            if torch.isfinite(v).all():
                o, A = torch.einsum("igk,kd->igd", p, v), torch.einsum("igk,kd->igd", p, v.abs())
            else:
                o, A = torch.zeros_like(qh), torch.zeros_like(qh)
                for i in range(n):
                    own = see[i].nonzero().flatten()
                    o[i] = p[i][:, own] @ v[own]
                    A[i] = p[i][:, own] @ v[own].abs()
            rel = 2.0 ** -8 + 4 * es[:, :, None] + 2 * (2.0 ** -20 + 2 * L * 2.0 ** -23)
            out[t:t + n, h * G:(h + 1) * G] = o
            bound[t:t + n, h * G:(h + 1) * G] = A * rel + 2.0 ** -8 * o.abs()
        t += n
    return out, bound
