"""Plain implementations, in 64 bits, of what include/lora_kv.h defines."""
import torch

GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
# every scale by its byte: 5 bits of exponent and 3 of fraction
SCALES = torch.tensor([m * 2.0 ** -17 if e == 0 else (1 + m / 8) * 2.0 ** (e - 15) for e in range(31) for m in range(8)],
                      dtype=torch.float64)


def padded(D):
    return 64 if D <= 64 else 128


def nearest(x, to):
    """Places of the entries of ascending `to` nearest to x, ties to even places."""
    hi = torch.searchsorted(to, x.contiguous()).clamp(1, to.numel() - 1)
    up, down = to[hi] - x, x - to[hi - 1]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x):
    """Codes [..., Dp] and scale bytes [..., Dp / 16] of bf16 rows x [..., D]."""
    D = x.shape[-1]
    x = torch.nn.functional.pad(x.double(), (0, padded(D) - D)).unflatten(-1, (-1, 16))
    a = x.abs().amax(-1)
    byte = nearest(a.nan_to_num(0, 1e300, 1e300) / 6, SCALES[:227])        # 226: 10240
    s = SCALES[byte][..., None]
    code = nearest((x.abs().nan_to_num(0, 1e300) / s.clamp(min=1e-30)).clamp(max=6), GRID)
    code = torch.where(s > 0, code + 8 * (x < 0), torch.zeros_like(code))
    nan = x.isnan().any(-1)
    byte[nan] = 255
    code[nan] = 0
    return code.flatten(-2), byte


def dequantise(code, byte):
    """What codes and scale bytes stand for (NaN for the byte 255)."""
    table = torch.cat([SCALES, torch.full((8,), float("nan"), dtype=torch.float64)])
    v = torch.where(code >= 8, -GRID[code % 8], GRID[code % 8]).unflatten(-1, (-1, 16)) * table[byte.long()][..., None]
    return v.flatten(-2)


def places(D, key):
    """For key (0 to 15) of a tile: bytes of the key codes' and value codes' pairs by element (the even element's
    code in the low half), and of the scales by group."""
    Dp = padded(D)
    d = torch.arange(Dp)
    g = torch.arange(Dp // 16)
    k = key * (Dp // 2) + d // 2
    v = 9 * Dp + ((((key // 8) * 8 + d // (Dp // 8)) * 4 + key % 8 // 2) * (Dp // 64) + d % (Dp // 8) // 8) * 8 + (key % 2) * 4 + d % 8 // 2
    return k, 8 * Dp + key * (Dp // 16) + g, v, 17 * Dp + (g * 4 + key % 8 // 2) * 4 + key // 8 * 2 + key % 2


def put(tile, key, k, v):
    """Write one head's key and value rows (bf16 [D]) as key `key` of a tile (uint8 [18 * Dp], host)."""
    kc, ks, vc, vs = places(k.shape[-1], key)
    for row, at, scale_at in ((k, kc, ks), (v, vc, vs)):
        code, byte = quantise(row)
        tile[at[0::2]] = (code[0::2] | code[1::2] << 4).to(torch.uint8)
        tile[scale_at] = byte.to(torch.uint8)


def get(tile, key, D):
    """The key's and value's rows [D] that a tile holds, fp64."""
    kc, ks, vc, vs = places(D, key)
    out = []
    for at, scale_at in ((kc, ks), (vc, vs)):
        nib = tile[at].long() >> (4 * (torch.arange(at.numel()) % 2)) & 15
        out.append(dequantise(nib, tile[scale_at])[:D])
    return out


def rope(x, w, eps, position, inv_freq, interleaved):
    """x [T, heads, D], position [T], inv_freq fp32 [rot / 2]: norms (w given) and rotation, and the size of the
    operands of each output element."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    half = 0 if inv_freq is None else inv_freq.numel()
    y, size = x.clone(), x.abs()
    if half:
        a = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
        b = a + 1 if interleaved else a + half
        f = (position.double()[:, None] * inv_freq.double()[None, :])[:, None]
        y[..., a] = x[..., a] * torch.cos(f) - x[..., b] * torch.sin(f)
        y[..., b] = x[..., b] * torch.cos(f) + x[..., a] * torch.sin(f)
        size = size.clone()
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


class Pages:
    """The state of the pages and what lora_kv_release, lora_kv_fork and lora_kv_compact do to it, in plain loops."""

    def __init__(self, table, ctx, ref, free, head, page):
        self.table, self.ctx, self.ref, self.free, self.head, self.page = table, ctx, ref, free, head, page

    def held(self, r):
        cap = len(self.table[r]) * self.page
        return -(-max(0, min(self.ctx[r], cap)) // self.page)

    def release(self, rows):
        freed, seen = [], set()
        for r in rows:
            if r < 0 or r >= len(self.ctx) or r in seen:
                continue
            seen.add(r)
            for p in self.table[r][:self.held(r)]:
                if 0 <= p < len(self.ref):
                    self.ref[p] -= 1
            self.ctx[r] = 0
        for p, n in enumerate(self.ref):
            if n < 0:
                freed.append(p)
                self.ref[p] = 0
        first = max(0, self.head - len(freed))
        self.free[first:self.head] = freed[:self.head - first]
        self.head = first

    def fork(self, parents, children):
        known = lambda r: 0 <= r < len(self.ctx)  # noqa: E731
        pairs, done, short = [], set(), False
        named = {f for f, c in zip(parents, children) if known(f) and known(c)}
        for f, c in zip(parents, children):
            if not known(f) or not known(c) or c in done or c in named:
                if known(f) and known(c):
                    done.add(c)
                pairs.append((-1, -1))
                continue
            done.add(c)
            n = max(0, min(self.ctx[f], len(self.table[f]) * self.page))
            whole, part = n // self.page, n % self.page > 0
            if part and (short or self.head >= len(self.free)):
                short = True
                self.ctx[c] = 0
                pairs.append((-1, -1))
                continue
            for j in range(whole):
                self.table[c][j] = self.table[f][j]
                if 0 <= self.table[f][j] < len(self.ref):
                    self.ref[self.table[f][j]] += 1
            if part:
                self.table[c][whole] = self.free[self.head]
                pairs.append((self.table[f][whole], self.free[self.head]))
                self.head += 1
            else:
                pairs.append((-1, -1))
            self.ctx[c] = n
        return pairs

    def compact(self, limit, most):
        n = len(self.ref)
        used = {p for r in range(len(self.ctx)) for p in self.table[r][:self.held(r)] if 0 <= p < n}
        free = {p for p in self.free[self.head:] if 0 <= p < n} - used
        pairs = list(zip(sorted(p for p in used if p >= limit), sorted(p for p in free if p < limit)))[:most]
        to = dict(pairs)
        for r in range(len(self.ctx)):
            for j in range(self.held(r)):
                self.table[r][j] = to.get(self.table[r][j], self.table[r][j])
        for a, b in pairs:
            self.ref[b], self.ref[a] = self.ref[a], 0
        left = sorted(free - set(to.values()) | set(to))
        self.head = len(self.free) - len(left)
        self.free[self.head:] = left
        return pairs + [(-1, -1)] * (most - len(pairs))
