"""Plain 64-bit forms of the paged-cache operators and of the prompt's attention weights, one
(request, head) at a time, and the caches the tests run on."""
import math

import torch

from mea_workloads import cu_seqlens, make_qkv, randn

# Half a rounding step of a 16-bit output (relative).
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# fp32 arithmetic: scores of up to 2^6 in log2 units carry an absolute error of a few 2^-18 (their
# products' sums, the multiplication by scale, the subtraction of the maximum), exp2 adds 2^-22.
F32 = 2.0 ** -14


class Cache:
    """A block cache of ``lens`` keys per request in shuffled blocks. Slots past a request's end and
    unused blocks hold NaN; block table entries past a request's last block hold an id that
    does not exist."""

    def __init__(self, lens, hq, hkv, d, dtype, bs, seed, extra=3):
        self.lens, self.hq, self.hkv, self.d, self.bs = lens, hq, hkv, d, bs
        self.dtype = dtype
        _, k, v = make_qkv([1], [sum(lens)], hq, hkv, d, dtype, seed)
        self.off = cu_seqlens(lens).tolist()
        self.k = [k[a:b] for a, b in zip(self.off, self.off[1:])]
        self.v = [v[a:b] for a, b in zip(self.off, self.off[1:])]
        nblk = [-(-x // bs) for x in lens]
        self.num_blocks = sum(nblk) + extra
        perm = torch.randperm(self.num_blocks, generator=torch.Generator().manual_seed(seed))
        self.kc = torch.full((self.num_blocks, bs, hkv, d), float("nan"), dtype=dtype)
        self.vc = torch.full_like(self.kc, float("nan"))
        self.table = torch.full((len(lens), max(max(nblk), 1)), 1 << 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(lens):
            for j in range(nblk[b]):
                blk = int(perm[at])
                at += 1
                m = min(bs, n - j * bs)
                self.table[b, j] = blk
                self.kc[blk, :m] = self.k[b][j * bs:j * bs + m]
                self.vc[blk, :m] = self.v[b][j * bs:j * bs + m]
        self.spare = perm[at:].tolist()
        self.cu = cu_seqlens(lens)
        self.max = max(lens)

    def gpu(self):
        return self.kc.cuda(), self.vc.cuda(), self.table.cuda(), self.cu.cuda()


def attend(q, k, v, x):
    """Scores x [rows, keys] (-inf: masked) -> weights, out, sum of weights times |v|, lse."""
    lse = torch.logsumexp(x, 1) if x.shape[1] else torch.full((x.shape[0],), -math.inf).double()
    p = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return p, p @ v, p @ v.abs(), lse


def decode(c, q, scale, slopes=None, keys=None):
    """One token per request over the keys ``keys[b][g]`` (index lists; None: all). Returns out, its
    sum of weights times |v|, lse [hq, n], and the group-summed weights of the keys by
    request and KV head."""
    n, hq, d = q.shape
    r = hq // c.hkv
    out, mag = torch.zeros(n, hq, d).double(), torch.zeros(n, hq, d).double()
    lse, w = torch.zeros(hq, n).double(), []
    for b in range(n):
        wb = []
        for g in range(c.hkv):
            idx = torch.arange(c.lens[b]) if keys is None else torch.tensor(keys[b][g]).long()
            k, v = c.k[b][idx, g].double(), c.v[b][idx, g].double()
            x = scale * (q[b, g * r:(g + 1) * r].double() @ k.t())
            if slopes is not None:
                x = x - slopes[g * r:(g + 1) * r, None].double() * (c.lens[b] - 1 - idx)
            p, o, m, z = attend(None, k, v, x)
            out[b, g * r:(g + 1) * r], mag[b, g * r:(g + 1) * r] = o, m
            lse[g * r:(g + 1) * r, b] = z
            wb.append(p.sum(0))
        w.append(wb)
    return out, mag, lse, w


def tree(c, q, nq, masks, scale, slopes=None):
    """Drafted tokens: ``masks[b]`` bool [n_b, n_b]."""
    tq, hq, d = q.shape
    r = hq // c.hkv
    out, mag = torch.zeros(tq, hq, d).double(), torch.zeros(tq, hq, d).double()
    lse = torch.zeros(hq, tq).double()
    off = 0
    for b, n in enumerate(nq):
        length = c.lens[b]
        ctx = length - n
        seen = torch.ones(n, length, dtype=torch.bool)
        seen[:, ctx:] = masks[b]
        other = masks[b] & ~torch.eye(n, dtype=torch.bool)
        pos = torch.arange(length).double()
        pos[ctx:] = ctx + other.sum(1)
        for h in range(hq):
            k, v = c.k[b][:, h // r].double(), c.v[b][:, h // r].double()
            x = scale * (q[off:off + n, h].double() @ k.t())
            if slopes is not None:
                x = x - float(slopes[h]) * (pos[ctx:, None] - pos[None, :]).abs()
            _, o, m, z = attend(None, k, v, x.masked_fill(~seen, -math.inf))
            out[off:off + n, h], mag[off:off + n, h], lse[h, off:off + n] = o, m, z
        off += n
    return out, mag, lse


def block_bounds(c):
    """[num_blocks, hkv, 2, d] of the blocks in use, and which blocks those are."""
    out = torch.zeros(c.num_blocks, c.hkv, 2, c.d, dtype=c.dtype)
    used = torch.zeros(c.num_blocks, dtype=torch.bool)
    for b, n in enumerate(c.lens):
        for j in range(-(-n // c.bs)):
            x = c.k[b][j * c.bs:(j + 1) * c.bs]
            blk = int(c.table[b, j])
            out[blk, :, 0], out[blk, :, 1] = x.amin(0), x.amax(0)
            used[blk] = True
    return out, used


def choose(c, q, bounds, n_select, n_first, n_last):
    """The blocks' choice: for each request and KV head the ascending list."""
    r = c.hq // c.hkv
    res = []
    for b, n in enumerate(c.lens):
        nblk = -(-n // c.bs)
        row = []
        for g in range(c.hkv):
            x = q[b, g * r:(g + 1) * r].double()
            lo, hi = bounds[c.table[b, :nblk].long(), g].double().unbind(1)
            # (for ranges with lo <= hi: the sum over heads and columns of max(x lo, x hi))
            up, down = x.clamp_min(0).sum(0), x.clamp_max(0).sum(0)
            score = (hi * up + lo * down).sum(1).float()
            order = sorted(range(nblk), key=lambda j: (
                not (j < n_first or j >= nblk - n_last),
                0.0 if (j < n_first or j >= nblk - n_last) else -float(score[j]), j))
            row.append(sorted(order[:n_select]))
        res.append(row)
    return res


def prompt_weights(q, k, lse, lens_q, lens_k, scale, causal, slopes, last, width):
    hq, hkv = q.shape[1], k.shape[1]
    r = hq // hkv
    out = torch.zeros(len(lens_q), hkv, width).double()
    qo = ko = 0
    for s, (lq, lk) in enumerate(zip(lens_q, lens_k)):
        i0 = max(0, lq - last) if last else 0
        pos = torch.arange(i0, lq) + lk - lq
        j = torch.arange(lk)
        for h in range(hq):
            x = scale * (q[qo + i0:qo + lq, h].double() @ k[ko:ko + lk, h // r].double().t())
            if slopes is not None:
                x = x - float(slopes[h]) * (pos[:, None] - j).abs()
            p = torch.exp(x - lse[h, qo + i0:qo + lq, None].double())
            if causal:
                p = torch.where(j[None, :] <= pos[:, None], p, torch.zeros_like(p))
            out[s, h // r, :lk] += p.sum(0)
        qo += lq
        ko += lk
    return out


def check_out(out, lse, ref, mag, rlse, dtype):
    """out: P and the result are each rounded to 16 bits once (half a step of the weighted sum of
    |v|, and of the result), the rest is fp32. lse: fp32."""
    u = UNIT[dtype]
    assert bool(torch.isfinite(out).all())
    err = (out.double() - ref).abs()
    bound = u * (mag + ref.abs()) + F32 * mag + 1e-30 + (2.0 ** -25 if u == 2.0 ** -11 else 0.0)
    assert bool((err <= bound).all()), f"out: {float((err / bound).max())} of the bound"
    empty = torch.isinf(rlse)
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all())
    e = (lse.double() - rlse)[~empty].abs()
    assert bool((e <= F32 * (1 + rlse[~empty].abs() / 16)).all()), f"lse: {float(e.max())}"
