"""Plain 64-bit forms of the operators between the token ids and the FP8
products (dropout, layer norm, router, embedding), with the error that fp32
arithmetic and one final rounding may add to each value.

The bounds are worst cases, fixed before any run, and count as ops_reference
does: 2^-24 of its result for an fp32 operation, (n - 1) * 2^-24 of the sum of
the magnitudes for a sum of n terms, 2 units in the last place (2^-22) for exp,
log and 1/sqrt.  Sums along a row are counted as 128 additions deep.
"""
import numpy as np
import torch

from ops_reference import F

DEEP = 128 * F


# ---- dropout
def philox(counter, key):
    """Philox4x32-10 of arrays of uint64 that hold 32-bit words."""
    mask = np.uint64(0xFFFFFFFF)
    shift = np.uint64(32)
    x = [np.asarray(v, np.uint64) for v in counter]
    k0, k1 = (int(k) for k in key)
    for _ in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> shift) ^ x[1] ^ np.uint64(k0), b & mask,
             (a >> shift) ^ x[3] ^ np.uint64(k1), a & mask]
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    return x


def cut_of(p):
    return int(np.floor(float(np.float32(p)) * 65536 + 0.5))


def drop_factor(rows, cols, p, seed, step, site):
    """What a dropout multiplies each element by (float64 [rows, cols])."""
    cut = cut_of(p)
    if cut == 0:
        return torch.ones(rows, cols, dtype=torch.float64)
    group, row = np.meshgrid(np.arange(-(-cols // 8)), np.arange(rows))
    words = philox((group, row, np.full_like(row, site), np.full_like(row, step % 2 ** 32)),
                   (seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32))
    bits = np.stack([h for w in words for h in (w % 65536, w // 65536)], 2).reshape(rows, -1)[:, :cols]
    return torch.from_numpy((bits >= cut) * float(np.float32(65536 / (65536 - cut))))


def dropped(x, factor):
    """x * factor, 0 where factor is 0 whatever x is."""
    return torch.where(factor > 0, x.double() * factor, 0.0)


# ---- layer norm
class LayerNorm:
    def __init__(self, u, res, weight, bias, eps, weight_offset, factor):
        self.res, self.eps, self.factor = res.double(), eps, factor
        self.u = None if u is None else dropped(u, factor)
        rows, self.H = res.shape
        self.w = (torch.ones(self.H, dtype=torch.float64) if weight is None
                  else weight_offset + weight.double())
        self.b = torch.zeros(self.H, dtype=torch.float64) if bias is None else bias.double()

    def forward(self):
        v = self.res if self.u is None else self.res + self.u
        err = torch.zeros_like(v) if self.u is None else F * self.u.abs() + F * v.abs()
        self.out, self.out_err = v, err
        self.mean = v.mean(1)
        self.mean_err = DEEP * v.abs().mean(1) + err.mean(1)
        away = v - self.mean[:, None]
        away_err = err + self.mean_err[:, None] + F * away.abs()
        var = away.square().mean(1)
        var_err = (2 * away.abs() * away_err + away_err.square()).mean(1) + DEEP * var
        self.rstd = (var + self.eps).rsqrt()
        # of 1 / sqrt: half the relative error of its argument, while that is small
        rel = var_err / (var + self.eps) + 6 * F
        self.rstd_err = self.rstd * rel
        hat = away * self.rstd[:, None]
        hat_err = away_err * self.rstd[:, None] * (1 + rel[:, None]) + hat.abs() * rel[:, None]
        self.y = hat * self.w + self.b
        self.y_err = (hat_err + 3 * F * hat.abs()) * self.w.abs() + 2 * F * (self.b.abs() + self.y.abs())
        return self

    def backward(self, dy, dres_out, res_out, mean, rstd):
        """Gradients from what the forward pass kept, and their bounds."""
        c = DEEP + 16 * F
        rows = len(res_out)
        s = rstd.double()[:, None]
        hat, g = (res_out.double() - mean.double()[:, None]) * s, dy.double() * self.w
        d = torch.zeros_like(hat) if dres_out is None else dres_out.double()
        size = d.abs() + s * (g.abs() + g.abs().mean(1, keepdim=True)
                              + hat.abs() * (g * hat).abs().mean(1, keepdim=True))
        d = d + s * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
        terms = dy.double() * hat
        return {"dres": (d, c * size),
                "du": (dropped(d, self.factor), (c + F) * size * self.factor),
                "dweight": (terms.sum(0), (rows + 6) * F * terms.abs().sum(0)),
                "dbias": (dy.double().sum(0), (rows + 2) * F * dy.double().abs().sum(0))}


# ---- router
class Router:
    def __init__(self, logits, mask, topk, normalize, balance, z):
        self.x = logits.double()
        self.T, self.E = logits.shape
        self.K, self.normalize, self.balance, self.z = topk, normalize, balance, z
        valid = torch.isnan(self.x).any(1) | (self.x > -np.inf).any(1)
        self.valid = valid if mask is None else valid & mask.bool()
        safe = torch.where(self.valid[:, None], self.x, 0.0)
        self.lse = torch.logsumexp(safe, 1)
        self.p = torch.softmax(safe, 1)
        away = (safe - safe.amax(1, keepdim=True)).abs()
        # the exponent's argument is rounded, exp itself, the sum, the division
        self.p_rel = F * torch.where(torch.isfinite(away), away, 0.0) + 8 * F
        self.p_rel = self.p_rel + (self.p * self.p_rel).sum(1, keepdim=True) + DEEP
        self.lse_err = 4 * F * self.lse.abs() + DEEP + 8 * F + (self.p * self.p_rel).sum(1)

    def forward(self):
        """Walks over the tokens; sorts by (-logit, index), NaN first."""
        idx = torch.full((self.T, self.K), -1, dtype=torch.int32)
        counts = torch.zeros(self.E + 1, dtype=torch.int32)
        for t in self.valid.nonzero()[:, 0].tolist():
            row = [(-np.inf if np.isnan(v) else -v, np.isnan(v), e)
                   for e, v in enumerate(self.x[t].tolist()) if v != -np.inf]
            row.sort(key=lambda r: (not r[1], r[0], r[2]))
            for k, (_, _, e) in enumerate(row[:self.K]):
                idx[t, k] = e
                counts[e] += 1
            counts[self.E] += 1
        self.idx, self.counts = idx, counts
        self.n = int(counts[self.E])
        at, chosen = idx.long().clamp(min=0), idx >= 0
        w = torch.where(chosen, self.p.gather(1, at), 0.0)
        rel = self.p_rel.gather(1, at)
        if self.normalize:
            w = torch.where(chosen, w / w.sum(1, keepdim=True), 0.0)
            rel = rel + rel.amax(1, keepdim=True) + 64 * F
        # Below 2^-126 fp32 has a fixed spacing of 2^-149: exp is off by at most two
        # of them, which a division by a sum of at least 1 (it has the largest
        # term, exp(0)) does not enlarge, and the division by half a one.
        self.weights, self.w_err = w, w * (rel + 2 * F) + 3 * 2.0 ** -149 * (w > 0)
        n = max(self.n, 1)
        f = counts[:self.E].double() / (n * self.K)
        p = torch.where(self.valid[:, None], self.p, 0.0)
        lse = torch.where(self.valid, self.lse, 0.0)
        a = self.balance * self.E * (f * p.sum(0)).sum() / n
        b = self.z * lse.square().sum() / n
        deep = (self.T + self.E + 32) * F
        rel_p = (p * self.p_rel).sum() / p.sum() if self.n else 0.0
        self.loss = a + b
        # the probabilities' errors are no larger than the largest relative one
        worst = (self.p_rel * (p > 0)).max() if self.T else 0.0
        self.loss_err = (abs(a) * (deep + worst + rel_p) + abs(b) * deep
                         + abs(self.z) * (2 * lse.abs() * self.lse_err).sum() / n)
        return self

    def backward(self, dweights, dloss):
        n = max(self.n, 1)
        f = self.counts[:self.E].double() / (n * self.K)
        chosen, at = self.idx >= 0, self.idx.long().clamp(min=0)
        dw = torch.zeros(self.T, self.K, dtype=torch.float64)
        if dweights is not None:
            dw = torch.where(chosen, dweights.double(), 0.0)
        each = (dloss * self.balance * self.E / n * f).expand(self.T, -1).clone()
        size_each = each.abs()
        extra, size_extra = torch.zeros_like(each), torch.zeros_like(each)
        w, rel = self.weights, self.p_rel
        if self.normalize:
            inner = w * (dw - (w * dw).sum(1, keepdim=True))
            extra.scatter_add_(1, at, torch.where(chosen, inner, 0.0))
            big = w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))
            size_extra.scatter_add_(1, at, torch.where(chosen, big, 0.0))
        else:
            each.scatter_add_(1, at, dw)
            size_each.scatter_add_(1, at, dw.abs())
        top = rel.amax(1, keepdim=True)
        zt = 2 * dloss * self.z / n * self.lse[:, None]
        d = self.p * (each - (self.p * each).sum(1, keepdim=True) + zt) + extra
        size = self.p * (size_each + (self.p * size_each).sum(1, keepdim=True) + zt.abs())
        err = (size * (2 * top + DEEP + 32 * F) + size_extra * (6 * top + 128 * F)
               + self.p * abs(2 * dloss * self.z / n) * self.lse_err[:, None])
        keep = self.valid[:, None]
        return torch.where(keep, d, 0.0), torch.where(keep, err, 0.0)


# ---- embedding
def embedding(idx, table, scale):
    inside = (idx >= 0) & (idx < len(table))
    out = torch.zeros(len(idx), table.shape[1], dtype=torch.float64)
    out[inside] = scale * table.double()[idx[inside].long()]
    return out, F * out.abs()


def embedding_backward(idx, dout, vocab, scale, old=None):
    inside = (idx >= 0) & (idx < vocab)
    at, rows = idx[inside].long(), dout.double()[inside]
    count = torch.zeros(vocab, 1, dtype=torch.float64).index_add_(0, at, torch.ones(len(at), 1, dtype=torch.float64))
    total = torch.zeros(vocab, dout.shape[1], dtype=torch.float64).index_add_(0, at, rows)
    size = torch.zeros_like(total).index_add_(0, at, rows.abs())
    out, err = scale * total, (count + 2) * F * abs(scale) * size
    if old is not None:
        out = out + old.double()
        err = err + torch.where(count > 0, F * out.abs(), 0.0)
    return out, err, count[:, 0] > 0
