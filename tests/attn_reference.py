"""Plain 64-bit restatements of the softmax-attention layer's operators (norm + rotary +
append, paged attention) and of the page tables, for the tests."""
import numpy as np
import torch

F64 = torch.float64


def norm_rotate(x, w, offset, eps, pos, inv_freq, R, interleaved, rope_scale):
    """x [rows][H][d], pos [rows] -> (result, magnitude of each element's pair), in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (offset + w.double())
    y, mag = x.clone(), x.abs()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        ang = pos.double() * float(inv_freq[i])
        c, s = (rope_scale * torch.cos(ang))[:, None], (rope_scale * torch.sin(ang))[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = rope_scale * (x[..., a].abs() + x[..., b].abs())
    return y, mag


def attention(q, k, v, past, scale, softcap, window, gate=None):
    """One sequence: q [n][Hq][d] at positions past.., k, v [past + n][Hkv][d] (any float
    type) -> out, lse, sum P|v| (times the gate), largest sum |q k| scale, in 64 bits. Keys
    outside a row's mask are never touched."""
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out, lse, mass, big = [], [], [], []
    for t in range(n):
        hi = past + t + 1
        lo = max(0, hi - window) if window else 0
        qq = q[t].double().view(Hkv, G, d)
        kk, vv = k[lo:hi].double(), v[lo:hi].double()
        x = torch.einsum("hgd,lhd->hgl", qq, kk) * scale
        big.append((torch.einsum("hgd,lhd->hgl", qq.abs(), kk.abs()) * scale).amax(-1).reshape(Hq))
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        P = torch.softmax(x, -1)
        o = torch.einsum("hgl,lhd->hgd", P, vv).reshape(Hq, d)
        m = torch.einsum("hgl,lhd->hgd", P, vv.abs()).reshape(Hq, d)
        if gate is not None:
            z = torch.sigmoid(gate[t].double())
            o, m = o * z, m * z
        out.append(o)
        mass.append(m)
        lse.append(torch.logsumexp(x, -1).reshape(Hq))
    return torch.stack(out), torch.stack(lse), torch.stack(mass), torch.stack(big)


class Tables:
    """The page tables as plain Python lists (a bad argument is not modelled)."""

    def __init__(self, table, lens, refs, page_size):
        self.table, self.lens, self.refs, self.ps = table.tolist(), lens.tolist(), refs.tolist(), page_size

    def _lowest(self):
        return next((i for i, r in enumerate(self.refs) if r == 0), None)

    def free(self, slots):
        for s in slots:
            for j, e in enumerate(self.table[s]):
                if e >= 0:
                    self.refs[e] -= 1
                    self.table[s][j] = -1
            self.lens[s] = 0

    def reserve(self, slots, counts):
        left = self.refs.count(0)
        flagged = False
        for s, c in zip(slots, counts):
            want = -(-(self.lens[s] + c) // self.ps)
            missing = [j for j in range(want) if self.table[s][j] < 0]
            if len(missing) > left:
                flagged, left = True, 0  # nothing more is given in this call
                continue
            left -= len(missing)
            for j in missing:
                self.table[s][j] = page = self._lowest()
                self.refs[page] = 1
        return flagged

    def fork(self, src, dst):
        pairs = []
        for a, z in zip(src, dst):
            full, part = divmod(self.lens[a], self.ps)
            if part:
                page = self._lowest()
                if page is None:
                    pairs.append((-1, -2))
                    continue
                self.refs[page] = 1
                self.table[z][full] = page
                pairs.append((self.table[a][full], page))
            else:
                pairs.append((-1, -1))
            for j in range(full):
                self.table[z][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            self.lens[z] = self.lens[a]
        return pairs

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [i for i in range(live) if self.refs[i] == 0]
        movers = [i for i in range(live, len(self.refs)) if self.refs[i] > 0]
        remap = [i if r > 0 else -1 for i, r in enumerate(self.refs)]
        for a, z in zip(movers, holes):
            remap[a] = z
            self.refs[z], self.refs[a] = self.refs[a], 0
        self.table = [[remap[e] if e >= 0 else e for e in row] for row in self.table]
        return movers, holes, remap

    def same(self, table, lens, refs):
        assert np.array_equal(np.array(self.table), table.cpu().numpy())
        assert self.lens == lens.tolist() and self.refs == refs.tolist()
