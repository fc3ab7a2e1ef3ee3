"""Trees of drafted tokens, page tables and adjusted logits from their
definitions: lists and float64, on the CPU, no code of the library."""
import numpy as np

import kv_ref

BAD_TOKEN, BAD_GAMMA, BAD_LENGTH, BAD_PAGE, NO_PAGES, BAD_TREE, BAD_PENALTY, BAD_FORK = (
    1 << 0, 1 << 4, 1 << 7, 1 << 8, 1 << 9, 1 << 10, 1 << 11, 1 << 12)


def random_parents(rng, B, G, bushy=0.6):
    """Parents [B, G] of nodes 1 .. G, any order that has parents first."""
    p = np.zeros((B, G), np.int32)
    for j in range(1, G + 1):
        p[:, j - 1] = np.minimum(j - 1, (rng.random(B) ** bushy * j).astype(int))
    return p


def ancestors(parents, n):
    """[n] lists: the nodes that each of nodes 0 .. n - 1 sees, itself last."""
    out = [[0]]
    for j in range(1, n):
        out.append(out[parents[j - 1]] + [j])
    return out


def sees(parents, gammas):
    """Truth values [B, N, N] and depths [B, N]."""
    B, G = parents.shape
    bits, depth = np.zeros((B, G + 1, G + 1), bool), np.zeros((B, G + 1), np.int32)
    for b in range(B):
        for i, way in enumerate(ancestors(parents[b], int(gammas[b]) + 1)):
            bits[b, i, way] = True
            depth[b, i] = len(way) - 1
    return bits, depth


def words(bits):
    """Truth values [..., n] -> int32 [..., ceil(n / 32)]."""
    n = bits.shape[-1]
    pad = np.zeros(bits.shape[:-1] + (-n % 32,), bool)
    b = np.concatenate([bits, pad], -1).reshape(*bits.shape[:-1], -1, 32)
    return (b.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def accept(target, draft, parents, gamma):
    """One sequence: (accepted_len, next_token, path)."""
    at, path = 0, [0]
    while True:
        t = int(target[at])
        if t < 0:
            return 0, -1, []
        child = [j for j in range(1, gamma + 1) if parents[j - 1] == at and draft[j - 1] == t]
        if not child:
            return len(path) - 1, t, path
        at = child[0]
        path.append(at)


def attend(q, kval, vval, table, kv_len, ptable, prefix, gammas, page_size, scale, bits):
    """As kv_ref.attend, with what the nodes see of the step [B, N, N]."""
    B, N, Hq, D = q.shape
    G = Hq // kval.shape[1]
    out, lse = np.zeros(q.shape), np.full((B, N, Hq), -np.inf)
    weight, size = np.zeros(q.shape), np.zeros((B, N, Hq))
    for b in range(B):
        before, n = int(kv_len[b]), int(gammas[b]) + 1
        k = kv_ref.tokens_of(kval, table, ptable, prefix, page_size, b, before + n)
        v = kv_ref.tokens_of(vval, table, ptable, prefix, page_size, b, before + n)
        for i in range(n):
            at = np.concatenate([np.arange(before), before + np.nonzero(bits[b, i, :n])[0]])
            if at.size == 0:
                continue
            for h in range(Hq):
                kk, vv = k[at, h // G], v[at, h // G]
                with np.errstate(invalid="ignore", over="ignore"):
                    z = scale * (kk @ q[b, i, h])
                    m = z.max()
                    e = np.exp(z - m)
                    s = e.sum()
                    out[b, i, h] = (e / s) @ vv
                    lse[b, i, h] = m + np.log(s)
                    weight[b, i, h] = (e / s) @ np.abs(vv)
                    size[b, i, h] = scale * (np.abs(kk) @ np.abs(q[b, i, h])).max()
    return out, lse, weight, size


class Pool:
    """Page tables over reference counts, as lists."""

    def __init__(self, refs, table, held, page_size, prefix=0):
        self.refs, self.table, self.held = list(refs), [list(r) for r in table], list(held)
        self.page, self.prefix = page_size, prefix

    def there(self, i):
        return 0 <= i < len(self.refs)

    def resize(self, kv_len, n_step):
        want, status = [], []
        wide = len(self.table[0])
        for b, x in enumerate(kv_len):
            t = x + n_step - self.prefix
            w = 0 if x == -1 else -(-t // self.page)
            bad = x < -1 or (x >= 0 and t < 0) or w > wide or not 0 <= self.held[b] <= wide
            want.append(self.held[b] if bad else w)
            status.append(BAD_LENGTH if bad else 0)
        for b, w in enumerate(want):
            for i in range(w, self.held[b] if not status[b] else w):
                if self.there(self.table[b][i]):
                    self.refs[self.table[b][i]] -= 1
                else:
                    status[b] |= BAD_PAGE
        free, at = [i for i, r in enumerate(self.refs) if r <= 0], 0
        for b, w in enumerate(want):
            need = max(0, w - self.held[b]) if not status[b] & BAD_LENGTH else 0
            at += need
            if need and at > len(free):
                status[b] |= NO_PAGES
                continue
            for i in range(need):
                page = free[at - need + i]
                self.table[b][self.held[b] + i] = page
                self.refs[page] = 1
            if not status[b] & BAD_LENGTH:
                self.held[b] = w
        return status

    def fork(self, kv_len, src, dst):
        """Updates kv_len; returns (copies, status)."""
        B, wide = len(self.table), len(self.table[0])
        before, held = list(kv_len), list(self.held)
        copies, status, plan = [[-1, -1, 0] for _ in src], [0] * len(src), []
        for j, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < B and 0 <= d < B) or s == d or d in list(dst)[:j] or held[d] != 0:
                status[j] = BAD_FORK
                continue
            t = 0 if before[s] == -1 else before[s] - self.prefix
            if before[s] < -1 or t < 0 or not 0 <= held[s] <= wide or -(-t // self.page) > held[s]:
                status[j] = BAD_LENGTH
                continue
            plan.append((j, s, d, t // self.page, t % self.page))
        free, at = [i for i, r in enumerate(self.refs) if r <= 0], 0
        for j, s, d, full, part in plan:
            at += part > 0
            if part and at > len(free):
                status[j] = NO_PAGES
                continue
            for i in range(full):
                page = self.table[s][i]
                self.table[d][i] = page
                if self.there(page):
                    self.refs[page] += 1
                else:
                    status[j] |= BAD_PAGE
            if part:
                new, old = free[at - 1], self.table[s][full]
                self.table[d][full] = new
                self.refs[new] = 1
                if self.there(old):
                    copies[j] = [old, new, part]
                else:
                    status[j] |= BAD_PAGE
            self.held[d], kv_len[d] = full + (part > 0), before[s]
        return copies, status


def adjust(z, seq, prompt, path, r, f, p, bias, allowed):
    """One position: float64 logits [V] -> (adjusted, the largest magnitude on the way, whether a step applied).
    bias: pairs (token, value); allowed: truth values [V] or None."""
    V = len(z)
    y, size, hit = z.copy(), np.abs(z), np.zeros(V, bool)
    made, seen = np.zeros(V, int), np.zeros(V, bool)
    for s, t in enumerate(list(seq) + list(path)):
        if 0 <= t < V:
            seen[t] = True
            made[t] += s >= prompt
    with np.errstate(invalid="ignore", over="ignore"):
        y[seen] = np.where(y > 0, y / r, y * r)[seen]
        size = np.maximum(size, np.abs(y))
        y[made > 0] = (y - f * made - p)[made > 0]
        size = size + (abs(f) * made + abs(p)) * (made > 0)
        hit |= seen
        for t, v in dict(bias).items():  # the last of several
            if 0 <= t < V:
                y[t] += v
                size[t] += abs(v)
                hit[t] = True
    if allowed is not None:
        y[~allowed] = -np.inf
    return y, size, hit
