"""A paged key/value cache in plain numpy loops: what each kv_* call has to do, for the tests."""
import numpy as np
import torch


class Model:
    """The cache's state on the host; K and V as bf16 bit patterns [n_pages, Hkv, page_size, D]."""

    def __init__(self, k, v, table, lens, ref):
        bits = lambda t: t.detach().cpu().contiguous().view(torch.int16).numpy().copy()  # noqa: E731
        self.k, self.v = bits(k), bits(v)
        self.table, self.lens, self.ref = (t.detach().cpu().numpy().copy() for t in (table, lens, ref))
        self.P = self.k.shape[2]

    def pages(self, n):
        return -(-n // self.P)

    def take(self):
        page = int(np.flatnonzero(self.ref == 0)[0])
        self.ref[page] = 1
        return page

    def free_pages(self):
        return int((self.ref == 0).sum())

    def append(self, k_new, v_new, cu):
        bits = lambda t: t.detach().cpu().contiguous().view(torch.int16).numpy()  # noqa: E731
        k_new, v_new = bits(k_new), bits(v_new)
        n = np.diff(cu)
        room = self.table.shape[1] * self.P
        own = all(m <= 0 or a % self.P == 0 or self.ref[self.table[b, a // self.P]] == 1
                  for b, (a, m) in enumerate(zip(self.lens, n)) if 0 <= a < room)
        if not own or (n < 0).any() or cu[0] < 0 or cu[-1] > len(k_new) or (self.lens < 0).any() or (self.lens + n > room).any():
            return -1
        want = sum(self.pages(a + m) - self.pages(a) for a, m in zip(self.lens, n))
        if want > self.free_pages():
            return int(want - self.free_pages())
        for b, m in enumerate(n):
            for p in range(self.pages(self.lens[b]), self.pages(self.lens[b] + m)):
                self.table[b, p] = self.take()
            for u in range(m):
                page, slot = self.table[b, self.lens[b] // self.P], self.lens[b] % self.P
                self.k[page, :, slot], self.v[page, :, slot] = k_new[cu[b] + u], v_new[cu[b] + u]
                self.lens[b] += 1
        return 0

    def fork(self, parents, children):
        rows = len(self.lens)
        ok = all(0 <= x < rows for x in (*parents, *children)) and len(set(children)) == len(children) and \
            not set(parents) & set(children) and all(self.lens[c] == 0 for c in children) and \
            all(0 <= self.lens[a] <= self.table.shape[1] * self.P for a in parents) and \
            all(0 <= self.table[a, self.lens[a] // self.P] < len(self.ref) for a in parents if self.lens[a] % self.P)
        if not ok:
            return -1
        want = sum(int(self.lens[a] % self.P != 0) for a in parents)
        if want > self.free_pages():
            return want - self.free_pages()
        for a, c in zip(parents, children):
            full, part = divmod(int(self.lens[a]), self.P)
            self.table[c] = -1
            self.table[c, :full] = self.table[a, :full]
            for p in self.table[a, :full]:
                self.ref[p] += 1
            if part:
                page, old = self.take(), self.table[a, full]
                self.table[c, full] = page
                self.k[page, :, :part], self.v[page, :, :part] = self.k[old, :, :part], self.v[old, :, :part]
            self.lens[c] = self.lens[a]
        return 0

    def drop(self, b, keep):
        for p in range(self.pages(keep), self.pages(int(self.lens[b]))):
            self.ref[self.table[b, p]] -= 1
            self.table[b, p] = -1
        self.lens[b] = keep

    def compact(self, cu, accepted, cu_acc):
        status, ref = np.zeros(len(self.lens), np.int32), self.ref.copy()
        for b in range(len(self.lens)):
            n, a0, a1 = int(cu[b + 1] - cu[b]), int(cu_acc[b]), int(cu_acc[b + 1])
            ctx = int(self.lens[b]) - n
            if n < 0 or ctx < 0 or a0 < 0 or a1 < a0 or a1 > len(accepted) or a1 - a0 > n:
                status[b] = -1
                continue
            acc = [int(x) for x in accepted[a0:a1]]
            place = lambda t: (self.table[b, t // self.P], t % self.P)  # noqa: E731
            end = ctx + len(acc)
            inside = len(acc) < n and end % self.P and ref[place(end)[0]] != 1  # ends in a shared page
            if inside or any(not 0 <= x < n for x in acc) or any(y <= x for x, y in zip(acc, acc[1:])) or \
                    any(x != i and ref[place(ctx + i)[0]] != 1 for i, x in enumerate(acc)):
                status[b] = -1
                continue
            for i, x in enumerate(acc):
                (sp, ss), (dp, ds) = place(ctx + x), place(ctx + i)
                self.k[dp, :, ds], self.v[dp, :, ds] = self.k[sp, :, ss], self.v[sp, :, ss]
            self.drop(b, ctx + len(acc))
        return status

    def free(self, rows):
        for b in rows:
            if 0 <= b < len(self.lens):
                self.drop(b, 0)


def i32(x, device="cuda"):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=device)


def pool(n_pages, Hkv, P, D, layout="heads", seed=0, device="cuda"):
    """K and V pages of random values in one of the layouts a user may have: page-head-slot, page-slot-head, or K and
    V side by side in each page."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(device)  # noqa: E731
    if layout == "heads":
        return draw(n_pages, Hkv, P, D), draw(n_pages, Hkv, P, D)
    if layout == "slots":
        return tuple(draw(n_pages, P, Hkv, D).transpose(1, 2) for _ in "kv")
    both = draw(n_pages, 2, Hkv, P, D)
    return both[:, 0], both[:, 1]


def empty_cache(n_pages, Hkv, P, D, rows, max_pages, layout="heads", seed=0, device="cuda"):
    k, v = pool(n_pages, Hkv, P, D, layout, seed, device)
    return (k, v, torch.full((rows, max_pages), -1, dtype=torch.int32, device=device),
            torch.zeros(rows, dtype=torch.int32, device=device),
            torch.zeros(n_pages, dtype=torch.int32, device=device))


def same(model, cache):
    k, v, table, lens, ref = cache
    now = Model(k, v, table, lens, ref)
    for name in ("lens", "ref", "table", "k", "v"):
        assert np.array_equal(getattr(model, name), getattr(now, name)), name
