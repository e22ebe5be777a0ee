"""Page bookkeeping row by row in plain Python: what the update and the compaction of a cache have to give."""
import random

PAGE = 64


def pages(n):
    return (n + PAGE - 1) // PAGE


class State:
    """A table, lengths and counts; `pins` are holders outside the table."""

    def __init__(self, rows, width, num_pages, lengths, seed=0, share=1, pins=(), live_low=False):
        rng = random.Random(seed)
        self.width, self.num_pages, self.lengths = width, num_pages, list(lengths)
        ids = list(range(num_pages))
        if not live_low:
            rng.shuffle(ids)
        self.refs, self.table, at = [0] * num_pages, [], 0
        for r in range(rows):
            n = pages(self.lengths[r])
            # rows of one group of `share` hold the same full pages, as far as both have them
            common = min(n, self.lengths[r] // PAGE, self.lengths[r - 1] // PAGE) if r % share else 0
            mine = self.table[-1][:common] if common else []
            mine = mine + ids[at:at + n - common]
            at += n - common
            assert at <= num_pages
            for x in mine:
                self.refs[x] += 1
            # entries past the held ones may hold anything
            self.table.append(mine + [rng.choice([-1, 7, 1 << 30]) for _ in range(width - n)])
        self.free = ids[at:]
        for k in pins:
            self.refs[ids[k]] += 1

    def update(self, parents, new):
        """(table, refs, copies as (from, to, positions)), or the name of the error."""
        held = [0] * self.num_pages
        for row, n in zip(self.table, self.lengths):
            for x in row[:pages(n)]:
                held[x] += 1
        count = [a - b for a, b in zip(self.refs, held)]
        rows, writers = [], {}
        for r, (p, n) in enumerate(zip(parents, new)):
            keep = min(self.lengths[p], n) if p >= 0 else 0
            mine = self.table[p][:keep // PAGE] if p >= 0 else []
            mine = list(mine)
            if keep % PAGE:
                tail = self.table[p][keep // PAGE]
                if n > keep:
                    writers.setdefault(tail, []).append((r, keep % PAGE))
                else:
                    mine.append(tail)
            for x in mine:
                count[x] += 1
            rows.append(mine)
        copies = {}
        for x, who in writers.items():
            if count[x] == 0:
                rows[who[0][0]].append(x)
                count[x] = 1
                who = who[1:]
            for r, n in who:
                copies[r] = (x, n)
        free = [x for x in range(self.num_pages) if count[x] == 0]
        if sum(pages(n) - len(mine) for mine, n in zip(rows, new)) > len(free):
            return "no pages"
        made = []
        for r, (mine, n) in enumerate(zip(rows, new)):
            while len(mine) < pages(n):
                x = free.pop(0)
                count[x] = 1
                if r in copies:
                    src, k = copies.pop(r)
                    made.append((src, x, k))
                mine.append(x)
        return [m + [-1] * (self.width - len(m)) for m in rows], count, made

    def compact(self):
        """(table, refs, map)."""
        n = sum(c > 0 for c in self.refs)
        to = [x if c > 0 else -1 for x, c in enumerate(self.refs)]
        holes = [x for x in range(n) if self.refs[x] == 0]
        refs = list(self.refs)
        for x in range(n, self.num_pages):
            if refs[x] > 0:
                to[x] = holes.pop(0)
                refs[to[x]], refs[x] = refs[x], 0
        table = [[to[x] if i < pages(k) else x for i, x in enumerate(row)] for row, k in zip(self.table, self.lengths)]
        return table, refs, to
