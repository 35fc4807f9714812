"""Who writes which rows in the attention kernel for many rows, restated on the CPU: what the host launches from the
sizes of a call, and what its CTAs and the join's make of the offsets that only they see."""
import random

import pytest

SMS, KEYS = 152, 128


def ceil(a, b):
    return -(-a // b)


class Call:
    def __init__(self, dim, heads, group, tokens, counts, lens, width, page, offsets, causal=True, window=0):
        self.rows, self.least = (128, 17) if dim == 256 else (256, 33)
        self.heads, self.group, self.tokens, self.width, self.page, self.offsets = heads, group, tokens, width, page, offsets
        self.counts, self.lens, self.causal, self.window = counts, lens, causal, window
        few = min(len(counts), tokens)
        self.most = heads * (tokens * group // self.rows + few if offsets else len(counts) * ceil(tokens // len(counts) * group, self.rows))

    def joined(self):
        """The host's decision: the keys may be cut, and the join follows."""
        return self.width * self.page > 2 * KEYS and 2 * self.all() <= SMS

    def all(self):
        """Row tiles at least if every token of the buffer belongs to a sequence."""
        mine = self.tokens * self.group - (self.least - 1) * len(self.counts)
        return self.heads * max(0, ceil(mine, self.rows)) if self.offsets else self.most

    def key_tiles(self, b, row0, rows):
        L, start = self.lens[b], self.lens[b] - self.counts[b]
        lo = max(0, start + row0 // self.group - self.window + 1) if self.window else 0
        hi = min(L, start + (row0 + rows - 1) // self.group + 1) if self.causal else L
        return max(1, ceil(max(hi, 0) - min(lo, L) // 16 * 16, KEYS))

    def plans(self):
        for b, n in enumerate(self.counts):
            rows = n * self.group
            if n and rows >= self.least:
                tiles = ceil(rows, self.rows)
                last = (tiles - 1) * self.rows
                yield b, tiles * self.heads, self.key_tiles(b, last, rows - last)

    def work(self, cut):
        """CTA -> (tile, part, parts, slot, key tiles), the join's CTA -> tile; most key tiles of a part, 0: not cut."""
        plans = list(self.plans())
        tiles, keys = sum(t for _, t, _ in plans), sum(t * k for _, t, k in plans)
        most = max(2, ceil(keys, SMS - tiles)) if cut and 2 * tiles <= SMS and tiles else 0
        ctas, joins, slot = [], [], 0
        for b, n, k in plans:
            parts = ceil(k, most) if most else 1
            for i in range(n):
                row0 = i // self.heads * self.rows
                rows = min(self.rows, self.counts[b] * self.group - row0)
                mine = self.key_tiles(b, row0, rows)
                own = min(parts, (mine + 1) // 2) if most else 1
                tile = (b, i % self.heads, row0, rows, own)
                joins.append(tile)
                for part in range(parts):
                    ctas.append((tile, part, slot + part, mine * part // own, mine * (part + 1) // own) if part < own else None)
                slot += parts
        return ctas, joins, most


def unwritten(call, cut, join):
    """Row tiles that no launched CTA writes."""
    ctas, joins, most = call.work(cut)
    grid = max(call.most, SMS) if cut else call.most
    assert len(ctas) <= grid
    written = set()
    parts = {}
    for w in ctas:
        if w is None:
            continue
        tile, part, slot, t0, t1 = w
        assert t0 < t1
        if tile[4] == 1:
            written.add(tile)
        else:
            assert cut and slot < SMS  # the workspace's parts
            parts.setdefault(tile, []).append((t0, t1))
    for tile, p in parts.items():
        assert len(p) == tile[4] and all(a[1] == b[0] for a, b in zip(p, p[1:])) and p[0][0] == 0
        assert p[-1][1] == call.key_tiles(tile[0], tile[2], tile[3])
        lines = min((call.tokens if call.offsets else max(call.counts)) * call.group, call.rows)  # that the join has CTAs for
        if join and most and joins.index(tile) < min(call.most, SMS // 2) and tile[3] <= ceil(lines, 32) * 32:
            written.add(tile)
    return [t for t in joins if t not in written]


def draw(rng):
    dim, heads, group = rng.choice((64, 128, 256)), rng.choice((1, 2, 4, 8)), rng.choice((1, 3, 5, 8, 40))
    tokens = rng.choice((17, 40, 512, 700, 4096))
    batch, page = rng.choice((1, 1, 2, 7, 40)), rng.choice((16, 64, 128))
    offsets = rng.random() < 0.8
    if offsets:
        named = rng.choice((0, 1, rng.randint(0, tokens), rng.randint(0, min(tokens, 100)), tokens))
        at = sorted(rng.randint(0, named) for _ in range(batch - 1))
        counts = [b - a for a, b in zip([0] + at, at + [named])]
    else:
        tokens = tokens // batch * batch or batch
        counts = [tokens // batch] * batch
    lens = [max(0, rng.choice((0, n - 3, n, n + rng.randint(0, 20000)))) for n in counts]
    width = ceil(max(lens) + rng.choice((0, 1, 5000)), page)
    causal = rng.random() < 0.8
    return Call(dim, heads, group, tokens, counts, lens, width, page, offsets, causal, rng.randint(1, 3000) if causal and rng.random() < 0.3 else 0)


def test_every_row_tile_is_written():
    rng = random.Random(1)
    cut = 0
    for _ in range(3000):
        call = draw(rng)
        join = call.joined()
        assert not unwritten(call, join, join)
        cut += any(w and w[0][4] > 1 for w in call.work(join)[0])
    assert cut > 300


@pytest.mark.parametrize("tokens,counts,lens", [(512, [100], [16000]), (4096, [64], [5000])])
def test_the_model_sees_a_join_left_out_for_the_buffers_size(tokens, counts, lens):
    """A kernel that may cut behind a host that takes all of the buffer's tokens for named: keys cut and never joined."""
    call = Call(128, 8, 5, tokens, counts, lens, ceil(lens[0], 64), 64, True)
    assert not call.joined() and len(unwritten(call, True, False)) == 8 * ceil(counts[0] * 5, 256)
    assert not unwritten(call, call.joined(), call.joined())
