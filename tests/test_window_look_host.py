"""Windowed prompts: the look at V and the products that do not wait for it, on the CPU.

In a window of 128 keys that hides some of them, one warp takes out of shared memory what is not
finite, while the products of the 16-key steps that every row of the pair sees run already (the others
wait).  So no key of such a step may be among those that are looked over.  This is the arithmetic of
tv_prompt_attn.cu (read_work, below, steps and the two roles), in Python."""
import pytest


class Pair:
    """Two tiles of `tile` tokens from t0 on, of a sequence of `length`, window W, K sinks."""

    def __init__(self, t0, length, tile, W, K):
        self.t0, self.length, self.tile, self.W, self.K = t0, length, tile, W, K
        self.hi, self.tiles = min(length, t0 + 2 * tile), 2 if t0 + tile < length else 1
        self.lo = t0 - W + 1 if t0 - W + 1 > K else 0
        self.low = self.windows = -(-(self.hi - self.lo) // 128)
        self.sink_steps = 0
        if self.lo > 0 and K > 0 and -(-K // 16) * 16 <= 128 * self.low - (self.hi - self.lo):
            self.sink_steps = -(-K // 16)
            self.lo = self.hi - 128 * self.low
        apart, hidden = self.lo > 0 and self.sink_steps == 0, self.hi - W - self.lo
        self.up = max(1, self.low - ((t0 + 1 - self.lo) >> 7))
        self.down = self.low - -(-hidden // 128) if hidden > 0 else self.low
        if apart:
            self.windows += -(-K // 128)
        if hidden <= 0 and (not apart or K % 16 == 0):
            self.down = self.windows
        self.skip0 = self.low - -(-(t0 + tile - self.lo) // 128) if self.tiles == 2 else 0

    def start(self, w):
        return self.lo + 128 * (self.low - 1 - w) if w < self.low else 128 * (self.windows - 1 - w)

    def steps(self, s, w):
        end = self.K if w >= self.low else min(self.length, self.t0 + (s + 1) * self.tile)
        return min(8, (end - self.start(w) + 15) >> 4)

    def below(self, w):
        at = self.start(w)
        if w >= self.low:
            return min(128, self.K - at), 16 * self.steps(0, w)
        first = (self.K if w == self.low - 1 else 0) if self.sink_steps else max(0, self.K - at)
        return first, min(128, self.hi - self.W - at)

    def looked_over(self, w, one_range=False):
        """Ranges of rows of window w; one_range: what lies between two of them, too."""
        at = self.start(w)
        first, last = max(0, self.t0 + 1 - at), min(128, self.hi - at)
        ranges, empty, end = [(first, last)], last, (last + 15) & ~15
        if w >= self.down:
            a, b = self.below(w)
            if w >= self.low:
                ranges, empty, end = [], a, b
            elif a < b:
                if first >= last:
                    ranges = [(a, b)]
                elif one_range or first <= b:
                    ranges = [(min(first, a), last)]
                else:
                    ranges.append((a, b))
        return [r for r in ranges + [(empty, end)] if r[0] < r[1]]

    def early(self, w):
        """Ranges of rows whose products do not wait for the look."""
        seen, low = min(8, max(0, self.t0 + 1 - self.start(w)) >> 4), 0
        if w >= self.down:
            low = (self.below(w)[1] + 15) >> 4
            if w >= self.low:
                seen = 8
        for s in range(self.tiles):
            f = self.skip0 if s == 0 else 0
            if w >= f:   # the first tile that has the window waits, the other comes behind it
                m = min(self.steps(s, w), seen)
                l = m if w == f and low > 0 else min(m, low)
                return [(16 * l, 16 * m)] if l < m else []
        return []

    def clashes(self, **kw):
        return [w for w in range(self.windows) if w < self.up or w >= self.down
                for a, b in self.early(w) for c, d in self.looked_over(w, **kw) if a < d and c < b]

    def hidden_rows(self, w):
        """Rows of window w that some row of the pair must not see and that its products have."""
        at, got = self.start(w), []
        for row in range(16 * max(self.steps(s, w) for s in range(self.tiles))):
            if self.sink_steps and w == self.low - 1 and row < 16 * self.sink_steps:
                j, seen = row, row < self.K
            elif w >= self.low:
                j, seen = at + row, at + row < self.K
            else:
                j = at + row
                # (sinks that the last window holds in its lowest steps are not counted here)
                seen = j <= self.t0 and (j > self.hi - 1 - self.W or (j < self.K and not self.sink_steps))
            if not seen:
                got.append(row)
        return got


def pairs(group):
    tile = 128 // group
    for K in (0, 1, 4, 16, 20, 33, 130):
        for W in [1, 16, 17, 64, 77, *range(90, 131, 3), 126, 127, 160, 161, 200, 205, 254, 255, 256, 300, 513]:
            for length in (400, 701, 1100):
                for t0 in {0, 2 * tile, *range(128 // (2 * tile) * 2 * tile, length, 6 * tile), (length - 1) // (2 * tile) * 2 * tile}:
                    yield Pair(t0, length, tile, W, K)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 8, 16, 24, 32, 128])
def test_products_that_do_not_wait_are_left_alone(group):
    for p in pairs(group):
        assert not p.clashes(), vars(p)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 8, 16, 24, 32, 128])
def test_what_a_row_must_not_see_is_looked_over(group):
    for p in pairs(group):
        for w in range(p.windows):
            looked = set(r for a, b in p.looked_over(w) for r in range(a, b)) if w < p.up or w >= p.down else set()
            early = set(r for a, b in p.early(w) for r in range(a, b)) if looked else set()
            hidden = set(p.hidden_rows(w))
            assert hidden <= looked and not hidden & early, (w, sorted(hidden - looked)[:5], vars(p))


def test_one_range_would_not_do():
    """What the two ranges are for: keys that every row sees lie between those that the window's ends hide."""
    assert any(p.clashes(one_range=True) for p in pairs(4))
