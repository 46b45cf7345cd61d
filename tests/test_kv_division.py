"""The attention's division of work where it keeps to units, and the kernels'
divisions by multiplication, over every value they meet.  The integer
expressions are the kernels'."""
import numpy as np
import pytest

ROWS, BLOCK, LEAST, UNEVEN = 16, 64, 4, 8


def tile_blocks(T, G, length, n, tree):
    """Blocks of a request's row tiles."""
    out = []
    for tile in range(-(-n * G // ROWS)):
        last = n - 1 if tree else (min((tile + 1) * ROWS, n * G) - 1) // G
        out.append(-(-(length + last + 1) // BLOCK))
    return out


def padding(units, B, H, T, G, grid):
    """The kernel's choice: blocks a unit is padded to a multiple of (1: none)."""
    most = B * H * -(-T * G // ROWS)
    total = sum(units)
    if 2 * most > grid or total >= 1 << 30:
        return 1
    room = grid - most
    q = max(LEAST, (total + room - 1) // room)
    return 1 if q > total // grid + UNEVEN else q


@pytest.mark.parametrize("seed", range(300))
def test_padded_division(seed):
    """Few units: every unit starts a part, no part holds two units, the parts
    fit the grid, and each block is some CTA's once."""
    rng = np.random.default_rng(seed)
    grid = int(rng.integers(1, 321))
    B, H = int(rng.integers(1, 9)), int(rng.integers(1, 9))
    T, G = int(rng.integers(1, 17)), int(rng.choice([1, 2, 3, 4, 8]))
    if T * G > 48:
        T = 48 // G
    tree = bool(rng.integers(0, 2))
    units = []
    for _ in range(B):
        length = int(np.exp(rng.uniform(0, np.log(rng.choice([64, 4000, 131072])))))
        n = int(rng.integers(0, T + 1))
        units += tile_blocks(T, G, length, n, tree) * H
    pad = padding(units, B, H, T, G, grid)
    if pad == 1 or not units:
        return
    padded = [-(-n // pad) * pad for n in units]
    total = sum(padded)
    count = total // pad
    assert count * pad == total and count <= grid
    starts = np.concatenate([[0], np.cumsum(padded)])
    held = [np.zeros(n, int) for n in units]
    firsts = set()
    for c in range(count):
        w0, n = c * pad, pad
        u = int(np.searchsorted(starts, w0, side="right")) - 1
        blk = w0 - starts[u]
        n = min(n, units[u] - blk)   # the part ends with its unit
        assert n > 0 and w0 + n <= starts[u + 1]
        held[u][blk:blk + n] += 1
        first, last = starts[u] // pad, (starts[u] + units[u] - 1) // pad
        assert first <= c <= last
        if blk == 0:
            assert c == first and c not in firsts
            firsts.add(c)
    assert all((h == 1).all() for h in held)
    assert len(firsts) == len(units)


def test_padded_parts_fit_the_grid_always():
    """sum ceil(n_u / q) <= total / q + units <= room + units = grid."""
    rng = np.random.default_rng(0)
    for _ in range(20000):
        grid = int(rng.integers(2, 321))
        most = int(rng.integers(1, grid // 2 + 1))
        units = rng.integers(1, rng.choice([2, 50, 5000]), rng.integers(1, most + 1))
        room = grid - most
        q = max(LEAST, (int(units.sum()) + room - 1) // room)
        assert (-(-units // q)).sum() <= grid


def test_read_divides_every_index():
    """A block's chunk index, idle threads' included, by the chunks of a token,
    for one and for eight chunks a thread."""
    threads = 256
    for heads in range(1, 257):
        for d in (4, 8):
            per = heads * d
            magic = np.uint64(2 ** 32 // per + 1)
            for chunks in (1, 8):
                tokens = max(1, threads * chunks // per)
                # turns of the loop: at0 below the block's chunks, in whole warps
                turns = -(-(tokens * per) // (threads * chunks))
                at = np.arange(0, turns * threads * chunks + threads, dtype=np.uint64)
                assert ((at * magic) >> np.uint64(32) == at // np.uint64(per)).all(), (per, chunks)
