"""Host models of what the cache kernels' warps wait for (CPU): every order in
which they can run, explored, for memory that one may still read while another
writes it."""
from __future__ import annotations

import pytest


def weights_orders(chunks, tiles, buffers):
    """Every order of the weights kernel's two sub-tiles and its product queue
    over ``chunks`` of rows by ``tiles`` key tiles.  A sub-tile, for each chunk:
    writes its half of the rows' constants, arrives on QF and waits for it (both
    arrive), reads the constants during each tile it owns (alternate ones, counted
    through the chunks) once the tile's products are done, waits for QD (all of
    the chunk's products).  Returns the first hazard found: a sub-tile writes a
    buffer that the other one reads, or None."""
    steps = []
    for t in range(2):
        own = []
        for c in range(chunks):
            own += [("write", c), ("written", c), ("qf", c)]
            for j in range(tiles):
                if (c * tiles + j) & 1 == t:
                    own += [("read", c, j), ("have read", c, j)]
            own += [("qd", c)]
        steps.append(own)

    def ready(step, pos, done):
        """Whether an agent at pos may begin this step: done products, sub-tiles' places."""
        if step[0] == "qf":  # both have written
            return all(("written", step[1]) in steps[t][: pos[t]] for t in range(2))
        if step[0] == "read":
            return done > step[1] * tiles + step[2]
        if step[0] == "qd":
            return done >= (step[1] + 1) * tiles
        return True

    seen, todo = set(), [(0, 0, 0)]
    while todo:
        a, b, done = state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        pos = (a, b)
        during = [steps[t][pos[t] - 1] if pos[t] else None for t in range(2)]
        for t in range(2):
            w, r = during[t], during[1 - t]
            if w and r and w[0] == "write" and r[0] == "read" and w[1] % buffers == r[1] % buffers:
                return w, r
        for t in range(2):
            if pos[t] < len(steps[t]) and ready(steps[t][pos[t]], pos, done):
                todo.append((a + (t == 0), b + (t == 1), done))
        # the next product: its chunk's queries are there, and its score buffer (of two) is read
        if done < chunks * tiles and all(("written", done // tiles) in steps[t][: pos[t]] for t in range(2)):
            before = done - 2
            if before < 0 or ("have read", before // tiles, before % tiles) in steps[before & 1][: pos[before & 1]]:
                todo.append((a, b, done + 1))
    assert any(s[0] == len(steps[0]) and s[1] == len(steps[1]) for s in seen), "the model comes to a stop"
    return None


@pytest.mark.parametrize("tiles", [1, 2, 3, 4])
def test_weights_row_constants_are_read_before_they_are_written_again(tiles):
    assert weights_orders(4, tiles, buffers=2) is None


@pytest.mark.parametrize("tiles", [1, 2, 3])
def test_one_buffer_of_row_constants_would_not_do(tiles):
    w, r = weights_orders(2, tiles, buffers=1)
    assert w == ("write", 1) and r[:2] == ("read", 0)
