"""A beam request whose rows are sequences of the host block manager: blocks are
allotted ahead, the device's tables go their own way from the first reordering on,
and all rows are freed together.  `copy(src, dst)`, `write(blocks, slot, tokens)`
and `reorder(tables, n, parents)` act on the caller's pool."""
import numpy as np

from paged_kv_attention_decode_gb300.block_manager import BlockManager

BS, AHEAD = 16, 5
NO_TOKEN = -1            # stands for decoded tokens, which the manager never learns


def search(n0, W, steps, seed, prefix_caching, copy, write, reorder, max_blocks):
    """Runs the request; returns (tables [W, max_blocks], tokens cached, every row's
    tokens), with the manager's checks made on the way."""
    rng = np.random.default_rng(seed)
    prompt = rng.integers(0, 1000, n0)
    bm = BlockManager(1 + W * max_blocks, BS, prefix_caching)
    free = bm.num_free_blocks
    assert bm.add_sequence(0, prompt) == 0 and bm.allocate_slots(0, n0) is None
    t0 = bm.block_table(0)
    for j in range(n0):
        write(t0[j // BS:j // BS + 1], j % BS, prompt[j:j + 1])
    for w in range(1, W):
        bm.fork(0, w)
    tables, have, room = np.zeros((W, max_blocks), np.int32), 0, n0
    hist, n = [list(prompt) for _ in range(W)], n0
    for step in range(steps):
        if n == room:                                    # the next AHEAD tokens' blocks
            for w in range(W):
                bm.append_tokens(w, [NO_TOKEN] * AHEAD)
                moved = bm.allocate_slots(w, AHEAD)
                if moved:                                # (the prompt's last block, before any reordering)
                    assert have == 0 and n % BS
                    copy(*moved)
            room += AHEAD
            mine = [bm.block_table(w) for w in range(W)]
            end = len(mine[0])
            for w in range(W):                           # new columns only: the device's tables are its own
                tables[w, have:end] = mine[w][have:end]
            have = end
        tokens = rng.integers(0, 1000, W)
        write(tables[:, n // BS], n % BS, tokens)
        for w in range(W):
            hist[w].append(tokens[w])
        n += 1
        parents = rng.integers(0, W, W) if step % 4 else np.full(W, rng.integers(0, W))
        tables = reorder(tables, n, parents)
        hist = [list(hist[p]) for p in parents]
    # the prompt's whole blocks are still a later request's; the others are no one's
    if prefix_caching and n0 >= BS:
        assert bm.add_sequence(99, np.concatenate([prompt, [5]])) == n0 // BS * BS
        bm.free_sequence(99)
    for w in range(W):
        bm.free_sequence(w)
    assert bm.num_free_blocks == free
    return tables, n, hist
