"""Batches that take each cut of an attention's work past what a wave holds of
its pages at a time, or past what the cut's rule asks for.  What each is for
(mode, heads to a workgroup, tiles that a wave goes through) is checked on the
CPU against the plan, the results on the GPU against the definition."""
FAR = 1 << 22  # a bound on the contexts that always asks for runs


def case(name, mode, hw, tiles, lens, ctx, G, heads, dim, bs, st, max_ctx, order="tokens", window=0, holes=True):
    """mode "runs" (equal runs of tiles) or "units" (a workgroup each); hw
    heads of a workgroup; tiles: at least so many to some wave."""
    return dict(locals())


def _spread(lo, hi, n, step):
    return [lo + (i * step) % (hi - lo + 1) for i in range(n)]


CASES = [
    # single tokens, in runs: a wave's pages are looked up anew more than once
    case("runs_1_head", "runs", 1, 65, [1, 1, 1], [40000, 100, 31000], 1, 64, 16, 16, 16, FAR, "heads"),
    case("runs_2_heads", "runs", 2, 33, [1, 2, 1], [30000, 77, 21000], 1, 62, 16, 32, 8, FAR),
    case("runs_4_heads", "runs", 4, 65, [1, 1, 1], [70000, 50, 34000], 1, 64, 16, 16, 16, FAR),
    case("runs_4_heads_fine", "runs", 4, 65, [1, 1, 1], [36001, 50, 68000], 2, 64, 16, 16, 1, FAR),
    case("runs_4_heads_window", "runs", 4, 65, [1, 2], [120001, 110000], 1, 64, 16, 64, 64, FAR, window=100000),
    case("runs_4_heads_192", "runs", 4, 65, [1, 1], [60000, 9000], 1, 64, 192, 16, 16, FAR),
    # a verification's tokens: blocks of several row tiles, in runs
    case("runs_5_tiles", "runs", 1, 65, [9, 8], [200000, 80001], 8, 16, 32, 16, 16, FAR),
    case("runs_3_tiles_fine", "runs", 1, 65, [6, 5], [90000, 50000], 8, 32, 80, 32, 2, FAR),
    # a full card of contexts of a few thousand tokens: a unit each, a wave to a head
    case("full_card", "units", 4, 100, [1] * 400, _spread(1025, 4096, 400, 977), 1, 16, 32, 16, 16, 4096),
    case("full_card_fine", "units", 4, 100, [i % 2 for i in range(800)], _spread(1000, 4000, 800, 131), 2, 8, 32, 16,
         4, 4096),
    case("full_card_2_heads", "units", 2, 60, [1] * 800, _spread(1, 4096, 800, 577), 1, 6, 16, 16, 16, 4096),
    # prompts: many blocks of rows, a unit each
    case("prompt_3_tiles", "units", 1, 65, [800, 600], [9001, 8500], 4, 8, 128, 64, 64, 16384),
    case("prompt_5_tiles", "units", 1, 65, [700, 650], [8400, 9011], 8, 8, 64, 16, 16, FAR),
    case("prompt_fine_window", "units", 1, 65, [500, 450], [20000, 15001], 8, 8, 96, 16, 1, FAR, window=8500),
    # more units than the runs' beginnings are searched for in
    case("many_units", "units", 1, 1, [i % 3 for i in range(66000)], _spread(0, 70, 66000, 37), 1, 1, 32, 16, 16, FAR,
         holes=False),
    case("many_units_2_heads", "units", 2, 1, [1] * 65537, _spread(0, 70, 65537, 41), 2, 2, 16, 16, 4, FAR,
         holes=False),
]
