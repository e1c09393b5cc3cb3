"""That the shapes of the GPU tests reach every kernel of the serving operators."""
import serving_rules as rules

CUS = 256


def test_every_tiling_of_the_product_is_reached():
    every = rules.tilings()
    for kind, shapes in (("stream", rules.STREAMED), ("any", rules.LOOSE)):
        reached = set()
        for T, M, N in shapes:
            got, t = rules.product_kernel(T, M, N, CUS)
            assert got == kind
            if N > 2 * t.stages * t.columns and N % t.columns and T % t.tokens and M % t.outputs:
                reached.add(t)
        assert reached == set(every[kind]), set(every[kind]) - reached


def test_large_tiles_are_reached_whole_and_halved():
    forms = set()
    for T, M, N in rules.LARGE:
        assert rules.product_kernel(T, M, N, CUS) == ("tiles", None)
        tiles = -(-T // 256) * -(-M // 256)
        left = tiles % CUS
        forms.add((tiles < CUS, tiles > CUS and 0 < left <= CUS // 2))
        assert N > 512      # more than two rounds of the buffers
    assert forms == {(True, False), (False, True), (False, False)}
    # of the halved ones, one ends in the first half of its last tile
    assert any(0 < M % 256 <= 128 and -(-T // 256) * -(-M // 256) > CUS for T, M, _ in rules.LARGE)
