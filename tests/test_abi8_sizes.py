"""The attention's workspace size, on the host: enough for every smaller call too."""
import ctypes
import random

import pytest


@pytest.fixture(scope="module")
def sb():
    from video_diffusion_mixed_b200 import build
    build.build()
    from video_diffusion_mixed_b200 import sixbit
    sixbit.lib()
    return sixbit


def size(sb, batch, heads_q, n_q, dim):
    n = ctypes.c_size_t(0)
    assert sb.lib().sb_kv8_workspace_size(batch, heads_q, n_q, dim, ctypes.byref(n)) == sb.SB_OK
    return n.value


@pytest.mark.parametrize("dim", [64, 128])
def test_size_never_falls_as_a_call_grows(sb, dim):
    rng = random.Random(dim)
    some = [(1, 30, 17776), (1, 30, 1350), (1, 30, 1), (4, 32, 8192), (1200, 1, 1), (100, 1, 1), (3, 16, 2047), (1, 1, 1),
            (16384, 16384, 4096)]
    for _ in range(300):
        some.append(tuple(int(2 ** rng.uniform(0, t)) for t in (14, 9, 16)))
    sizes = [size(sb, *s, dim) for s in some]
    for a, na in zip(some, sizes):
        for b, nb in zip(some, sizes):
            if all(x <= y for x, y in zip(a, b)):
                assert na <= nb, (a, na, b, nb)
