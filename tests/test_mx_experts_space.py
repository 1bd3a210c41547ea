"""Rows that the experts' layer lays its (token, choice) pairs out in, against
the space of lutq_mx_experts_workspace_bytes, without a GPU."""
import random

import pytest

D, F = 32, 32


def _rows(space, e, pairs):
    """The rows in a workspace, from its size: per row, codes and scales of x and of the hidden
    values, the hidden values in bf16 and the output in fp32."""
    up = lambda v, m=256: -(-v // m) * m  # noqa: E731
    per_128 = 2 * (128 * D // 2 + 1024) + 2 * 128 * F + 4 * 128 * D  # (D = F, one chunk each)
    fixed = 2 * up(4 * e) + up(4 * pairs)
    return (space - fixed) // per_128 * 128


def _needed(ids, t, e, nt):
    """Tiles of nt pairs begin at multiples of 128 rows."""
    count = [0] * e
    for i in ids:
        if 0 <= i < e:
            count[i] += 1
    return sum(-(-c // nt) * 128 for c in count)


@pytest.mark.parametrize("k", [1, 2, 5, 8, 64])
def test_every_layout_fits(k):
    import dequant_gemv_group_b200 as lq
    rng = random.Random(k)
    for t in [1, 2, 3, 15, 16, 17, 31, 32, 33, 50, 63, 64, 65, 128, 129, 300]:
        nt = 16 if t <= 16 else 32 if t <= 32 else 64 if t <= 64 else 128
        for e in (1, 2, 3, 8, 40, 1024):
            rows = _rows(lq.lutq_mx_experts_workspace_bytes(t, k, e, D, F, "mxfp4"), e, t * k)
            assert rows % 128 == 0
            layouts = [[0] * (t * k), [i % e for i in range(t * k)],
                       [rng.randrange(e) for _ in range(t * k)]]
            # one pair over a full tile in as many experts as there are pairs for
            layouts.append([min(i // (nt + 1), e - 1) for i in range(t * k)])
            # a pair to every expert, the others to the first
            layouts.append([i if i < e else 0 for i in range(t * k)])
            for ids in layouts:
                for tile in {nt, 128}:
                    assert _needed(ids, t, e, tile) <= rows, (t, e, tile)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_space_for_a_batch_holds_a_smaller_one(fmt):
    import dequant_gemv_group_b200 as lq
    for k in (1, 3, 8):
        for e in (1, 7, 64, 1024):
            need = [lq.lutq_mx_experts_workspace_bytes(t, k, e, 256, 96, fmt) for t in range(400)]
            assert need == sorted(need)
