"""GPU parity: how prompt attention hands out its work."""

import pytest
import torch

from stream_helpers import Prompt

pytestmark = pytest.mark.gpu


def was_split(ws):
    """The plan's third word: whether units were cut into parts."""
    return int(ws[8:12].view(torch.int32).item())


def ends_late(units, rows, ctas):
    """Whether the CTA with the most work of units of two tokens, dealt out there and back by size, has more than ten
    tiles of 128 rows above the mean."""
    costs = sorted(((rows - 2 * u - 1) // 128 + 1 for u in range(units)), reverse=True)
    load = [0] * ctas
    for j, cost in enumerate(costs):
        r, c = divmod(j, ctas)
        load[ctas - 1 - c if r % 2 else c] += cost
    return max(load) - sum(costs) // ctas > 10


# units of 2 tokens per SM (and as many more), rows; for 152 SMs the longest CTA and the mean are
@pytest.mark.parametrize("per_sm,more,rows", [
    (0, 50, 2500),  # 20 tiles and 6
    (1, 0, 2500),   # 20 and 18
    (1, 8, 2500),   # 36 and 19
    (2, 0, 2500),   # 36 and 35
    (2, 40, 2500),  # 51 and 39
    (1, 8, 1250),   # 16 and 9
    (3, 20, 1700),  # 37 and 31
    (3, 8, 3500),   # 92 and 71
])
def test_units_are_split_where_a_cta_would_end_late(kvc, per_sm, more, rows):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    units = per_sm * sms + more
    p = Prompt([2 * units], [rows], 128, 1, 64, 16, "bf16", None, 0, seed=units, pad=0)
    ws = p.workspace(kvc)
    p.run(kvc, ws)
    p.check()
    assert was_split(ws) == ends_late(units, rows, sms) and kvc.get_error_flags() == 0


def test_a_workspace_for_the_largest_call_serves_all(kvc):
    """A serving loop makes its workspace once. Sizes never fall with the batch, the tokens or the table, and a call finds
    what it needs in a workspace made for more."""
    def size(batch, tokens, blocks):
        return kvc.prompt_workspace_size(batch, tokens, 8, 2, 128, 16, blocks)

    tokens = (0, 1, 40, 500, 2000, 9000, 16384, 70000, 300000)
    batches, tables = (1, 3, 64, 300, 4096), (1, 70, 72, 73, 500, 9000)
    for t in tables:
        for b in batches:
            assert [size(b, n, t) for n in tokens] == sorted(size(b, n, t) for n in tokens)
        for n in tokens:
            assert [size(b, n, t) for b in batches] == sorted(size(b, n, t) for b in batches)
    for b in batches:
        for n in tokens:
            assert [size(b, n, t) for t in tables] == sorted(size(b, n, t) for t in tables)

    p = Prompt([70, 3], [5000, 40], 8, 2, 128, 16, "bf16", None, 0, seed=33)
    ws = torch.full((size(64, 300000, 500),), 255, dtype=torch.uint8, device="cuda")
    p.run(kvc, ws)
    p.check()
    assert kvc.get_error_flags() == 0
