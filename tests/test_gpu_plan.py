"""Page plans (tq_plan_step, tq_release_pages) against lists on the host:
whole numbers, so equal."""
import random

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


def tq():
    import block_quantized_matmul_repack_amd as m
    return m


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def state(rng, B, page, width, most_len, most_new, spare):
    lens, new, owned = [], [], []
    for _ in range(B):
        c = rng.choice([0, 0, rng.randint(0, most_len), page, 2 * page - 1])
        n = rng.choice([0, 1, 1, rng.randint(0, most_new), page])
        lens.append(min(c, width * page))
        new.append(n)
        owned.append(min(-(-lens[-1] // page) + rng.choice([0, 0, 1]), width))
    want = sum(max(0, min(-(-(c + n) // page), width) - o) for c, n, o in zip(lens, new, owned))
    ids = list(range(sum(owned) + max(want + spare, 0)))
    rng.shuffle(ids)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, o in enumerate(owned):
        table[b, :o] = torch.tensor(ids[at:at + o], dtype=torch.int32)
        at += o
    free = ids[at:]
    return lens, new, owned, table, free


def check(lens, new, owned, table, free, page, tokens, count=None, pad=3):
    count = len(free) if count is None else count
    B, width = table.shape
    want_table = table.numpy().copy()
    want = ref.plan(lens, new, owned, want_table, free, count, page, tokens)
    wide = torch.full((max(B, 1), width + pad), 77, dtype=torch.int32, device="cuda")  # a row stride
    t = wide[:B, :width]
    t.copy_(table)
    got = tq().plan_step(dev(lens), dev(new), dev(owned), t, dev(free), dev([count]), page, tokens)
    for name, g, w in zip(("starts", "positions", "slots", "lens", "owned", "free"), got, want):
        assert g.tolist() == w, name
    assert (t.cpu().numpy() == want_table).all()
    assert (wide[:, width:] == 77).all()
    return got, t


@pytest.mark.parametrize("B", [0, 1, 2, 63, 64, 65, 500, 1023, 1024, 1025, 3000])
def test_batches(B):
    rng = random.Random(B)
    page = rng.choice([16, 64])
    lens, new, owned, table, free = state(rng, B, page, 9, 8 * page, 3 * page, 5)
    check(lens, new, owned, table, free, page, sum(new) + rng.choice([0, 1, 70]))


@pytest.mark.parametrize("page", [16, 128, 1024])
@pytest.mark.parametrize("tokens", [0, 1, 1024, 1025, 5000])
def test_rows_short_of_the_tokens(page, tokens):
    """Tokens that there are no rows for are left out, and take no pages."""
    rng = random.Random(page + tokens)
    lens, new, owned, table, free = state(rng, 40, page, 12, 10 * page, 400, 5)
    check(lens, new, owned, table, free, page, tokens)


@pytest.mark.parametrize("spare", [-1, -7, -1000])
def test_pages_run_out(spare):
    rng = random.Random(3)
    lens, new, owned, table, free = state(rng, 200, 16, 20, 100, 150, spare)
    got, _ = check(lens, new, owned, table, free, 16, sum(new) + 9)
    assert got[5].item() < 0 and (got[2] == -1).sum() > 9


def test_long_prompts_and_full_tables():
    """One prompt of many pages, one past its row of the table."""
    lens, new, owned = [0, 500, 130], [40000, 200, 1], [0, 32, 9]
    table = torch.full((3, 2504), -1, dtype=torch.int32)
    table[1, :32] = torch.arange(32)
    table[2, :9] = torch.arange(40, 49)
    check(lens, new, owned, table, list(range(100, 2700)), 16, 40201)
    short = table[:, :40].contiguous()
    got, _ = check(lens, new, owned, short, list(range(100, 2700)), 16, 40201)
    assert (got[2][640:40000] == -1).all()


def test_numbers_out_of_range():
    """Negative numbers count as 0, a count past the stack as its size, ids that
    give no slot of 31 bits as none; nothing is read or written outside."""
    table = torch.full((4, 6), -1, dtype=torch.int32)
    table[0, :2] = torch.tensor([-5, 2 ** 31 - 1])
    free = [2 ** 31 - 1, 7, 8, 9]
    lens, new, owned = [20, -3, 5, 90], [3, 17, -4, 40], [2, -1, 1, 99]
    table[2, 0] = 3
    table[3] = torch.tensor([10, 11, 12, 13, 14, 15])
    t = table.cuda()
    got = tq().plan_step(dev(lens), dev(new), dev(owned), t, dev(free), dev([1000]), 16, 64)
    starts, pos, slots, new_lens, new_owned, left = (g.tolist() for g in got)
    assert starts == [0, 3, 20, 20, 60]
    assert pos[:20] == [20, 21, 22] + list(range(17)) and pos[60:] == [0] * 4
    # 2^31 - 1 names no slot; request 1 takes pages 9 and 8
    assert slots[:20] == [-1] * 3 + [9 * 16 + i for i in range(16)] + [8 * 16]
    assert slots[20:60] == [15 * 16 + i for i in range(10, 16)] + [-1] * 34
    assert new_lens == [23, 17, 5, 130] and new_owned == [2, 2, 1, 6] and left == [2]
    got = tq().plan_step(dev(lens), dev(new), dev(owned), t, dev(free), dev([-4]), 16, 64)
    assert got[5].item() == -2 and t[1, :2].tolist() == [-1, -1]


@pytest.mark.parametrize("B", [1, 64, 1500])
def test_release(B):
    rng = random.Random(B + 1)
    lens, new, owned, table, free = state(rng, B, 16, 70, 1000, 50, 11)
    done = [rng.choice([0, 1, -1]) for _ in range(B)]
    for extra in (sum(owned), 3):                # room for all of them, or for three
        count = len(free)
        want_table, stack = table.numpy().copy(), free + [-9] * extra
        want_owned, want_count = ref.release(done, owned, want_table, stack, count)
        t, f = table.cuda(), dev(free + [-9] * extra)
        got_owned, got_count = tq().release_pages(dev(done), dev(owned), t, f, dev([count]))
        assert got_owned.tolist() == want_owned and got_count.tolist() == want_count
        assert (t.cpu().numpy() == want_table).all() and f.tolist() == stack


def test_requests_come_and_go():
    """Many steps: no page is ever owned twice, none is lost."""
    rng = random.Random(9)
    B, page, width, pages = 24, 16, 12, 150
    lens, owned = dev([0] * B), dev([0] * B)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = dev(rng.sample(range(pages), pages)), dev([pages])
    for step in range(30):
        host = lens.tolist()
        new = [rng.choice([0, 1, 1, 40]) if c < 140 else 0 for c in host]
        starts, pos, slots, lens, owned, count = tq().plan_step(
            lens, dev(new), owned, table, free, count, page, 1024)
        assert count.item() >= 0
        live = slots[:sum(new)]
        assert (live >= 0).all() and len(set(live.tolist())) == sum(new)
        # drafts refused, requests done
        lens = (lens - dev([rng.choice([0, 0, 1]) if n else 0 for n in new])).clamp(min=0)
        done = dev([int(c > 100 and rng.random() < 0.5) for c in lens.tolist()])
        owned, count = tq().release_pages(done, owned, table, free, count)
        lens = lens * (1 - done)
        held = [e for row, o in zip(table.tolist(), owned.tolist()) for e in row[:o]]
        assert sorted(held + free[:count.item()].tolist()) == list(range(pages))
