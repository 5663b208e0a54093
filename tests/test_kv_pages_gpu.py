"""mx_kv_truncate where rows of the table have holes: pages in front of a
window that were given back early, which the attention accepts as -1."""
import numpy as np
import pytest
import torch

import block_scaled_quantized_mx_gb300 as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    mx.build()
    mx.lib()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _truncate(lens, keep, table, stack, count, page):
    """The definition: entries behind what is kept become -1; of the n pages
    among them, in request order, then table order, the i-th goes to
    stack[count + n - 1 - i]."""
    table, stack, out, freed = table.copy(), list(stack), [], []
    for b, n in enumerate(lens):
        k = min(max(keep[b], 0), n)
        out.append(k)
        cut = slice(-(-k // page), -(-n // page))
        freed += [int(p) for p in table[b, cut] if p >= 0]
        table[b, cut] = -1
    for i, p in enumerate(freed):
        if count + len(freed) - 1 - i < len(stack):
            stack[count + len(freed) - 1 - i] = p
    total = count + len(freed)
    return table, stack, out, [min(total, len(stack)), max(0, total - len(stack))]


@pytest.mark.parametrize("B,width", [(1, 9), (3, 300), (64, 70), (700, 40), (2500, 140), (16384, 4)])
@pytest.mark.parametrize("holes", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_truncate_rows_with_holes(B, width, holes, in_place):
    rng = np.random.default_rng(B)
    page, pages = 16, B * width + 7
    lens = rng.integers(0, width * page + 1, B)
    drop = rng.choice([0, 1, 3, 40, 10 ** 6], B, p=[0.2, 0.3, 0.2, 0.2, 0.1])
    keep = np.where(rng.random(B) < 0.1, -5, lens - drop)
    table = np.full((B, width), -1, np.int32)
    ids = rng.permutation(pages)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = ids[at:at + m]
        at += m
        gone = rng.random(m) < holes              # any of them, the last one apart now and then
        gone[-1:] &= rng.random() < holes
        table[b, :m][gone] = -1
    count = len(ids) - at
    stack = list(ids[at:]) + [-9] * (pages - count)
    want = _truncate(lens.tolist(), keep.tolist(), table, stack, count, page)
    t, s, n, c = _i32(table), _i32(stack), _i32(lens), _i32([count, 0])
    out = mx.KVCut(n, c) if in_place else None
    cut = mx.mx_kv_truncate(n, _i32(keep), t, s, c, page, out=out)
    torch.cuda.synchronize()
    assert cut.lens.tolist() == want[2] and cut.counts.tolist() == want[3]
    assert s.tolist() == want[1] and (t.cpu().numpy() == want[0]).all()


def test_a_finished_request_with_pages_behind_its_window():
    """It gives back what it still has; the pages that follow are pages."""
    page = 16
    table, stack = _i32([[-1, -1, 7, 8, 9]]), _i32([1, 2, 0, 0, 0, 0, 0, 0, 0, 0])
    cut = mx.mx_kv_truncate(_i32([70]), _i32([0]), table, stack, _i32([2]), page)
    assert cut.counts.tolist() == [5, 0]
    plan = mx.mx_kv_extend(cut.lens, _i32([80]), table, stack, cut.counts, page, 80)
    assert table.tolist() == [[7, 8, 9, 2, 1]] and plan.counts.tolist() == [0, 0]
    assert (plan.slots >= 0).all()


def test_truncate_where_the_stack_has_no_room_for_all():
    table = _i32([[3, -1, 4, 5], [6, 7, -1, 8]])
    stack = _i32([0, 1, -9, -9])
    cut = mx.mx_kv_truncate(_i32([64, 64]), _i32([0, 0]), table, stack, _i32([2]), 16)
    # freed: 3 4 5 6 7 8; the i-th to stack[7 - i], of which there are four
    assert cut.counts.tolist() == [4, 4] and stack.tolist() == [0, 1, 8, 7] and (table == -1).all()


def test_extend_from_two_threads():
    """Calls of very different size at the same time: neither changes what the
    other may launch."""
    import threading

    wrong = []

    def calls(B, times):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                lens, new = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
                table, stack = torch.full((B, 1), -1, dtype=torch.int32, device="cuda"), _i32(np.arange(B))
                count = _i32([B])
                plan = mx.mx_kv_extend(lens, new, table, stack, count, 16, B)
                call, args = mx.lib().mx_kv_extend, (
                    lens.data_ptr(), new.data_ptr(), B, table.data_ptr(), 1, 1, stack.data_ptr(), B,
                    count.data_ptr(), 16, plan.lens.data_ptr(), plan.cu.data_ptr(), plan.slots.data_ptr(), B,
                    plan.counts.data_ptr(), stream.cuda_stream)
                status = [call(*args) for _ in range(times)]
                stream.synchronize()
                assert set(status) == {0}
                assert plan.counts.tolist() == [0, 0] and (plan.slots == (B - 1 - torch.arange(B).cuda()) * 16).all()
        except Exception as e:  # noqa: BLE001 -- shown below, by the thread that can fail the test
            wrong.append((B, repr(e)))

    threads = [threading.Thread(target=calls, args=a) for a in ((16384, 20000), (5000, 20000), (9000, 20000))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
