"""The order in which launch 2 of moe_layer_few hands out its down items (csrc/few_order.h, compiled here by the host's
compiler): every item once, the runs of a row block in one list with run 0 last, and a model of the
workgroups that take them -- a few resident or all, in any order of arrival -- that always comes to its end."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = """
#include "few_order.h"
extern "C" {
int lists() { return moe::kLists; }
int items(int blocks, int runs, int c) { return moe::list_items(blocks, runs, c); }
int block_of(int id, int blocks, int runs) { return moe::down_item(id, blocks, runs).block; }
int run_of(int id, int blocks, int runs) { return moe::down_item(id, blocks, runs).run; }
int row_blocks(int T, int f, int k, int shared, int w) { return moe::few_row_blocks(T, f, k, shared, (moe_dtype)w); }
int runs(int T, int d, int f, int E, int k, int shared, int w) { return moe::few_splits(T, d, f, E, k, shared, (moe_dtype)w); }
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    where = tmp_path_factory.mktemp("few_order")
    src, so = where / "order.cpp", where / "order.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "expert_offload_cache_amd", "csrc"), str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def lists_of(order, blocks, runs):
    """-> the (block, run) of every list in the order in which its counter hands them out."""
    n = order.lists()
    return [[(order.block_of(c + n * v, blocks, runs), order.run_of(c + n * v, blocks, runs))
             for v in range(order.items(blocks, runs, c))] for c in range(n)]


def shapes(order):
    """Every (row blocks, runs) that some call has."""
    seen = set()
    for code, q in ((0, 32), (1, 32), (2, 128), (3, 128)):  # F32, BF16, INT4_G128, FP8_B128
        for d in range(64 if q == 32 else 128, 16385, 64 if q == 32 else 128):
            for f in (64 if q == 32 else 128, 768, 2048, 16384):
                for T, k, shared in ((1, 1, 0), (1, 8, 0), (3, 4, 0), (5, 4, 1), (16, 2, 0), (16, 8, 1), (16, 32, 0)):
                    rb = order.row_blocks(T, f, k, shared, code)
                    seen.add((d // 16 // rb, order.runs(T, d, f, 256, k, shared, code)))
    return sorted(seen)


def test_a_row_block_is_handed_out_in_one_list_run_0_last(order):
    pairs = shapes(order)
    assert {(45, 4), (44, 4), (18, 8), (4, 2)} <= set(pairs) and max(r for _, r in pairs) == 16 and len(pairs) > 500
    for blocks, runs in pairs:
        lists = lists_of(order, blocks, runs)
        every = [i for l in lists for i in l]
        assert len(every) == blocks * runs and set(every) == {(b, r) for b in range(blocks) for r in range(runs)}, (blocks, runs)
        for l in lists:
            left = {}
            for b, r in l:
                assert r == left.setdefault(b, runs) - 1, (blocks, runs, b)  # runs - 1, runs - 2, .., 0
                left[b] = r
            assert all(r == 0 for r in left.values())


def ends(lists, runs, workgroups, rng):
    """The workgroups as launch 2 has them: each asks for its next item (its home list first, then any that has one left) while
    it has the last one still to finish, and one that holds run 0 finishes when the other runs of the block are
    stored.  -> whether all of them come to their end in a random order of steps."""
    taken = [0] * len(lists)
    stored = {}

    def ask(home):
        for o in range(len(lists)):
            c = (home + o) % len(lists)
            if taken[c] < len(lists[c]):
                taken[c] += 1
                return lists[c][taken[c] - 1]
        return None

    # a workgroup: home list, item, next item, whether that has been asked for; it starts when there is room
    waiting = list(range(256))
    active = []
    while waiting or active:
        while waiting and len(active) < workgroups:
            home = waiting.pop(0) % len(lists)
            active.append([home, ask(home), None, False])
        able = []
        for w in active:
            _, item, _, asked = w
            if item is None or not asked or item[1] > 0 or stored.get(item[0], 0) == runs - 1:
                able.append(w)
        if not able:
            return False
        w = rng.choice(able)
        home, item, nxt, asked = w
        if item is None:
            active.remove(w)
        elif not asked:
            w[2], w[3] = ask(home), True
        else:
            stored[item[0]] = stored.get(item[0], 0) + (item[1] > 0)
            w[1], w[2], w[3] = nxt, None, False
    return sum(taken) == sum(len(l) for l in lists)


@pytest.mark.parametrize("blocks,runs", [(45, 4), (44, 4), (18, 8), (17, 8), (36, 4), (23, 8), (10, 2), (9, 16), (7, 16), (4, 2), (1, 16), (64, 4),
                                         (128, 2)])
def test_every_wait_of_the_join_ends(order, blocks, runs):
    rng = random.Random(blocks * 100 + runs)
    lists = lists_of(order, blocks, runs)
    for workgroups in (1, 2, 3, 4, 6, 8, 12, 16, 64, 256):
        for _ in range(3):
            assert ends(lists, runs, workgroups, rng), workgroups


def test_the_model_sees_a_closed_circle():
    """Items dealt to the lists one by one, whatever block they belong to: run 0 is then handed out before runs it waits for."""
    blocks, runs = 45, 4
    lists = [[(i % blocks, runs - 1 - i // blocks) for i in range(c, blocks * runs, 8)] for c in range(8)]
    rng = random.Random(1)
    assert not any(ends(lists, runs, n, rng) for n in (1, 2, 4, 6) for _ in range(3))
