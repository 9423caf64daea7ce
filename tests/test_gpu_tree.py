"""tree_plan and tree_attn on the GPU against their 64-bit definitions, element by element."""
import numpy as np
import pytest
import torch

import drafts_reference as dr
import paged_reference as ref
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda
from test_gpu_index_data import reported
from test_gpu_prefix_attn import Batch

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


# ---- tree_plan ---------------------------------------------------------------------------

def plan_case(sizes, width, seed=0, cached=50, max_tree=None, pad=0, pos0=0):
    rng = np.random.default_rng(seed)
    parent = sum((dr.random_forest(rng, n, width) for n in sizes), [])
    cu = np.concatenate([[0], np.cumsum(sizes)]).tolist()
    kv = [n + int(rng.integers(0, cached)) for n in sizes]
    most = max_tree or max(max(sizes), 1)
    T = cu[-1] + pad
    want = dr.tree_plan(parent, cu, kv, -(-most // 32), T, pos0)
    return (i32(parent + [9] * pad), i32(cu), i32(kv), most), dict(pos0=pos0), want


def assert_plan(got, want):
    assert got.positions.dtype == torch.int64 and got.mask.dtype == torch.int32
    assert np.array_equal(got.positions.cpu().numpy(), want[0])
    assert np.array_equal(got.mask.cpu().numpy(), want[1])


@pytest.mark.parametrize("sizes,width,kw", [
    ([1], 1, {}), ([32], 1, {}), ([33], 4, {}), ([64], 1, dict(pad=3)), ([1, 1, 1], 2, dict(pos0=7)), ([0, 5, 0, 0, 7, 0], 3, dict(pad=1)),
    ([16] * 8, 3, dict(cached=32768)), ([1024], 1, {}), ([1024, 3, 1023], 5, dict(pad=200)), ([200, 129, 1, 31], 8, dict(max_tree=1000)),
    ([0] * 40 + [3] + [0] * 70 + [2], 2, {}), ([1] * 300, 1, {}), ([100] * 30, 100, dict(pos0=1 << 40)), ([5], 2, dict(max_tree=1024)),
])
def test_plan_matches_the_definition(sizes, width, kw):
    need_cuda()
    args, opts, want = plan_case(sizes, width, **kw)
    assert_plan(rsa.tree_plan(*args, **opts), want)
    rsa.check_device_error()


@pytest.mark.parametrize("seed", range(8))
def test_random_plans(seed):
    need_cuda()
    rng = np.random.default_rng(seed)
    sizes = rng.integers(0, rng.choice([2, 8, 70, 300]), int(rng.choice([1, 30, 33, 1100])))
    sizes[rng.integers(0, len(sizes))] += 1
    args, opts, want = plan_case(sizes.tolist(), int(rng.choice([1, 2, 6, 50])), seed, pad=int(rng.integers(0, 140)))
    assert_plan(rsa.tree_plan(*args, **opts), want)
    rsa.check_device_error()


def test_plan_rows_before_the_first_request_and_outputs_given():
    need_cuda()
    (parent, cu, kv, most), _, want = plan_case([4, 3], 2)
    parent, cu = torch.cat([i32([5] * 6), parent]), cu + 6
    out = rsa.TreePlan(torch.full((13,), 77, device="cuda"), i32([[55]] * 13))
    got = rsa.tree_plan(parent, cu, kv, most, out=out)
    assert got is out
    assert (out.positions[:6] == 0).all() and (out.mask[:6] == 0).all()
    assert_plan(rsa.TreePlan(out.positions[6:], out.mask[6:]), want)
    rsa.check_device_error()
    for bad in (rsa.TreePlan(out.positions[:12], out.mask), rsa.TreePlan(out.positions, out.mask[:, :0]), (1,), 5,
                rsa.TreePlan(out.positions.int(), out.mask), rsa.TreePlan(out.positions, out.mask.long())):
        with pytest.raises((ValueError, TypeError)):
            rsa.tree_plan(parent, cu, kv, most, out=bad)
    for args in ((parent.long(), cu, kv, most), (parent, cu[:-1], kv, most), (parent, cu, kv, 0), (parent, cu, kv, 1025),
                 (parent[::2], cu, kv, most), (parent[None], cu, kv, most)):
        with pytest.raises((ValueError, TypeError, rsa.RsaError)):
            rsa.tree_plan(*args)
    with pytest.raises(rsa.RsaError):
        rsa.tree_plan(parent[:0], cu, kv, most)


def test_plan_reports_what_it_cannot_follow():
    need_cuda()
    # a parent that is no earlier token counts as none
    for bad in (3, 2, 1 << 30, -2, -(1 << 31)):
        got = rsa.tree_plan(i32([-1, 0, bad, 2]), i32([0, 4]), i32([14]), 4)
        assert f"site code 0x98, first bad index {bad})" in reported()
        assert got.mask[:, 0].tolist() == [1, 3, 4, 12] and got.positions.tolist() == [10, 11, 10, 11]
    # more tokens than the mask has bits: those past it get nothing
    chain = list(range(-1, 69))
    got = rsa.tree_plan(i32(chain), i32([0, 70]), i32([70]), 64)
    assert "site code 0x99, first bad index 64)" in reported()
    want = dr.tree_plan(chain, [0, 70], [70], 3, 70)
    assert np.array_equal(got.mask[:64].cpu().numpy(), want[1][:64, :2]) and (got.mask[64:] == 0).all()
    assert got.positions.tolist() == list(range(64)) + [0] * 6
    # fewer tokens in the cache than drafted ones: they count from 0
    got = rsa.tree_plan(i32([-1, 0, 1]), i32([0, 3]), i32([2]), 3)
    assert "site code 0x97, first bad index 2)" in reported() and got.positions.tolist() == [0, 1, 2]
    # rows past the batch, and rows that do not ascend: nothing outside is read, request 0 stays right
    got = rsa.tree_plan(i32([-1, 0, 1]), i32([0, 2, 90]), i32([2, 99]), 3)
    assert "site code 0x96, first bad index 90)" in reported() and got.positions.tolist()[:2] == [0, 1]
    got = rsa.tree_plan(i32([-1, 0, 1]), i32([0, 2, -5]), i32([2, 99]), 3)
    assert "site code 0x96, first bad index -5)" in reported()
    got = rsa.tree_plan(i32([-1, 0, -1, 0]), i32([0, 2, 1, 4]), i32([2, 9, 9]), 4)
    assert "site code 0x96, first bad index 1)" in reported()
    assert got.positions[0] == 0  # (row 1 lies in [0, 2) and in [1, 4): either may have it)


@pytest.mark.parametrize("sizes", [[100], [60, 300, 5], [1000, 90]])
def test_plan_of_long_trees_with_runs_and_bad_parents(sizes):
    # chains that break off at many places, among them parents that are none, across words and blocks
    need_cuda()
    rng = np.random.default_rng(sum(sizes))
    for often in (0.02, 0.3):
        parent, good = [], []
        for n in sizes:
            for i in range(n):
                j = i - 1 if rng.random() > often else int(rng.integers(-1, i)) if i else -1
                bad = rng.random() < 0.02
                parent.append(int(rng.choice([i, i + 1, 2000, -2, -(1 << 31)])) if bad else j)
                good.append(-1 if bad else j)
        cu, lens = np.concatenate([[0], np.cumsum(sizes)]), [n + 7 for n in sizes]
        want = dr.tree_plan(good, cu.tolist(), lens, -(-max(sizes) // 32), len(parent))
        got = rsa.tree_plan(i32(parent), i32(cu.tolist()), i32(lens), max(sizes))
        assert_plan(got, want)
        assert parent == good or "site code 0x98" in reported()


def test_long_plans_whose_rows_do_not_ascend():
    # what is right of it does not matter, but nothing else is read or written, and it is reported
    need_cuda()
    parent = i32(list(range(-1, 299)))
    for cu in ([0, 290, 40, 300], [200, 290, 0, 300], [300, 0, 250, 10], [0, 130, 129, 300]):
        got = rsa.tree_plan(parent, i32(cu), i32([400] * 3), 300)
        assert "site code 0x9" in reported()  # (0x96; or 0x98 first, a parent that is none among the rows of another request)
        assert (got.positions >= 0).all() and (got.positions < 700).all()


# ---- tree_attn ---------------------------------------------------------------------------

class TreeBatch(Batch):
    """Batch whose newest tokens are drafted; lens count them."""

    def __init__(self, new, lens, *args, width=3, words=None, mask=None, seed=0, **kw):
        super().__init__(new, lens, *args, seed=seed, **kw)
        rng = np.random.default_rng(seed)
        words = words or max(1, -(-max(new) // 32))
        parent = sum((dr.random_forest(rng, n, width) for n in new), [])
        T = self.q.shape[0]
        if mask is None:
            self.mask = torch.from_numpy(dr.tree_plan(parent, self.cu.tolist(), [max(n, 0) for n in lens], words, T)[1])
        elif mask == "random":  # a row need not see itself, nor anything
            bits = rng.integers(0, 1 << 32, (T, words), dtype=np.uint64).astype(np.uint32)
            bits[rng.random(T) < 0.2] = 0
            self.mask = torch.from_numpy(bits.view(np.int32))
        else:
            self.mask = torch.full((T, words), mask, dtype=torch.int32)

    def reference(self):
        return dr.tree_attn(ref.to64(self.q), ref.to64(self.kc), ref.to64(self.vc), self.cu.tolist(), self.table.numpy(),
                            self.lens.tolist(), self.mask.numpy(), self.prefix_pages.numpy(), self.prefix)

    def device(self):
        return [t.cuda() for t in (self.q, self.kc, self.vc, self.cu, self.table, self.lens, self.mask, self.prefix_pages)]

    def run(self, **kw):
        dev = self.device()
        out, lse = rsa.tree_attn(*dev[:7], prefix_pages=dev[7], prefix_len=self.prefix, **kw)
        torch.cuda.synchronize()
        return out, lse


CASES = [
    # new, lens, prefix, Hq, Hkv, d, page, dtype
    ([1], [1], 0, 1, 1, 128, 16, BF),
    ([8], [8], 0, 8, 1, 64, 64, BF),                                        # nothing cached
    ([8], [1008], 0, 64, 8, 128, 64, BF),
    ([16], [128], 0, 8, 2, 128, 64, BF),                                    # the tree ends with a tile
    ([17], [128 + 9], 0, 8, 2, 128, 16, BF),                                # it lies in two tiles, the last one short
    ([33], [128 + 33], 1, 5, 1, 128, 16, BF),                               # it begins with a tile
    ([40], [64 + 40], 0, 3, 1, 64, 128, BF),                                # ... with a half
    ([200], [1000], 0, 4, 2, 128, 64, BF),                                  # over three tiles, several row groups
    ([3, 0, 1, 25, 0, 64], [10, 4, 1, 525, 0, 300], 50, 6, 2, 128, 16, BF),
    ([5 + i % 20 for i in range(40)], [40 + 13 * i for i in range(40)], 1000, 8, 8, 128, 16, BF),
    ([7, 7], [200, 100], 40, 256, 2, 128, 64, BF),                          # 128 query heads a key head
    ([9, 12], [100, 257], 65, 198, 2, 64, 16, BF),                          # 99
    ([64], [20064], 0, 16, 2, 128, 16, BF),                                 # over every worker
    ([12], [12], 20000, 2, 1, 128, 128, BF),
    ([1], [1], 0, 1, 1, 64, 16, F),
    ([9] * 6, [9, 31, 32, 41, 500, 1000], 600, 8, 2, 64, 16, F),
    ([3, 0, 33], [10, 3, 300], 33, 6, 3, 128, 32, F),
    ([150], [182], 0, 2, 1, 64, 64, F),
    ([5, 13], [77, 200], 129, 128, 1, 128, 128, F),
    ([32], [5000], 0, 2, 1, 128, 16, F),
]
IDS = ["R{}n{}P{}q{}k{}d{}p{}{}".format(len(c[0]), sum(c[0]), *c[2:7], "bf" if c[7] == BF else "f") for c in CASES]


@pytest.mark.parametrize("mask", [None, "random"], ids=["tree", "any"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_attn_matches_the_definition(case, mask):
    need_cuda()
    TreeBatch(*case, mask=mask).check()


@pytest.mark.parametrize("case", [
    ([152], [160], 300, 256, 2, 64, 64, BF),                # a unit of the prefix for every SM, none over
    ([101, 60], [110, 300], 140, 256, 2, 128, 16, BF),      # ... and a few over
    ([300, 20, 1], [300, 25, 200], 129, 256, 2, 64, 32, BF),  # two for every SM
    ([7, 9, 2, 1, 4], [7, 300, 140, 1, 5], 0, 256, 2, 64, 16, BF),       # pairs of token groups with and without one over
    ([64, 0, 33, 5, 96], [2064, 3, 700, 5, 129], 0, 16, 2, 128, 64, BF),
    ([70] * 9, [70 + 90 * i for i in range(9)], 20, 8, 1, 128, 32, BF),
    ([5] * 40, [6 + 7 * i for i in range(40)], 0, 128, 1, 64, 16, BF),    # more requests than a warp
], ids=lambda c: f"R{len(c[0])}n{sum(c[0])}P{c[2]}")
@pytest.mark.parametrize("mask", [None, "random"], ids=["tree", "any"])
def test_units_side_by_side(case, mask):
    need_cuda()
    b = TreeBatch(*case, mask=mask)
    first = b.check()
    again = b.run()
    assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("prefix", [0, 200])
def test_more_requests_than_threads_with_pairs(prefix):
    # the blocks look at the lengths in several turns
    need_cuda()
    rng = np.random.default_rng(8)
    new = rng.integers(0, 6, 800)
    lens = new + rng.integers(0, 40, 800)
    TreeBatch(new.tolist(), lens.tolist(), prefix, 128, 1, 64, 16, BF).check()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
@pytest.mark.parametrize("seed", range(10))
def test_random_trees(dtype, seed):
    need_cuda()
    rng = np.random.default_rng(5000 + 1000 * (dtype == F) + seed)
    R = int(rng.integers(1, 20))
    new = rng.integers(0, rng.choice([2, 9, 70, 140]), R)
    new[rng.integers(0, R)] += 1
    lens = new + rng.integers(0, rng.choice([3, 200, 1000]), R)
    G, Hkv = int(rng.choice([1, 2, 3, 5, 8, 12])), int(rng.choice([1, 2, 3]))
    TreeBatch(new.tolist(), lens.tolist(), int(rng.choice([0, 1, 100, 128, 1111])), G * Hkv, Hkv, int(rng.choice([64, 128])),
              int(rng.choice([16, 32, 64, 128])), dtype, seed=seed, scale=float(rng.choice([0.1, 1, 4])), wide=int(rng.integers(0, 3)),
              width=int(rng.choice([1, 2, 8])), words=None if rng.random() < 0.5 else 6, mask=None if rng.random() < 0.6 else "random").check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", [c for c in CASES if c[7] == BF and c[5] == 128][:9], ids=lambda c: f"n{sum(c[0])}P{c[2]}")
def test_a_chain_sees_what_the_causal_attention_sees(case, d):
    # every token the child of the one before, and a mask of ones (bits of later tokens are none of a row's): the causal
    # definition, and the same bits whichever way it is said
    need_cuda()
    case = (*case[:5], d, *case[6:])
    want, n, first = Batch(*case).reference(), int(sum(case[0])), None
    for kw in (dict(width=1), dict(mask=-1), dict(mask=-1, words=32)):
        got = TreeBatch(*case, **kw).run()
        ref.assert_prefix_attn(*got, want, BF, n)
        first = first or got
        assert torch.equal(got[0][:n], first[0][:n]) and torch.equal(got[1][:n], first[1][:n])
    rsa.check_device_error()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
def test_rows_that_see_nothing_and_rows_behind_the_batch(dtype):
    need_cuda()
    # empty masks: without a cached token or prefix such rows see nothing; request 1 has fewer keys than rows
    for prefix, lens in ((0, [6, 3, 0]), (20, [6, 3, 0]), (0, [40, 3, 5])):
        b = TreeBatch([6, 5, 2], lens, prefix, 4, 2, 64, 16, dtype, extra=5, mask=0)
        out, lse = torch.full((18, 4, 64), 7.0, dtype=dtype, device="cuda"), torch.full((18, 4), 8.0, device="cuda")
        b.check(out=out, lse=lse)
        assert (out[13:] == 7).all() and (lse[13:] == 8).all()
        if prefix == 0 and lens[0] == 6:
            assert torch.isneginf(lse[:13]).all() and (out[:13] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
@pytest.mark.parametrize("rows", [2, 60, 900])
def test_one_request_whose_rows_begin_later(dtype, rows):
    # rows before the first request are none of its, with one request as with several
    need_cuda()
    for cls in (Batch, TreeBatch):
        for prefix in (0, 40):
            b = cls([rows], [rows + 50], prefix, 6, 2, 64, 32, dtype, extra=5)
            b.cu += 3
            out, lse = torch.full((rows + 5, 6, 64), 7.0, dtype=dtype, device="cuda"), torch.full((rows + 5, 6), 8.0, device="cuda")
            if cls is TreeBatch:
                b.mask[3:rows + 3] = b.mask[:rows].clone()
            b.run(out=out, lse=lse)
            rsa.check_device_error()
            if rows < 100:
                ref.assert_prefix_attn(out[3:rows + 3], lse[3:rows + 3], tuple(x[3:rows + 3] for x in b.reference()), dtype)
            for at in (slice(0, 3), slice(rows + 3, None)):
                assert (out[at] == 7).all() and (lse[at] == 8).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
def test_masked_keys_may_hold_anything(dtype):
    # keys of tokens that a row does not see: infinite, NaN or huge (values within the lengths have to be finite)
    need_cuda()
    b = TreeBatch([20, 3], [150, 10], 30, 8, 2, 128, 32, dtype, width=4)
    base, at = 130, 7
    want, wl = b.run()
    hidden = [i for i in range(20) if not dr.sees(b.mask[i].numpy(), i, at)] + [20, 21, 22]
    assert len(hidden) > 3
    for x in (float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max, torch.finfo(dtype).min):
        b.kc[int(b.table[0, (base + at) // 32]), :, (base + at) % 32] = x
        out, lse = b.run()
        assert torch.equal(out[hidden], want[hidden]) and torch.equal(lse[hidden], wl[hidden])
    rsa.check_device_error()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
def test_more_tokens_than_the_mask_has_bits(dtype):
    # bits past the mask count as not set
    need_cuda()
    b = TreeBatch([70, 2], [200, 9], 17, 4, 2, 64, 16, dtype, width=1, words=3)
    b.mask = b.mask[:, :2].contiguous()
    b.check()


def test_strided_masks_and_refusals():
    need_cuda()
    b = TreeBatch(*CASES[8])
    want, wl = b.run()
    dev = b.device()
    kw = dict(prefix_pages=dev[7], prefix_len=b.prefix)
    wide = torch.full((dev[6].shape[0], 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:6] = dev[6]
    got = rsa.tree_attn(*dev[:6], wide[:, 4:6], **kw)
    assert torch.equal(got[0], want) and torch.equal(got[1], wl)
    for bad in (dev[6][:-1], dev[6].long(), dev[6][:, 0], dev[6].cpu(), wide[:, ::4], dev[6][:, :0], None,
                torch.zeros(dev[6].shape[0], 33, dtype=torch.int32, device="cuda"), dev[6][:1].expand(dev[6].shape[0], 2)):
        with pytest.raises((ValueError, TypeError, rsa.RsaError)):
            rsa.tree_attn(*dev[:6], bad, **kw)
    with pytest.raises(rsa.RsaError):
        rsa.tree_attn(*dev[:6], wide[:, :2], **kw, lse=wide.view(-1)[:6 * wide.shape[0]].view(-1, 6).view(torch.float32))
    rsa.check_device_error()


def test_same_bits_whatever_the_workspace_held_and_on_streams():
    need_cuda()
    b = TreeBatch(*CASES[9])
    dev = b.device()
    kw = dict(prefix_pages=dev[7], prefix_len=b.prefix)
    n = rsa.tree_attn_workspace_size(BF, *b.q.shape[:2], CASES[9][4], CASES[9][5], len(b.lens))
    want = b.run(workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    for fill in (255, 127):
        got = b.run(workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    for shift in (16, 48, 240):  # (a workspace need not begin on more than 16 bytes)
        got = b.run(workspace=torch.zeros(n + shift, dtype=torch.uint8, device="cuda")[shift:])
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [rsa.tree_attn(*dev[:7], **kw, stream=s[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g in got for x, y in zip(g, want))


def test_captured_plan_and_attention_replay_with_other_trees():
    need_cuda()
    b = TreeBatch([16] * 4, [300, 20, 130, 64], 200, 8, 2, 128, 32, BF)
    dev = b.device()
    rng = np.random.default_rng(3)
    parent = torch.zeros(64, dtype=torch.int32, device="cuda")

    def call():
        tree = rsa.tree_plan(parent, dev[3], dev[5], 16)
        return tree, rsa.tree_attn(*dev[:6], tree.mask, prefix_pages=dev[7], prefix_len=b.prefix)
    parent.copy_(i32(sum((dr.random_forest(rng, 16, 3) for _ in range(4)), [])))
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tree, (out, lse) = call()
    for lens, cu in (([300, 20, 130, 64], [0, 16, 32, 48, 64]), ([64, 18, 17, 64], [0, 1, 17, 33, 40]), ([17, 16, 130, 33], [0, 16, 16, 17, 20])):
        p = sum((dr.random_forest(rng, cu[r + 1] - cu[r], 3) for r in range(4)), [])
        b.lens, b.cu = torch.tensor(lens, dtype=torch.int32), torch.tensor(cu, dtype=torch.int32)
        parent[:len(p)] = i32(p)
        dev[5].copy_(b.lens)
        dev[3].copy_(b.cu)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        pos, mask = dr.tree_plan(p, cu, lens, 1, 64)
        assert_plan(tree, (pos, mask))
        b.mask = torch.from_numpy(mask)
        ref.assert_prefix_attn(out, lse, b.reference(), BF, cu[-1])
    rsa.check_device_error()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
def test_bad_lengths_and_pages_are_reported_and_harmless(dtype):
    need_cuda()
    b = TreeBatch([9, 9, 9], [40, 150, 60], 30, 4, 2, 64, 16, dtype)
    want, wl = b.check()
    keep = [*range(9), *range(18, 27)]
    lens, table = b.lens.clone(), b.table.clone()
    for n in (-3, 1000, 2147483647):
        b.lens = lens.clone()
        b.lens[1] = n
        b.table = table.clone()
        b.table[1, 3:] = table[1, 0]  # (a clamped length reads the whole row)
        out, lse = b.run()
        assert f"site code 0x94, first bad index {n})" in reported()
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wl[keep])
    b.lens = lens
    for page in (-1, b.kc.shape[0], 2147483647):
        b.table = table.clone()
        b.table[1, 9] = page
        out, lse = b.run()
        assert f"site code 0x95, first bad index {page})" in reported()
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wl[keep])
    b.table, cu = table, b.cu
    b.cu = torch.tensor([0, 9, 1 << 30, 27], dtype=torch.int32)
    out, lse = b.run()
    assert "site code 0x93, first bad index" in reported()
    assert torch.equal(out[:9], want[:9])
    b.cu = cu
    b.check()


def test_injected_launch_failure_touches_nothing():
    need_cuda()
    b = TreeBatch(*CASES[8])
    out = torch.full(b.q.shape, 5.0, dtype=BF, device="cuda")
    rsa.inject_launch_failure(0)
    with pytest.raises(rsa.RsaError) as e:
        b.run(out=out)
    assert e.value.status == 3 and "injected launch failure" in str(e.value)
    torch.cuda.synchronize()
    assert (out == 5).all()
    b.check(out=out)
