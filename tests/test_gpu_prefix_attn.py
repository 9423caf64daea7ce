"""prefix_attn on the GPU against the 64-bit definition, element by element."""
import numpy as np
import pytest
import torch

import paged_reference as ref
import context_attention_rsa_gb300 as rsa
from gpu_helpers import need_cuda

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


class Batch:
    """A paged cache with shuffled pages; cache rows that no request owns are NaN."""

    def __init__(self, new, lens, prefix, Hq, Hkv, d, page, dtype, seed=0, scale=1.0, extra=0, wide=0):
        g = torch.Generator().manual_seed(seed)
        R = len(lens)
        counts = [-(-max(n, 0) // page) for n in lens]
        npre = -(-prefix // page)
        n_pages = npre + sum(counts) + 2
        ids = torch.randperm(n_pages, generator=g).to(torch.int32)
        self.kc = torch.full((n_pages, Hkv, page, d), float("nan"), dtype=dtype)
        self.vc = self.kc.clone()
        self.prefix_pages, at = ids[:npre].contiguous(), npre
        max_pages = max(max(counts), 1) + wide
        self.table = torch.full((R, max_pages), -(1 << 30), dtype=torch.int32)  # entries past the keys are never read
        owners = [(self.prefix_pages, prefix)]
        for r in range(R):
            self.table[r, :counts[r]] = ids[at:at + counts[r]]
            owners.append((ids[at:at + counts[r]], lens[r]))
            at += counts[r]
        for pages, n in owners:
            for j in range(0, max(n, 0), page):
                m = min(page, n - j)
                p = int(pages[j // page])
                self.kc[p, :, :m] = torch.randn(Hkv, m, d, generator=g).to(dtype)
                self.vc[p, :, :m] = torch.randn(Hkv, m, d, generator=g).to(dtype)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        T = int(self.cu[-1]) + extra
        self.q = (scale * torch.randn(max(T, 1), Hq, d, generator=g)).to(dtype)
        self.lens, self.prefix, self.dtype = torch.tensor(lens, dtype=torch.int32), prefix, dtype

    def reference(self):
        return ref.prefix_attn(ref.to64(self.q), ref.to64(self.kc), ref.to64(self.vc), self.cu.tolist(), self.table.numpy(),
                               self.lens.tolist(), self.prefix_pages.numpy(), self.prefix)

    def run(self, **kw):
        dev = [t.cuda() for t in (self.q, self.kc, self.vc, self.cu, self.table, self.lens, self.prefix_pages)]
        out, lse = rsa.prefix_attn(*dev[:6], prefix_pages=dev[6], prefix_len=self.prefix, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, **kw):
        out, lse = self.run(**kw)
        rsa.check_device_error()
        ref.assert_prefix_attn(out, lse, self.reference(), self.dtype, int(self.cu[-1]))
        return out, lse


CASES = [
    # new, lens, prefix, Hq, Hkv, d, page, dtype
    ([1], [1], 0, 1, 1, 128, 16, BF),
    ([1], [1], 0, 8, 1, 64, 64, BF),
    ([1], [1000], 0, 64, 8, 128, 64, BF),
    ([1], [129], 1, 5, 1, 128, 16, BF),
    ([1, 1, 1], [1, 127, 128], 128, 14, 2, 128, 32, BF),
    ([1] * 9, [5, 300, 17, 1, 129, 64, 33, 1000, 2], 777, 32, 4, 128, 64, BF),
    ([1] * 40, [7 + 13 * i for i in range(40)], 1000, 8, 8, 128, 16, BF),
    ([1] * 70, [3 + i for i in range(70)], 2500, 16, 2, 64, 16, BF),        # several row groups on the prefix
    ([3, 0, 1, 5, 0], [10, 4, 1, 5, 0], 50, 6, 2, 128, 16, BF),             # requests without tokens, prompts without a past
    ([40, 200], [1000, 200], 0, 8, 2, 128, 128, BF),                        # more rows than a unit
    ([300], [300], 300, 4, 4, 64, 32, BF),
    ([17, 1], [333, 5000], 129, 7, 1, 64, 64, BF),
    ([2, 2], [200, 100], 40, 256, 2, 128, 64, BF),                          # 128 query heads a key head
    ([1, 2], [100, 257], 65, 198, 2, 64, 16, BF),                           # 99
    ([1], [20000], 0, 2, 1, 128, 16, BF),                                   # one row over every worker
    ([1], [1], 20000, 2, 1, 128, 128, BF),
    ([1], [1], 0, 1, 1, 64, 16, F),
    ([1] * 6, [1, 31, 32, 33, 500, 1000], 600, 8, 2, 64, 16, F),
    ([3, 0, 9], [10, 3, 300], 33, 6, 3, 128, 32, F),
    ([150], [150], 0, 2, 1, 64, 64, F),
    ([1, 3], [77, 200], 129, 128, 1, 128, 128, F),
    ([1], [5000], 0, 2, 1, 128, 16, F),
]
IDS = ["R{}n{}P{}q{}k{}d{}p{}{}".format(len(c[0]), sum(c[0]), *c[2:7], "bf" if c[7] == BF else "f") for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_matches_the_definition(case):
    need_cuda()
    Batch(*case).check()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
@pytest.mark.parametrize("seed", range(10))
def test_random_batches(dtype, seed):
    need_cuda()
    rng = np.random.default_rng(1000 * (dtype == F) + seed)
    R = int(rng.integers(1, 30))
    new = rng.integers(0, rng.choice([2, 4, 60]), R)
    new[rng.integers(0, R)] += 1
    lens = new + rng.integers(0, rng.choice([3, 200, 1500]), R)
    G, Hkv = int(rng.choice([1, 2, 3, 5, 8, 12, 33])), int(rng.choice([1, 2, 3]))
    prefix = int(rng.choice([0, 1, 100, 128, 1111]))
    Batch(new.tolist(), lens.tolist(), prefix, G * Hkv, Hkv, int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128])), dtype,
          seed=seed, scale=float(rng.choice([0.1, 1, 4])), wide=int(rng.integers(0, 3))).check()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
def test_rows_that_see_nothing_and_rows_behind_the_batch(dtype):
    need_cuda()
    # request 1 has more new rows than cached tokens: its first rows see nothing; request 2 has no key at all
    for prefix in (0, 20):
        b = Batch([1, 5, 2], [9, 3, 0], prefix, 4, 2, 64, 16, dtype, extra=6)
        out = torch.full((14, 4, 64), 7.0, dtype=dtype, device="cuda")
        lse = torch.full((14, 4), 8.0, device="cuda")
        b.check(out=out, lse=lse)
        assert (out[8:] == 7).all() and (lse[8:] == 8).all()
        if prefix == 0:
            assert torch.isneginf(lse[1:3]).all() and torch.isneginf(lse[6:8]).all() and (out[6:8] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
def test_long_runs_of_rows_that_see_nothing(dtype):
    # far more new rows than cached tokens: most of the request's row groups have no key to see, dozens of them one
    # after the other in one worker's share, between groups and requests that do
    need_cuda()
    for prefix, G in ((0, 8), (100, 3), (0, 1)):
        new, lens = [1, 3000, 1, 700, 2], [40, 130, 300, 0, 9]
        b = Batch(new, lens, prefix, 2 * G, 2, 64, 32, dtype)
        out, lse = b.run()
        rsa.check_device_error()
        if prefix == 0:
            hidden = 3000 - 130
            assert torch.isneginf(lse[1:1 + hidden]).all() and (out[1:1 + hidden] == 0).all()
        # rows at both ends of every run against the definition
        keep = torch.tensor([0, 1, 1 + 3000 - 131, 1 + 3000 - 130, 3000, 3001, 3002, 3701, 3702, 3703])
        r = b.reference()
        ref.assert_prefix_attn(out[keep.cuda()], lse[keep.cuda()], tuple(x[keep.numpy()] for x in r), dtype)


def test_large_scores_and_infinite_values_in_masked_rows():
    need_cuda()
    # (rows past kv_len and prefix_len are NaN in every batch); scores of thousands do not overflow
    for dtype in (BF, F):
        b = Batch([1, 1], [70, 200], 130, 8, 2, 128, 64, dtype, scale=1.0)
        b.q *= 300
        out, lse = b.run()
        r = b.reference()
        # near one-hot rows: the scores' own error (relative to |q||k|) decides, which the bound counts
        ref.assert_prefix_attn(out, lse, r, dtype)
        rsa.check_device_error()


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
def test_a_request_of_nan_stays_by_itself(dtype, prefix):
    # the others' rows keep their bits; its own are NaN, their lse too unless only the values are
    need_cuda()
    for what in ("q", "k", "v"):
        b = Batch([1, 3, 1, 2], [70, 300, 5, 129], prefix, 8, 2, 128, 32, dtype)
        want, wl = b.run()
        if what == "q":
            b.q[1:4] = float("nan")
        else:
            (b.kc if what == "k" else b.vc)[int(b.table[1, 2]), :, 7] = float("nan")
        out, lse = b.run()
        keep = [0, 4, 5, 6]
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wl[keep])
        assert out[1:4].isnan().all()
        assert torch.equal(lse[1:4], wl[1:4]) if what == "v" else lse[1:4].isnan().all()
    rsa.check_device_error()


@pytest.mark.parametrize("prefix", [0, 100])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
def test_more_requests_than_threads(dtype, prefix):
    # a block looks at the lengths in several turns; requests without tokens and without keys among them
    need_cuda()
    rng = np.random.default_rng(7)
    new = rng.integers(0, 3, 1100)
    lens = np.where(rng.integers(0, 9, 1100) == 0, 0, new + rng.integers(0, 60, 1100))
    Batch(new.tolist(), lens.tolist(), prefix, 4, 2, 64, 16, dtype).check()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf", "f"])
def test_rows_before_the_first_request(dtype):
    need_cuda()
    for prefix in (0, 150):
        b = Batch([1, 2], [100, 40], prefix, 6, 2, 64, 32, dtype, extra=5)
        b.cu += 3
        out, lse = torch.full((8, 6, 64), 7.0, dtype=dtype, device="cuda"), torch.full((8, 6), 8.0, device="cuda")
        b.run(out=out, lse=lse)
        rsa.check_device_error()
        ref.assert_prefix_attn(out[3:6], lse[3:6], tuple(x[3:6] for x in b.reference()), dtype)
        for rows in (slice(0, 3), slice(6, 8)):
            assert (out[rows] == 7).all() and (lse[rows] == 8).all()


def test_one_request_equals_the_dense_decode():
    # the same keys as a dense cache of the library's own decode
    need_cuda()
    H, T, d = 4, 2048, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(1, H, n, d, generator=g, device="cuda").to(BF) for n in (3, T, T))
    o, l = rsa.decode_attn(q, k, v, 4, True)
    page = 64
    kc, vc = (x[0].view(H, T // page, page, d).transpose(0, 1).contiguous() for x in (k, v))
    table = torch.arange(T // page, dtype=torch.int32, device="cuda")[None]
    cu, n = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.tensor([T], dtype=torch.int32, device="cuda")
    o2, l2 = rsa.prefix_attn(q[0].transpose(0, 1), kc, vc, cu, table, n)
    # half of the keys as a prefix: the same rows again
    o3, l3 = rsa.prefix_attn(q[0].transpose(0, 1), kc, vc, cu, table[:, 16:].contiguous(), n - 16 * page,
                             prefix_pages=table[0, :16], prefix_len=16 * page)
    for oo, ll in ((o2, l2), (o3, l3)):
        assert (oo.float() - o[0].transpose(0, 1).float()).abs().max() <= 2e-2
        assert (ll - l[0].transpose(0, 1)).abs().max() <= 1e-3


def test_same_bits_every_time_whatever_the_workspace_held():
    need_cuda()
    case = CASES[5]
    b = Batch(*case)
    n = rsa.prefix_attn_workspace_size(BF, *b.q.shape[:2], case[4], case[5], len(b.lens))
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        out, lse = b.run(workspace=ws)
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_captured_call_replays_with_other_lengths():
    need_cuda()
    b = Batch([1] * 5, [300, 20, 7, 129, 64], 200, 8, 2, 128, 32, BF)
    dev = [t.cuda() for t in (b.q, b.kc, b.vc, b.cu, b.table, b.lens, b.prefix_pages)]
    kw = dict(prefix_pages=dev[6], prefix_len=b.prefix)
    rsa.prefix_attn(*dev[:6], **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = rsa.prefix_attn(*dev[:6], **kw)
    for lens in ([300, 20, 7, 129, 64], [1, 20, 3, 5, 64], [300, 1, 1, 128, 33]):
        b.lens = torch.tensor(lens, dtype=torch.int32)
        dev[5].copy_(b.lens)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref.assert_prefix_attn(out, lse, b.reference(), BF)
    rsa.check_device_error()


def test_two_calls_at_once_on_two_streams():
    need_cuda()
    a, b = Batch(*CASES[5], seed=1), Batch(*CASES[6], seed=2)
    want = [x.run() for x in (a, b)]
    dev = [[t.cuda() for t in (x.q, x.kc, x.vc, x.cu, x.table, x.lens, x.prefix_pages)] for x in (a, b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, x in enumerate((a, b)):
            got[i].append(rsa.prefix_attn(*dev[i][:6], prefix_pages=dev[i][6], prefix_len=x.prefix, stream=s[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_bad_lengths_and_pages_are_reported_and_harmless():
    need_cuda()
    b = Batch([1, 1, 1], [40, 50, 60], 30, 4, 2, 64, 16, BF)
    want, wl = b.check()
    keep = [0, 2]

    def bad(**kw):
        for n, v in kw.items():
            setattr(b, n, v)
        out, lse = b.run()
        with pytest.raises(rsa.RsaError) as e:
            rsa.check_device_error()
        assert e.value.status == 3 and "bounds check" in str(e.value)
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wl[keep])
    lens, table = b.lens.clone(), b.table.clone()
    for n in (-3, 1000, 2147483647):
        x = lens.clone()
        x[1] = n
        t = table.clone()
        t[1, 3:] = t[1, 0]  # (a clamped length reads the whole row)
        bad(lens=x, table=t)
    for page in (-1, b.kc.shape[0], 2147483647):
        t = table.clone()
        t[1, 2] = page
        bad(lens=lens, table=t)
    # rows that do not ascend: forced into the batch, other requests stay right
    b.table = table
    b.lens = lens
    cu = b.cu
    b.cu = torch.tensor([0, 1, 1 << 30, 3], dtype=torch.int32)
    b.run()
    with pytest.raises(rsa.RsaError):
        rsa.check_device_error()
    b.cu = cu
    b.check()


def test_strided_queries_and_refusals():
    need_cuda()
    b = Batch(*CASES[4])
    want, wl = b.run()
    T, Hq, d = b.q.shape
    packed = torch.zeros(T, Hq + 3, d, dtype=BF)
    packed[:, 1:Hq + 1] = b.q
    dev = [t.cuda() for t in (packed, b.kc, b.vc, b.cu, b.table, b.lens, b.prefix_pages)]
    kw = dict(prefix_pages=dev[6], prefix_len=b.prefix)
    out, lse = rsa.prefix_attn(dev[0][:, 1:Hq + 1], *dev[1:6], **kw)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    heads_first = b.q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    out, lse = rsa.prefix_attn(heads_first, *dev[1:6], **kw)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    q = b.q.cuda()
    for bad in (dict(out=torch.empty(T, Hq, d, device="cuda")), dict(lse=torch.empty(T, device="cuda")),
                dict(prefix_pages=dev[6][:0]), dict(workspace=torch.empty(10, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, TypeError, rsa.RsaError)):
            rsa.prefix_attn(q, *dev[1:6], **{**kw, **bad})
    for at, t in [(0, q[:, :, ::2]), (0, q.half()), (0, q[:, :9].contiguous()), (1, dev[1].float()), (2, dev[2][:, :, :, :64]),
                  (3, dev[3][:-1]), (3, dev[3].long()), (4, dev[4].long()), (5, dev[5][:-1])]:
        args = [q, *dev[1:6]]
        args[at] = t
        with pytest.raises((ValueError, TypeError, rsa.RsaError)):
            rsa.prefix_attn(*args, **kw)


def test_injected_launch_failure_touches_nothing():
    need_cuda()
    b = Batch(*CASES[4])
    out = torch.full(b.q.shape, 5.0, dtype=BF, device="cuda")
    rsa.inject_launch_failure(0)
    with pytest.raises(rsa.RsaError) as e:
        b.run(out=out)
    assert e.value.status == 3 and "injected launch failure" in str(e.value)
    torch.cuda.synchronize()
    assert (out == 5).all()
    b.check(out=out)


def test_offsets_beyond_32_bits():
    # a cache of more than 2^32 bytes and 2^31 elements; the request's pages lie at its far end
    need_cuda()
    page, Hkv, d = 128, 2, 128
    n_pages = (1 << 31) // (page * Hkv * d) + 40
    kc, vc = (torch.zeros(n_pages, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    far = torch.arange(n_pages - 6, n_pages, device="cuda")
    kc[far], vc[far] = (torch.randn(6, Hkv, page, d, generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(1, 8, d, generator=g, device="cuda").to(BF)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = far[:3].flip(0).to(torch.int32)[None].contiguous()
    out, lse = rsa.prefix_attn(q, kc, vc, i32(0, 1), table, i32(300), prefix_pages=far[3:].to(torch.int32), prefix_len=260)
    torch.cuda.synchronize()
    rsa.check_device_error()
    small = lambda c: ref.to64(c[far])  # noqa: E731
    r = ref.prefix_attn(ref.to64(q), small(kc), small(vc), [0, 1], table.cpu().numpy() - (n_pages - 6), [300],
                        np.array([3, 4, 5]), 260)
    ref.assert_prefix_attn(out, lse, r, BF)
    # ... and rows written there
    k = torch.randn(2, Hkv, d, generator=g, device="cuda").to(BF)
    slots = torch.tensor([(n_pages - 1) * page + 5, (n_pages - 2) * page], device="cuda")
    ko = torch.empty_like(k)
    rsa.qk_norm_rope(q.expand(2, 8, d).contiguous(), k, None, None, torch.zeros(2, dtype=torch.int64, device="cuda"), None, v=k,
                     slot_map=slots, k_cache=kc, v_cache=vc, k_out=ko)
    assert torch.equal(kc[n_pages - 1, :, 5], ko[0]) and torch.equal(vc[n_pages - 2, :, 0], k[1])
