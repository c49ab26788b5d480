"""The paged-cache operators against the fp64 oracle (oracle/paged.py).

Tolerances, from the formats.  u = 2^-8 and e = 2^-24 are the unit roundoffs of bf16 (8
significant bits) and fp32 (24).  A score is a sum of head_dim products, so with
S = scale sum |q_i||k_i| it is off by at most d = (head_dim + 8) e S; fp32 inputs go through
products of split operands, which adds 2^-20 S.  An exponential is then off by the factor
1 +- (d + 4e) and, with bf16 inputs, by u from its rounding; numerator and denominator both
carry the former: with A = sum p |v| / sum p the result is off by at most
A (2 d + u [bf16] + (L + 16) 2 e) before its own rounding of |o| u [bf16] or |o| e, L keys
summed.  fp32 values are split like the scores: A 2^-20 more.  lse is off by d + (L + 8) e + 4 e |lse|.
"""
import numpy as np
import pytest
import torch

from oracle import paged as oracle
from speculative_decoding_tree_spec_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U, E = 2.0 ** -8, 2.0 ** -24


def _np(t):
    return t.detach().cpu().double().numpy()


def _table(rng, total, page, extra=2, pad=1):
    """Distinct pages in random order for `total` positions per sequence, -1 after them."""
    need = [-(-int(t) // page) for t in total]
    pool = rng.permutation(sum(need) + extra)
    table = np.full((len(total), max(need + [1]) + pad), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = pool[at:at + n]
        at += n
    return table, len(pool)


def _tree_masks(rng, B, N):
    mask = np.zeros((B, N, N), dtype=np.uint8)
    depth = np.zeros((B, N), dtype=np.int32)
    for b in range(B):
        mask[b, 0, 0] = 1
        for n in range(1, N):
            p = int(rng.integers(0, n))
            mask[b, n] = mask[b, p]
            mask[b, n, n] = 1
            depth[b, n] = depth[b, p] + 1
    return mask, depth


class Case:
    room = 0  # positions every table row has columns for at least

    def __init__(self, prefix, N, hq=4, hkv=2, d=64, page=16, dtype=BF, seed=0, mask=None,
                 counts=None, shared=0, spread=2.0, heads_first=False, pad_nan=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        B = len(prefix)
        prefix = np.asarray(prefix, dtype=np.int32)
        self.table, pool = _table(rng, prefix + N, page)
        more = -(-self.room // page) - self.table.shape[1]
        if more > 0:
            self.table = np.pad(self.table, ((0, 0), (0, more)), constant_values=-1)
        if shared:
            self.table[:, :shared // page] = self.table[0, :shared // page]
        shape = (pool, hkv, page, d) if heads_first else (pool, page, hkv, d)
        self.k = torch.randn(shape, generator=g).to(dtype)
        self.v = torch.randn(shape, generator=g).to(dtype)
        if heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.q = (torch.randn((B, N, hq, d), generator=g) * spread).to(dtype)
        self.prefix, self.counts, self.shared = prefix, counts, shared
        self.mask = _tree_masks(rng, B, N)[0] if isinstance(mask, str) else mask
        self.scale = d ** -0.5
        if pad_nan:  # what no query sees may hold anything
            used = np.zeros((pool, page), dtype=bool)
            for b in range(B):
                cnt = N if counts is None else counts[b]
                for t in range(int(prefix[b]) + cnt):
                    used[self.table[b, t // page], t % page] = True
            self.k[torch.from_numpy(~used)] = float("nan")
            self.v[torch.from_numpy(~used)] = float("nan")

    def device(self, t):
        if isinstance(t, np.ndarray):
            return torch.as_tensor(t, device=DEV)
        out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=DEV)
        return out.copy_(t)

    def run(self, **kw):
        counts = None if self.counts is None else np.asarray(self.counts, dtype=np.int32)
        kw = dict(dict(scale=self.scale, shared_len=self.shared,
                       mask=None if self.mask is None else self.device(self.mask),
                       counts=None if counts is None else self.device(counts)), **kw)
        return binding.tree_attention_paged(self.device(self.q), self.device(self.k),
                                            self.device(self.v), self.device(self.table),
                                            self.device(self.prefix), **kw)

    def check(self, got=None):
        got = got or self.run()
        want, lse, A, S = oracle.attention(_np(self.q), _np(self.k), _np(self.v), self.table,
                                           self.prefix, self.scale, self.mask, self.counts,
                                           self.shared)
        D, L = self.q.shape[3], int(self.prefix.max()) + self.q.shape[1]
        out, got_lse = _np(got["out"]), _np(got["lse"])
        bf = self.q.dtype == BF
        d = S * ((D + 8) * E + (0 if bf else 2.0 ** -20))
        tol = A * (2 * d[..., None] + (L + 16) * 2 * E + (U if bf else 2.0 ** -20))
        tol += np.abs(want) * (U if bf else E) + 1e-30
        assert np.array_equal(np.isnan(out), np.isnan(want))
        assert np.array_equal(np.isneginf(got_lse), np.isneginf(lse))
        fine = np.isfinite(want)
        assert np.array_equal(out[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
        over = np.abs(out - want)[fine] / tol[fine]
        assert over.size == 0 or over.max() <= 1, over.max()
        some = np.isfinite(lse)
        assert np.array_equal(np.isnan(got_lse), np.isnan(lse))
        assert (np.abs(got_lse - lse) <= d + (L + 8) * E + 4 * E * np.abs(lse))[some].all()
        return got


@pytest.fixture(autouse=True, params=[0, 5000], ids=["tight", "roomy"])
def _room(request, monkeypatch):
    """A short table lets a call of few tiles go to clusters of the few-rows kernel; a table
    with room for thousands of positions does not, whatever the lengths are."""
    monkeypatch.setattr(Case, "room", request.param)


HEADS = [(4, 4, 64), (8, 2, 128), (8, 1, 64), (6, 3, 96), (2, 1, 8), (32, 8, 128), (5, 1, 104)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_one_token(dtype, hq, hkv, d):
    Case([0, 1, 15, 16, 63, 64, 65, 300], 1, hq, hkv, d, dtype=dtype).check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("N", [2, 11, 60])
def test_trees(dtype, hq, hkv, d, N):
    Case([0, 1, 127, 130, 40], N, hq, hkv, d, dtype=dtype, mask="tree", seed=N).check()


@pytest.mark.parametrize("page", [1, 3, 5, 8, 16, 24, 40, 64, 128, 200])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_page_lengths(page, dtype):
    Case([3, 131, 0, 260], 33, 8, 2, 64, page, dtype, seed=page, mask="tree").check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 7, 129, 200])
def test_prompts_with_padding(dtype, N):
    Case([0, 77, 5, 200, 9], N, 8, 2, 64, 24, dtype, seed=N,
         counts=[N, 0, 1, max(1, N - 1), N // 2 + 1]).check()


@pytest.mark.parametrize("hq,hkv,d,N,B", [(8, 2, 128, 1, 5), (8, 2, 128, 20, 9), (4, 4, 64, 3, 3),
                                          (8, 1, 96, 40, 4)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_shared_prefix(dtype, hq, hkv, d, N, B):
    shared = 160
    prefix = [shared + 13 * b for b in range(B)]
    c = Case(prefix, N, hq, hkv, d, 16, dtype, mask="tree", shared=shared)
    got = c.check()
    plain = c.run(shared_len=0)
    torch.testing.assert_close(got["out"].float(), plain["out"].float(), rtol=2 * U, atol=2 * U)
    c.prefix = c.prefix.copy()
    c.prefix[1] = shared - 1  # not a sequence behind the shared positions
    c.check()


def test_shared_prefix_alone():
    """A prefix that ends with the shared positions, and one that is all there is to see."""
    Case([64, 64, 65], 4, 8, 2, 64, 32, mask="tree", shared=64).check()
    mask = np.zeros((3, 4, 4), dtype=np.uint8)
    Case([64, 64, 65], 4, 8, 2, 64, 32, mask=mask, shared=64).check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [5, 70])
def test_rows_that_see_nothing(dtype, N):
    mask = np.tril(np.ones((3, N, N), dtype=np.uint8))
    mask[:, 1] = 0
    mask[2] = 0
    got = Case([0, 9, 0], N, 4, 1, 64, 16, dtype, mask=mask).check()
    assert (got["out"][0, 1] == 0).all() and (got["out"][2] == 0).all()
    assert torch.isneginf(got["lse"][2]).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [6, 60])
def test_values_that_are_not_finite_reach_only_those_who_see_them(dtype, N):
    """Drafts with NaN and infinite keys or values: the rows whose mask leaves them out are
    untouched, the rows that see them get what the formula gives."""
    c = Case([10, 140, 0], N, 4, 2, 64, 16, dtype, mask="tree", seed=4)
    for b in range(3):
        for j, (kx, vx) in {2: (1.0, np.inf), 3: (np.nan, 1.0), 4: (1.0, np.nan)}.items():
            t = int(c.prefix[b]) + j
            at = int(c.table[b, t // 16]), t % 16
            if not np.isfinite(kx):
                c.k[at] = kx
            if not np.isfinite(vx):
                c.v[at][..., 5] = vx
    c.check()


@pytest.mark.parametrize("N", [1, 40])
def test_infinite_values_of_the_prefix_reach_everyone(N):
    c = Case([200, 20], N, 4, 2, 64, 16, seed=4, mask="tree")
    c.v[int(c.table[0, 1]), 3, 0, 7] = float("inf")
    c.v[int(c.table[1, 0]), 3, 1, 9] = float("nan")
    c.check()


@pytest.mark.parametrize("N", [1, 50])
def test_pages_the_table_lacks_are_masked(N):
    c = Case([150, 90], N, 8, 2, 64, 16, seed=2, mask="tree")
    c.table[0, 2] = -1
    c.table[0, 4] = 1 << 20
    c.table[1, 5] = c.k.shape[0]
    c.check()
    c.table[:] = -1
    got = c.check()
    assert (got["out"] == 0).all()


@pytest.mark.parametrize("N", [1, 50])
def test_lengths_beyond_the_table_and_below_zero(N):
    c = Case([150, 90, 20], N, 8, 2, 64, 16, seed=2, mask="tree", pad_nan=False)
    c.prefix = np.array([len(c.table[0]) * 16 - 2, 1 << 30, -5], dtype=np.int32)
    c.table[:] = np.arange(c.table.size).reshape(c.table.shape) % c.k.shape[0]
    got = c.run()
    c.prefix[1] = len(c.table[0]) * 16  # the oracle's loops: no position beyond it exists
    c.check(got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_strided_queries_outputs_and_head_major_caches(dtype):
    c = Case([150, 31], 20, 8, 2, 64, 16, dtype, seed=6, mask="tree", heads_first=True)
    c.check()
    wide = torch.randn((2, 20, 3, 12, 64), generator=torch.Generator().manual_seed(1)).to(dtype)
    c.q = wide[:, :, 1, 2:10]
    out = torch.full((20, 2, 8, 72), 7.0, dtype=dtype, device=DEV)
    got = c.run(out=out.permute(1, 0, 2, 3)[..., :64])
    c.check(got)
    assert (out[..., 64:] == 7).all()


def test_long_context_is_cut_and_joined_reproducibly():
    c = Case([20011, 5], 3, 4, 1, 128, 16, seed=8)
    a, b = c.run(), c.run()
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    c.check(a)


@pytest.mark.parametrize("B,N,hq,hkv,d", [(1, 70, 4, 1, 128), (3, 40, 2, 1, 128), (2, 33, 8, 2, 64),
                                          (1, 300, 2, 2, 96)])
def test_many_blocks_of_many_rows(B, N, hq, hkv, d):
    """Long runs of key blocks in one tile, rising and falling scores."""
    c = Case([4000 + 777 * b for b in range(B)], N, hq, hkv, d, 16, seed=N, mask="tree")
    ramp = torch.linspace(0.1, 2.5, c.k.shape[0])[torch.randperm(c.k.shape[0],
                                                               generator=torch.Generator().manual_seed(1))]
    c.k = (c.k.float() * ramp[:, None, None, None]).to(BF)
    c.check()


def test_large_scores_and_flat_rows():
    Case([90, 300], 20, 4, 2, 64, 16, mask="tree", spread=60.0).check()
    Case([90, 300], 20, 4, 2, 64, 16, mask="tree", spread=0.0).check()


def test_offsets_beyond_32_bits():
    """A pool whose last pages start past 2^32 elements."""
    n_pages, page, hkv, d = 4200000, 16, 1, 64
    if torch.cuda.mem_get_info()[0] < 3 * 2 * n_pages * page * d:
        pytest.skip("needs 26 GB of device memory")
    small = Case([100], 5, 2, 1, 64, 16, seed=3)
    k = torch.zeros((n_pages, page, hkv, d), dtype=BF, device=DEV)
    v = torch.zeros_like(k)
    high = n_pages - small.k.shape[0]
    k[high:], v[high:] = small.k.to(DEV), small.v.to(DEV)
    table = np.where(small.table >= 0, small.table + high, -1).astype(np.int32)
    got = binding.tree_attention_paged(small.q.to(DEV), k, v, small.device(table),
                                       small.device(small.prefix), small.scale)
    small.check(got)


def test_other_streams():
    c = Case([150, 90], 50, 8, 2, 64, 16, seed=2, mask="tree")
    s = torch.cuda.Stream()
    dev = [c.device(x) for x in (c.q, c.k, c.v, c.table, c.prefix, c.mask)]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = binding.tree_attention_paged(*dev[:5], c.scale, mask=dev[5])
    torch.cuda.current_stream().wait_stream(s)
    c.check(got)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-6])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 50])
def test_scales(scale, dtype, N):
    c = Case([150, 90], N, 8, 2, 64, 16, dtype, seed=2, mask="tree")
    c.scale = scale
    c.check()


@pytest.mark.parametrize("shared", [96, 4608])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (6, 2)])  # with and without a tensor map of the queries
def test_shared_prefix_with_padding_and_strided_queries(hq, hkv, shared):
    N, B = 30, 4
    c = Case([shared, shared + 4, shared + 35, shared], N, hq, hkv, 64, 16, seed=5, mask="tree",
             shared=shared, counts=[N, 0, 1, N - 3])
    c.check()
    wide = torch.randn((N, B, hq + 3, 64), generator=torch.Generator().manual_seed(1)).to(BF)
    c.q = wide.permute(1, 0, 2, 3)[:, :, 1:hq + 1]  # batches and nodes are no one direction
    c.check()


def test_a_captured_call_replays_on_new_lengths():
    c = Case([150, 90, 0], 40, 8, 2, 64, 16, seed=2, mask="tree", pad_nan=False)
    dev = [c.device(x) for x in (c.q, c.k, c.v, c.table, c.prefix, c.mask)]
    out = {"out": torch.empty_like(dev[0]), "lse": torch.empty((3, 40, 8), device=DEV)}
    ws = torch.empty(binding.tree_attention_workspace_size(3, 40, 8, 2, 64), dtype=torch.uint8,
                     device=DEV)
    call = lambda: binding.tree_attention_paged(*dev[:5], c.scale, mask=dev[5], workspace=ws, **out)
    call()  # the kernels' one-time set-up stays out of the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for prefix in ([100, 3, 0], [150, 90, 0]):
        c.prefix = np.array(prefix, dtype=np.int32)
        dev[4].copy_(torch.as_tensor(c.prefix))
        graph.replay()
        c.check(out)


def test_empty_calls():
    for B, N in ((0, 3), (2, 0)):
        q = torch.zeros((B, N, 4, 64), dtype=BF, device=DEV)
        kv = torch.zeros((2, 16, 2, 64), dtype=BF, device=DEV)
        table = torch.zeros((B, 1), dtype=torch.int32, device=DEV)
        pre = torch.zeros(B, dtype=torch.int32, device=DEV)
        assert binding.tree_attention_paged(q, kv, kv, table, pre)["out"].shape == (B, N, 4, 64)


def test_binding_refuses():
    q = torch.zeros((2, 3, 4, 64), dtype=BF, device=DEV)
    kv = torch.zeros((4, 16, 2, 64), dtype=BF, device=DEV)
    table = torch.zeros((2, 1), dtype=torch.int32, device=DEV)
    pre = torch.zeros(2, dtype=torch.int32, device=DEV)
    ok = dict(q=q, k_cache=kv, v_cache=kv, page_table=table, prefix_len=pre)
    bad = [dict(q=q.float()), dict(q=q[..., :32]), dict(v_cache=kv.float()),
           dict(page_table=table.long()), dict(prefix_len=pre[:1]), dict(prefix_len=pre.cpu()),
           dict(mask=torch.ones((2, 3, 4), dtype=torch.uint8, device=DEV)),
           dict(counts=pre.float()), dict(lse=torch.zeros((2, 3, 3), device=DEV)),
           dict(out=torch.zeros((2, 3, 4, 32), dtype=BF, device=DEV))]
    for kw in bad:
        with pytest.raises((TypeError, ValueError)):
            binding.tree_attention_paged(**{**ok, **kw})
    for kw in (dict(shared_len=8), dict(scale=float("nan")),
               dict(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)),
               dict(q=q[:, :, :3])):
        with pytest.raises(binding.SpecError):
            binding.tree_attention_paged(**{**ok, **kw})


# ---------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------
def _cos_sin(n, rot):
    a = torch.arange(n, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))
    return torch.cat([a.cos(), a.sin()], dim=1).float()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("hq,hkv,d,rot,page,N", [(8, 2, 64, 64, 16, 7), (4, 4, 128, 64, 5, 1),
                                                 (3, 1, 40, 32, 3, 60), (32, 8, 128, 128, 16, 5),
                                                 (2, 1, 1024, 512, 8, 3), (4, 2, 64, 0, 16, 9)])
def test_append(dtype, inter, hq, hkv, d, rot, page, N):
    """A rotated element is two products and a sum in fp32 (3 e of their magnitudes), then
    rounded; everything else is copied."""
    rng = np.random.default_rng(d + N)
    g = torch.Generator().manual_seed(N)
    prefix = np.array([0, 17, 3, 40], dtype=np.int32)
    counts = np.array([N, max(N - 1, 0), 0, N], dtype=np.int32)
    table, pool = _table(rng, prefix + N, page)
    table[3, -2 if table.shape[1] > 1 else 0] = -1
    kc, vc = (torch.randn((pool, page, hkv, d), generator=g).to(dtype) for _ in range(2))
    qkv = torch.randn((4, N, hq + 2 * hkv, d), generator=g).to(dtype)
    q, k, v = qkv.split([hq, hkv, hkv], dim=2)
    ids = _tree_masks(rng, 4, N)[1]
    ids[3, 0] = 1000  # a rotary position the table lacks
    cs = _cos_sin(90, rot)
    want = oracle.append(_np(q), _np(k), _np(v), _np(kc), _np(vc), table, prefix, _np(cs), ids,
                         counts, inter)
    dq, dk, dv = qkv.to(DEV).split([hq, hkv, hkv], dim=2)
    dkc, dvc = kc.to(DEV), vc.to(DEV)
    t = lambda x: torch.as_tensor(x, device=DEV)
    out = binding.paged_append_rope(dq, dk, dv, dkc, dvc, t(table), t(prefix),
                                    cs.to(DEV) if rot else None, position_ids=t(ids),
                                    counts=t(counts), interleaved=inter)
    size = {"q": np.abs(_np(q)).max(), "k": max(np.abs(_np(k)).max(), np.abs(_np(kc)).max())}
    half = U if dtype == BF else E
    for got, ref, m in ((out, want[0], size["q"]), (dkc, want[1], size["k"])):
        err = np.abs(_np(got) - ref)
        assert (err <= np.abs(ref) * half * (1 + 2 ** -10) + 3 * E * 2 * m).all(), err.max()
    np.testing.assert_array_equal(_np(dvc), want[2])
    same = _np(kc) == want[1]  # untouched entries keep their bits
    np.testing.assert_array_equal(_np(dkc)[same], want[1][same])
    # in place, on another stream, without queries
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k2, v2 = kc.to(DEV), vc.to(DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        same_q = binding.paged_append_rope(dq, dk, dv, k2, v2, t(table), t(prefix),
                                           cs.to(DEV) if rot else None, position_ids=t(ids),
                                           counts=t(counts), interleaved=inter, out_q=dq)
        none = binding.paged_append_rope(None, dk, dv, k2, v2, t(table), t(prefix),
                                         cs.to(DEV) if rot else None, position_ids=t(ids),
                                         counts=t(counts), interleaved=inter)
    s.synchronize()
    assert none is None and torch.equal(same_q, out)
    assert torch.equal(k2, dkc) and torch.equal(v2, dvc)


def test_append_positions_without_a_place():
    d, page = 64, 16
    kc = torch.zeros((3, page, 1, d), dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    k = torch.ones((3, 4, 1, d), dtype=BF, device=DEV)
    table = torch.tensor([[0], [1], [2]], dtype=torch.int32, device=DEV)
    prefix = torch.tensor([14, 2 ** 31 - 2, -9], dtype=torch.int32, device=DEV)
    out = binding.paged_append_rope(k, k, k, kc, vc, table, prefix)
    assert kc[0, 14:].eq(1).all() and kc[0, :14].eq(0).all()  # two of four fit
    assert kc[1].eq(0).all() and kc[2, :4].eq(1).all()        # none; from position 0
    assert torch.equal(kc, vc) and out.eq(1).all()


def test_append_refuses():
    kv = torch.zeros((4, 16, 2, 64), dtype=BF, device=DEV)
    x = torch.zeros((2, 3, 2, 64), dtype=BF, device=DEV)
    table = torch.zeros((2, 1), dtype=torch.int32, device=DEV)
    pre = torch.zeros(2, dtype=torch.int32, device=DEV)
    ok = dict(q=x, k=x, v=x, k_cache=kv, v_cache=kv.clone(), page_table=table, prefix_len=pre)
    for kw in (dict(k=x[:, :, :1]), dict(q=x.float()), dict(cos_sin=torch.zeros((9, 64), device=DEV,
               dtype=BF)), dict(out_q=x[:, :2]), dict(position_ids=pre), dict(k_cache=kv.float())):
        with pytest.raises((TypeError, ValueError)):
            binding.paged_append_rope(**{**ok, **kw})
    with pytest.raises(binding.SpecError):
        binding.paged_append_rope(**ok, cos_sin=torch.zeros((9, 24), device=DEV))


# ---------------------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("planes,B,N,page,heads,row,heads_first",
                         [(4, 5, 30, 16, 8, 128, False), (1, 9, 60, 5, 1, 24, False),
                          (3, 2, 26, 7, 3, 40, True), (64, 3, 60, 64, 2, 64, True)])
def test_commit(planes, B, N, page, heads, row, heads_first):
    rng = np.random.default_rng(planes + B)
    W = 10
    prefix = rng.integers(0, 90, B).astype(np.int32)
    table, pool = _table(rng, prefix + N, page)
    path = np.full((B, W), -1, dtype=np.int32)
    path[:, 0] = 0
    acc = rng.integers(0, W, B).astype(np.int32)
    for b in range(B):
        path[b, 1:acc[b] + 1] = np.sort(rng.choice(np.arange(1, N), acc[b], replace=False))
    acc[0] = -1
    if B > 2:
        table[2, (int(prefix[2]) + int(path[2, 1])) // page] = -1
    shape = (planes, pool, heads, page, row) if heads_first else (planes, pool, page, heads, row)
    cache = torch.from_numpy(rng.integers(-30000, 30000, shape).astype(np.int16))
    if heads_first:
        cache = cache.transpose(2, 3)
    want = oracle.commit(cache.numpy(), table, prefix, path, acc)
    dev = torch.empty_strided(cache.shape, cache.stride(), dtype=cache.dtype, device=DEV)
    dev.copy_(cache)
    t = lambda x: torch.as_tensor(x, device=DEV)
    binding.commit_accepted_path_paged(dev, t(table), t(prefix), t(path), t(acc))
    np.testing.assert_array_equal(dev.cpu().numpy(), want)


def test_commit_refuses():
    cache = torch.zeros((2, 4, 16, 2, 64), dtype=BF, device=DEV)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    for args in ((cache[0, 0, 0], i(2, 1), i(2), i(2, 3), i(2)), (cache, i(1, 1), i(2), i(2, 3), i(2)),
                 (cache, i(2, 1), i(2).long(), i(2, 3), i(2))):
        with pytest.raises((TypeError, ValueError)):
            binding.commit_accepted_path_paged(*args)
    with pytest.raises(binding.SpecError):
        binding.commit_accepted_path_paged(cache[..., :4].contiguous()[..., :1, :], i(2, 1), i(2),
                                           i(2, 3), i(2))
