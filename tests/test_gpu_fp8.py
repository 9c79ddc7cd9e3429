"""Attention over the 8-bit cache on the GPU against 64 bits: every grouping of
heads, block size and length at which the kernels take another path."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from fp8_reference import F8, RefCache8, attention64, attention_tolerance

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
NAN_CODE = 0x7F


class Case8:
    """A cache of random codes and scales, block tables in random order; rows
    behind each context hold NaN codes and unused blocks NaN scales."""

    def __init__(self, dev, ctx, H, Hkv, d, B, dtype="f16", seed=0, scale_exp=(-9, -4), width=None, free_scales=False):
        rng = np.random.default_rng(seed)
        self.ctx = np.asarray(ctx, np.int32)
        nblk = -(-self.ctx // B)
        width = width or max(1, int(nblk.max()))
        NB = int(nblk.sum()) + 5
        order = rng.permutation(NB).astype(np.int32)
        self.tables = np.full((len(ctx), width), -1, np.int32)
        at = 0
        codes = [torch.randn(NB, Hkv, B, d, generator=torch.Generator().manual_seed(seed + i)).mul(100).clamp(-448, 448)
                 .to(F8).view(torch.uint8).numpy() for i in range(2)]
        sc = 2.0 ** rng.integers(*scale_exp, (NB, Hkv + Hkv % 2, 2))
        if free_scales:
            sc = sc * rng.uniform(1, 2, sc.shape)
        sc = sc.astype(np.float32)
        used = np.zeros(NB, bool)
        for s, n in enumerate(self.ctx):
            b = order[at:at + nblk[s]]
            at += nblk[s]
            self.tables[s, :nblk[s]] = b
            used[b] = True
            if n % B:
                for c in codes:
                    c[b[-1], :, n % B:] = NAN_CODE
        for c in codes:
            c[~used] = NAN_CODE
        sc[~used] = np.nan
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.kc, self.vc = t(codes[0]).view(F8), t(codes[1]).view(F8)
        self.sc = t(sc)
        self.ref = RefCache8(self.kc, self.vc, self.sc)
        self.kvals, self.vvals = self.ref.values(0), self.ref.values(1)
        self.H, self.Hkv, self.d, self.B, self.dtype, self.dev = H, Hkv, d, B, dtype, dev
        self.dt_, self.dc = t(self.tables), t(self.ctx)
        self.q = torch.randn(len(ctx), H, d, generator=torch.Generator().manual_seed(seed + 9)).to(DT[dtype])

    def decode(self, q=None, **kw):
        q = (self.q if q is None else q).to(self.dev)
        out = torch.full_like(q, math.nan)
        pkv.paged_attention_decode_fp8(out, q, self.kc, self.vc, self.sc, self.dt_, self.dc, **kw)
        return out

    def check(self, out, seqs=None, scale=None, q=None):
        q = self.q if q is None else q
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        eps = torch.finfo(q.dtype).eps
        for s in range(len(self.ctx)) if seqs is None else seqs:
            got = out[s].double().cpu().numpy()
            n = int(self.ctx[s])
            if n == 0:
                assert not got.any()
                continue
            want, mag, vmax = attention64(q[s:s + 1].double().numpy(), self.kvals, self.vvals, self.tables[s], n, scale)
            tol = attention_tolerance(want[0], mag, vmax, n, self.d, eps, 21)
            assert np.all(np.abs(got - want[0]) <= tol), (s, n, np.abs(got - want[0]).max(), tol.min())


LENGTHS = (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 200, 0, 511, 513, 1030)


@pytest.mark.parametrize("B", [4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_block_and_head_sizes(cuda_device, B, d, dtype):
    c = Case8(cuda_device, LENGTHS, 4, 2, d, B, dtype, seed=B)
    for P in (0, 64, 192):
        out = c.decode(partition_size=P)
        pkv.check()
        c.check(out)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (6, 2), (5, 1), (8, 1), (7, 7), (16, 2), (9, 1), (12, 1), (16, 1),
                                   (17, 1), (48, 3), (40, 40)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_head_groupings(cuda_device, H, Hkv, dtype):
    c = Case8(cuda_device, (3, 64, 777), H, Hkv, 128, 16, dtype, seed=H)
    out = c.decode(partition_size=128)
    pkv.check()
    c.check(out)


@pytest.mark.parametrize("parts", [1, 2, 15, 16, 17, 33, 65])
def test_decode_merges(cuda_device, parts):
    """Splits merged in the kernel (to 16 partitions) and by the merge kernel."""
    c = Case8(cuda_device, (64 * parts, 64 * parts - 63, 5), 8, 2, 64, 16, "bf16", seed=parts)
    out = c.decode(partition_size=64)
    pkv.check()
    c.check(out)


def test_decode_scales_of_all_sizes(cuda_device):
    """Blocks whose scales lie sixty binades apart combine, and scales need not be powers of two."""
    for exp, free in (((-30, 31), False), ((-9, -4), True)):
        c = Case8(cuda_device, (40, 300, 1000), 4, 1, 128, 16, "bf16", seed=4, scale_exp=exp, free_scales=free)
        c.sc[:, :, 0] = torch.where(c.sc[:, :, 0].isnan(), c.sc[:, :, 0], torch.full_like(c.sc[:, :, 0], 2.0 ** -7))
        c.ref.scales = c.sc.cpu().numpy()
        c.kvals, c.vvals = c.ref.values(0), c.ref.values(1)
        out = c.decode()
        pkv.check()
        c.check(out)


def test_decode_queries_of_all_sizes(cuda_device):
    """bf16 queries far outside fp16's range, with keys that bring the scores back."""
    for q_exp in (-60, -20, 40, 90):
        c = Case8(cuda_device, (5, 64, 321), 3, 1, 64, 16, "bf16", seed=6)
        q = (c.q.double() * 2.0 ** q_exp).to(torch.bfloat16)
        out = c.decode(q=q, scale=2.0 ** (-3 - q_exp))
        pkv.check()
        c.check(out, q=q, scale=2.0 ** (-3 - q_exp))
    for what in (math.inf, -math.inf, math.nan):                 # one head of one sequence: its row alone is NaN
        q = c.q.clone()
        q[1, 2, 7] = what
        out = c.decode(q=q)
        bad = out.isnan()
        assert bool(bad[1, 2].all()) and int(bad.sum()) == c.d
        out[1, 2] = c.decode()[1, 2]
        c.check(out)
    z = c.decode(q=torch.zeros_like(c.q))
    c.check(z, q=torch.zeros_like(c.q))


def test_decode_nan_in_the_context_shows_and_beyond_it_does_not(cuda_device):
    c = Case8(cuda_device, (40, 40, 40), 2, 2, 64, 16, seed=8)
    c.kc.view(torch.uint8)[int(c.tables[1, 1]), 0, 3, 5] = NAN_CODE
    c.vc.view(torch.uint8)[int(c.tables[2, 2]), 1, 7, 9] = NAN_CODE
    out = c.decode()
    pkv.check()
    c.check(out, seqs=[0])
    assert bool(out[1, 0].isnan().all()) and not bool(out[1, 1].isnan().any())
    assert bool(out[2, 1, 9].isnan()) and int(out[2].isnan().sum()) == 1


@pytest.mark.parametrize("H,ctx,parts", [(2, 700, 64), (12, 700, 256), (2, 5000, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_nan_in_a_split_context_shows(cuda_device, H, ctx, parts, d):
    """In one of its partitions, or all through one."""
    c = Case8(cuda_device, (ctx, ctx, ctx), H, 2, d, 16, seed=14)
    keys = c.kc.view(torch.uint8)
    keys[int(c.tables[1, 20]), 0, 3, 5] = NAN_CODE
    keys[torch.from_numpy(c.tables[2, parts // 16:parts // 8].astype(np.int64)).to(cuda_device), 1] = NAN_CODE
    out = c.decode(partition_size=parts)
    pkv.check()
    c.check(out, seqs=[0])
    g = H // 2
    assert bool(out[1, :g].isnan().all()) and not bool(out[1, g:].isnan().any())
    assert bool(out[2, g:].isnan().all()) and not bool(out[2, :g].isnan().any())


def test_decode_zero_scales_are_zeros(cuda_device):
    c = Case8(cuda_device, (100,), 2, 1, 128, 16, seed=10)
    c.sc[int(c.tables[0, 0])] = 0.0
    c.ref.scales = c.sc.cpu().numpy()
    c.kvals, c.vvals = c.ref.values(0), c.ref.values(1)
    out = c.decode()
    c.check(out)
    c.sc.zero_()
    assert not bool(c.decode().any())
    pkv.check()


def test_decode_many_sequences(cuda_device):
    """More than one launch holds, with a split context in the second."""
    rng = np.random.default_rng(1)
    ctx = rng.integers(0, 20, 2500)
    ctx[2300], ctx[1] = 700, 500
    c = Case8(cuda_device, ctx, 2, 1, 64, 4, seed=11)
    out = c.decode(partition_size=64)
    pkv.check()
    c.check(out, seqs=[0, 1, 7, 2047, 2048, 2300, 2499])


def test_decode_long_context_is_independent_of_the_split(cuda_device):
    c = Case8(cuda_device, (20000, 9999), 8, 2, 128, 32, "bf16", seed=12)
    out = c.decode()
    c.check(out)
    again = c.decode()
    assert torch.equal(out, again)
    c.check(c.decode(partition_size=4096))
    pkv.check()


def test_decode_latches_bad_indexes(cuda_device):
    c = Case8(cuda_device, (100, 100), 2, 1, 64, 16, seed=13)
    good = c.decode()
    for bad in (c.kc.shape[0], -1):
        t = c.dt_.clone()
        t[1, 3] = bad
        out = torch.zeros_like(good)
        pkv.paged_attention_decode_fp8(out, c.q.to(cuda_device), c.kc, c.vc, c.sc, t, c.dc)
        with pytest.raises(pkv.PkvError) as e:
            pkv.check()
        assert e.value.status_name == "PKV_EINDEX" and "block" in str(e.value)
        assert torch.equal(out[0], good[0])
    for n in (-1, 113):
        out = torch.zeros_like(good)
        dc = torch.tensor([100, n], dtype=torch.int32, device=cuda_device)
        pkv.paged_attention_decode_fp8(out, c.q.to(cuda_device), c.kc, c.vc, c.sc, c.dt_, dc)
        with pytest.raises(pkv.PkvError) as e:
            pkv.check()
        assert "context" in str(e.value) or "block" in str(e.value)
        assert torch.equal(out[0], good[0])
    assert torch.equal(c.decode(), good)
    pkv.check()


def test_workspaces_of_the_other_kind_are_refused(cuda_device):
    c = Case8(cuda_device, (100,), 2, 1, 64, 16, seed=14)
    n = pkv.paged_attention_decode_fp8_workspace_size(1, 2, 1, 64, 112, 0)
    for ws in (pkv.make_workspace(cuda_device, n), torch.zeros(n, dtype=torch.uint8, device=cuda_device)):
        c.decode(workspace=ws)
        with pytest.raises(pkv.PkvError) as e:
            pkv.check()
        assert e.value.status_name == "PKV_EINVAL" and "workspace" in str(e.value)
    with pytest.raises(pkv.PkvError):
        c.decode(workspace=pkv.make_fp8_workspace(cuda_device, 0)[:128])
    # an 8-bit workspace does not serve the 16-bit calls either
    q = torch.zeros(1, 2, 64, dtype=torch.float16, device=cuda_device)
    kc = torch.zeros(8, 1, 16, 64, dtype=torch.float16, device=cuda_device)
    pkv.paged_attention_decode(q, q.clone(), kc, kc, torch.zeros(1, 8, dtype=torch.int32, device=cuda_device),
                               torch.tensor([100], dtype=torch.int32, device=cuda_device),
                               workspace=pkv.make_fp8_workspace(cuda_device, 1 << 20))
    with pytest.raises(pkv.PkvError) as e:
        pkv.check()
    assert e.value.status_name == "PKV_EINVAL"
    c.check(c.decode())
    pkv.check()


def test_graphs_of_different_sizes_share_a_workspace(cuda_device):
    """Two captured calls whose partials lie where the other's would, replayed in any order, and an eager prompt-phase
    call between them."""
    a = Case8(cuda_device, (1000, 900), 8, 2, 128, 16, "bf16", seed=15)
    b = Case8(cuda_device, (300, 1, 2000, 40, 999), 4, 4, 128, 16, "bf16", seed=16)
    ws = pkv.make_fp8_workspace(cuda_device, 1 << 25)
    graphs = []
    for c in (a, b):
        c.gq = c.q.to(cuda_device)
        c.gout = torch.empty_like(c.gq)
        args = (c.gout, c.gq, c.kc, c.vc, c.sc, c.dt_, c.dc)
        pkv.paged_attention_decode_fp8(*args, partition_size=128, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_attention_decode_fp8(*args, partition_size=128, workspace=ws)
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1, 0):
        c = (a, b)[i]
        c.gout.fill_(math.nan)
        graphs[i].replay()
        torch.cuda.synchronize()
        c.check(c.gout)
        p = Case8(cuda_device, (70, 20), 4, 2, 64, 16, seed=17)
        qs = torch.tensor([0, 1, 2], dtype=torch.int32, device=cuda_device)
        out = torch.empty_like(p.q.to(cuda_device))
        pkv.paged_attention_prefill_fp8(out, p.q.to(cuda_device), p.kc, p.vc, p.sc, p.dt_, p.dc, qs, workspace=ws)
    pkv.check()


def test_decode_on_two_streams_with_a_workspace_each(cuda_device):
    cases = [Case8(cuda_device, (700, 33, 2000), 8, 2, 64, 16, seed=s) for s in (18, 19)]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [pkv.make_fp8_workspace(cuda_device, 1 << 24) for _ in cases]
    qs = [c.q.to(cuda_device) for c in cases]
    outs = [[torch.empty_like(q) for _ in range(5)] for q in qs]
    torch.cuda.synchronize()
    for r in range(5):
        for c, s, w, q, o in zip(cases, streams, ws, qs, outs):
            pkv.paged_attention_decode_fp8(o[r], q, c.kc, c.vc, c.sc, c.dt_, c.dc, partition_size=128, workspace=w, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o[0])
        assert all(torch.equal(x, o[0]) for x in o)
    pkv.check()


# -- prompt phase -------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,d,B,dtype", [(4, 4, 128, 16, "f16"), (8, 2, 128, 32, "bf16"), (6, 2, 64, 8, "bf16"),
                                             (5, 1, 64, 4, "f16"), (2, 1, 128, 128, "f16")])
def test_prefill(cuda_device, H, Hkv, d, B, dtype):
    new = (1, 7, 130, 0, 300, 64)
    ctx = (40, 7, 500, 33, 301, 129)
    c = Case8(cuda_device, ctx, H, Hkv, d, B, dtype, seed=d + B)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.randn(int(start[-1]) + 2, H, d, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    out = torch.full((len(q), H, d), 5.0, dtype=DT[dtype], device=cuda_device)
    dq = q.to(cuda_device)
    pkv.paged_attention_prefill_fp8(out, dq, c.kc, c.vc, c.sc, c.dt_, c.dc, torch.from_numpy(start).to(cuda_device),
                                    max_context_len=max(ctx))
    pkv.check()
    eps = torch.finfo(DT[dtype]).eps
    got = out.double().cpu().numpy()
    assert (got[int(start[-1]):] == 5.0).all()              # rows behind the last sequence stay
    for s, n in enumerate(ctx):
        if new[s]:
            rows = slice(int(start[s]), int(start[s + 1]))
            want, mag, vmax = attention64(q[rows].double().numpy(), c.kvals, c.vvals, c.tables[s], n, 1 / math.sqrt(d))
            # the prompt-phase kernel's probabilities: 11 bits in fp16, 16 in bf16
            tol = attention_tolerance(want, mag, vmax, n, d, eps, 11 if dtype == "f16" else 15)
            assert np.all(np.abs(got[rows] - want) <= tol), (s, np.abs(got[rows] - want).max())


def test_prefill_latches_what_does_not_fit(cuda_device):
    c = Case8(cuda_device, (40, 100), 2, 1, 64, 16, seed=20)
    q = torch.zeros(4, 2, 64, dtype=torch.float16, device=cuda_device)
    out = torch.zeros_like(q)
    qs = torch.tensor([0, 2, 4], dtype=torch.int32, device=cuda_device)
    pkv.paged_attention_prefill_fp8(out, q, c.kc, c.vc, c.sc, c.dt_, c.dc, qs, max_context_len=48)
    with pytest.raises(pkv.PkvError) as e:
        pkv.check()
    assert e.value.status_name == "PKV_EINDEX"
    t = c.dt_.clone()
    t[1, 2] = c.kc.shape[0] + 3
    pkv.paged_attention_prefill_fp8(out, q, c.kc, c.vc, c.sc, t, c.dc, qs)
    with pytest.raises(pkv.PkvError) as e:
        pkv.check()
    assert "block" in str(e.value)
    with pytest.raises(pkv.PkvError):                       # a workspace of the 16-bit calls
        pkv.paged_attention_prefill_fp8(out, q, c.kc, c.vc, c.sc, c.dt_, c.dc, qs,
                                        workspace=pkv.make_workspace(cuda_device, 1 << 22))
        pkv.check()
    pkv.paged_attention_prefill_fp8(out, q, c.kc, c.vc, c.sc, c.dt_, c.dc, qs)
    pkv.check()


def test_prefill_shared_prefix(cuda_device):
    """Sequences that share full blocks in the same place, in another place, and a partly filled one; in a workspace that
    held NaN."""
    B, d, H, Hkv = 16, 64, 4, 2
    ctx = (100, 77, 100, 52, 41)
    c = Case8(cuda_device, ctx, H, Hkv, d, B, "f16", seed=30)
    t = c.tables
    t[1, :3] = t[0, :3]                       # a prefix of three blocks
    t[2, :2] = t[0, :2]
    t[2, 3] = t[0, 4]                         # a block of another place
    t[3, :3] = t[1, :3]
    t[3, 3] = t[1, 3]                         # shared, but sequence 3 ends in it (52 = 3 * 16 + 4)
    t[4, :2] = t[0, :2]
    t[4, 2] = t[0, 2]                         # sequence 4 ends in it
    c.dt_ = torch.from_numpy(t).to(cuda_device)
    new = (5, 1, 30, 7, 41)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.randn(int(start[-1]), H, d, generator=torch.Generator().manual_seed(1)).to(torch.float16)
    ws = pkv.make_fp8_workspace(cuda_device, 1 << 22)
    ws[256:].fill_(0xFF)
    out = torch.empty(q.shape, dtype=q.dtype, device=cuda_device)
    pkv.paged_attention_prefill_fp8(out, q.to(cuda_device), c.kc, c.vc, c.sc, c.dt_, c.dc,
                                    torch.from_numpy(start).to(cuda_device), workspace=ws)
    pkv.check()
    got = out.double().cpu().numpy()
    for s, n in enumerate(ctx):
        rows = slice(int(start[s]), int(start[s + 1]))
        want, mag, vmax = attention64(q[rows].double().numpy(), c.kvals, c.vvals, c.tables[s], n, 1 / math.sqrt(d))
        tol = attention_tolerance(want, mag, vmax, n, d, torch.finfo(q.dtype).eps, 11)
        assert np.all(np.abs(got[rows] - want) <= tol), (s, np.abs(got[rows] - want).max())


def test_decode_very_long_context(cuda_device):
    """More than a thousand partitions of one sequence beside a short one."""
    c = Case8(cuda_device, (300001, 7), 2, 1, 64, 64, "f16", seed=31)
    out = c.decode()
    pkv.check()
    c.check(out)


@pytest.mark.parametrize("fp8", [True, False])
def test_pools_past_32_bits(cuda_device, fp8):
    """Writes, decode and prompt phase at the end of pools whose offsets pass 2^32 give what a small pool gives."""
    Hkv, H, B, d, T = 8, 16, 128, 128, 150
    dt = torch.bfloat16
    far = (1 << 32) // (Hkv * B * d) + 40
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(T, h, d, generator=g).to(dt).to(cuda_device) for h in (H, Hkv, Hkv))
    cs = pkv.rotary_table(512, d, device=cuda_device)
    pos = torch.arange(T, dtype=torch.int32, device=cuda_device)
    got = []
    for NB, blocks in ((3, (2, 0)), (far, (far - 1, far - 9))):
        pool = lambda: torch.empty(NB, Hkv, B, d, dtype=torch.float8_e4m3fn if fp8 else dt, device=cuda_device)  # noqa: E731
        kc, vc = pool(), pool()
        slots = torch.tensor([blocks[t // B] * B + t % B for t in range(T)], device=cuda_device)
        table = torch.tensor([blocks], dtype=torch.int32, device=cuda_device)
        ctx = torch.tensor([T], dtype=torch.int32, device=cuda_device)
        start = torch.tensor([0, T], dtype=torch.int32, device=cuda_device)
        if fp8:
            sc = pkv.kv_scales(NB, Hkv, cuda_device)
            r = pkv.kv_rotary_and_cache_fp8(q, k, v, cs, pos, kc, vc, sc, slots)
            a = pkv.paged_attention_decode_fp8(torch.empty_like(r[-1:]), r[-1:].contiguous(), kc, vc, sc, table, ctx)
            b = pkv.paged_attention_prefill_fp8(torch.empty_like(r), r, kc, vc, sc, table, ctx, start)
            got.append([r, a, b, sc[list(blocks)]])
        else:
            r = pkv.kv_rotary_and_cache(q, k, v, cs, pos, kc, vc, slots)
            a = pkv.paged_attention_decode(torch.empty_like(r[-1:]), r[-1:].contiguous(), kc, vc, table, ctx)
            got.append([r, a])
        pkv.check()
        got[-1] += [kc[list(blocks)].view(torch.uint8)[0], vc[blocks[1], :, :T - B].view(torch.uint8)]
        del kc, vc
        torch.cuda.empty_cache()
    for x, y in zip(*got):
        assert torch.equal(x, y)
