"""Rotary and 8-bit calls at the edges of what their definitions allow."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_139_gb300 as pkv
from fp8_reference import F8, RefCache8, attention64, attention_tolerance, rotate32
from paged_kv_cache_139_gb300.engine import PagedKVCache
from test_gpu_fp8 import Case8
from test_gpu_rotary import DT, Inputs, _random_cache8, _same8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,rot,layout", [(64, 0, "half"), (128, 0, "half"), (128, 32, "half"), (64, 48, "interleaved"),
                                          (128, 128, "half"), (64, 64, "interleaved")])
@pytest.mark.parametrize("B", [4, 16, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append8_nan_rows_do_not_count(cuda_device, dtype, B, d, rot, layout):
    """Whole rows of NaN among the tokens that one call writes to a block: scales and the other rows' codes are those of
    the numbers alone, in blocks begun anew and in partly filled ones, also where nothing but NaN is written."""
    H, Hkv, NB = 2, 3, 12
    # block 0 anew, 1 and 2 from their second row, 3 anew and all NaN, 4 partly filled and all NaN, 5 and 6 one token each
    slots = np.concatenate([np.arange(B), B + 1 + np.arange(B - 1), 2 * B + 1 + np.arange(2), 3 * B + np.arange(B),
                            4 * B + 2 + np.arange(2), [5 * B, 6 * B + 3]]).astype(np.int64)
    T = len(slots)
    x = Inputs(cuda_device, T, H, Hkv, d, B, dtype, B + d, rot, NB=NB, strided=False)
    block = slots // B
    k, v = x.k.clone(), x.v.clone()
    k[1], v[0] = math.nan, math.nan                             # whole tokens
    k[B, 1], v[B + 1, 2], k[B + 2, 0, :32] = math.nan, math.nan, math.nan       # a head's row; the first part of one
    v[torch.from_numpy(block == 2)] = math.nan
    for b in (3, 4):
        k[torch.from_numpy(block == b)] = v[torch.from_numpy(block == b)] = math.nan
    k[-1] = v[-2] = math.nan
    k0, v0, s0 = _random_cache8(NB, Hkv, B, d, B)
    kc, vc, sc = k0.to(cuda_device), v0.to(cuda_device), s0.to(cuda_device)
    dk, dv = k.to(cuda_device), v.to(cuda_device)
    args = (x.dq, dk, dv, x.dcs, x.dpos) if rot else (None, dk, dv, None, None)
    pkv.kv_rotary_and_cache_fp8(*args, kc, vc, sc, torch.from_numpy(slots).to(cuda_device), layout=layout)
    pkv.check()
    ref = RefCache8(k0, v0, s0)
    ref.append(rotate32(k, x.cs, x.positions, rot, layout).numpy(), v.float().numpy(), slots)
    _same8(ref, kc, vc, sc, "NaN rows")


def test_chunks_of_a_long_prompt_hold_a_bounded_workspace(cuda_device):
    H, Hkv, d, B, chunk, n = 4, 2, 64, 16, 128, 64
    eng = PagedKVCache(n * chunk // B, Hkv, d, B, F8, cuda_device, n * chunk // B)
    seq = eng.new_sequence(0)
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(chunk, h, d, generator=g).half().to(cuda_device) for h in (H, Hkv, Hkv))
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(n):
        eng.prefill(q, k, v, eng.upload_prefill(eng.plan_prefill([seq], [chunk])), out=out)
    pkv.check()
    need = pkv.paged_attention_prefill_fp8_workspace_size(1, Hkv, d, B, n * chunk)
    assert torch.cuda.memory_allocated() - before <= 2 * need


def test_growing_calls_without_a_workspace_hold_a_bounded_one(cuda_device):
    H, Hkv, d, B, NB = 2, 2, 128, 16, 2048
    kc, vc = (torch.zeros(NB, Hkv, B, d, device=cuda_device).to(F8) for _ in range(2))
    sc = pkv.kv_scales(NB, Hkv, cuda_device)
    q = torch.randn(8, H, d, device=cuda_device).half()
    out = torch.empty_like(q)
    bt = torch.arange(NB, dtype=torch.int32, device=cuda_device)[None]
    start = torch.tensor([0, 8], dtype=torch.int32, device=cuda_device)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for n in range(512, NB * B + 1, 512):
        pkv.paged_attention_prefill_fp8(out, q, kc, vc, sc, bt, torch.tensor([n], dtype=torch.int32, device=cuda_device), start,
                                        max_context_len=n)
    pkv.check()
    need = pkv.paged_attention_prefill_fp8_workspace_size(1, Hkv, d, B, NB * B)
    assert torch.cuda.memory_allocated() - before <= 2 * need


def test_a_captured_call_keeps_its_workspace(cuda_device):
    """A graph replays into the workspace that it was captured with, after larger calls have taken another."""
    eng = PagedKVCache(600, 2, 64, 16, F8, cuda_device, 300)
    for pool in eng._pools():
        pool.zero_()
    g = torch.Generator().manual_seed(1)
    seqs = [eng.new_sequence(0), eng.new_sequence(0)]
    new = lambda n: [torch.randn(n, h, 64, generator=g).half().to(cuda_device) for h in (4, 2, 2)]  # noqa: E731
    small = eng.upload_prefill(eng.plan_prefill(seqs, [70, 50]))
    q, k, v = new(120)
    eng.prefill(q, k, v, small)
    small.pairs = small.pairs[:0]
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eng.prefill(q, k, v, small, out=out)
    graph.replay()
    torch.cuda.synchronize()
    first = out.clone()
    eng.prefill(*new(4000), eng.upload_prefill(eng.plan_prefill([eng.new_sequence(0)], [4000])))
    junk = [torch.full((1 << 18,), 0xFF, dtype=torch.uint8, device=cuda_device) for _ in range(64)]
    out.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    pkv.check()
    assert torch.equal(out, first) and all(bool((x == 0xFF).all()) for x in junk)


def test_layers_that_share_a_workspace_give_what_they_give_alone(cuda_device):
    g = torch.Generator().manual_seed(2)
    make = lambda **kw: PagedKVCache(64, 2, 64, 16, F8, cuda_device, 32, **kw)  # noqa: E731
    first = make()
    shared, alone = [first, make(workspace_of=first)], [make(), make()]
    new = lambda n: [torch.randn(n, h, 64, generator=g).half().to(cuda_device) for h in (4, 2, 2)]  # noqa: E731
    seqs = [c.new_sequence(0) for c in shared + alone]
    for n in (40, 300, 1):
        inputs = [new(n), new(n)]                           # of the two layers
        outs = []
        for i, c in enumerate(shared + alone):
            if n == 1:
                outs.append(c.decode(*inputs[i % 2], c.upload(c.plan_step([seqs[i]]))))
            else:
                outs.append(c.prefill(*inputs[i % 2], c.upload_prefill(c.plan_prefill([seqs[i]], [n]))))
        pkv.check()
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert shared[1]._workspace(0) is first._workspace(0)


def test_prefill_of_large_fp16_numbers(cuda_device):
    """Cached numbers past fp16's range (65,504 in 8 bits is 65,536; a turned pair of them reaches 92,682) leave earlier
    rows of the same tiles as they are, and keys keep their scores: the prompt phase gives what the definition gives."""
    H, Hkv, d, B, T = 2, 1, 64, 16, 100
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(T, Hkv, d, generator=g).half() for _ in range(2))
    q = (torch.randn(T, H, d, generator=g) * 2.0 ** -10).half()
    # rows 40 and 70 turn by an eighth of a turn: (65504, 65504) becomes (0, 92637)
    cs = torch.zeros(2, d // 2, 2)
    cs[0, :, 0] = 1.0
    cs[1] = math.sqrt(0.5)
    pos = torch.zeros(T, dtype=torch.int32)
    pos[[40, 70]] = 1
    k[40] = 0
    k[40, 0, 3] = k[40, 0, 3 + d // 2] = 65504
    k[70] = 0
    k[70, 0, 5] = k[70, 0, 5 + d // 2] = -65504
    v[50, 0, 7], v[60, 0, 8], v[70, 0, :4] = 65504, -65504, 64000
    dev = cuda_device
    kc, vc = (torch.zeros(8, Hkv, B, d, device=dev).to(F8) for _ in range(2))
    sc = pkv.kv_scales(8, Hkv, dev)
    pkv.kv_rotary_and_cache_fp8(None, k.to(dev), v.to(dev), cs.to(dev), pos.to(dev), kc, vc, sc, torch.arange(T, device=dev))
    ref = RefCache8(kc, vc, sc)
    assert np.abs(ref.values(0)).max() > 85000 and np.abs(ref.values(1)).max() == 65536
    out = torch.empty(T, H, d, dtype=torch.float16, device=dev)
    tables = np.arange(8, dtype=np.int32)[None, :7]
    pkv.paged_attention_prefill_fp8(out, q.to(dev), kc, vc, sc, torch.from_numpy(tables).to(dev),
                                    torch.tensor([T], dtype=torch.int32, device=dev),
                                    torch.tensor([0, T], dtype=torch.int32, device=dev))
    pkv.check()
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    for lo, hi in ((0, 40), (40, 50), (50, T)):             # rows by the numbers that they may see
        want, mag, vmax = attention64(q[lo:hi].double().numpy(), ref.values(0), ref.values(1), tables[0], hi, 1 / math.sqrt(d))
        # beside the probabilities' 11 bits, 65,536 itself is off by half a step of fp16 (2^-11)
        tol = attention_tolerance(want, mag, vmax, hi, d, torch.finfo(q.dtype).eps, 10)
        assert np.all(np.abs(got[lo:hi] - want) <= tol), (lo, np.abs(got[lo:hi] - want).max())


def _prefill(c, new, dtype, seed=1):
    """The prompt phase over a Case8 of the last new[s] tokens of each sequence: outputs, queries and where they start."""
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.randn(int(start[-1]), c.H, c.d, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])
    out = torch.empty(q.shape, dtype=q.dtype, device=c.dev)
    pkv.paged_attention_prefill_fp8(out, q.to(c.dev), c.kc, c.vc, c.sc, c.dt_, c.dc, torch.from_numpy(start).to(c.dev))
    pkv.check()
    return out.double().cpu().numpy(), q.double().numpy(), start


@pytest.mark.parametrize("dtype,scale_exp,free", [("bf16", (-11, -8), True), ("f16", (-11, -8), True), ("f16", (-20, -14), False),
                                                  ("bf16", (-40, -14), False)])
def test_prefill_rounds_what_16_bits_do_not_hold(cuda_device, dtype, scale_exp, free):
    """Scales that are no powers of two, and in fp16 scales whose least codes lie below its range."""
    new, ctx = (3, 40, 150), (30, 40, 400)
    c = Case8(cuda_device, ctx, 4, 2, 64, 16, dtype, seed=40, scale_exp=scale_exp, free_scales=free)
    got, q, start = _prefill(c, new, dtype)
    eps, s = torch.finfo(DT[dtype]).eps, 1 / math.sqrt(64)
    for i, n in enumerate(ctx):
        rows = slice(int(start[i]), int(start[i + 1]))
        want, mag, vmax = attention64(q[rows], c.kvals, c.vvals, c.tables[i], n, s)
        # each key and value off by half a step of 16 bits: eps / 2 of itself, or in fp16 half of 2^-23 and 2^-24
        dx = (eps / 2 * mag if free else 0) + (2.0 ** -24 * s * np.abs(q[rows]).sum(-1).max() if dtype == "f16" else 0)
        dv = (eps / 2 * vmax if free else 0) + (2.0 ** -25 if dtype == "f16" else 0)
        tol = attention_tolerance(want, mag, vmax, n, 64, eps, 11 if dtype == "f16" else 15) + vmax * math.expm1(2 * dx) + dv
        tol = tol + (2.0 ** -25 if dtype == "f16" else 0)                     # the output's own least step
        assert np.all(np.abs(got[rows] - want) <= tol), (i, np.abs(got[rows] - want).max())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prefill_nan_in_the_context_shows(cuda_device, dtype):
    """In the rows that see it and in no other sequence or kv head."""
    c = Case8(cuda_device, (200, 200, 200), 4, 2, 64, 16, dtype, seed=41)
    c.kc.view(torch.uint8)[int(c.tables[0, 3]), 0, 2, 5] = 0x7F            # token 50
    c.vc.view(torch.uint8)[int(c.tables[1, 3]), 1, 2, 9] = 0x7F
    got, _, start = _prefill(c, (100, 100, 100), dtype)
    nan = np.isnan(got)
    assert nan[:100, :2].all() and not nan[:100, 2:].any()
    assert nan[100:200, 2:, 9].all() and nan[100:200].sum() == 2 * 100
    assert not nan[200:].any()


def test_decode_in_one_huge_partition(cuda_device):
    """Partition sizes up to the largest number are one partition."""
    c = Case8(cuda_device, (1, 100, 700), 4, 2, 64, 16, seed=3)
    one = c.decode(partition_size=1 << 20)
    for P in (1 << 30, 2 ** 31 - 64):
        assert torch.equal(c.decode(partition_size=P), one)
        pkv.check()
    c.check(one)


def test_16_bit_decode_in_one_huge_partition(cuda_device):
    S, H, Hkv, d, B = 2, 4, 2, 64, 16
    g = torch.Generator().manual_seed(0)
    kc, vc = (torch.randn(20, Hkv, B, d, generator=g).half().to(cuda_device) for _ in range(2))
    q = torch.randn(S, H, d, generator=g).half().to(cuda_device)
    bt = torch.arange(20, dtype=torch.int32, device=cuda_device).view(2, 10)
    cl = torch.tensor([3, 150], dtype=torch.int32, device=cuda_device)
    a, b = torch.empty_like(q), torch.empty_like(q)
    pkv.paged_attention_decode(a, q, kc, vc, bt, cl, partition_size=1 << 20)
    pkv.paged_attention_decode(b, q, kc, vc, bt, cl, partition_size=2 ** 31 - 32)
    pkv.check()
    assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [True, False])
def test_sequences_without_tokens_attend_to_nothing(cuda_device, fp8):
    eng = PagedKVCache(70, 2, 64, 16, F8 if fp8 else torch.float16, cuda_device, 64)
    seqs = [eng.new_sequence(0) for _ in range(3)]
    step = eng.upload(eng.plan_tables(seqs))
    q = torch.ones(3, 4, 64, dtype=torch.float16, device=cuda_device)
    out = eng.attend(q, step, out=torch.full_like(q, 5.0))
    pkv.check()
    assert not bool(out.any())
    kv = torch.zeros(0, 2, 64, dtype=torch.float16, device=cuda_device)
    out.fill_(5.0)
    eng.prepare(q, kv, kv, step, out)()
    pkv.check()
    assert not bool(out.any())


@pytest.mark.parametrize("parts", [31, 32, 33])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_merges_on_both_sides_of_its_two_kernels(cuda_device, parts, d):
    """Splits of up to 32 partitions take a warp each, longer ones a CTA; shorter contexts beside them."""
    c = Case8(cuda_device, (64 * parts, 64 * parts - 63, 64 * parts - 64, 65, 64, 0), 8, 2, d, 16, "bf16", seed=parts)
    out = c.decode(partition_size=64)
    pkv.check()
    c.check(out)


def test_decode_launches_of_512_sequences(cuda_device):
    """Split contexts at the last and first sequences of the launches that a large batch takes."""
    rng = np.random.default_rng(5)
    ctx = rng.integers(0, 20, 1200)
    at = [0, 1, 510, 511, 512, 513, 1022, 1023, 1024, 1025, 1199]
    ctx[at] = rng.integers(100, 900, len(at))
    c = Case8(cuda_device, ctx, 4, 2, 64, 8, seed=12)
    out = c.decode(partition_size=64)
    pkv.check()
    c.check(out, seqs=at + [2, 509, 514, 1021, 1026, 1198])


@pytest.mark.parametrize("n,rot", [(33, 48), (1, 16), (2049, 128), (5000, 256)])
def test_table_rows_are_on_the_unit_circle_and_nothing_else_is_written(cuda_device, n, rot):
    """Cosine and sine are each off by under 2^-22 (see test_gpu_rotary's test_table), so their squares' sum by under
    2 sqrt(2) times that and its own rounding."""
    buf = torch.full((n + 7, rot // 2, 2), 7.0, device=cuda_device)
    pkv.rotary_table(n, rot, out=buf[:n])
    pkv.check()
    off = (buf[:n].double().square().sum(-1) - 1).abs()
    assert float(off.max()) < 3 * 2.0 ** -22 and bool((buf[n:] == 7.0).all())
    assert bool((buf[0, :, 0] == 1).all()) and bool((buf[0, :, 1] == 0).all())


def test_a_plain_8_bit_cache_takes_slices_of_keys_and_values(cuda_device):
    """Without rotary positions the queries go to the attention as they are, which takes them contiguous."""
    eng = PagedKVCache(16, 2, 64, 16, F8, cuda_device, 8)
    seq = eng.new_sequence(0)
    qkv = torch.randn(20, 8, 64, generator=torch.Generator().manual_seed(3)).half().to(cuda_device)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    step = eng.upload_prefill(eng.plan_prefill([seq], [20]))
    out = eng.prefill(q.contiguous(), k, v, step)
    with pytest.raises(ValueError, match="contiguous"):
        eng.prefill(q, k, v, step)
    other = PagedKVCache(16, 2, 64, 16, F8, cuda_device, 8)
    step2 = other.upload_prefill(other.plan_prefill([other.new_sequence(0)], [20]))
    assert torch.equal(out, other.prefill(q.contiguous(), k.contiguous(), v.contiguous(), step2))
    pkv.check()


@pytest.mark.parametrize("fp8", [True, False])
def test_steps_after_a_reported_timeout_are_whole(cuda_device, fp8):
    """A call that gives up waiting may leave its workspace's counters mid-count (written here by hand, with the self-test's
    timeout beside them): once check has reported it, the engine's and the bindings' own workspaces serve again."""
    S, H, Hkv, d, B, n = 40, 4, 2, 64, 16, 700
    g = torch.Generator().manual_seed(4)
    eng = PagedKVCache(S * 45, Hkv, d, B, F8 if fp8 else torch.float16, cuda_device, 45)
    seqs = [eng.new_sequence(0) for _ in range(S)]
    new = [torch.randn(S * n, h, d, generator=g).half().to(cuda_device) for h in (H, Hkv, Hkv)]
    eng.prefill(*new, eng.upload_prefill(eng.plan_prefill(seqs, [n] * S)))
    step = eng.upload(eng.plan_tables(seqs))
    q = torch.randn(S, H, d, generator=g).half().to(cuda_device)
    out = torch.empty_like(q)
    none = new[1][:0]
    prep = eng.prepare(q, none, none, step, out, partition_size=64)
    if fp8:
        own = lambda o: pkv.paged_attention_decode_fp8(o, q, eng.key_cache, eng.value_cache, eng.scales, step.tables,  # noqa: E731
                                                       step.context_lens, partition_size=64)
    else:
        own = lambda o: pkv.paged_attention_decode(o, q, eng.key_cache, eng.value_cache, step.tables, step.context_lens,  # noqa: E731
                                                   partition_size=64)
    prep()
    want = out.clone()
    assert torch.equal(own(torch.empty_like(q)), want)
    pkv.check()
    bindings = pkv._ws8_cache[0]._buf if fp8 else pkv._ws_cache[torch.device("cuda", 0)]
    for ws in (eng._workspace(0), bindings):
        ws[:8].view(torch.int32).copy_(torch.tensor([50, 3], dtype=torch.int32))         # tickets taken, pipelines done
    torch.cuda.synchronize()
    L = pkv.load()
    assert L.pkv_selftest_wait_timeout(100000, torch.cuda.current_stream().cuda_stream) == 0
    with pytest.raises(pkv.PkvError) as e:
        pkv.check()
    assert e.value.status_name == "PKV_ETIMEOUT"
    out.fill_(5.0)
    prep()
    mine = own(torch.full_like(q, 5.0))
    pkv.check()
    assert torch.equal(out, want) and torch.equal(mine, want)
