"""Block tables, context slots and the paged append on the GPU."""
import numpy as np
import pytest

import csa2_synth as syn
from tests import _verify as V
from tests._cases import bf16_dev, bf16_host, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import compressed_sparse_attention_step_gb300 as c  # noqa: E402


def _pool(g, old, P, mp, spare):
    B = len(old)
    held = [V.pages(o, P) for o in old]
    perm = g.permutation(sum(held) + spare).astype(np.int32)
    table = np.full((B, mp), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(B * mp + spare, -9, np.int32)
    free[:spare] = perm[at:]
    return table, free


def _run(old, new, P, table, free, state, n_new):
    granted = torch.full((len(old),), -5, dtype=torch.int32, device="cuda")
    slots = torch.full((len(old), n_new), -5, dtype=torch.int32, device="cuda") if n_new else None
    c.csa2_block_tables(to_dev(np.array(old, np.int32)), to_dev(np.array(new, np.int32)), P, table, free, state, granted,
                        slots=slots)
    return granted, slots


@pytest.mark.parametrize("B,P,mp,n_new,spare,kind", [
    (1, 16, 1, 1, 1, "mix"), (1, 64, 4, 3, 0, "mix"), (5, 16, 9, 20, 4, "mix"), (33, 32, 12, 7, 1000, "grow"),
    (300, 16, 20, 70, 900, "mix"), (1025, 16, 6, 9, 40, "mix"), (64, 64, 70, 4096, 2000, "admit"),
    (8192, 16, 3, 2, 100, "mix"), (40, 1024, 3, 5, 3, "shrink"), (7, 128, 4, 0, 9, "mix"),
])
def test_block_tables(B, P, mp, n_new, spare, kind):
    g = np.random.default_rng(B * 1000 + P)
    cap = mp * P
    old = g.integers(0, cap + 1, B) if kind != "admit" else np.zeros(B, np.int64)
    if kind == "grow":
        new = np.minimum(old + g.integers(0, n_new + 1, B), cap + 3)          # some past the table
    elif kind == "shrink":
        new = (old * g.random(B)).astype(np.int64)
    elif kind == "admit":
        new = g.integers(1, n_new + 1, B)
    else:
        new = np.where(g.random(B) < 0.3, g.integers(0, cap + 1, B), np.minimum(old + g.integers(0, 2 * P, B), cap))
    old, new = old.tolist(), new.tolist()
    table, free = _pool(g, old, P, mp, spare)
    dt, df = to_dev(table), to_dev(free)
    state = torch.tensor([spare, 0, 0, 0], dtype=torch.int32, device="cuda")
    c.csa2_device_flags()
    granted, slots = _run(old, new, P, dt, df, state, n_new)
    flags = c.csa2_device_flags()
    lt, lf = table.tolist(), free.tolist()
    eg, es, n = V.block_tables(old, new, P, lt, lf, spare, n_new)
    assert granted.tolist() == eg
    assert (slots.tolist() if n_new else es) == es
    assert dt.tolist() == lt and df.tolist() == lf and state.tolist() == [n, 0, 0, 0]
    assert flags == (c.FLAG_PAGES_OUT if eg != new else 0)
    # the undo gives every page back where it was
    undone, _ = _run(eg, old, P, dt, df, state, 0)
    eu, _, n = V.block_tables(eg, old, P, lt, lf, n, 0)
    assert undone.tolist() == old == eu and state.tolist() == [spare, 0, 0, 0]
    assert df.tolist()[:spare] == free[:spare].tolist()
    for b in range(B):
        h = V.pages(old[b], P)
        assert dt[b, :h].tolist() == table[b, :h].tolist()
    assert c.csa2_device_flags() == 0


def test_block_tables_bad_lengths():
    """Negative lengths count as 0, an old length past the table as its end, bad page numbers give slot -1."""
    table = torch.tensor([[3, 4], [5, -1], [6, 7]], dtype=torch.int32, device="cuda")
    free = torch.tensor([9, 8, -2, 0], dtype=torch.int32, device="cuda")
    state = torch.tensor([3, 0, 0, 0], dtype=torch.int32, device="cuda")
    c.csa2_device_flags()
    granted, slots = _run([-3, 16, 1000], [-1, 18, 32], 16, table, free, state, 4)
    assert granted.tolist() == [0, 18, 32]
    assert slots.tolist() == [[-1] * 4, [-1] * 4, [-1] * 4]       # sequence 1's new page is number -2
    assert c.csa2_device_flags() == c.FLAG_INDEX_OOB
    assert state.tolist() == [2, 0, 0, 0]


def test_block_tables_captured_and_on_another_stream():
    g = np.random.default_rng(5)
    B, P, mp = 50, 16, 8
    old = g.integers(0, mp * P - 8, B).tolist()
    new = [o + 8 for o in old]
    table, free = _pool(g, old, P, mp, 60)
    dt, df = to_dev(table), to_dev(free)
    state = torch.tensor([60, 0, 0, 0], dtype=torch.int32, device="cuda")
    do, dn = to_dev(np.array(old, np.int32)), to_dev(np.array(new, np.int32))
    granted, undone = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    slots = torch.empty((B, 8), dtype=torch.int32, device="cuda")

    def step():
        c.csa2_block_tables(do, dn, P, dt, df, state, granted, slots=slots)
        c.csa2_block_tables(granted, do, P, dt, df, state, undone)
    lt, lf = table.tolist(), free.tolist()
    _, es, _ = V.block_tables(old, new, P, lt, lf, 60, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert slots.tolist() == es
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        slots.fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        assert slots.tolist() == es and state.tolist() == [60, 0, 0, 0]


@pytest.mark.parametrize("B,N,P,T,extra,paged,drafts", [
    (1, 1, 16, 0, 0, True, True), (1, 5, 16, 1, 3, True, True), (3, 64, 64, 300, 5, True, True), (2, 7, 32, 4096, 0, True, True),
    (4, 3, 128, 999, 2, False, True), (3, 2, 16, 65, 1, True, False), (2, 9, 1024, 2000, 7, True, True),
])
def test_context_slots(B, N, P, T, extra, paged, drafts):
    g = np.random.default_rng(B * 100 + N)
    lens = g.integers(0, T + 1, B)
    lens[0] = T
    nn = g.integers(0, N + 1, B)
    nn[0] = N
    parent = V.random_parents(g, B, N)
    mp = V.pages(T + N, P)
    table = g.permutation(B * mp).astype(np.int32).reshape(B, mp)
    ld = T + N + extra
    slots = torch.full((B * N, ld), -5, dtype=torch.int32, device="cuda")
    ns = torch.full((B * N,), -5, dtype=torch.int32, device="cuda")
    c.csa2_device_flags()
    c.csa2_context_slots(to_dev(lens.astype(np.int32)), slots, ns, block_table=to_dev(table) if paged else None,
                         page_size=P if paged else 0, parent=to_dev(parent) if drafts else None,
                         n_nodes=to_dev(nn.astype(np.int32)))
    exp = np.full((B * N, ld), -1, np.int64)
    en = np.zeros(B * N, np.int64)
    for b in range(B):
        for i in range(int(nn[b])):
            pos = np.concatenate((np.arange(lens[b]), [lens[b] + j for j in V.path(parent[b], i)] if drafts else []))
            pos = pos.astype(np.int64)
            exp[b * N + i, :len(pos)] = table[b][pos // P].astype(np.int64) * P + pos % P if paged else pos
            en[b * N + i] = len(pos)
    assert np.array_equal(slots.cpu().numpy(), exp) and np.array_equal(ns.cpu().numpy(), en)
    assert c.csa2_device_flags() == 0


def test_context_slots_flags():
    """A list that does not fit is cut, a position past the table is -1, a parent out of order a root."""
    lens = torch.tensor([30], dtype=torch.int32, device="cuda")
    table = torch.tensor([[2]], dtype=torch.int32, device="cuda")
    slots = torch.empty((2, 20), dtype=torch.int32, device="cuda")
    ns = torch.empty(2, dtype=torch.int32, device="cuda")
    parent = torch.tensor([[-1, 1]], dtype=torch.int32, device="cuda")
    c.csa2_device_flags()
    c.csa2_context_slots(lens, slots, ns, block_table=table, page_size=16, parent=parent)
    row = list(range(32, 48)) + [-1] * 4
    assert slots.tolist() == [row, row] and ns.tolist() == [20, 20]
    assert c.csa2_device_flags() == c.FLAG_INDEX_OOB
    lens.fill_(3)
    c.csa2_context_slots(lens, slots, ns, block_table=table, page_size=16, parent=parent)
    assert slots.tolist() == [[32, 33, 34, 35] + [-1] * 16, [32, 33, 34, 36] + [-1] * 16] and ns.tolist() == [4, 4]
    assert c.csa2_device_flags() == c.FLAG_INDEX_OOB


@pytest.mark.parametrize("n,S,what", [(1, 4, "both"), (37, 100, "both"), (513, 600, "kv"), (64, 64, "ki")])
def test_paged_append(orc, n, S, what):
    g = np.random.default_rng(n)
    kv, ki = syn.outlier_bf16(n, syn.T_X, 0, (n, 512)), syn.normal_bf16(n, syn.T_KI_NEW, 0, (n, 128))
    slots = g.permutation(S)[:n].astype(np.int32)
    if n > 1:
        slots[g.random(n) < 0.2] = -1
        slots[0], slots[1] = S, S + 7          # outside the pool
    codes = torch.full((S, 256), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((S, 32), 0x5A, dtype=torch.uint8, device="cuda")
    KI = torch.full((S, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ec, es = orc.fp4_quantize(kv)
    rc, rs, rk = codes.cpu().numpy(), scales.cpu().numpy(), bf16_host(KI)
    ok = (slots >= 0) & (slots < S)
    if what != "ki":
        rc[slots[ok]], rs[slots[ok]] = ec[ok], es[ok]
    if what != "kv":
        rk[slots[ok]] = ki[ok]
    c.csa2_device_flags()
    kw = {}
    if what != "ki":
        kw.update(kv_new=bf16_dev(kv), codes=codes, scales=scales)
    if what != "kv":
        kw.update(ki_new=bf16_dev(ki), KI=KI)
    c.csa2_paged_append(to_dev(slots), **kw)
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(bf16_host(KI), rk)
    assert c.csa2_device_flags() == (c.FLAG_APPEND_OOB if n > 1 else 0)


def test_paged_append_every_value_scale_and_tie(orc):
    """The paged append's codes are the oracle's for every finite bf16 value against 16 group maxima, every
    positive maximum, and, under every scale, every midpoint of two codes with its neighbours."""
    from tests.test_gpu_fp4 import _sweep_rows
    rows = [_sweep_rows()]
    ties = []
    for sb in range(1, 0x7F):
        s = V.e4m3(np.uint8(sb))
        mids = syn.f32_to_bf16_bits((np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5]) * s).astype(np.float32)).astype(np.int64)
        top = int(syn.f32_to_bf16_bits(np.array([6 * s], np.float32))[0])      # makes the scale s, exactly
        for sign in (0, 0x8000):
            ties.append([top] + [(v | sign) for v in mids] + [(v - 1) | sign for v in mids] + [top | sign])
            ties.append([top] + [(v + 1) | sign for v in mids] + [0, 0x8000] + [(v | (sign ^ 0x8000)) for v in mids[:6]])
    ties = np.array(ties, np.int64).astype(np.uint16)
    pad = np.zeros(((-len(ties)) % 32, 16), np.uint16)
    rows.append(np.concatenate((ties, pad)).reshape(-1, 512))
    x = np.concatenate(rows)
    n = x.shape[0]
    codes = torch.zeros((n, 256), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((n, 32), dtype=torch.uint8, device="cuda")
    order = np.random.default_rng(8).permutation(n).astype(np.int32)
    c.csa2_paged_append(to_dev(order), kv_new=bf16_dev(x), codes=codes, scales=scales)
    ec, es = orc.fp4_quantize(x)
    assert np.array_equal(scales.cpu().numpy()[order], es)
    assert np.array_equal(codes.cpu().numpy()[order], ec)
    ref_c, ref_s = torch.empty((1, n, 256), dtype=torch.uint8, device="cuda"), torch.empty((1, n, 32), dtype=torch.uint8, device="cuda")
    c.csa2_fp4_quantize_append(bf16_dev(x)[None], ref_c, ref_s)
    assert torch.equal(codes[to_dev(order).long()], ref_c[0]) and torch.equal(scales[to_dev(order).long()], ref_s[0])


@pytest.mark.parametrize("kv_off,ki_off", [(8, 0), (16, 8), (24, 8)])
def test_paged_append_sources_at_any_16_bytes(kv_off, ki_off):
    """Sources that start on 16 bytes and no more (a view into a larger buffer) append the same bytes."""
    g = torch.Generator(device="cuda").manual_seed(kv_off)
    n, n_slots = 37, 64
    kv = torch.randn((n, 512), generator=g, device="cuda").bfloat16()
    ki = torch.randn((n, 128), generator=g, device="cuda").bfloat16()
    order = torch.randperm(n_slots, generator=g, device="cuda")[:n].int()
    got = []
    for a, b in ((0, 0), (kv_off, ki_off)):
        src = torch.zeros(n * 512 + 32, dtype=torch.bfloat16, device="cuda")[a:a + n * 512].view(n, 512).copy_(kv)
        key = torch.zeros(n * 128 + 32, dtype=torch.bfloat16, device="cuda")[b:b + n * 128].view(n, 128).copy_(ki)
        codes, scales = (torch.zeros((n_slots, w), dtype=torch.uint8, device="cuda") for w in (256, 32))
        KI = torch.zeros((n_slots, 128), dtype=torch.bfloat16, device="cuda")
        c.csa2_paged_append(order, kv_new=src, codes=codes, scales=scales, ki_new=key, KI=KI)
        got.append((codes, scales, KI))
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert torch.equal(got[0][2][order.long()], ki)


def test_paged_append_of_infinities_and_nan():
    """Infinities and NaN (any payload, any channel) are stored as csa2_fp4_quantize_append stores them."""
    x = np.zeros((64, 512), np.uint16)
    rng = np.random.default_rng(5)
    x[:] = syn.f32_to_bf16_bits(rng.standard_normal(x.shape).astype(np.float32))
    for i, v in enumerate([0x7F80, 0xFF80, 0x7FC0, 0xFFC0, 0x7F81, 0xFFFF, 0x7FFF, 0x7F7F]):
        for j in range(16):
            x[8 * i + j // 2, 16 * j + j::64] = v
    codes, scales = (torch.zeros((64, w), dtype=torch.uint8, device="cuda") for w in (256, 32))
    c.csa2_paged_append(torch.arange(64, dtype=torch.int32, device="cuda"), kv_new=bf16_dev(x), codes=codes, scales=scales)
    ref_c, ref_s = (torch.zeros((1, 64, w), dtype=torch.uint8, device="cuda") for w in (256, 32))
    c.csa2_fp4_quantize_append(bf16_dev(x)[None], ref_c, ref_s)
    assert torch.equal(scales, ref_s[0]) and torch.equal(codes, ref_c[0])


def test_block_tables_a_full_list_loses_pages_with_a_flag():
    """More pages given back than the list holds: the first ones are kept, the rest flagged, none written past it."""
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    free = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    state = torch.zeros(4, dtype=torch.int32, device="cuda")
    c.csa2_device_flags()
    granted, _ = _run([64, 64], [0, 0], 16, table, free[:3], state, 0)
    assert granted.tolist() == [0, 0] and state.tolist() == [3, 0, 0, 0]
    assert free.tolist() == [7, 6, 5, -1, -1, -1]
    assert c.csa2_device_flags() == c.FLAG_INDEX_OOB


def test_binding_refuses_strides_types_and_places():
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, slots, ns = torch.zeros(2, **i32), torch.zeros((2, 8), **i32), torch.zeros(2, **i32)
    with pytest.raises(ValueError, match="contiguous"):
        c.csa2_context_slots(lens, torch.zeros((8, 2), **i32).t(), ns)
    with pytest.raises(TypeError, match="dtype"):
        c.csa2_context_slots(lens.long(), slots, ns)
    with pytest.raises(ValueError, match="CUDA"):
        c.csa2_context_slots(lens.cpu(), slots, ns)
    with pytest.raises(ValueError, match="shape"):
        c.csa2_context_slots(lens, slots, ns[:1])
    with pytest.raises(TypeError):
        c.csa2_context_slots([0, 0], slots, ns)
    with pytest.raises(c.Csa2Error):                      # rows of 16 bytes start at a multiple of 16
        c.csa2_context_slots(lens, torch.zeros(17, **i32)[1:].view(2, 8), ns)
    with pytest.raises(c.Csa2Error):
        c.csa2_block_tables(lens, ns, 24, slots, torch.zeros(4, **i32), torch.zeros(4, **i32), torch.zeros(2, **i32))


def test_no_free_list_and_no_columns():
    """A pool without a free list still moves pages between sequences; lists of no columns count nothing and say so."""
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[5, 3], [-1, -1]], **i32)
    state, granted = torch.zeros(4, **i32), torch.zeros(2, **i32)
    c.csa2_device_flags()
    c.csa2_block_tables(torch.tensor([32, 0], **i32), torch.tensor([16, 16], **i32), 16, table, torch.empty(0, **i32), state,
                        granted)
    assert granted.tolist() == [16, 16] and table[1].tolist() == [3, -1] and state.tolist() == [0, 0, 0, 0]
    assert c.csa2_device_flags() == 0
    n = torch.full((2,), -5, **i32)
    c.csa2_context_slots(torch.tensor([0, 0], **i32), torch.empty((2, 0), **i32), n)
    assert n.tolist() == [0, 0] and c.csa2_device_flags() == 0
    c.csa2_context_slots(torch.tensor([0, 3], **i32), torch.empty((2, 0), **i32), n)
    assert n.tolist() == [0, 0] and c.csa2_device_flags() == c.FLAG_INDEX_OOB


def test_paged_append_into_far_rows():
    """Rows whose byte offsets pass 32 bits hold what near rows hold."""
    n, n_slots = 48, (1 << 24) + 64
    g = torch.Generator(device="cuda").manual_seed(2)
    kv = torch.randn((n, 512), generator=g, device="cuda").bfloat16()
    ki = torch.randn((n, 128), generator=g, device="cuda").bfloat16()
    codes, scales = (torch.empty((n_slots, w), dtype=torch.uint8, device="cuda") for w in (256, 32))
    KI = torch.empty((n_slots, 128), dtype=torch.bfloat16, device="cuda")
    for first in (0, (1 << 24) + 64 - n):
        c.csa2_paged_append(torch.arange(first, first + n, dtype=torch.int32, device="cuda"), kv_new=kv, codes=codes,
                            scales=scales, ki_new=ki, KI=KI)
    assert torch.equal(codes[:n], codes[-n:]) and torch.equal(scales[:n], scales[-n:])
    assert torch.equal(KI[-n:], ki) and torch.equal(KI[:n], ki)


def test_context_slots_of_many_long_rows():
    """Lists of more than 2^31 entries together."""
    B, N, T = 33, 64, 1_050_000
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    parent = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").repeat(B, 1)
    slots = torch.empty((B * N, T + N), dtype=torch.int32, device="cuda")
    assert slots.numel() > 2 ** 31
    n_slots = torch.empty(B * N, dtype=torch.int32, device="cuda")
    c.csa2_device_flags()
    c.csa2_context_slots(lens, slots, n_slots, parent=parent)
    want = torch.arange(T + N, dtype=torch.int32, device="cuda")
    for r in (0, N - 1, B * N - N, B * N - 2, B * N - 1):
        k = T + r % N + 1
        assert int(n_slots[r]) == k and torch.equal(slots[r, :k], want[:k]) and bool((slots[r, k:] == -1).all())
    assert c.csa2_device_flags() == 0


def test_block_tables_of_the_widest_lists():
    """Lists of 2^31 - 1 columns, the most that the call takes: every column is written, the last ones too."""
    n_new = 2 ** 31 - 1
    i32 = dict(dtype=torch.int32, device="cuda")
    table, free = torch.full((1, 4), -1, **i32), torch.tensor([9, 5, 7], **i32)
    state, granted = torch.tensor([3, 0, 0, 0], **i32), torch.zeros(1, **i32)
    slots = torch.full((1, n_new), -5, **i32)
    c.csa2_device_flags()
    c.csa2_block_tables(torch.tensor([0], **i32), torch.tensor([40], **i32), 16, table, free, state, granted, slots=slots)
    want = [p * 16 + i for p in (7, 5, 9) for i in range(16)][:40]
    assert granted.tolist() == [40] and slots[0, :40].tolist() == want
    for a in range(40, n_new, 1 << 28):
        assert bool((slots[0, a:a + (1 << 28)] == -1).all())
    assert state.tolist() == [0, 0, 0, 0] and c.csa2_device_flags() == 0
