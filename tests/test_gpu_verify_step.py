"""The verify step's operators together, as a serving program runs them: pages for the drafts, the append,
the drafted nodes' candidates, the indexer and the Top-K over the pool, the tree attention, an output
projection with a 4-bit weight, and the pages of the rejected drafts back.  Each node is checked against the
oracle's decode of its own path: the same selection, bit for bit, and the same attention."""
import numpy as np
import pytest

import csa2_synth as syn
from tests import _verify as V
from tests._cases import SCALE, assert_attn_close, bf16_dev, bf16_host, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import compressed_sparse_attention_step_gb300 as c  # noqa: E402


def test_verify_step(orc):
    g = np.random.default_rng(17)
    B, N, P, K, W, mp = 3, 6, 16, 64, 24, 40
    lens = [500, 37, 0]
    n_nodes = [6, 6, 4]
    parent = np.array([[-1, 0, 0, 1, -1, 4], [-1, 0, 1, 2, 3, 4], [-1, -1, 0, 2, 3, 4]], np.int32)
    n_pages = 60
    S = n_pages * P
    # the committed rows and the drafts' (FP4 main KV, indexer keys, window rows)
    kv = [syn.normal_bf16(1, syn.T_KV, b, (lens[b] + N, 512)) for b in range(B)]
    ki = [syn.normal_bf16(1, syn.T_KI, b, (lens[b] + N, 128)) for b in range(B)]
    swa = np.stack([syn.normal_bf16(1, syn.T_SWA, b, (W - 1 + N, 512)) for b in range(B)])
    q = np.stack([syn.normal_bf16(1, syn.T_Q, b, (N, 16, 512)) for b in range(B)])
    qI = np.stack([syn.normal_bf16(1, syn.T_QI, b, (N, 4, 128)) for b in range(B)])
    w = np.stack([syn.normal_f32(1, syn.T_W, b, (N, 4)) for b in range(B)])

    codes = torch.zeros((S, 256), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((S, 32), dtype=torch.uint8, device="cuda")
    KI = torch.full((S, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    free = to_dev(g.permutation(n_pages).astype(np.int32))
    state = torch.tensor([n_pages, 0, 0, 0], dtype=torch.int32, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    d_lens, d_nodes, d_parent = to_dev(np.array(lens, np.int32)), to_dev(np.array(n_nodes, np.int32)), to_dev(parent)
    granted, drafted, accepted = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(3))
    c.csa2_device_flags()

    def append(slots, rows):
        rows_kv = np.concatenate([kv[b][r] for b, r in rows])
        rows_ki = np.concatenate([ki[b][r] for b, r in rows])
        c.csa2_paged_append(slots, kv_new=bf16_dev(rows_kv), codes=codes, scales=scales, ki_new=bf16_dev(rows_ki), KI=KI)

    # the prompts: a padded batch
    slots0 = torch.empty((B, max(lens)), dtype=torch.int32, device="cuda")
    c.csa2_block_tables(zero, d_lens, P, table, free, state, granted, slots=slots0)
    pad = [(b, np.concatenate((np.arange(lens[b]), np.zeros(max(lens) - lens[b], np.int64)))) for b in range(B)]
    append(slots0.view(-1), pad)
    # the drafts
    slots1 = torch.empty((B, N), dtype=torch.int32, device="cuda")
    c.csa2_block_tables(granted, d_lens + d_nodes, P, table, free, state, drafted, slots=slots1)
    append(slots1.view(-1), [(b, lens[b] + np.arange(N)) for b in range(B)])
    assert drafted.tolist() == [a + n for a, n in zip(lens, n_nodes)]

    # selection over the pool as one sequence: candidates and map are the nodes' slots
    ld = max(lens) + N
    cand = torch.empty((B * N, ld), dtype=torch.int32, device="cuda")
    n_cand = torch.empty(B * N, dtype=torch.int32, device="cuda")
    c.csa2_context_slots(d_lens, cand, n_cand, block_table=table, page_size=P, parent=d_parent, n_nodes=d_nodes)
    scores = torch.empty((B * N, ld), dtype=torch.float32, device="cuda")
    n_valid = torch.empty(B * N, dtype=torch.int32, device="cuda")
    c.csa2_index_score(bf16_dev(qI).view(1, B * N, 4, 128), to_dev(w).view(1, B * N, 4), KI[None],
                       torch.tensor([S], dtype=torch.int32, device="cuda"), scores, cand=cand, cand_len=n_cand,
                       q_pos=torch.full((B * N,), S - 1, dtype=torch.int32, device="cuda"), n_valid=n_valid)
    assert torch.equal(n_valid, n_cand)
    idx = torch.empty((B * N, K), dtype=torch.int32, device="cuda")
    n_sel = torch.empty(B * N, dtype=torch.int32, device="cuda")
    c.csa2_topk(scores, K, idx, n_valid=n_valid, map_=cand, n_sel=n_sel)
    out = torch.zeros((B, N, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((B, N, 16), dtype=torch.float32, device="cuda")
    win_len = np.array([min(n, W - 1) for n in lens], np.int32)
    c.csa2_tree_attn(bf16_dev(q), d_parent, codes, scales, idx, out, n_nodes=d_nodes, n_valid=n_sel, swa=bf16_dev(swa),
                     win_len=to_dev(win_len), W=W, softmax_scale=SCALE, lse=lse)

    # every node against the oracle's decode of its path
    cand_h, idx_h, sel_h = cand.cpu().numpy(), idx.cpu().numpy(), n_sel.cpu().numpy()
    for b in range(B):
        ec, es = orc.fp4_quantize(kv[b])
        for i in range(n_nodes[b]):
            r = b * N + i
            p = V.path(parent[b], i)
            pos = np.concatenate((np.arange(lens[b]), lens[b] + np.array(p))).astype(np.int64)
            sc = orc.index_score(qI[b, i], w[b, i], ki[b][pos])
            top, n = orc.topk(sc, K)
            assert n == sel_h[r] and np.array_equal(idx_h[r, :n], cand_h[r, top[:n]])
            d = len(p) - 1
            win = np.concatenate((swa[b, max(d, W - 1 - win_len[b]):W - 1], swa[b, [W - 1 + j for j in p]]))
            o, el = orc.sparse_attn(q[b, i], ec[pos], es[pos], top[:n], win, SCALE)
            assert_attn_close(bf16_host(out[b, i]), o, f"sequence {b} node {i}")
            assert np.abs(lse[b, i].cpu().numpy() - el).max() <= 1e-2
        for i in range(n_nodes[b], N):
            assert (out[b, i] == 0).all()

    # an output projection of the first sequence's heads with a 4-bit weight
    wc, wsc = V.random_fp4(g, 96, 512)
    packed = c.fp4_weight_alloc(96, 512)
    c.csa2_fp4_pack_weight(to_dev(wc), to_dev(wsc), packed)
    y = torch.empty((16, 96), dtype=torch.float32, device="cuda")
    c.csa2_fp4_matvec(out[0, 0], packed, y)
    ref = V.f64(bf16_host(out[0, 0])) @ V.dequant(wc, wsc).T
    assert np.abs(y.cpu().numpy() - ref).max() <= 1e-4 * np.abs(ref).max()

    # two drafts accepted, the rest of the pages back: the pool holds what the accepted lengths need
    c.csa2_block_tables(drafted, d_lens + 2, P, table, free, state, accepted)
    held = sum(V.pages(n + 2, P) for n in lens)
    assert state.tolist() == [n_pages - held, 0, 0, 0]
    in_use = torch.cat([table[b, :V.pages(lens[b] + 2, P)] for b in range(B)])
    all_pages = torch.cat((in_use, free[:n_pages - held])).sort().values
    assert all_pages.tolist() == list(range(n_pages))
    assert c.csa2_device_flags() == 0


def test_accepted_paths_that_are_not_the_first_nodes(orc):
    """Two verify steps.  Of the first one's trees, paths that skip nodes are accepted: their rows are appended once
    more, to the first drafted positions, before the lengths are cut.  The second step's nodes then select and attend
    the accepted context, as the oracle's decode of it does; without that append the positions hold rejected rows."""
    g = np.random.default_rng(29)
    B, N, P, K, W, mp = 3, 6, 16, 48, 12, 12
    lens = [61, 15, 0]
    parent = np.array([[-1, 0, 0, 2, 2, 4], [-1, -1, 1, 2, 0, 4], [-1, 0, 1, 2, 3, 4]], np.int32)
    accepted = [[0, 2, 4, 5], [1, 2, 3], [0, 1]]                # the last: its first nodes
    n_pages = 40
    S = n_pages * P
    kv = [syn.normal_bf16(3, syn.T_KV, b, (lens[b], 512)) for b in range(B)]
    ki = [syn.normal_bf16(3, syn.T_KI, b, (lens[b], 128)) for b in range(B)]
    draft_kv = [[syn.normal_bf16(5 + s, syn.T_KV, b, (N, 512)) for b in range(B)] for s in range(2)]
    draft_ki = [[syn.normal_bf16(5 + s, syn.T_KI, b, (N, 128)) for b in range(B)] for s in range(2)]
    codes = torch.zeros((S, 256), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((S, 32), dtype=torch.uint8, device="cuda")
    KI = torch.full((S, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    free = to_dev(g.permutation(n_pages).astype(np.int32))
    state = torch.tensor([n_pages, 0, 0, 0], dtype=torch.int32, device="cuda")
    i32 = lambda v: to_dev(np.array(v, np.int32))  # noqa: E731
    held, drafted = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    c.csa2_device_flags()

    def append(slots, rows_kv, rows_ki):
        c.csa2_paged_append(slots, kv_new=bf16_dev(rows_kv), codes=codes, scales=scales, ki_new=bf16_dev(rows_ki), KI=KI)

    def draft(step, n):
        slots = torch.empty((B, N), dtype=torch.int32, device="cuda")
        c.csa2_block_tables(i32(n), i32(n) + N, P, table, free, state, drafted, slots=slots)
        assert drafted.tolist() == [x + N for x in n]
        append(slots.view(-1), np.concatenate(draft_kv[step]), np.concatenate(draft_ki[step]))
        return slots

    slots0 = torch.empty((B, max(lens)), dtype=torch.int32, device="cuda")
    c.csa2_block_tables(i32([0] * B), i32(lens), P, table, free, state, held, slots=slots0)
    pad = [np.concatenate((np.arange(n), np.full(max(lens) - n, -1))) for n in lens]
    at = lambda x, r, w: np.concatenate((x, np.zeros((1, w), np.uint16)))[r]  # noqa: E731  (-1: a row of zeros)
    append(slots0.view(-1), np.concatenate([at(kv[b], pad[b], 512) for b in range(B)]),
           np.concatenate([at(ki[b], pad[b], 128) for b in range(B)]))
    slots1 = draft(0, lens)

    def holds(b, i, j):  # the slot of drafted position i holds node j's row and key
        ec, es = orc.fp4_quantize(draft_kv[0][b][j:j + 1])
        s = int(slots1[b, i])
        return (np.array_equal(codes[s].cpu().numpy(), ec[0]) and np.array_equal(scales[s].cpu().numpy(), es[0])
                and np.array_equal(bf16_host(KI[s]), draft_ki[0][b][j]))
    assert holds(0, 1, 1) and not holds(0, 1, 2)                # a rejected node's row, in an accepted position
    # the accepted rows once more; nodes in place already, and the rest, are padding
    move = np.array([(b, i, j) for b in range(B) for i, j in enumerate(accepted[b])])
    to = slots1[i32(move[:, 0]).long(), i32(move[:, 1]).long()]
    to = torch.where(i32(move[:, 1]) == i32(move[:, 2]), torch.full_like(to, -1), to)
    append(to, np.stack([draft_kv[0][b][j] for b, _, j in move]), np.stack([draft_ki[0][b][j] for b, _, j in move]))
    assert all(holds(b, i, j) for b, i, j in move)
    lens2 = [n + len(a) for n, a in zip(lens, accepted)]
    c.csa2_block_tables(drafted, i32(lens2), P, table, free, state, held)
    assert held.tolist() == lens2 and int(state[0]) == n_pages - sum(V.pages(n, P) for n in lens2)
    kv = [np.concatenate((kv[b], draft_kv[0][b][accepted[b]])) for b in range(B)]
    ki = [np.concatenate((ki[b], draft_ki[0][b][accepted[b]])) for b in range(B)]

    # the second step
    draft(1, lens2)
    q = np.stack([syn.normal_bf16(7, syn.T_Q, b, (N, 16, 512)) for b in range(B)])
    qI = np.stack([syn.normal_bf16(7, syn.T_QI, b, (N, 4, 128)) for b in range(B)])
    w = np.stack([syn.normal_f32(7, syn.T_W, b, (N, 4)) for b in range(B)])
    swa = np.stack([syn.normal_bf16(7, syn.T_SWA, b, (W - 1 + N, 512)) for b in range(B)])
    rows, ld = B * N, max(lens2) + N
    cand, n_cand = torch.empty((rows, ld), dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda")
    c.csa2_context_slots(i32(lens2), cand, n_cand, block_table=table, page_size=P, parent=to_dev(parent))
    scores, n_valid = torch.empty((rows, ld), device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda")
    c.csa2_index_score(bf16_dev(qI).view(1, rows, 4, 128), to_dev(w).view(1, rows, 4), KI[None], i32([S]), scores, cand=cand,
                       cand_len=n_cand, q_pos=i32([S - 1] * rows), n_valid=n_valid)
    idx, n_sel = torch.empty((rows, K), dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda")
    c.csa2_topk(scores, K, idx, n_valid=n_valid, map_=cand, n_sel=n_sel)
    out, lse = torch.zeros((B, N, 16, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, N, 16), device="cuda")
    win_len = [min(n, W - 1) for n in lens2]
    c.csa2_tree_attn(bf16_dev(q), to_dev(parent), codes, scales, idx, out, n_valid=n_sel, swa=bf16_dev(swa),
                     win_len=i32(win_len), W=W, softmax_scale=SCALE, lse=lse)
    cand_h, idx_h, sel_h = cand.cpu().numpy(), idx.cpu().numpy(), n_sel.cpu().numpy()
    for b in range(B):
        all_kv, all_ki = np.concatenate((kv[b], draft_kv[1][b])), np.concatenate((ki[b], draft_ki[1][b]))
        ec, es = orc.fp4_quantize(all_kv)
        for i in range(N):
            r, p = b * N + i, V.path(parent[b], i)
            pos = np.concatenate((np.arange(lens2[b]), lens2[b] + np.array(p))).astype(np.int64)
            top, n = orc.topk(orc.index_score(qI[b, i], w[b, i], all_ki[pos]), K)
            assert n == sel_h[r] and np.array_equal(idx_h[r, :n], cand_h[r, top[:n]])
            d = len(p) - 1
            win = np.concatenate((swa[b, max(d, W - 1 - win_len[b]):W - 1], swa[b, [W - 1 + j for j in p[-W:]]]))
            o, el = orc.sparse_attn(q[b, i], ec[pos], es[pos], top[:n], win, SCALE)
            assert_attn_close(bf16_host(out[b, i]), o, f"sequence {b} node {i}")
            assert np.abs(lse[b, i].cpu().numpy() - el).max() <= 1e-2
    assert c.csa2_device_flags() == 0
