"""Refusals of the verify step's operators: answered from the arguments alone, nothing is launched."""
import ctypes

import pytest

import compressed_sparse_attention_step_gb300 as csa2
from compressed_sparse_attention_step_gb300 import _build

FAKE, FAKE2, ODD, ODD4 = (ctypes.c_void_p(v) for v in (0x100000, 0x900000, 0x100001, 0x100004))


@pytest.fixture(scope="module")
def L():
    _build.build()
    return csa2.lib()


def _p(i):  # distinct, aligned, never dereferenced on a rejected call
    return ctypes.c_void_p(0x10000000 * (i + 1))


def test_block_tables(L):
    def call(old=_p(0), new=_p(1), B=4, page=64, table=_p(2), mp=8, free=_p(3), cap=16, state=_p(4), granted=_p(5),
             slots=_p(6), n_new=8):
        return L.csa2_block_tables(old, new, B, page, table, mp, free, cap, state, granted, slots, n_new, None)
    for page in (0, -64, 8, 2048, 48):
        assert call(page=page) == csa2.ERR_INVALID_ARG
    assert call(B=-1) == 1 and call(B=csa2.MAX_SEQS + 1) == 1 and call(mp=0) == 1 and call(cap=-1) == 1
    assert call(n_new=-1) == 1
    assert call(B=8192, mp=1 << 18) == 1 and call(B=8192, n_new=1 << 18) == 1   # 2^31 entries
    assert call(mp=1 << 25) == 1                                                # positions past 31 bits
    for name in ("old", "new", "table", "free", "state", "granted", "slots"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: ODD}) == 1, name
    # granted and slots overlap no input, nor each other
    assert call(granted=_p(0)) == 1 and call(granted=_p(1)) == 1 and call(granted=_p(4)) == 1
    assert call(slots=_p(2)) == 1 and call(slots=_p(5)) == 1
    assert call(granted=ctypes.c_void_p(_p(2).value + 4 * 8 * 4 - 4)) == 1
    assert call(B=0) == csa2.OK


def test_context_slots(L):
    def call(lens=_p(0), parent=_p(1), nn=None, B=2, N=4, table=_p(2), mp=8, page=64, slots=_p(3), ld=64, ns=_p(4)):
        return L.csa2_context_slots(lens, parent, nn, B, N, table, mp, page, slots, ld, ns, None)
    assert call(N=csa2.MAX_TREE + 1) == 1 and call(N=-1) == 1 and call(B=-1) == 1 and call(B=65536) == 1
    assert call(ld=-1) == 1 and call(ld=1 << 31) == 1 and call(mp=0) == 1 and call(page=24) == 1
    assert call(lens=None) == 1 and call(slots=None) == 1 and call(ns=None) == 1
    assert call(slots=ODD4) == 1 and call(lens=ODD) == 1 and call(parent=ODD) == 1
    assert call(B=0) == 0 and call(N=0) == 0


def test_paged_append(L):
    def call(kv=_p(0), ki=_p(1), slots=_p(2), n=3, codes=_p(3), scales=_p(4), KI=_p(5), rows=64):
        return L.csa2_paged_append(kv, ki, slots, n, codes, scales, KI, rows, None)
    assert call(n=-1) == 1 and call(rows=-1) == 1 and call(slots=None) == 1 and call(slots=ODD) == 1
    for name in ("kv", "ki", "codes", "scales", "KI"):
        assert call(**{name: None}) == 1, name       # half a pair
        assert call(**{name: ODD4}) == 1, name
    assert call(n=0) == 0
    assert call(kv=None, codes=None, scales=None, ki=None, KI=None) == 0   # nothing to write


def test_tree_attn(L):
    def call(q=_p(0), B=2, N=4, parent=_p(1), nn=None, codes=_p(2), scales=_p(3), cap=64, pool=1, idx=_p(4), nv=None,
             k=8, swa=_p(5), wl=None, W=16, out=_p(6), lse=None):
        return L.csa2_tree_attn(q, B, N, parent, nn, codes, scales, cap, pool, idx, nv, k, swa, wl, W, 0.1, out, lse, None)
    assert call(N=csa2.MAX_TREE + 1) == 1 and call(k=513) == 1 and call(W=129) == 1 and call(cap=-1) == 1
    assert call(B=-1) == 1 and call(N=-1) == 1 and call(k=-1) == 1 and call(W=-1) == 1
    for name in ("q", "parent", "codes", "scales", "idx", "swa", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "codes", "scales", "swa", "out"):
        assert call(**{name: ODD4}) == 1, name
    assert call(B=0) == 0 and call(N=0) == 0


def test_fp4_weight(L):
    assert L.csa2_fp4_packed_bytes(16, 128) == 2304 and L.csa2_fp4_packed_bytes(33, 144) == 4 * 2304
    assert L.csa2_fp4_packed_bytes(16, 100) == 0 and L.csa2_fp4_packed_bytes(-1, 128) == 0
    assert L.csa2_fp4_pack_weight(_p(0), _p(1), 4, 24, _p(2), None) == 1
    assert L.csa2_fp4_pack_weight(None, _p(1), 4, 32, _p(2), None) == 1
    assert L.csa2_fp4_pack_weight(_p(0), _p(1), 4, 32, ODD4, None) == 1
    assert L.csa2_fp4_pack_weight(_p(0), _p(1), 0, 32, _p(2), None) == 0

    def call(x=_p(0), m=2, w=_p(1), n_out=8, n_in=32, rs=None, y=_p(2)):
        return L.csa2_fp4_matvec(x, m, w, n_out, n_in, rs, y, 0, None)
    assert call(m=csa2.MAX_MV_ROWS + 1) == 1 and call(m=-1) == 1 and call(n_in=40) == 1 and call(n_in=0) == 1
    assert call(n_out=-1) == 1
    assert call(x=None) == 1 and call(w=None) == 1 and call(y=None) == 1
    assert call(x=ODD4) == 1 and call(w=ODD4) == 1 and call(y=ODD4) == 1 and call(rs=ODD) == 1
    assert call(m=0) == 0 and call(n_out=0) == 0
    # y over x's last bytes, packed over its sources
    assert call(y=_p(0)) == 1 and call(y=ctypes.c_void_p(_p(0).value + 2 * 32 * 2 - 16)) == 1
    assert call(x=ctypes.c_void_p(_p(2).value + 2 * 8 * 2 - 16)) == 1
    assert L.csa2_fp4_pack_weight(_p(0), _p(1), 4, 32, _p(0), None) == 1
    assert L.csa2_fp4_pack_weight(_p(0), ctypes.c_void_p(_p(2).value + 2304 - 16), 4, 32, _p(2), None) == 1


def test_binding_checks_shapes_and_types():
    torch = pytest.importorskip("torch")
    i32 = torch.int32
    with pytest.raises(ValueError):   # not on a GPU
        csa2.csa2_block_tables(torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32), 64, torch.zeros((2, 4), dtype=i32),
                               torch.zeros(8, dtype=i32), torch.zeros(4, dtype=i32), torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError):   # granted of another batch
        csa2.csa2_block_tables(torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32), 64, torch.zeros((2, 4), dtype=i32),
                               torch.zeros(8, dtype=i32), torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32))
    with pytest.raises(ValueError):
        csa2.fp4_weight_alloc(16, 24, device="cpu")
    with pytest.raises(ValueError):   # channels not a multiple of 16
        csa2.csa2_fp4_matvec(torch.zeros((1, 24), dtype=torch.bfloat16), torch.zeros(2304, dtype=torch.uint8),
                             torch.zeros((1, 16), dtype=torch.bfloat16))
    with pytest.raises(ValueError):   # a weight of another size
        csa2.csa2_fp4_matvec(torch.zeros((1, 32), dtype=torch.bfloat16), torch.zeros(2304, dtype=torch.uint8),
                             torch.zeros((1, 33), dtype=torch.bfloat16))
    with pytest.raises(ValueError):   # scales of another width
        csa2.csa2_tree_attn(torch.zeros((1, 2, 16, 512), dtype=torch.bfloat16), torch.zeros((1, 2), dtype=i32),
                            torch.zeros((8, 256), dtype=torch.uint8), torch.zeros((8, 16), dtype=torch.uint8),
                            torch.zeros((2, 4), dtype=i32), torch.zeros((1, 2, 16, 512), dtype=torch.bfloat16))


def test_tree_attn_alignment_of_lists_it_may_not_need(L):
    """n_valid is read with k = 0 too, and win_len with W = 0: both on 4 bytes whatever the sizes."""
    def call(nv, wl, k, W, N=4):
        return L.csa2_tree_attn(_p(0), 2, N, _p(1), None, _p(2), _p(3), 64, 1, _p(4), nv, k, _p(5), wl, W, 0.1, _p(6),
                                None, None)
    assert call(ODD, None, 0, 16) == 1 and call(ODD, None, 8, 16) == 1
    assert call(None, ODD, 8, 0) == 1 and call(None, ODD, 8, 16) == 1
    assert call(ODD, ODD, 0, 0, N=0) == 0                # nothing to do: nothing is looked at


def _over(i, nbytes):  # the last 4, 16 or fewer bytes of buffer i
    return ctypes.c_void_p(_p(i).value + nbytes)


def test_overlap_of_context_slots(L):
    """What the call writes shares no byte with what it reads: n_slots may not be lens, though N = 1 gives both B
    entries; the lists may not lie over a table, the parents or the counts."""
    def call(lens=_p(0), parent=_p(1), nn=_p(5), B=2, N=4, table=_p(2), mp=8, slots=_p(3), ld=64, ns=_p(4)):
        return L.csa2_context_slots(lens, parent, nn, B, N, table, mp, 64, slots, ld, ns, None)
    assert call(ns=_p(0), N=1) == 1 and call(ns=_p(0), N=1, parent=None, nn=None, table=None) == 1
    for i in (0, 1, 2, 3, 5):
        assert call(ns=_p(i)) == 1, i
    for i in (0, 1, 2, 5):
        assert call(slots=_p(i)) == 1, i
    assert call(ns=_over(3, 2 * 4 * 64 * 4 - 4)) == 1            # the lists' last entry
    assert call(lens=_over(3, 2 * 4 * 64 * 4 - 4)) == 1 and call(table=_over(4, 2 * 4 * 4 - 4)) == 1


def test_overlap_of_block_tables(L):
    def call(old=_p(0), new=_p(1), table=_p(2), free=_p(3), state=_p(4), granted=_p(5), slots=_p(6)):
        return L.csa2_block_tables(old, new, 4, 64, table, 8, free, 16, state, granted, slots, 8, None)
    for name in ("table", "free", "state"):                      # changed in place
        for i in range(7):
            if _p(i).value != dict(table=_p(2), free=_p(3), state=_p(4))[name].value:
                assert call(**{name: _p(i)}) == 1, (name, i)
    assert call(free=_over(2, 4 * 8 * 4 - 4)) == 1 and call(state=_over(3, 16 * 4 - 4)) == 1


def test_overlap_of_paged_append(L):
    def call(kv=_p(0), ki=_p(1), slots=_p(2), codes=_p(3), scales=_p(4), KI=_p(5)):
        return L.csa2_paged_append(kv, ki, slots, 3, codes, scales, KI, 64, None)
    own = dict(codes=3, scales=4, KI=5)
    for name, at in own.items():
        for i in range(6):
            if i != at:
                assert call(**{name: _p(i)}) == 1, (name, i)
    assert call(kv=_over(5, 64 * 256 - 16)) == 1 and call(slots=_over(3, 64 * 256 - 4)) == 1


def test_overlap_of_tree_attn(L):
    """out may be q itself, not q moved by some rows, and nothing else that the call reads or writes."""
    row = 16 * 512 * 2

    def call(q=_p(0), parent=_p(1), nn=_p(7), codes=_p(2), scales=_p(3), idx=_p(4), nv=_p(8), swa=_p(5), wl=_p(9), out=_p(6),
             lse=_p(10), cap=64, pool=1, k=8, W=16):
        return L.csa2_tree_attn(q, 2, 4, parent, nn, codes, scales, cap, pool, idx, nv, k, swa, wl, W, 0.1, out, lse, None)
    for i in (1, 2, 3, 4, 5, 7, 8, 9, 10):
        assert call(out=_p(i)) == 1, i
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9):
        assert call(lse=_p(i)) == 1, i
    assert call(out=_over(0, row)) == 1 and call(out=_over(0, 8 * row - 16)) == 1 and call(q=_over(6, row)) == 1
    assert call(out=_p(0), lse=_over(0, row)) == 1
    assert call(out=_over(2, 64 * 256 - 16)) == 1                                    # a pool's last row
    assert call(out=_over(2, 2 * 64 * 256 - 16), pool=0) == 1                        # the last sequence's last row
    assert call(out=_over(5, 2 * 19 * 1024 - 16)) == 1                               # the window's last row
    assert call(out=_p(2), cap=(1 << 63) - 1, pool=0) == 1                           # sizes past 64 bits


def test_overlap_of_fp4_matvec(L):
    def call(x=_p(0), w=_p(1), rs=_p(3), y=_p(2), fp32=0):
        return L.csa2_fp4_matvec(x, 2, w, 8, 32, rs, y, fp32, None)
    assert call(y=_p(1)) == 1 and call(y=_over(1, 2304 - 16)) == 1 and call(y=_p(3)) == 1
    assert call(w=_over(2, 16)) == 1 and call(rs=_over(2, 2 * 8 * 2 - 4)) == 1
    assert call(rs=_over(2, 2 * 8 * 4 - 4), fp32=1) == 1


def test_what_does_not_overlap_is_not_refused(L):
    """Arrays that touch, an array given twice as an input, and arrays that the sizes leave without a byte pass the
    checks (what comes behind them needs a GPU: not an invalid argument here, or done)."""
    old = _p(0)
    ok = (csa2.OK, csa2.ERR_CUDA)
    if csa2._torch().cuda.is_available():
        pytest.skip("the calls would run")
    assert L.csa2_block_tables(old, old, 4, 64, _p(1), 8, _over(1, 4 * 8 * 4), 16, _p(2), _p(3), None, 0, None) in ok
    assert L.csa2_context_slots(old, None, old, 2, 4, None, 0, 0, _p(1), 64, _over(1, 2 * 4 * 64 * 4), None) in ok
    assert L.csa2_paged_append(None, _p(0), _p(1), 3, None, None, _over(0, 3 * 256), 64, None) in ok
    assert L.csa2_tree_attn(_p(0), 2, 4, _p(1), None, _p(2), _p(2), 64, 1, _p(4), None, 8, None, None, 0, 0.1, _p(0),
                            None, None) in ok
    assert L.csa2_tree_attn(_p(0), 2, 4, _p(1), None, _p(6), _p(6), 64, 1, _p(6), None, 0, _p(6), None, 0, 0.1, _p(6),
                            None, None) in ok                       # k = 0 and W = 0: neither cache nor window
    assert L.csa2_fp4_matvec(_p(0), 2, _p(1), 8, 32, None, _over(1, 2304), 0, None) in ok
