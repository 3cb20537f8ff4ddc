"""q4_0_kv_append against a 64-bit rotation (GPU).

Tolerance.  The kernel rotates in fp32 (each result is two products and a sum
of fp32 values: an error of at most 3 * 2^-24 (|a| + |b|) for |cos|, |sin| <=
1) and rounds once to bfloat16 (relative error 2^-8).  Values are only
rounded, so they equal torch's conversion bit for bit, as does everything the
rotation leaves alone.
"""
import pytest
import torch

import serving_ref as ref
from gpu_common import lib

pytestmark = pytest.mark.gpu


def table(positions, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def run(b, q_heads, rot, interleaved, dtype, positions=None, pad=0, seed=1):
    q4 = lib()
    width = (q_heads + 2 * b.kv_heads) * b.dim
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(b.rows, width + pad, generator=g).to(dtype).cuda()
    qkv = wide[:, :width]
    cs = table(max(b.kv + [1]) + 64, rot)
    before = [t.clone() for t in b.cuda()[:2]]
    q = q4.kv_append(qkv, cs.cuda(), *b.dev, q_heads=q_heads, interleaved=interleaved,
                     positions=None if positions is None else positions.cuda())
    return q4, qkv.cpu(), cs, q, before


def check(b, q_heads, rot, interleaved, qkv, cs, q, before, positions=None):
    x = qkv.double().view(b.rows, q_heads + 2 * b.kv_heads, b.dim)
    k_want, v_want = (t.cpu().clone() for t in before)
    k_err = torch.zeros(k_want.shape, dtype=torch.float64)
    k_exact = k_want.double()
    q_exact, q_size = torch.zeros(b.rows, q_heads, b.dim, dtype=torch.float64), None
    q_size = torch.zeros_like(q_exact)
    inside = torch.zeros(b.rows, dtype=torch.bool)
    for s, n in enumerate(b.new):
        for i in range(n):
            r, pos = int(b.q_start[s]) + i, b.kv[s] - n + i
            turn = pos if positions is None else int(positions[r])
            c, sn = cs[turn, :rot // 2].double(), cs[turn, rot // 2:].double()
            turned = x[r, :q_heads + b.kv_heads].clone()
            turned[:, :rot] = ref.rotate(turned[:, :rot], c, sn, interleaved)
            # |a| + |b| of each pair
            size = ref.rotate(x[r, :q_heads + b.kv_heads, :rot].abs(), torch.ones(rot // 2), -torch.ones(rot // 2),
                              interleaved)
            sizes = torch.zeros_like(turned)
            sizes[:, :rot] = size.abs()
            if not interleaved:
                sizes[:, rot // 2:rot] = sizes[:, :rot // 2]
            else:
                sizes[:, 1:rot:2] = sizes[:, 0:rot:2]
            q_exact[r], q_size[r] = turned[:q_heads], sizes[:q_heads]
            page, off = b.place(s, pos)
            k_exact[page, :, off] = turned[q_heads:]
            k_err[page, :, off] = 2 ** -8 * turned[q_heads:].abs() + 3 * 2 ** -24 * sizes[q_heads:]
            v_want[page, :, off] = x[r, q_heads + b.kv_heads:].float().bfloat16()
            inside[r] = True
    tol = 2 ** -8 * q_exact.abs() + 3 * 2 ** -24 * q_size
    assert ((q.double().cpu() - q_exact).abs() <= tol)[inside].all()
    # elements that are not rotated are only rounded
    assert torch.equal(q[..., rot:].cpu()[inside], qkv.view(x.shape)[:, :q_heads, rot:].bfloat16()[inside])
    k_got, v_got = b.dev[0].cpu(), b.dev[1].cpu()
    assert ((k_got.double() - k_exact).abs() <= k_err).all()   # exact where nothing was appended
    assert torch.equal(v_got, v_want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q_heads,kv_heads,dim,rot,interleaved,page,token_major", [
    (40, 8, 128, 128, False, 16, False),
    (40, 8, 128, 64, True, 16, True),
    (4, 1, 64, 64, True, 1, False),
    (3, 3, 80, 24, False, 7, True),
    (2, 2, 256, 0, False, 128, False),
    (5, 1, 8, 8, True, 3, False),
])
def test_rotation_and_places(dtype, q_heads, kv_heads, dim, rot, interleaved, page, token_major):
    b = ref.Batch([1, 0, 5, 1, 33], [1, 4, 5, 100, 70], page, kv_heads, dim, seed=3, token_major=token_major)
    q4, qkv, cs, q, before = run(b, q_heads, rot, interleaved, dtype)
    check(b, q_heads, rot, interleaved, qkv, cs, q, before)
    assert q4.device_error() == q4.OK


def test_rows_in_several_pieces():
    """A row wider than one block of threads holds (32 KB): 96 heads of 128."""
    b = ref.Batch([2, 3], [2, 90], 16, 16, 128, seed=4)
    q4, qkv, cs, q, before = run(b, 64, 128, False, torch.float32)
    check(b, 64, 128, False, qkv, cs, q, before)
    assert q4.device_error() == q4.OK


def test_strided_rows_given_positions_and_rows_of_no_sequence():
    b = ref.Batch([3, 2], [10, 2], 16, 2, 64, seed=5, extra_rows=2)
    positions = torch.tensor([7, 0, 3, 3, 40, 0, 0], dtype=torch.int32)
    q4, qkv, cs, q, before = run(b, 4, 32, False, torch.float32, positions=positions, pad=8)
    check(b, 4, 32, False, qkv, cs, q, before, positions)
    assert q4.device_error() == q4.OK


def test_many_sequences():
    n = 600
    b = ref.Batch([i % 3 for i in range(n)], [i % 3 + i % 20 for i in range(n)], 16, 1, 64, seed=6)
    q4, qkv, cs, q, before = run(b, 2, 64, False, torch.bfloat16)
    check(b, 2, 64, False, qkv, cs, q, before)
    assert q4.device_error() == q4.OK


def test_writes_past_32_bit_offsets():
    """A cache of more than 2^32 bytes: the last page's slots are reached."""
    q4 = lib()
    pages, page, heads, dim = 140000, 16, 8, 128          # 2.3e9 elements
    cache = torch.zeros(pages, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(pages, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    qkv = torch.randn(1, (2 + 2 * heads) * dim, device="cuda")
    q4.kv_append(qkv, torch.zeros(8, 0, device="cuda"), cache, v, torch.tensor([[pages - 1]], dtype=torch.int32).cuda(),
                 torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([6], dtype=torch.int32).cuda(), q_heads=2)
    x = qkv.view(18, dim).bfloat16()
    assert torch.equal(cache[pages - 1, :, 5], x[2:10]) and torch.equal(v[pages - 1, :, 5], x[10:])
    assert int(cache.count_nonzero()) == int(x[2:10].count_nonzero())
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("what", ["page", "page past the end", "long", "short", "turn"])
def test_bad_places_are_reported_and_skipped(what):
    q4 = lib()
    b = ref.Batch([1, 1], [9, 5], 4, 1, 64, seed=7)
    k, v, page_table, q_start, kv_len = b.cuda()
    positions = None
    if what == "page":
        page_table[0, 2] = -5
    elif what == "page past the end":
        page_table[0, 2] = b.pages
    elif what == "long":
        kv_len[0] = 10 ** 6
    elif what == "short":
        kv_len[0] = 0
    else:
        positions = torch.tensor([10 ** 6, 0], dtype=torch.int32).cuda()
    qkv = torch.randn(2, 3 * 64).cuda()
    q4.kv_append(qkv, table(64, 64).cuda(), k, v, page_table, q_start, kv_len, q_heads=1, positions=positions)
    assert q4.device_error() == q4.ERR_DEVICE_INDEX
    assert q4.device_error() == q4.OK
    page, off = b.place(1, 4)
    want = torch.zeros_like(v)
    want[page, 0, off] = qkv[1, 128:].bfloat16()
    assert torch.equal(v, want)                            # the good row was written, nothing else


def test_refusals():
    q4 = lib()
    b = ref.Batch([1], [1], 4, 2, 64)
    dev = b.cuda()
    qkv, cs = torch.zeros(1, 6 * 64, device="cuda"), table(4, 64).cuda()
    good = lambda **k: q4.kv_append(k.pop("qkv", qkv), k.pop("cs", cs), *k.pop("dev", dev),  # noqa: E731
                                    q_heads=k.pop("q_heads", 2), **k)
    good()
    with pytest.raises(TypeError):
        good(qkv=qkv.half())
    with pytest.raises(ValueError):
        good(qkv=qkv.cpu())
    with pytest.raises(ValueError):
        good(q_heads=3)
    with pytest.raises(TypeError):
        good(cs=cs.double())
    with pytest.raises(TypeError):
        good(dev=(*dev[:2], dev[2].long(), *dev[3:]))
    with pytest.raises(ValueError):
        good(dev=(*dev[:3], dev[3][:1], dev[4]))
    with pytest.raises(ValueError):
        good(positions=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        good(out=torch.zeros(1, 3, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(q4.Q4Error):
        good(cs=torch.zeros(4, 4, device="cuda"))          # rot % 8
    assert good(qkv=qkv[:0]).shape == (0, 2, 64)
    assert q4.device_error() == q4.OK
